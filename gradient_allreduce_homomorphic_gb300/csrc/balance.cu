// balance.cu -- a router's choices, per-expert counts and balance loss over P
// workers' tokens, with its gradient: gar_balance_loss.
//
// Token t of worker w chooses the k experts with the largest logits (ties to
// the lowest index).  With c_e the number of choices of expert e over all
// workers, N the number of tokens that count and p_t = softmax(z_t),
//   L       = alpha E sum_e f_e P_e,   f_e = c_e / (k N),  P_e = sum_t p_te / N
//           = coef sum_t d_t,          coef = alpha E / (k N^2), d_t = sum_e p_te c_e
//   dL/dz_te = coef p_te (c_e - d_t)   (the counts carry no gradient)
// so the only quantity that needs every token before the gradient is c: one
// pass over z takes the choices and counts (integer atomics, whose order does
// not matter), a second the gradient and d_t.  sum_e p_te = 1, so c may be
// shifted by any constant; the mean k N / E is taken off, which removes the
// cancellation of c_e - d_t for a router near balance.
#include "common.cuh"
#include "fp8.cuh"

namespace gar {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxExperts = 1024;
constexpr int kPerLane = kMaxExperts / 32;
constexpr int kMaxChoices = 32;
constexpr int kMaxBlocks = 4096;

struct BalanceParams {
    const void *z[GAR_MAX_WORKERS];
    void *dz[GAR_MAX_WORKERS];
    int32_t *choice[GAR_MAX_WORKERS];
    const uint8_t *valid[GAR_MAX_WORKERS];
    int64_t tokens, ldz, lddz;
    int32_t P, experts, k, has_valid, has_grad;
    float alpha;
    int32_t *counts;      // [P, experts]
    int32_t *n_tokens;    // workspace: tokens that count, per worker
    double *partial;      // workspace: sum of d_t per CTA
    float *loss;
};

// A token's logits: lane l holds experts l, l + 32, ...; -inf past the end.
template <typename T>
__device__ __forceinline__ void load_token(const BalanceParams &p, int w, int64_t t, int lane, int per, float *v) {
    const T *z = static_cast<const T *>(p.z[w]) + t * p.ldz;
    for (int i = 0; i < per; ++i) {
        const int e = i * 32 + lane;
        v[i] = e < p.experts ? load_f32(z + e) : -INFINITY;
    }
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) balance_count_kernel(const __grid_constant__ BalanceParams p) {
    __shared__ int32_t cnt[kMaxExperts];
    __shared__ int32_t seen;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = blockIdx.y;
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) cnt[e] = 0;
    if (threadIdx.x == 0) seen = 0;
    __syncthreads();
    const int per = (p.experts + 31) / 32;
    float v[kPerLane];
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < p.tokens;
         t += static_cast<int64_t>(gridDim.x) * kWarps) {
        const bool valid = !p.has_valid || p.valid[w][t] != 0;
        int32_t *out = p.choice[w] + t * p.k;
        if (!valid) {
            if (lane < p.k) out[lane] = -1;
            continue;
        }
        load_token<T>(p, w, t, lane, per, v);
        bool some = false;
        for (int i = 0; i < per; ++i) some |= !(v[i] == -INFINITY);
        some = __any_sync(0xFFFFFFFFu, some);
        if (some && lane == 0) atomicAdd(&seen, 1);
        for (int c = 0; c < p.k; ++c) {
            float best = -INFINITY;
            int at = 0x7FFFFFFF;
            for (int i = 0; i < per; ++i)
                if (v[i] > best) best = v[i], at = i * 32 + lane;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float u = __shfl_xor_sync(0xFFFFFFFFu, best, o);
                const int a = __shfl_xor_sync(0xFFFFFFFFu, at, o);
                if (u > best || (u == best && a < at)) best = u, at = a;
            }
            const bool found = at != 0x7FFFFFFF;
            if (lane == 0) {
                out[c] = found ? at : -1;
                if (found) atomicAdd(&cnt[at], 1);
            }
            if (found && (at & 31) == lane) v[at >> 5] = -INFINITY;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x)
        if (cnt[e]) atomicAdd(&p.counts[w * p.experts + e], cnt[e]);
    if (threadIdx.x == 0 && seen) atomicAdd(&p.n_tokens[w], seen);
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) balance_grad_kernel(const __grid_constant__ BalanceParams p) {
    __shared__ float c[kMaxExperts];
    __shared__ double wsum[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = blockIdx.y;
    int64_t n = 0;
    for (int i = 0; i < p.P; ++i) n += p.n_tokens[i];
    int64_t all = 0;  // choices made: k N, or fewer where a token had fewer experts to choose from
    for (int e = 0; e < p.experts; ++e)
        for (int i = 0; i < p.P; ++i) all += p.counts[i * p.experts + e];
    const double mean = static_cast<double>(all) / p.experts;
    for (int e = threadIdx.x; e < p.experts; e += blockDim.x) {
        int64_t s = 0;
        for (int i = 0; i < p.P; ++i) s += p.counts[i * p.experts + e];
        c[e] = static_cast<float>(static_cast<double>(s) - mean);
    }
    __syncthreads();
    const int per = (p.experts + 31) / 32;
    const double coef = n > 0 ? static_cast<double>(p.alpha) * p.experts / (static_cast<double>(p.k) * n * n) : 0.0;
    const float fcoef = static_cast<float>(coef);
    float v[kPerLane];
    double sum = 0.0;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < p.tokens;
         t += static_cast<int64_t>(gridDim.x) * kWarps) {
        T *dz = p.has_grad ? static_cast<T *>(p.dz[w]) + t * p.lddz : nullptr;
        bool live = !p.has_valid || p.valid[w][t] != 0;
        float m = -INFINITY;
        if (live) {
            load_token<T>(p, w, t, lane, per, v);
            bool some = false;
            for (int i = 0; i < per; ++i) m = fmaxf(m, v[i]), some |= !(v[i] == -INFINITY);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            live = __any_sync(0xFFFFFFFFu, some);
        }
        if (!live) {
            if (dz)
                for (int e = lane; e < p.experts; e += 32) store_f32(dz + e, 0.0f);
            continue;
        }
        float s = 0.0f, d = 0.0f;
        for (int i = 0; i < per; ++i) {
            const int e = i * 32 + lane;
            v[i] = expf(v[i] - m);
            s += v[i];
            if (e < p.experts) d += v[i] * c[e];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
        }
        d /= s;
        sum += d;
        const float f = fcoef / s;
        if (dz)
            for (int i = 0; i < per; ++i) {
                const int e = i * 32 + lane;
                if (e < p.experts) store_f32(dz + e, f * v[i] * (c[e] - d));
            }
    }
    if (lane == 0) wsum[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int i = 0; i < kWarps; ++i) s += wsum[i];
        p.partial[blockIdx.y * gridDim.x + blockIdx.x] = s;
    }
}

__global__ void balance_loss_kernel(const __grid_constant__ BalanceParams p, int blocks) {
    __shared__ double acc[256];
    int64_t n = 0, all = 0;
    for (int i = 0; i < p.P; ++i) n += p.n_tokens[i];
    for (int i = 0; i < p.P * p.experts; ++i) all += p.counts[i];
    double s = 0.0;
    for (int i = threadIdx.x; i < blocks; i += 256) s += p.partial[i];
    acc[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int i = 0; i < 256; ++i) t += acc[i];
        const double mean = static_cast<double>(all) / p.experts;
        const double coef = n > 0 ? static_cast<double>(p.alpha) * p.experts / (static_cast<double>(p.k) * n * n) : 0.0;
        *p.loss = static_cast<float>(coef * (t + mean * static_cast<double>(n)));
    }
}

template <typename T>
int launch(const BalanceParams &p, int blocks, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(p.P));
    balance_count_kernel<T><<<grid, kWarps * 32, 0, stream>>>(p);
    if (int rc = check_launch("balance_count_kernel")) return rc;
    balance_grad_kernel<T><<<grid, kWarps * 32, 0, stream>>>(p);
    if (int rc = check_launch("balance_grad_kernel")) return rc;
    balance_loss_kernel<<<1, 256, 0, stream>>>(p, blocks * p.P);
    return check_launch("balance_loss_kernel");
}

}  // namespace
}  // namespace gar

using namespace gar;

extern "C" size_t gar_balance_workspace_bytes(int32_t P) {
    return P < 1 || P > GAR_MAX_WORKERS ? 0 : static_cast<size_t>(kMaxBlocks) * 8 + GAR_MAX_WORKERS * 4;
}

extern "C" int gar_balance_loss(const void *const *z, int32_t P, int64_t tokens, int32_t experts, int64_t ldz,
                                int32_t dtype, int32_t k, const uint8_t *const *valid, float alpha,
                                int32_t *const *choice, int32_t *counts, float *loss, void *const *dz, int64_t lddz,
                                void *d_workspace, size_t workspace_bytes, gar_stream_t stream_) {
    if (P < 1 || P > GAR_MAX_WORKERS) return fail(GAR_EINVAL, "P=%d outside 1..%d", P, GAR_MAX_WORKERS);
    if (elem_bytes(dtype) < 0) return fail(GAR_EDTYPE, "unknown dtype %d", dtype);
    if (tokens < 0 || tokens * P > 0x7FFFFFFF / kMaxChoices || experts < 1 || experts > kMaxExperts || k < 1 ||
        k > kMaxChoices || k > experts)
        return fail(GAR_EINVAL, "tokens=%lld experts=%d (1..%d) k=%d (1..%d, at most the experts)",
                    static_cast<long long>(tokens), experts, kMaxExperts, k, kMaxChoices);
    if (!(alpha - alpha == 0.0f)) return fail(GAR_EINVAL, "alpha must be finite");
    if (!counts || !loss || !d_workspace || workspace_bytes < gar_balance_workspace_bytes(P))
        return fail(GAR_EINVAL, "NULL argument, or the workspace is too small");
    if (!aligned(counts, 4) || !aligned(loss, 4) || !aligned(d_workspace, 8)) return fail(GAR_EALIGN, "misaligned pointer");
    if (tokens > 0 && (!z || !choice || ldz < experts || (dz && lddz < experts)))
        return fail(GAR_EINVAL, "NULL pointer table, or a row stride below the experts");
    BalanceParams p{};
    for (int i = 0; tokens > 0 && i < P; ++i) {
        if (!z[i] || !choice[i] || (dz && !dz[i]) || (valid && !valid[i])) return fail(GAR_EINVAL, "NULL worker pointer");
        if (!aligned(z[i], elem_bytes(dtype)) || !aligned(choice[i], 4) || (dz && !aligned(dz[i], elem_bytes(dtype))))
            return fail(GAR_EALIGN, "misaligned worker pointer");
        if (dz && dz[i] == z[i] && lddz != ldz) return fail(GAR_EINVAL, "dz in place of z needs the same row stride");
        p.z[i] = z[i], p.choice[i] = choice[i];
        p.dz[i] = dz ? dz[i] : nullptr;
        p.valid[i] = valid ? valid[i] : nullptr;
    }
    p.tokens = tokens, p.ldz = ldz, p.lddz = lddz;
    p.P = P, p.experts = experts, p.k = k, p.has_valid = valid != nullptr, p.has_grad = dz != nullptr;
    p.alpha = alpha, p.counts = counts, p.loss = loss;
    p.partial = static_cast<double *>(d_workspace);
    p.n_tokens = reinterpret_cast<int32_t *>(p.partial + kMaxBlocks);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * P * experts, stream);
    if (e == cudaSuccess) e = cudaMemsetAsync(p.n_tokens, 0, sizeof(int32_t) * GAR_MAX_WORKERS, stream);
    if (e != cudaSuccess) return fail(GAR_ECUDA, "gar_balance_loss: %s", cudaGetErrorString(e));
    int64_t blocks = ceil_div(tokens, kWarps);
    const int64_t cap = ceil_div(static_cast<int64_t>(sm_count()) * 8, P);
    if (blocks > cap) blocks = cap;
    if (blocks > kMaxBlocks / P) blocks = kMaxBlocks / P;
    if (blocks < 1) blocks = 1;
    return dtype == GAR_F32 ? launch<float>(p, static_cast<int>(blocks), stream)
                            : launch<uint16_t>(p, static_cast<int>(blocks), stream);
}
