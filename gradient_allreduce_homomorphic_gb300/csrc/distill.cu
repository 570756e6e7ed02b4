// distill.cu -- distillation from a teacher's top logits: gar_distill_loss and
// gar_distill_grad.
//
// Row t has the student's logits z_v and the teacher's entries (i_j, t_j):
//   p_j  = softmax over the row's present entries of t_j / tau
//   lse  = log sum_v exp(z_v / tau)
//   loss = sum_j p_j (log p_j + lse - z_{i_j} / tau)
//   dz_v = w / tau (exp(z_v / tau - lse) - sum_{j: i_j = v} p_j)
// An entry is present if its index lies in [0, V) and its logit is above -inf.
// Everything is computed in fp32 and rounded once, when dz is stored.
#include "common.cuh"
#include "fp8.cuh"

namespace gar {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxTop = 1024;

struct DistillParams {
    const void *z;
    int64_t rows, ldz, lddz;
    int32_t vocab, k;
    const int32_t *index;
    const float *teacher;
    const float *weight;  // NULL: 1
    float inv_tau;
    float *loss, *lse;         // gar_distill_loss
    const float *lse_in;       // gar_distill_grad
    void *dz;                  // NULL: no gradient
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The block's sum (or maximum), the same value in every thread.
template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float *scratch) {
    v = kMax ? warp_max(v) : warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[threadIdx.x & (kThreads / 32 - 1)];
#pragma unroll
    for (int o = kThreads / 64; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = kMax ? fmaxf(v, u) : v + u;
    }
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) distill_kernel(const __grid_constant__ DistillParams p) {
    __shared__ float scratch[kThreads / 32];
    __shared__ float top_p[kMaxTop], top_z[kMaxTop];
    __shared__ int32_t top_i[kMaxTop];
    const int64_t row = blockIdx.x;
    const T *z = static_cast<const T *>(p.z) + row * p.ldz;
    T *dz = p.dz ? static_cast<T *>(p.dz) + row * p.lddz : nullptr;
    const float w = p.weight ? p.weight[row] : 1.0f;
    const int tid = threadIdx.x;

    float tmax = -INFINITY;
    for (int j = tid; j < p.k; j += kThreads) {
        const int32_t i = p.index[row * p.k + j];
        const float t = p.teacher[row * p.k + j] * p.inv_tau;
        const bool on = i >= 0 && i < p.vocab && !(t == -INFINITY);
        top_i[j] = on ? i : -1;
        top_p[j] = t;
        if (on) tmax = fmaxf(tmax, t);
    }
    tmax = block_reduce<true>(tmax, scratch);
    float tsum = 0.0f;
    for (int j = tid; j < p.k; j += kThreads) {
        const float e = top_i[j] >= 0 ? expf(top_p[j] - tmax) : 0.0f;
        tsum += e;
    }
    tsum = block_reduce<false>(tsum, scratch);
    const bool live = w != 0.0f && tsum != 0.0f;
    if (!live) {  // nothing to learn in this row: z is not read
        if (dz)
            for (int v = tid; v < p.vocab; v += kThreads) store_f32(dz + v, 0.0f);
        if (tid == 0 && p.loss) p.loss[row] = 0.0f;
        if (tid == 0 && p.lse) p.lse[row] = 0.0f;
        return;
    }
    const float log_tsum = logf(tsum);
    float lse;
    if (p.lse_in) {
        lse = p.lse_in[row];
    } else {
        float m = -INFINITY;
        for (int v = tid; v < p.vocab; v += kThreads) m = fmaxf(m, load_f32(z + v));
        m = block_reduce<true>(m, scratch);
        float s = 0.0f;
        for (int v = tid; v < p.vocab; v += kThreads) s += expf((load_f32(z + v) - m) * p.inv_tau);
        s = block_reduce<false>(s, scratch);
        lse = m == -INFINITY ? -INFINITY : m * p.inv_tau + logf(s);
    }
    float part = 0.0f;
    for (int j = tid; j < p.k; j += kThreads) {
        float pj = 0.0f;
        if (top_i[j] >= 0) {
            const float logp = top_p[j] - tmax - log_tsum;
            pj = expf(logp);
            const float zj = load_f32(z + top_i[j]) * p.inv_tau;
            top_z[j] = zj;
            if (pj > 0.0f) part += lse == -INFINITY ? INFINITY : pj * (logp + lse - zj);
            else if (pj != pj) part = pj;
        }
        top_p[j] = pj;
    }
    part = block_reduce<false>(part, scratch);
    if (tid == 0 && p.loss) p.loss[row] = part;
    if (tid == 0 && p.lse) p.lse[row] = lse;
    if (!dz) return;
    const float g = w * p.inv_tau;
    for (int v = tid; v < p.vocab; v += kThreads) {
        const float q = lse == -INFINITY ? 0.0f : expf(load_f32(z + v) * p.inv_tau - lse);
        store_f32(dz + v, g * q);
    }
    __syncthreads();
    for (int j = tid; j < p.k; j += kThreads) {
        const int32_t i = top_i[j];
        if (i < 0) continue;
        float sum = 0.0f;
        bool first = true;
        for (int o = 0; o < p.k; ++o)
            if (top_i[o] == i) {
                if (o < j) first = false;
                sum += top_p[o];
            }
        if (!first) continue;
        const float q = lse == -INFINITY ? 0.0f : expf(top_z[j] - lse);
        store_f32(dz + i, g * (q - sum));
    }
}

int check(const void *z, int32_t dtype, int64_t rows, int64_t vocab, int64_t ldz, const int32_t *index,
          const float *teacher, int32_t k, float tau, const void *dz, int64_t lddz) {
    if (elem_bytes(dtype) < 0) return fail(GAR_EDTYPE, "unknown dtype %d", dtype);
    if (rows < 0 || rows > 0x7FFFFFFF || vocab < 1 || vocab > 0x7FFFFFFF || k < 1 || k > kMaxTop)
        return fail(GAR_EINVAL, "rows=%lld vocab=%lld k=%d (1 <= k <= %d)", static_cast<long long>(rows),
                    static_cast<long long>(vocab), k, kMaxTop);
    if (!(tau > 0.0f) || !(tau <= 3.0e38f)) return fail(GAR_EINVAL, "tau must be positive and finite");
    if (rows == 0) return GAR_OK;
    if (!z || !index || !teacher) return fail(GAR_EINVAL, "NULL argument");
    if (ldz < vocab || (dz && lddz < vocab)) return fail(GAR_EINVAL, "a row stride is below the vocabulary");
    if (dz == z && dz && lddz != ldz) return fail(GAR_EINVAL, "dz in place of z needs the same row stride");
    if (!aligned(z, elem_bytes(dtype)) || !aligned(dz, elem_bytes(dtype)) || !aligned(index, 4) || !aligned(teacher, 4))
        return fail(GAR_EALIGN, "misaligned pointer");
    return GAR_OK;
}

int run(const DistillParams &p, int32_t dtype, cudaStream_t stream) {
    if (p.rows == 0) return GAR_OK;
    const unsigned blocks = static_cast<unsigned>(p.rows);
    if (dtype == GAR_F32)
        distill_kernel<float><<<blocks, kThreads, 0, stream>>>(p);
    else
        distill_kernel<uint16_t><<<blocks, kThreads, 0, stream>>>(p);
    return check_launch("distill_kernel");
}

}  // namespace
}  // namespace gar

using namespace gar;

extern "C" int gar_distill_loss(const void *z, int32_t dtype, int64_t rows, int64_t vocab, int64_t ldz,
                                const int32_t *index, const float *teacher, int32_t k, float tau, const float *weight,
                                float *loss, float *lse, void *dz, int64_t lddz, gar_stream_t stream) {
    if (int rc = check(z, dtype, rows, vocab, ldz, index, teacher, k, tau, dz, lddz)) return rc;
    if (rows > 0 && (!loss || !lse)) return fail(GAR_EINVAL, "loss or lse is NULL");
    if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(weight, 4)) return fail(GAR_EALIGN, "misaligned pointer");
    DistillParams p{};
    p.z = z, p.rows = rows, p.ldz = ldz, p.lddz = lddz, p.vocab = static_cast<int32_t>(vocab), p.k = k;
    p.index = index, p.teacher = teacher, p.weight = weight, p.inv_tau = 1.0f / tau;
    p.loss = loss, p.lse = lse, p.dz = dz;
    return run(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int gar_distill_grad(const void *z, int32_t dtype, int64_t rows, int64_t vocab, int64_t ldz,
                                const int32_t *index, const float *teacher, int32_t k, float tau, const float *weight,
                                const float *lse, void *dz, int64_t lddz, gar_stream_t stream) {
    if (int rc = check(z, dtype, rows, vocab, ldz, index, teacher, k, tau, dz, lddz)) return rc;
    if (rows > 0 && (!lse || !dz)) return fail(GAR_EINVAL, "lse or dz is NULL");
    if (!aligned(lse, 4) || !aligned(weight, 4)) return fail(GAR_EALIGN, "misaligned pointer");
    DistillParams p{};
    p.z = z, p.rows = rows, p.ldz = ldz, p.lddz = lddz, p.vocab = static_cast<int32_t>(vocab), p.k = k;
    p.index = index, p.teacher = teacher, p.weight = weight, p.inv_tau = 1.0f / tau;
    p.lse_in = lse, p.dz = dz;
    return run(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}
