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
//
// A token is held by L lanes of a warp, V of its logits each, in runs of 16
// bytes that neighbouring lanes hold in turn.  A warp works on 32 / L tokens at
// a time: with V = 32 most instructions serve several tokens and a warp has 4
// KB of loads in flight; with V = 8 few tokens spread over more warps.  Logits
// are loaded as they are stored and unpacked where they are used: unpacked at
// once, each load's wait would hold up the next (8 workers of 16384 tokens and
// 256 bf16 experts: 93 us, 69 so).
//
// 8 x 16384 x 256 fp32, 8 choices: 86 us, of which the counting pass 40 (the
// selection's instructions, 714 for a warp's four tokens, issued in 53 % of the
// cycles) and the gradient 46 (HBM: its logits read a second time).  Few tokens
// cost their launches: 4 x 2000 x 60 bf16 18 us a call, 64 x 8 12 us, one launch.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "fp8.cuh"
#include "launch.cuh"
#include "tensorcore.cuh"

namespace gar {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 32;
constexpr int kMaxBlocks = 4096;
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kOneThreads = 512;           // a CTA of the one-cluster kernel
constexpr int kOneCounts = 4096;           // its counts: workers x experts
constexpr float kLog2e = 1.44269504088896340736f;

struct BalanceParams {
    const void *z[GAR_MAX_WORKERS];
    void *dz[GAR_MAX_WORKERS];
    int32_t *choice[GAR_MAX_WORKERS];
    const uint8_t *valid[GAR_MAX_WORKERS];
    int64_t tokens, ldz, lddz;
    int32_t P, experts, k, has_valid, has_grad;
    int32_t align, dalign;  // every row of z, of dz starts on that many bytes (2 to 16)
    float alpha;
    int32_t *counts;     // [P, experts]
    uint32_t *seen;      // workspace: CTAs done; each worker's tokens that count
    float *partial;      // workspace: sum of d_t per CTA
    float *loss;
};

template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// The lanes that share a lane's token.
template <int L>
__device__ __forceinline__ uint32_t group_mask(int lane) {
    return L == 32 ? 0xFFFFFFFFu : ((1u << (L & 31)) - 1u) << (lane & ~(L - 1));
}

// Expert of a lane's i-th value, the values being of type T.
template <typename T, int L>
__device__ __forceinline__ int expert(int sub, int i) {
    constexpr int kRun = 16 / sizeof(T);
    return i / kRun * (kRun * L) + sub * kRun + i % kRun;
}

// A lane's logits of one token as they are stored, a run in each; -inf past the last expert.
template <typename T, int V>
using Runs = uint4[V * sizeof(T) / 16];
// kWide: all rows start on 16 bytes.  Else (`align`: on how many they do), and
// where the last expert cuts a run, it is accessed in the largest pieces that fit.
template <typename T, int L, int V, bool kWide>
__device__ __forceinline__ void load_runs(const T *z, int sub, int experts, int align, Runs<T, V> &g) {
    constexpr int kRun = 16 / sizeof(T), kWord = 4 / sizeof(T);
#pragma unroll
    for (int r = 0; r < V / kRun; ++r) {
        const int e0 = expert<T, L>(sub, r * kRun);
        if ((kWide || align == 16) && e0 + kRun <= experts) {
            g[r] = *reinterpret_cast<const uint4 *>(z + e0);
            continue;
        }
        uint32_t x[4];
#pragma unroll
        for (int h = 0; h < 4; h += 2) {
            const int e1 = e0 + h * kWord;
            if (!kWide && align >= 8 && e1 + 2 * kWord <= experts) {
                const uint2 u = *reinterpret_cast<const uint2 *>(z + e1);
                x[h] = u.x, x[h + 1] = u.y;
                continue;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int e = e1 + j * kWord;
                if ((kWide || align >= 4) && e + kWord <= experts)
                    x[h + j] = *reinterpret_cast<const uint32_t *>(z + e);
                else if constexpr (sizeof(T) == 2)
                    x[h + j] = (e < experts ? z[e] : 0xFF80u) | (e + 1 < experts ? z[e + 1] : 0xFF80u) << 16;
                else
                    x[h + j] = 0xFF800000u;
            }
        }
        g[r] = make_uint4(x[0], x[1], x[2], x[3]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void unpack_runs(const Runs<T, V> &g, float (&v)[V]) {
    constexpr int kRun = 16 / sizeof(T);
#pragma unroll
    for (int r = 0; r < V / kRun; ++r) {
        float *x = v + r * kRun;
        if constexpr (sizeof(T) == 2) {
            x[0] = bf16_lo(g[r].x), x[1] = bf16_hi(g[r].x), x[2] = bf16_lo(g[r].y), x[3] = bf16_hi(g[r].y);
            x[4] = bf16_lo(g[r].z), x[5] = bf16_hi(g[r].z), x[6] = bf16_lo(g[r].w), x[7] = bf16_hi(g[r].w);
        } else {
            x[0] = __uint_as_float(g[r].x), x[1] = __uint_as_float(g[r].y);
            x[2] = __uint_as_float(g[r].z), x[3] = __uint_as_float(g[r].w);
        }
    }
}
template <typename T, int L, int V, bool kWide>
__device__ __forceinline__ void store_token(T *dz, int sub, int experts, int align, const float (&v)[V]) {
    constexpr int kRun = 16 / sizeof(T), kWord = 4 / sizeof(T);
#pragma unroll
    for (int r = 0; r < V; r += kRun) {
        const int e0 = expert<T, L>(sub, r);
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 2)
                x[j] = pack_bf16x2(v[r + 2 * j], v[r + 2 * j + 1]);
            else
                x[j] = __float_as_uint(v[r + j]);
        }
        if ((kWide || align == 16) && e0 + kRun <= experts) {
            st16(dz + e0, make_uint4(x[0], x[1], x[2], x[3]));  // streaming: z, which is read again, is worth more in L2
            continue;
        }
#pragma unroll
        for (int h = 0; h < 4; h += 2) {
            const int e1 = e0 + h * kWord;
            if (!kWide && align >= 8 && e1 + 2 * kWord <= experts) {
                *reinterpret_cast<uint2 *>(dz + e1) = make_uint2(x[h], x[h + 1]);
                continue;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int e = e1 + j * kWord;
                if ((kWide || align >= 4) && e + kWord <= experts) {
                    *reinterpret_cast<uint32_t *>(dz + e) = x[h + j];
                } else if constexpr (sizeof(T) == 2) {
                    if (e < experts) dz[e] = static_cast<uint16_t>(x[h + j]);
                    if (e + 1 < experts) dz[e + 1] = static_cast<uint16_t>(x[h + j] >> 16);
                }
            }
        }
    }
}

// A NaN compares false and is passed over by fmaxf, so it is never chosen.

// A token's choices by k rounds of: the group's largest value, its lowest
// expert, that value taken out.  v is used up.  About 3 V + 2 log2 L + 15
// instructions a round for 32 / L tokens.
template <typename T, int L, int V>
__device__ __forceinline__ void choose_by_rounds(float (&v)[V], int sub, int lane, int k, bool live, int32_t *out, int32_t *cnt) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);
    for (int c = 0; c < k; ++c) {
        const float best = group_max<L>(m);
        const bool some = best > -INFINITY;
        uint32_t at = 0xFFFFFFFFu;
        if (some && m == best) {
#pragma unroll
            for (int i = V - 1; i >= 0; --i)
                if (v[i] == best) at = expert<T, L>(sub, i);
        }
        uint32_t lowest = at;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) lowest = min(lowest, __shfl_xor_sync(0xFFFFFFFFu, lowest, o));
        if (some && at == lowest) {
            m = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (expert<T, L>(sub, i) == static_cast<int>(at)) v[i] = -INFINITY;
                m = fmaxf(m, v[i]);
            }
            out[c] = static_cast<int32_t>(at);
            atomicAdd(cnt + at, 1);
        }
        if (!some && live && sub == 0) out[c] = -1;
    }
}

// The same in fewer instructions where a token takes four lanes or more: the
// k-th largest of its 4 L maxima of 8 values bounds the k-th largest value from
// below, so the few values that reach it (k and a half in the mean, for k = 8
// of 256) hold the choices; they are listed in shared memory and each is
// ranked against the others.  Tokens with more of them than the list holds
// (many equal values), or with fewer such maxima than choices, are reported
// for choose_by_rounds.
constexpr int kList = 32;
// Order of choice as an integer: larger value first, then the lower expert.
__device__ __forceinline__ uint64_t choice_key(float v, uint32_t e) {
    uint32_t u = __float_as_uint(v + 0.0f);  // one zero
    u ^= u >> 31 ? 0xFFFFFFFFu : 0x80000000u;
    return static_cast<uint64_t>(u) << 32 | (0xFFFFFFFFu - e);
}
template <typename T, int L>
__device__ __forceinline__ bool choose_by_bound(const float (&v)[32], const T *z, int sub, int lane, int k, bool live, int32_t *out,
                                                int32_t *cnt, uint64_t *list) {
    float g[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        g[j] = v[8 * j];
#pragma unroll
        for (int i = 1; i < 8; ++i) g[j] = fmaxf(g[j], v[8 * j + i]);
    }
    float bound = 0.0f;
    for (int c = 0; c < k; ++c) {
        bound = group_max<L>(fmaxf(fmaxf(g[0], g[1]), fmaxf(g[2], g[3])));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (g[j] == bound) g[j] = -INFINITY;
    }
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (v[i] >= bound) mask |= 1u << i;
    const int n = __popc(mask);
    int upto = n;
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, upto, o, L);
        if (sub >= o) upto += u;
    }
    const int total = __shfl_sync(0xFFFFFFFFu, upto, L - 1, L);
    const bool good = live && bound > -INFINITY && total <= kList;
    list += lane / L * kList;
    if (good) {
        int at = upto - n;
        while (mask) {
            const int i = __ffs(mask) - 1;
            mask &= mask - 1;
            const int e = expert<T, L>(sub, i);
            list[at++] = choice_key(load_f32(z + e), e);
        }
    }
    __syncwarp();
    if (good) {
        for (int own = sub; own < total; own += 2 * L) {  // two of the list at a time in each lane
            const bool second = own + L < total;
            const uint64_t a = list[own], b = list[second ? own + L : own];
            int rank_a = 0, rank_b = 0;
            for (int j = 0; j < total; ++j) {
                const uint64_t x = list[j];
                rank_a += x > a;
                rank_b += x > b;
            }
            if (rank_a < k) {
                const uint32_t e = 0xFFFFFFFFu - static_cast<uint32_t>(a);
                out[rank_a] = static_cast<int32_t>(e);
                atomicAdd(cnt + e, 1);
            }
            if (second && rank_b < k) {
                const uint32_t e = 0xFFFFFFFFu - static_cast<uint32_t>(b);
                out[rank_b] = static_cast<int32_t>(e);
                atomicAdd(cnt + e, 1);
            }
        }
    }
    __syncwarp();
    return good;
}

// A lane's logits of token t (-inf where it does not count), and whether it does.
template <typename T, int L, int V, bool kWide>
__device__ __forceinline__ bool fetch(const BalanceParams &p, int w, int64_t t, int sub, Runs<T, V> &g) {
    const bool live = t < p.tokens && (!p.has_valid || p.valid[w][t] != 0);
    if (live) {
        load_runs<T, L, V, kWide>(static_cast<const T *>(p.z[w]) + t * p.ldz, sub, p.experts, p.align, g);
    } else {
        constexpr uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
        for (uint4 &r : g) r = make_uint4(none, none, none, none);
    }
    return live;
}
// Choices of the tokens of one warp, from their logits; adds to cnt (shared
// memory) and returns, in each lane that leads a group, whether its token counts.
template <typename T, int L, int V>
__device__ __forceinline__ bool choose(const BalanceParams &p, int w, int64_t t, int sub, int lane, const Runs<T, V> &g, bool live,
                                       int32_t *cnt, uint64_t *list) {
    const bool here = t < p.tokens;
    int32_t *out = here ? p.choice[w] + t * p.k : nullptr;
    const T *z = static_cast<const T *>(p.z[w]) + (live ? t : 0) * p.ldz;
    float v[V];
    unpack_runs<T, V>(g, v);
    for (int c = sub; here && !live && c < p.k; c += L) out[c] = -1;
    float m = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);
    const bool some = (__ballot_sync(0xFFFFFFFFu, m > -INFINITY) & group_mask<L>(lane)) != 0;
    if constexpr (L >= 4 && V == 32) {
        bool good = !live;
        if (p.k > 2) good |= choose_by_bound<T, L>(v, z, sub, lane, p.k, live, out, cnt, list);
        if (__any_sync(0xFFFFFFFFu, !good)) {
            if (good) {  // done: nothing left to choose
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = -INFINITY;
            }
            choose_by_rounds<T, L, V>(v, sub, lane, p.k, live && !good, out, cnt);
        }
    } else {
        choose_by_rounds<T, L, V>(v, sub, lane, p.k, live, out, cnt);
    }
    return some && sub == 0;
}

// Gradient of one warp's tokens, from their logits; returns d_t in each lane that leads a group.
template <typename T, int L, int V, bool kWide>
__device__ __forceinline__ float gradient(const BalanceParams &p, int w, int64_t t, int sub, const Runs<T, V> &g, bool live,
                                          const float (&c)[V], float coef) {
    const bool here = t < p.tokens;
    float v[V];
    unpack_runs<T, V>(g, v);
    float m = v[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);
    m = group_max<L>(m);
    live = live && m > -INFINITY;
    const float r = live ? m : 0.0f;
    float s = 0.0f, d = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float x;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"((v[i] - r) * kLog2e));
        v[i] = x;
        s += x;
        d = fmaf(x, c[i], d);
    }
    s = group_sum<L>(s);
    d = group_sum<L>(d);
    d = live ? d / s : 0.0f;
    const float f = live ? coef / s : 0.0f, fd = f * d;
    if (here && p.has_grad) {
        if (!live) {  // powers of nothing, or of NaN alone
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= fmaf(f, c[i], -fd);
        store_token<T, L, V, kWide>(static_cast<T *>(p.dz[w]) + t * p.lddz, sub, p.experts, p.dalign, v);
    }
    return sub == 0 ? d : 0.0f;
}

// A CTA's sum of integers, the same value in every thread.
__device__ __forceinline__ int64_t cta_count(int64_t v, int64_t *scratch) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if (lane == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < static_cast<int>(blockDim.x >> 5) ? scratch[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// alpha E / (k N^2), and the loss from the sum of d_t in which c_e lacked its
// mean (choices / E).  In fp32: GB300 has few fp64 units, and one division on
// them takes longer than a launch's other arithmetic.
__device__ __forceinline__ float loss_scale(const BalanceParams &p, int64_t n) {
    const float f = static_cast<float>(n);
    return n > 0 ? p.alpha * static_cast<float>(p.experts) / static_cast<float>(p.k) / f / f : 0.0f;
}
__device__ __forceinline__ float loss_of(const BalanceParams &p, float sum, int64_t n, int64_t choices) {
    return loss_scale(p, n) * (sum + static_cast<float>(choices) / static_cast<float>(p.experts) * static_cast<float>(n));
}
// c_e less its mean: the integer E c_e - choices, rounded once, over E.
__device__ __forceinline__ float centred(int32_t count, int64_t choices, int experts) {
    return __fdividef(static_cast<float>(static_cast<int64_t>(count) * experts - choices), static_cast<float>(experts));
}

// Two or three launches.  With kTogether, blockIdx.y's CTAs are one cluster,
// which adds its counts in distributed shared memory and stores a worker's whole
// counts; else the counts are zeroed by a kernel ahead and added with atomics
// (integers: their order does not matter).  Each kernel waits for the one ahead
// before it reads z too: that a kernel further ahead, which wrote z, has ended
// orders the two, but only a wait of its own makes those writes visible to it
// (8 x 16384 tokens of 64 fp32 experts 44 us, 41 with the first logits read ahead).
__global__ void __launch_bounds__(kThreads) balance_zero_kernel(int32_t *counts, int n, uint32_t *seen, int workers) {
    let_next_begin();
    after_previous();
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i < n) counts[i] = 0;
    if (i <= workers) seen[i] = 0;
}

template <typename T, int L, int V, bool kTogether, bool kWide>
__global__ void __launch_bounds__(kThreads) balance_count_kernel(const __grid_constant__ BalanceParams p) {
    __shared__ int32_t cnt[kMaxExperts];
    __shared__ uint64_t list[L >= 4 && V == 32 ? kWarps : 1][32 / L * kList];
    __shared__ uint32_t seen;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = blockIdx.y, sub = lane & (L - 1);
    for (int e = threadIdx.x; e < p.experts; e += kThreads) cnt[e] = 0;
    if (threadIdx.x == 0) seen = 0;
    __syncthreads();
    let_next_begin();
    after_previous();
    constexpr int kPerWarp = 32 / L;
    uint32_t mine = 0;
    int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kPerWarp + lane / L;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps * kPerWarp;
    Runs<T, V> g;
    if constexpr (V == 32) {
        for (; t - lane / L < p.tokens; t += stride) {
            const bool live = fetch<T, L, V, kWide>(p, w, t, sub, g);
            mine += choose<T, L, V>(p, w, t, sub, lane, g, live, cnt, list[L >= 4 ? warp : 0]);
        }
    } else {  // few registers a token: the next tokens' logits come while these are worked on
        Runs<T, V> coming;
        bool live = fetch<T, L, V, kWide>(p, w, t, sub, g);
        for (; t - lane / L < p.tokens; t += stride) {
            const bool live_next = fetch<T, L, V, kWide>(p, w, t + stride, sub, coming);
            mine += choose<T, L, V>(p, w, t, sub, lane, g, live, cnt, list[0]);
#pragma unroll
            for (int i = 0; i < static_cast<int>(V * sizeof(T) / 16); ++i) g[i] = coming[i];
            live = live_next;
        }
    }
    mine = __reduce_add_sync(0xFFFFFFFFu, mine);
    if (lane == 0 && mine) atomicAdd(&seen, mine);
    __syncthreads();
    if (kTogether) {
        const int C = gridDim.x;
        cluster_barrier();
        for (int e = blockIdx.x * kThreads + threadIdx.x; e < p.experts; e += C * kThreads) {
            int32_t sum = 0;
            for (int r = 0; r < C; ++r) sum += cluster_load_int(cluster_map(smem_u32(cnt + e), r));
            p.counts[w * p.experts + e] = sum;
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            uint32_t sum = 0;
            for (int r = 0; r < C; ++r) sum += cluster_load_int(cluster_map(smem_u32(&seen), r));
            p.seen[1 + w] = sum;
            if (w == 0) p.seen[0] = 0;
        }
        cluster_barrier();  // no CTA leaves while another reads its shared memory
    } else {
        for (int e = threadIdx.x; e < p.experts; e += kThreads)
            if (cnt[e]) atomicAdd(&p.counts[w * p.experts + e], cnt[e]);
        if (threadIdx.x == 0 && seen) atomicAdd(p.seen + 1 + w, seen);
    }
}

template <typename T, int L, int V, bool kWide>
__global__ void __launch_bounds__(kThreads, V == 32 ? 2 : 1) balance_grad_kernel(const __grid_constant__ BalanceParams p) {
    __shared__ int32_t all[kMaxExperts];
    __shared__ float dsum[kWarps];
    __shared__ int64_t isum[kWarps];
    __shared__ float coef;
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = blockIdx.y, sub = lane & (L - 1);
    let_next_begin();
    constexpr int kPerWarp = 32 / L;
    // backwards: what the counting pass read last is still in L2
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps * kPerWarp;
    const int64_t own = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kPerWarp;
    int64_t t = own < p.tokens ? own + (p.tokens - 1 - own) / stride * stride : -1;
    Runs<T, V> g, coming;
    after_previous();
    bool live = t >= 0 && fetch<T, L, V, kWide>(p, w, t + lane / L, sub, g), live_next = false;
    int64_t n = 0;
    for (int i = 0; i < p.P; ++i) n += p.seen[1 + i];
    if (threadIdx.x == 0) coef = loss_scale(p, n);
    int64_t choices = 0;
    for (int e = threadIdx.x; e < p.experts; e += kThreads) {
        int32_t s = 0;
        for (int i = 0; i < p.P; ++i) s += p.counts[i * p.experts + e];
        all[e] = s;
        choices += s;
    }
    choices = cta_count(choices, isum);
    float c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = expert<T, L>(sub, i);
        c[i] = e < p.experts ? centred(all[e], choices, p.experts) : 0.0f;
    }
    float sum = 0.0f;
    for (; t >= 0; t -= stride) {  // the next tokens' logits on their way while these are worked on
        if (t >= stride) live_next = fetch<T, L, V, kWide>(p, w, t - stride + lane / L, sub, coming);
        sum += gradient<T, L, V, kWide>(p, w, t + lane / L, sub, g, live, c, coef);
#pragma unroll
        for (int i = 0; i < static_cast<int>(V * sizeof(T) / 16); ++i) g[i] = coming[i];
        live = live_next;
    }
    sum = group_sum<32>(sum);
    if (lane == 0) dsum[warp] = sum;
    __syncthreads();
    const uint32_t blocks = gridDim.x * gridDim.y;
    if (threadIdx.x == 0) {
        float s = 0.0f;
        for (int i = 0; i < kWarps; ++i) s += dsum[i];
        p.partial[blockIdx.y * gridDim.x + blockIdx.x] = s;
        __threadfence();
        last = atomicAdd(p.seen, 1u) == blocks - 1;
    }
    __syncthreads();
    if (last) {  // the sums of all CTAs, in their order
        __threadfence();
        float s = 0.0f;
        for (uint32_t i = threadIdx.x; i < blocks; i += kThreads) s += __ldcg(p.partial + i);
        s = group_sum<32>(s);
        if (lane == 0) dsum[warp] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kWarps; ++i) s += dsum[i];
            *p.loss = loss_of(p, s, n, choices);
        }
    }
}

// Few tokens: everything in one cluster of up to 16 CTAs (one launch, and its
// barriers, cost less than three launches).  The CTAs' counts and sums meet in
// distributed shared memory; every CTA adds them in rank order.
template <typename T, int L, int V, bool kWide>
__global__ void __launch_bounds__(kOneThreads) balance_one_kernel(const __grid_constant__ BalanceParams p) {
    constexpr int threads = kOneThreads, warps = threads / 32;
    __shared__ int32_t cnt[kOneCounts];
    __shared__ int32_t all[kMaxExperts];
    __shared__ float dsum[kOneThreads / 32];
    __shared__ int64_t isum[kOneThreads / 32];
    __shared__ float coef;
    __shared__ int32_t seen;
    __shared__ float total;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & (L - 1);
    const int C = gridDim.x, rank = blockIdx.x, P = p.P, E = p.experts;
    for (int e = threadIdx.x; e < P * E; e += threads) cnt[e] = 0;
    __syncthreads();
    let_next_begin();
    after_previous();
    constexpr int kPerWarp = 32 / L;
    const int chunks = static_cast<int>((p.tokens + kPerWarp - 1) / kPerWarp), items = chunks * P;
    int64_t n = 0;
    for (int i = warp * C + rank; i < items; i += warps * C) {
        const int w = i / chunks;
        const int64_t t = static_cast<int64_t>(i - w * chunks) * kPerWarp + lane / L;
        Runs<T, V> g;
        const bool live = fetch<T, L, V, kWide>(p, w, t, sub, g);
        n += choose<T, L, V>(p, w, t, sub, lane, g, live, cnt + w * E, nullptr);
    }
    n = cta_count(n, isum);
    if (C > 1) {
        if (threadIdx.x == 0) seen = static_cast<int32_t>(n);
        cluster_barrier();
        n = 0;
        for (int r = 0; r < C; ++r) n += cluster_load_int(cluster_map(smem_u32(&seen), r));
    }
    if (threadIdx.x == 0) coef = loss_scale(p, n);
    int64_t choices = 0;
    for (int e = threadIdx.x; e < E; e += threads) {
        int32_t s = 0;
        for (int i = 0; i < P; ++i) {
            int32_t of_worker = cnt[i * E + e];
            if (C > 1) {
                of_worker = 0;
                for (int r = 0; r < C; ++r) of_worker += cluster_load_int(cluster_map(smem_u32(cnt + i * E + e), r));
            }
            if (rank == 0) p.counts[i * E + e] = of_worker;
            s += of_worker;
        }
        all[e] = s;
        choices += s;
    }
    choices = cta_count(choices, isum);
    float c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = expert<T, L>(sub, i);
        c[i] = e < E ? centred(all[e], choices, E) : 0.0f;
    }
    float sum = 0.0f;
    for (int i = warp * C + rank; i < items; i += warps * C) {
        const int w = i / chunks;
        const int64_t t = static_cast<int64_t>(i - w * chunks) * kPerWarp + lane / L;
        Runs<T, V> g;
        const bool live = fetch<T, L, V, kWide>(p, w, t, sub, g);
        sum += gradient<T, L, V, kWide>(p, w, t, sub, g, live, c, coef);
    }
    sum = group_sum<32>(sum);
    if (lane == 0) dsum[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.0f;
        for (int i = 0; i < warps; ++i) sum += dsum[i];
        total = sum;
    }
    if (C > 1) {
        __syncthreads();
        cluster_barrier();
        if (rank == 0 && threadIdx.x == 0) {
            sum = 0.0f;
            for (int r = 0; r < C; ++r) sum += cluster_load(cluster_map(smem_u32(&total), r));
        }
        cluster_barrier();  // no CTA leaves while another reads its shared memory
    }
    if (rank == 0 && threadIdx.x == 0) *p.loss = loss_of(p, sum, n, choices);
}

// Whether clusters of 16 CTAs of a kernel (above the portable size) can be had
// on this device; known: a static array of the caller, 1: yes, 2: no, 0: not
// looked up yet.
template <typename Kernel>
bool wide_clusters(Kernel kernel, unsigned threads, std::atomic<int> *known) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    int have = known[dev & 63].load(std::memory_order_relaxed);
    if (have == 0) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(threads);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 16;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        const bool good = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                          cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess && clusters > 0;
        if (!good) cudaGetLastError();  // not an error of this call: clusters of eight do
        have = good ? 1 : 2;
        known[dev & 63].store(have, std::memory_order_relaxed);
    }
    return have == 1;
}

template <typename T, int L, int V, bool kWide>
int launch_as(const BalanceParams &p, cudaStream_t stream) {
    const unsigned P = static_cast<unsigned>(p.P);
    bool together = false;
    unsigned ctas = 1;
    if constexpr (V == 8) {
        // One launch of one cluster up to two passes of its 256 warps; two launches, of a cluster a worker, up to four
        // passes of its 128 warps; else three over the whole device.  (8000 tokens of 60 experts, GPU time: 20, 14.5
        // and 13.5 us; but a launch takes the host 3 us.)
        const int64_t items = ceil_div(p.tokens, int64_t{32 / L});  // of a worker
        if (items * p.P <= 16 * 16 * 2 && p.P * p.experts <= kOneCounts) {
            const auto kernel = balance_one_kernel<T, L, V, kWide>;
            static std::atomic<int> known[64];
            while (ctas < 16 && items * p.P > static_cast<int64_t>(ctas) * 16 * 2) ctas *= 2;
            if (ctas == 16 && !wide_clusters(kernel, kOneThreads, known)) ctas = 8;
            return launch_early("balance_one_kernel", kernel, dim3(ctas), kOneThreads, 0, ctas, stream, p);
        }
        if (items <= 16 * kWarps * 4) {
            const auto kernel = balance_count_kernel<T, L, V, true, kWide>;
            static std::atomic<int> known[64];
            while (ctas < 16 && items > static_cast<int64_t>(ctas) * kWarps) ctas *= 2;
            if (ctas == 16 && !wide_clusters(kernel, kThreads, known)) ctas = 8;
            if (int rc = launch_early("balance_count_kernel", kernel, dim3(ctas, P), kThreads, 0, ctas, stream, p)) return rc;
            together = true;
        }
    }
    // as many CTAs as the SMs hold (registers), for each begins with the totals of all counts
    const auto blocks = [&](int per_sm) {
        const int64_t work = ceil_div(p.tokens, int64_t{kWarps} * (32 / L));
        const int64_t most = std::min(ceil_div(static_cast<int64_t>(sm_count()) * per_sm, p.P), int64_t{kMaxBlocks} / p.P);
        return static_cast<unsigned>(std::max(std::min(work, most), int64_t{1}));
    };
    if (!together) {
        const int n = p.P * p.experts;
        if (int rc = launch_early("balance_zero_kernel", balance_zero_kernel, dim3(static_cast<unsigned>(ceil_div(std::max(n, p.P + 1), kThreads))),
                                  kThreads, 0, 1, stream, p.counts, n, p.seen, p.P))
            return rc;
        if (int rc = launch_early("balance_count_kernel", balance_count_kernel<T, L, V, false, kWide>, dim3(blocks(V == 32 ? 3 : 6), P), kThreads, 0,
                                  1, stream, p))
            return rc;
    }
    return launch_early("balance_grad_kernel", balance_grad_kernel<T, L, V, kWide>, dim3(blocks(V == 32 ? 2 : 4), P), kThreads, 0, 1, stream, p);
}

// Kernels for aligned rows alone: 8 x 8192 x 512 fp32 83 us, 105 with the other pieces' code in
// its way; 8 x 16384 x 250 fp32 (rows on 8 bytes) 107, element by element 123.
template <typename T, int L, int V>
int launch(const BalanceParams &p, cudaStream_t stream) {
    if (p.align == 16 && p.dalign == 16) return launch_as<T, L, V, true>(p, stream);
    return launch_as<T, L, V, false>(p, stream);
}

template <typename T>
int dispatch(const BalanceParams &p, cudaStream_t stream) {
    // 32 logits a lane once that leaves every SM sixteen warps
    const bool many = p.tokens * p.P * p.experts >= static_cast<int64_t>(sm_count()) * 16 * 32 * 32;
    if (p.experts <= 8) return launch<T, 1, 8>(p, stream);
    if (p.experts <= 16) return many ? launch<T, 1, 16>(p, stream) : launch<T, 2, 8>(p, stream);
    if (p.experts <= 32) return many ? launch<T, 1, 32>(p, stream) : launch<T, 4, 8>(p, stream);
    if (p.experts <= 64) return many ? launch<T, 2, 32>(p, stream) : launch<T, 8, 8>(p, stream);
    if (p.experts <= 128) return many ? launch<T, 4, 32>(p, stream) : launch<T, 16, 8>(p, stream);
    if (p.experts <= 256) return many ? launch<T, 8, 32>(p, stream) : launch<T, 32, 8>(p, stream);
    if (p.experts <= 512) return launch<T, 16, 32>(p, stream);
    return launch<T, 32, 32>(p, stream);
}

// How many bytes every row of every worker starts on, 16 at most.
int rows_align(const void *const *rows, int P, int64_t ld, int elem) {
    uint64_t bits = static_cast<uint64_t>(ld) * elem | 16;
    for (int i = 0; i < P; ++i) bits |= reinterpret_cast<uintptr_t>(rows[i]);
    return static_cast<int>(bits & (~bits + 1));
}

}  // namespace
}  // namespace gar

using namespace gar;

extern "C" size_t gar_balance_workspace_bytes(int32_t P) {
    return P < 1 || P > GAR_MAX_WORKERS ? 0 : static_cast<size_t>(kMaxBlocks) * 4 + (GAR_MAX_WORKERS + 1) * 4;
}

extern "C" int gar_balance_loss(const void *const *z, int32_t P, int64_t tokens, int32_t experts, int64_t ldz,
                                int32_t dtype, int32_t k, const uint8_t *const *valid, float alpha,
                                int32_t *const *choice, int32_t *counts, float *loss, void *const *dz, int64_t lddz,
                                void *d_workspace, size_t workspace_bytes, gar_stream_t stream_) {
    if (P < 1 || P > GAR_MAX_WORKERS) return fail(GAR_EINVAL, "P=%d outside 1..%d", P, GAR_MAX_WORKERS);
    if (elem_bytes(dtype) < 0) return fail(GAR_EDTYPE, "unknown dtype %d", dtype);
    if (tokens < 0 || tokens > 0x7FFFFFFF / kMaxChoices / P || experts < 1 || experts > kMaxExperts || k < 1 ||
        k > kMaxChoices || k > experts)
        return fail(GAR_EINVAL, "tokens=%lld (P tokens <= %d) experts=%d (1..%d) k=%d (1..%d, at most the experts)",
                    static_cast<long long>(tokens), 0x7FFFFFFF / kMaxChoices, experts, kMaxExperts, k, kMaxChoices);
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
    p.partial = static_cast<float *>(d_workspace);
    p.seen = reinterpret_cast<uint32_t *>(p.partial + kMaxBlocks);
    if (tokens > 0) {
        p.align = rows_align(p.z, P, ldz, elem_bytes(dtype));
        p.dalign = dz ? rows_align(p.dz, P, lddz, elem_bytes(dtype)) : 16;
    }
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    return dtype == GAR_F32 ? dispatch<float>(p, stream) : dispatch<uint16_t>(p, stream);
}
