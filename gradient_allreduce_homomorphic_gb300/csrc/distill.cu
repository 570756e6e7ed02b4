// distill.cu -- distillation from a teacher's top logits: gar_distill_loss and
// gar_distill_grad.
//
// Row t has the student's logits z_v and the teacher's entries (i_j, t_j):
//   p_j  = softmax over the row's present entries of t_j / tau
//   lse  = log sum_v exp(z_v / tau)
//   loss = sum_j p_j (log p_j + lse - z_{i_j} / tau)
//   dz_v = w / tau (exp(z_v / tau - lse) - sum_{j: i_j = v} p_j)
// An entry is present if its index lies in [0, V) and its logit is not -inf.
// Everything is computed in fp32 and rounded once, when dz is stored.  Powers
// are taken as 2^((z - m) c), c = log2(e) / tau: the difference from the row's
// maximum m is formed first, so a row of equal values, however large, stays
// exact, and the product's rounding is relative to a small number.  A maximum
// of -inf is replaced by 0 in the difference, which makes the powers 0.
//
// Bound by HBM: a row is read once and, with dz, written once.  Short rows, or
// few, are held in the registers of one CTA (distill_row_kernel); others go
// through shared memory (distill_stream_kernel).  Loss and gradient in one call:
// 4096 x 50001 bf16 144 us, 5.7 TB/s; 4096 x 50001 fp32 244 us, 6.7 TB/s;
// 4096 x 4096 bf16 16.4 us, 4.1 TB/s (the rows' reductions); 8 x 32000 bf16 5 us
// (one row's latency).  The loss alone of bf16 rows is bound by its pass's
// instructions and powers: 4096 x 32768 65 us, 4.1 TB/s (fp32 82 us, 6.6 TB/s).
#include <atomic>

#include "common.cuh"
#include "fp8.cuh"
#include "launch.cuh"
#include "tensorcore.cuh"

namespace gar {
namespace {

constexpr int kMaxTop = 1024;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// bf16 rows with |m c| up to this take (z - m) c as one fma of z, c and the rounded m c.  That adds 2^-16 to an exponent
// at most, in the sum (2^-17 from rounding m c, as much from rounding the fma: a fraction 1.1e-5 of it), and 2^-15 in the
// gradient, whose subtrahend has the sum and the weight in it (2.1e-5, where rounding dz to bf16 takes 2e-3).
constexpr float kPlain = 256.0f;

struct DistillParams {
    const void *z;
    int64_t rows, ldz, lddz;
    int32_t vocab, k;
    const int32_t *index;
    const float *teacher;
    const float *weight;  // NULL: 1
    float inv_tau, inv_tau_rest;  // 1 / tau, and what its rounding left
    float *loss, *lse;         // gar_distill_loss
    const float *lse_in;       // gar_distill_grad
    void *dz;                  // NULL: no gradient
    int32_t stages, stage_bytes, slots, log_cluster, log_parts;  // distill_stream_kernel
    unsigned int *status;
};

__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.0f : m; }

// A maximum and the sum of 2^((z - maximum) c) over the values seen.
struct MaxSum {
    float m, s;
};
__device__ __forceinline__ MaxSum merge(MaxSum a, MaxSum b, float c) {
    const float m = fmaxf(a.m, b.m), r = finite_or_0(m);
    return {m, a.s * pow2((a.m - r) * c) + b.s * pow2((b.m - r) * c)};
}
__device__ __forceinline__ float warp_max(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(v));
    return m;
}
template <int kWidth>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int o = kWidth / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ float warp_sum(float v) { return lane_sum<32>(v); }
// The merge of kWidth lanes' pairs (each held by 32 / kWidth lanes).
template <int kWidth>
__device__ __forceinline__ MaxSum merge_lanes(MaxSum a, float c) {
    const float m = warp_max(a.m);
    return {m, lane_sum<kWidth>(a.s * pow2((a.m - finite_or_0(m)) * c))};
}

// exp((t - tmax) / tau) of a teacher's entry, and its exponent.  The difference
// and the product keep what their rounding leaves (the sum of two floats is
// exact as a pair, [K]; a product by fma), for a teacher's spread over tens of
// units would cost its small probabilities four bits otherwise; entries are few.
//   [K] Knuth, The Art of Computer Programming vol. 2, 4.2.2: two-sum.
struct Entry {
    float power, exponent;
};
__device__ __forceinline__ Entry entry_power(const DistillParams &p, float t, float tmax) {
    const float d = t - tmax, x = d * p.inv_tau;
    if (x < -200.0f) return {0.0f, x};  // 0 in fp32; a mask's lowest value would overflow below
    const float b = d - t, lost = (t - (d - b)) + (-tmax - b);
    const float rest = fmaf(d, p.inv_tau_rest, fmaf(lost, p.inv_tau, fmaf(d, p.inv_tau, -x)));
    const float e = expf(x);
    return {fmaf(e, rest, e), x + rest};
}

// Where the gradient of a student logit z comes from: the row's maximum and
// log2 of its sum (loss), or its saved lse (grad).
template <bool kSaved>
struct Softmax {
    float ref, sub, c;  // probability 2^((z - ref) c - sub), or exp(z c - sub)
    __device__ __forceinline__ float operator()(float z) const {
        return kSaved ? pow2(fmaf(z, c, -sub) * kLog2e) : pow2(fmaf(z - ref, c, -sub));
    }
};

// ------------------------------------------------------------ a row's vectors
template <typename T>
struct Row {  // one row's split into head, vectors and tail
    int32_t head, vectors, v0, v1;  // this CTA: vectors v0 .. v1
    __device__ __forceinline__ Row(const T *z, int32_t vocab, int32_t rank, int32_t log_cluster) {
        constexpr int32_t n = 16 / sizeof(T);
        const int32_t off = static_cast<int32_t>((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / static_cast<int32_t>(sizeof(T));
        head = off < vocab ? off : vocab;
        vectors = (vocab - head) / n;
        v0 = (vectors * rank) >> log_cluster;  // a row that is taken this way has fewer than 2^16 vectors
        v1 = (vectors * (rank + 1)) >> log_cluster;
    }
    // Element of the i-th place outside the vectors, which are the first CTA's; -1 past the last.
    __device__ __forceinline__ int32_t edge(int32_t i, int32_t vocab, int32_t rank) const {
        const int32_t at = i < head ? i : i + vectors * static_cast<int32_t>(16 / sizeof(T));
        return rank == 0 && at < vocab ? at : -1;
    }
    __device__ __forceinline__ bool holds(int32_t i, int32_t rank) const {
        constexpr int32_t n = 16 / sizeof(T);
        const int32_t v = i - head;
        if (v < 0 || v >= vectors * n) return rank == 0;
        return v >= v0 * n && v < v1 * n;
    }
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4 &g, float (&x)[16 / sizeof(T)]) {
    if constexpr (sizeof(T) == 2) {
        x[0] = bf16_lo(g.x), x[1] = bf16_hi(g.x), x[2] = bf16_lo(g.y), x[3] = bf16_hi(g.y);
        x[4] = bf16_lo(g.z), x[5] = bf16_hi(g.z), x[6] = bf16_lo(g.w), x[7] = bf16_hi(g.w);
    } else {
        x[0] = __uint_as_float(g.x), x[1] = __uint_as_float(g.y);
        x[2] = __uint_as_float(g.z), x[3] = __uint_as_float(g.w);
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[16 / sizeof(T)]) {
    if constexpr (sizeof(T) == 2)
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    else
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

template <int n>
__device__ __forceinline__ float tree_max(const float (&x)[n]) {
    float m[n / 2];
#pragma unroll
    for (int j = 0; j < n / 2; ++j) m[j] = fmaxf(x[j], x[j + n / 2]);
    if constexpr (n == 2)
        return m[0];
    else
        return tree_max(m);
}
template <int n>
__device__ __forceinline__ float tree_sum(const float (&x)[n]) {
    float m[n / 2];
#pragma unroll
    for (int j = 0; j < n / 2; ++j) m[j] = x[j] + x[j + n / 2];
    if constexpr (n == 2)
        return m[0];
    else
        return tree_sum(m);
}

// ---------------------------------------------------------------- short rows
// A CTA holds its row in registers, kHold vectors a thread, so z is read once
// and the maximum is known before the powers; the other rows' CTAs on the SM
// hide its barriers.  Rows too long for the stages of eight CTAs (above 880 KB)
// are taken here too, with kHold = 0: they are read from memory each time.

// Sums (or maxima) of both over the block.  The scratch is the call's own: one barrier.
template <bool kMax, int kWarps>
__device__ __forceinline__ float2 block_reduce(float2 v, float2 (&scratch)[kWarps]) {
    v = kMax ? make_float2(warp_max(v.x), warp_max(v.y)) : make_float2(warp_sum(v.x), warp_sum(v.y));
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) {
        const float2 o = scratch[i];
        v = kMax ? make_float2(fmaxf(v.x, o.x), fmaxf(v.y, o.y)) : make_float2(v.x + o.x, v.y + o.y);
    }
    return v;
}

template <typename T, bool kSaved, int kHold, int kThreads>
__global__ void __launch_bounds__(kThreads) distill_row_kernel(const __grid_constant__ DistillParams p) {
    constexpr int n = 16 / sizeof(T);
    __shared__ float2 scratch[3][kThreads / 32];
    __shared__ float top_p[kMaxTop], top_z[kMaxTop];
    __shared__ int32_t top_i[kMaxTop];
    __shared__ uint32_t seen[((kHold * kThreads + 2) * n + 31) / 32];  // a bit for each element: entries that repeat one
    __shared__ int repeated;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const T *z = static_cast<const T *>(p.z) + row * p.ldz;
    T *dz = p.dz ? static_cast<T *>(p.dz) + row * p.lddz : nullptr;
    const Row<T> part(z, p.vocab, 0, 0);
    const int odd = part.edge(tid, p.vocab, 0);
    if (kHold)
        for (int i = tid; i * 32 < p.vocab; i += kThreads) seen[i] = 0;
    if (tid == 0) repeated = kHold == 0;
    let_next_begin();
    after_previous();
    uint4 held[kHold ? kHold : 1];
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
        const int i = tid + h * kThreads;
        const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf: in no maximum and in no sum
        held[h] = make_uint4(none, none, none, none);
        if (i < part.vectors) held[h] = ld16(z + part.head + i * n);
    }
    // every vector of this thread's: f(which, its values)
    const auto each = [&](auto &&f) {
        float x[n];
        if constexpr (kHold > 0) {
#pragma unroll
            for (int h = 0; h < kHold; ++h) {
                unpack<T>(held[h], x);
                f(tid + h * kThreads, x);
            }
        } else {
#pragma unroll 2
            for (int i = tid; i < part.vectors; i += kThreads) {
                unpack<T>(*reinterpret_cast<const uint4 *>(z + part.head + static_cast<int64_t>(i) * n), x);
                f(i, x);
            }
        }
    };
    const float z_odd = odd >= 0 ? load_f32(z + odd) : -INFINITY;
    const float w = p.weight ? p.weight[row] : 1.0f;
    const float saved = kSaved ? p.lse_in[row] : 0.0f;

    float2 top = make_float2(-INFINITY, z_odd);  // maxima of the entries' logits and of z
    for (int j = tid; j < p.k; j += kThreads) {
        const int32_t i = p.index[row * p.k + j];
        const float t = p.teacher[row * p.k + j];
        const bool on = i >= 0 && i < p.vocab && !(t == -INFINITY);
        top_i[j] = on ? i : -1;
        top_p[j] = t;
        top_z[j] = on ? load_f32(z + i) : 0.0f;
        if (on) top.x = fmaxf(top.x, t);
    }
    const float c = kLog2e * p.inv_tau;
    if (!kSaved) each([&](int, float(&x)[n]) { top.y = fmaxf(top.y, tree_max(x)); });
    top = block_reduce<true>(top, scratch[0]);
    const float tmax = top.x, r = finite_or_0(top.y);
    float2 sum = make_float2(0.0f, 0.0f);  // of the entries' powers and of z's
    for (int j = tid; j < p.k; j += kThreads) {
        const int32_t i = top_i[j];
        if (i < 0) continue;
        sum.x += entry_power(p, top_p[j], tmax).power;
        if (kHold && dz && (atomicOr(seen + (i >> 5), 1u << (i & 31)) >> (i & 31) & 1)) repeated = 1;
    }
    if (!kSaved) {
        sum.y = pow2((z_odd - r) * c);
        const float rc = r * c;
        if (sizeof(T) == 2 && fabsf(rc) <= kPlain) {
            each([&](int, float(&x)[n]) {
#pragma unroll
                for (int j = 0; j < n; ++j) x[j] = pow2(fmaf(x[j], c, -rc));
                sum.y += tree_sum(x);
            });
        } else {
            each([&](int, float(&x)[n]) {
#pragma unroll
                for (int j = 0; j < n; ++j) x[j] = pow2((x[j] - r) * c);
                sum.y += tree_sum(x);
            });
        }
    }
    sum = block_reduce<false>(sum, scratch[1]);
    const bool live = w != 0.0f && sum.x != 0.0f;  // NaN: live, and it spreads
    Softmax<kSaved> q{0.0f, 0.0f, kSaved ? p.inv_tau : c};
    bool none;
    if (kSaved)
        q.sub = saved, none = saved == -INFINITY;
    else
        q.ref = r, q.sub = log2f(sum.y), none = top.y == -INFINITY && sum.y == 0.0f;
    float2 cross = make_float2(0.0f, 0.0f);
    if (live) {
        const float log_tsum = logf(sum.x);
        for (int j = tid; j < p.k; j += kThreads) {
            float pj = 0.0f;
            if (top_i[j] >= 0) {
                const Entry t = entry_power(p, top_p[j], tmax);
                pj = t.power / sum.x;
                if (!(pj == 0.0f)) cross.x += pj * (t.exponent - log_tsum - (top_z[j] - q.ref) * p.inv_tau);
            }
            top_p[j] = pj;
        }
    }
    if (!kSaved) {
        cross = block_reduce<false>(cross, scratch[2]);
        if (tid == 0) {
            p.loss[row] = !live ? 0.0f : none ? INFINITY : cross.x + q.sub * kLn2;
            p.lse[row] = !live ? 0.0f : none ? -INFINITY : q.ref * p.inv_tau + q.sub * kLn2;
        }
    }
    if (!dz) return;
    const float g = live && !none ? w * p.inv_tau : 0.0f;
    const bool zero = g == 0.0f;  // whatever z holds
    T *out = dz + part.head;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    if (odd >= 0) store_f32(dz + odd, zero ? 0.0f : g * q(z_odd));
    if (sizeof(T) == 2 && !kSaved && wide && g > 0.0f && fabsf(q.ref * c) <= kPlain) {
        const float sub = fmaf(q.ref, c, q.sub) - log2f(g);  // g too goes into the exponent
        each([&](int i, float(&x)[n]) {
            if (i >= part.vectors) return;
#pragma unroll
            for (int j = 0; j < n; ++j) x[j] = pow2(fmaf(x[j], c, -sub));
            st16(out + static_cast<int64_t>(i) * n, pack<T>(x));
        });
    } else {
        each([&](int i, float(&x)[n]) {
            if (i >= part.vectors) return;
#pragma unroll
            for (int j = 0; j < n; ++j) x[j] = zero ? 0.0f : g * q(x[j]);
            T *at = out + static_cast<int64_t>(i) * n;
            if (wide) {
                st16(at, pack<T>(x));
            } else {
#pragma unroll
                for (int j = 0; j < n; ++j) store_f32(at + j, x[j]);
            }
        });
    }
    if (!live) return;
    __syncthreads();
    for (int j = tid; j < p.k; j += kThreads) {  // dz at the entries, over what the pass stored there
        const int32_t i = top_i[j];
        if (i < 0) continue;
        float pj = top_p[j];
        if (repeated) {
            pj = 0.0f;
            bool earlier = false;
            for (int o = 0; o < p.k; ++o)
                if (top_i[o] == i) {
                    earlier |= o < j;
                    pj += top_p[o];
                }
            if (earlier) continue;
        }
        store_f32(dz + i, fmaf(-(w * p.inv_tau), pj, zero ? 0.0f : g * q(top_z[j])));
    }
}

// ----------------------------------------------------------------- long rows
// A cluster of K CTAs takes a row at a time, each CTA a K-th of its 16-byte
// vectors, in shared memory, as a pipeline of warps:
//   one warp copies the CTA's part of the coming rows there (bulk copies, up to
//   eight stages);
//   kPrepare warps take turns preparing the coming rows' teacher entries
//   (slots), a chain of dependent loads and reductions of microseconds a row;
//   the first group passes over a row for the maximum and the sum of powers,
//   which its CTAs send one another as one pair each;
//   the second group, a row or more behind, takes the pairs and passes over the
//   row again for the gradient, then writes dz at the entries.
// So copies, reductions and exchanges of some rows hide behind the passes over
// others.  The elements before a row's first 16-byte boundary and after its last
// one (a vocabulary of odd size) are the cluster's first CTA's; they come with the
// teacher entries.  The loss alone leaves the second group one warp, and takes the
// parts of a row one after another where there are rows for all SMs; the gradient
// alone, from a saved lse, needs no first group and no cluster.
enum { kFused, kLossOnly, kGradOnly };
constexpr int first_warps(int mode) { return mode == kGradOnly ? 0 : 8; }  // as many with the gradient as without: the same loss
constexpr int second_warps(int mode) { return mode == kFused ? 8 : mode == kLossOnly ? 1 : 16; }
constexpr int kPrepare = 3;  // more take issue slots: 4096 x 50001 bf16 144 us, 159 with five
constexpr int stream_threads(int mode) { return 32 * (first_warps(mode) + second_warps(mode) + 1 + kPrepare); }
constexpr int kMaxStages = 8, kMaxSlots = 8, kMaxCluster = 8;
// Exchanges under way.  A CTA's first group is at most kMaxStages rows ahead of its second; to send row i + n it has
// seen its second group finish row i + n - kMaxStages, for which every CTA's first group sent that row and its second
// group finished one kMaxStages before: the pair of row i has been read if n = 2 kMaxStages.
constexpr int kMeets = 2 * kMaxStages;

// A slot's row.  The slot's entries follow it in dynamic shared memory: their
// indices (-1: absent), probabilities, and the student's logits at those that
// this CTA's part holds (at all of them in the first CTA, for the loss).
struct Header {
    float weight, cross;  // cross: sum of p_j (log p_j - (z_j - zref) / tau)
    float zref;
    int32_t live, repeated;
    float edge[16];  // the first CTA's logits outside the vectors (up to 14), in order
};

// `bytes` (a multiple of 16) to shared memory, counted on the mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    if (bytes > 0)
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                     "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
                     : "memory");
}

template <int kThreads>
__device__ __forceinline__ void bar_group(int id) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}

// Dynamic shared memory: of a CTA that has its SM to itself, and of each of two CTAs that share one (of_warps below is the
// loss-only kernel's).
constexpr int kSmBytes = 228 * 1024, kCtaBytes = 227 * 1024, kReserved = 1024;  // shared memory; a CTA's most; what each CTA costs besides
constexpr int kSharedBytes = 220 * 1024;
constexpr int two_room(int mode) { return kSharedBytes / 2 - 2048 - (mode == kLossOnly ? 1408 : 0); }

template <typename T, int kMode>
__global__ void __launch_bounds__(stream_threads(kMode), 2) distill_stream_kernel(const __grid_constant__ DistillParams p) {
    constexpr int n = 16 / sizeof(T);
    constexpr bool kSaved = kMode == kGradOnly;
    constexpr int kFirst = first_warps(kMode), kSecond = second_warps(kMode), kMainWarps = kFirst + kSecond;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 2 * kMaxSlots + kMeets];
    __shared__ Header header[kMaxSlots];
    __shared__ MaxSum partial[2][16];
    // (the first group is at most kMaxSlots rows ahead: a row's slot is free once the second group is done with it)
    __shared__ MaxSum of_warps[kMode == kLossOnly ? kMaxSlots : 1][kMaxCluster][8];
    __shared__ __align__(8) MaxSum pairs[kMeets][kMaxCluster];
    __shared__ int failed;
    __shared__ uint32_t exchanged;  // rows whose pairs this CTA's cluster exchanged
    constexpr int kArrays =
        sizeof(bars) + sizeof(header) + sizeof(partial) + sizeof(of_warps) + sizeof(pairs) + sizeof(failed) + sizeof(exchanged);
    constexpr int kStatic = (kArrays + 127) / 128 * 128;  // the dynamic part behind them starts on 128 bytes
    static_assert(kSharedBytes + kStatic <= kCtaBytes && 2 * (two_room(kMode) + kStatic + kReserved) <= kSmBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t K = 1u << p.log_cluster, rank = blockIdx.x & (K - 1);
    const uint32_t own = kMode == kLossOnly ? 1u << (p.log_parts - p.log_cluster) : 1u;  // this CTA's parts of a row
    // With the loss alone and no cluster, the second group's warp adds the first group's warps too, so that those need not
    // meet after each part (4096 x 50001 bf16: 99 us, 108 where they do).
    const bool apart = kMode == kLossOnly && K == 1;
    const int64_t first = blockIdx.x >> p.log_cluster, step = gridDim.x >> p.log_cluster;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxStages, slot_full = empty + 8 * kMaxStages,
                   slot_empty = slot_full + 8 * kMaxSlots, met = slot_empty + 8 * kMaxSlots;
    const uint32_t S = p.stages, E = p.slots;
    // dynamic shared memory: the stages, the slots, each preparing warp's table for finding repeated indices
    const int entries = (p.k + 3) & ~3;
    uint8_t *slots = smem + S * p.stage_bytes;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, kMode == kLossOnly ? kFirst : kMainWarps);
        }
        for (int i = 0; i < kMaxSlots; ++i) {
            mbar_init(slot_full + 8 * i, 1);
            mbar_init(slot_empty + 8 * i, kMainWarps);
        }
        for (int i = 0; i < kMeets; ++i) mbar_init(met + 8 * i, apart ? kFirst * own : 1);
        failed = 0;
        mbar_init_fence();
    }
    __syncthreads();
    const bool exchange = !kSaved && K > 1;
    if (exchange) cluster_barrier();
    let_next_begin();
    after_previous();

    if (warp == kMainWarps) {
        if (lane == 0) {
            uint32_t s = 0, turn = 1, issued = 0;
            bool ok = true;
            for (int64_t row = first; row < p.rows; row += step) {
                const T *z = static_cast<const T *>(p.z) + row * p.ldz;
                for (uint32_t u = 0; u < own; ++u) {
                    const Row<T> part(z, p.vocab, rank * own + u, p.log_parts);
                    const uint32_t bytes = static_cast<uint32_t>((part.v1 - part.v0) * 16);
                    if (!(ok = mbar_wait(empty + 8 * s, turn, &failed))) break;
                    mbar_expect_tx(full + 8 * s, bytes);
                    bulk_load(smem_u32(smem + s * p.stage_bytes), z + part.head + part.v0 * n, bytes, full + 8 * s);
                    issued = issued < S ? issued + 1 : S;
                    if (++s == S) s = 0, turn ^= 1;
                }
                if (!ok) break;
            }
            if (!ok)  // leave no copy in flight
                for (; issued > 0; --issued) {
                    if (s == 0) s = S, turn ^= 1;
                    --s;
                    int given_up = 0;
                    mbar_wait(full + 8 * s, turn ^ 1, &given_up);
                }
        }
    } else if (warp > kMainWarps) {
        const uint32_t mine = warp - kMainWarps - 1;
        uint32_t buckets = 32, shift = 27;  // a bucket is the top bits of the index times an odd constant
        while (buckets < 2 * static_cast<uint32_t>(p.k)) buckets *= 2, --shift;
        uint32_t *table = reinterpret_cast<uint32_t *>(slots + E * 12 * entries) + mine * buckets;
        uint32_t e = mine % E, turn = 1 ^ (mine / E & 1);
        for (int64_t row = first + mine * step; row < p.rows; row += kPrepare * step) {
            const T *z = static_cast<const T *>(p.z) + row * p.ldz;
            const Row<T> part(z, p.vocab, rank, p.log_cluster);
            mbar_wait(slot_empty + 8 * e, turn, &failed);
            __syncwarp();
            int32_t *top_i = reinterpret_cast<int32_t *>(slots + e * 12 * entries);
            float *top_p = reinterpret_cast<float *>(top_i + entries), *top_z = top_p + entries;
            const float w = p.weight ? p.weight[row] : 1.0f;
            const int odd = lane < 16 ? part.edge(lane, p.vocab, rank) : -1;
            const float z_odd = odd >= 0 ? load_f32(z + odd) : 0.0f;
            float tmax = -INFINITY, tsum = 0.0f, zref = -INFINITY;
            constexpr int kAtOnce = 4;  // entries of a lane whose loads are in flight together
            for (int j0 = lane; j0 < p.k; j0 += 32 * kAtOnce) {
                int32_t at[kAtOnce];
                float t[kAtOnce], zj[kAtOnce];
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                    const int j = j0 + 32 * u;
                    at[u] = j < p.k ? p.index[row * p.k + j] : -1;
                    t[u] = j < p.k ? p.teacher[row * p.k + j] : -INFINITY;
                }
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                    if (at[u] < 0 || at[u] >= p.vocab || t[u] == -INFINITY) at[u] = -1;
                    zj[u] = at[u] >= 0 && ((!kSaved && rank == 0) || part.holds(at[u], rank)) ? load_f32(z + at[u]) : 0.0f;
                }
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                    const int j = j0 + 32 * u;
                    if (j >= p.k) continue;
                    top_i[j] = at[u];
                    top_p[j] = t[u];
                    top_z[j] = zj[u];
                    if (at[u] >= 0) tmax = fmaxf(tmax, t[u]), zref = fmaxf(zref, zj[u]);
                }
            }
            tmax = warp_max(tmax);
            zref = finite_or_0(warp_max(zref));
            for (uint32_t j = lane; j < buckets; j += 32) table[j] = 0xFFFFFFFFu;
            for (int j = lane; j < p.k; j += 32)
                if (top_i[j] >= 0) tsum += entry_power(p, top_p[j], tmax).power;
            tsum = warp_sum(tsum);
            const bool live = w != 0.0f && tsum != 0.0f;  // NaN: live, and it spreads
            float cross = 0.0f;
            bool twice = false;
            __syncwarp();
            if (live) {
                const float log_tsum = logf(tsum);
                for (int j = lane; j < p.k; j += 32) {
                    const int32_t i = top_i[j];
                    float pj = 0.0f;
                    if (i >= 0) {
                        const Entry t = entry_power(p, top_p[j], tmax);
                        pj = t.power / tsum;
                        if (!(pj == 0.0f)) cross += pj * (t.exponent - log_tsum - (top_z[j] - zref) * p.inv_tau);
                        uint32_t at = (static_cast<uint32_t>(i) * 0x9E3779B1u) >> shift;
                        while (true) {  // ends: at most half of the buckets are taken
                            const uint32_t was = atomicCAS(table + at, 0xFFFFFFFFu, static_cast<uint32_t>(i));
                            if (was == 0xFFFFFFFFu) break;
                            if (was == static_cast<uint32_t>(i)) {
                                twice = true;
                                break;
                            }
                            at = (at + 1) & (buckets - 1);
                        }
                    }
                    top_p[j] = pj;
                }
                cross = warp_sum(cross);
                twice = __any_sync(0xFFFFFFFFu, twice);
            }
            Header &h = header[e];
            if (lane < 16) h.edge[lane] = z_odd;
            if (lane == 0) h.weight = w, h.cross = cross, h.zref = zref, h.live = live, h.repeated = twice;
            __syncwarp();
            if (lane == 0) mbar_arrive(slot_full + 8 * e);
            for (int i = 0; i < kPrepare; ++i)
                if (++e == E) e = 0, turn ^= 1;
        }
    } else if (warp < kFirst) {
        const float c = kLog2e * p.inv_tau;
        constexpr int kThreads = 32 * (kFirst > 0 ? kFirst : 1);
        uint32_t s = 0, turn = 0, e = 0, eturn = 0, meet = 0, flip = 0;
        for (int64_t row = first; row < p.rows; row += step) {
            const T *z = static_cast<const T *>(p.z) + row * p.ldz;
            mbar_wait(slot_full + 8 * e, eturn, &failed);
            // One decision for the warp, and barriers that every row passes: after a wait that ran out the header may change
            // as it is read.
            const bool live = __any_sync(0xFFFFFFFFu, header[e].live != 0);
            for (uint32_t u = 0; u < own; ++u) {
                const Row<T> part(z, p.vocab, rank * own + u, p.log_parts);
                const uint4 *v = reinterpret_cast<const uint4 *>(smem + s * p.stage_bytes);
                const int count = part.v1 - part.v0, odd = part.edge(threadIdx.x, p.vocab, rank * own + u);
                mbar_wait(full + 8 * s, turn, &failed);
                MaxSum a{-INFINITY, 0.0f};
                if (live) {
                    if (odd >= 0) a.m = header[e].edge[threadIdx.x], a.s = pow2((a.m - finite_or_0(a.m)) * c);
                    // two vectors at a time: a thread's maximum, powers and sum are chains of dependent instructions
                    for (int i = threadIdx.x; i < count; i += 2 * kThreads) {
                        float x[2][n];
                        unpack<T>(v[i], x[0]);
                        unpack<T>(v[i + kThreads < count ? i + kThreads : i], x[1]);
                        const float kept = i + kThreads < count ? 1.0f : 0.0f;  // of the second one's powers
                        const float m = fmaxf(a.m, fmaxf(tree_max(x[0]), tree_max(x[1]))), r = finite_or_0(m);
                        if (m > a.m) {  // a new maximum: seldom, after the first values
                            a.s *= pow2((a.m - r) * c);
                            a.m = m;
                        }
                        if (sizeof(T) == 2 && fabsf(r * c) <= kPlain) {
                            const float rc = r * c;
#pragma unroll
                            for (int j = 0; j < n; ++j) x[0][j] = pow2(fmaf(x[0][j], c, -rc)), x[1][j] = pow2(fmaf(x[1][j], c, -rc));
                        } else {
#pragma unroll
                            for (int j = 0; j < n; ++j) x[0][j] = pow2((x[0][j] - r) * c), x[1][j] = pow2((x[1][j] - r) * c);
                        }
                        a.s += fmaf(kept, tree_sum(x[1]), tree_sum(x[0]));
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(empty + 8 * s);
                    if (u == own - 1) mbar_arrive(slot_empty + 8 * e);
                }
                if (++s == S) s = 0, turn ^= 1;
                if (!live && apart) continue;
                a = merge_lanes<32>(a, c);
                if (apart) {
                    if (lane == 0) {
                        of_warps[kMode == kLossOnly ? meet % kMaxSlots : 0][u][warp] = a;
                        mbar_arrive(met + 8 * (meet % kMeets));
                    }
                    continue;
                }
                if (lane == 0) partial[flip & 1][warp] = a;
                bar_group<kThreads>(1);
                if (live && warp == 0) {
                    const uint32_t at = meet % kMeets, bar = met + 8 * at;
                    a = merge_lanes<(kFirst > 0 ? kFirst : 1)>(partial[flip & 1][lane & (kFirst > 0 ? kFirst - 1 : 0)], c);
                    if (K == 1) {
                        if (lane == 0) {
                            pairs[at][0] = a;
                            mbar_arrive(bar);
                        }
                    } else {
                        if (lane == 0) mbar_expect_tx(bar, 8 * K);
                        __syncwarp();
                        if (lane < static_cast<int>(K))
                            asm volatile(
                                "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                                    cluster_map(smem_u32(&pairs[at][rank]), lane)),
                                "f"(a.m), "f"(a.s), "r"(cluster_map(bar, lane))
                                : "memory");
                    }
                }
                ++flip;
            }
            if (live) ++meet;
            if (++e == E) e = 0, eturn ^= 1;
        }
        if (threadIdx.x == 0) exchanged = meet;
    } else {
        const float c = kLog2e * p.inv_tau;
        constexpr int kThreads = 32 * kSecond;
        const int tid = threadIdx.x - 32 * kFirst;
        uint32_t s = 0, turn = 0, e = 0, eturn = 0, meet = 0;
        for (int64_t row = first; row < p.rows; row += step) {
            const T *z = static_cast<const T *>(p.z) + row * p.ldz;
            T *dz = kMode == kLossOnly ? nullptr : static_cast<T *>(p.dz) + row * p.lddz;
            const Row<T> part(z, p.vocab, rank, p.log_cluster);
            mbar_wait(slot_full + 8 * e, eturn, &failed);
            const Header &h = header[e];
            if (kMode != kLossOnly) mbar_wait(full + 8 * s, turn, &failed);
            const bool live = __any_sync(0xFFFFFFFFu, h.live != 0);  // as in the first group
            Softmax<kSaved> q{0.0f, 0.0f, kSaved ? p.inv_tau : c};
            float g = 0.0f;
            if (live) {
                bool none;
                if (kSaved) {
                    q.sub = p.lse_in[row];
                    none = q.sub == -INFINITY;
                } else {
                    const uint32_t at = meet % kMeets;
                    mbar_wait(met + 8 * at, (meet / kMeets) & 1, &failed);
                    MaxSum a{};
                    if (apart) {
                        for (uint32_t u = 0; u < own; ++u) {
                            const MaxSum of_part = merge_lanes<8>(of_warps[kMode == kLossOnly ? meet % kMaxSlots : 0][u][lane & 7], c);
                            a = u == 0 ? of_part : merge(a, of_part, c);
                        }
                    } else {
                        a = pairs[at][0];
                        for (uint32_t i = 1; i < K; ++i) a = merge(a, pairs[at][i], c);
                    }
                    ++meet;
                    none = a.m == -INFINITY && a.s == 0.0f;
                    q.ref = finite_or_0(a.m), q.sub = log2f(a.s);
                    if (rank == 0 && tid == 0) {
                        p.loss[row] = none ? INFINITY : h.cross + (q.ref - h.zref) * p.inv_tau + q.sub * kLn2;
                        p.lse[row] = none ? -INFINITY : q.ref * p.inv_tau + q.sub * kLn2;
                    }
                }
                if (none)
                    q.ref = q.sub = 0.0f;  // probabilities 0 by g = 0
                else
                    g = h.weight * p.inv_tau;
            } else if (!kSaved && rank == 0 && tid == 0) {
                p.loss[row] = 0.0f, p.lse[row] = 0.0f;
            }
            if (kMode != kLossOnly) {
                const uint4 *v = reinterpret_cast<const uint4 *>(smem + s * p.stage_bytes);
                T *out = dz + part.head + part.v0 * n;
                const int count = part.v1 - part.v0, odd = part.edge(tid, p.vocab, rank);
                const bool wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
                const bool zero = g == 0.0f;  // whatever z holds
                if (odd >= 0) store_f32(dz + odd, zero ? 0.0f : g * q(h.edge[tid]));
                if (wide && zero) {
                    for (int i = tid; i < count; i += kThreads) st16(out + i * n, make_uint4(0, 0, 0, 0));
                } else if (sizeof(T) == 2 && !kSaved && wide && g > 0.0f && fabsf(q.ref * c) <= kPlain) {
                    const float sub = fmaf(q.ref, c, q.sub) - log2f(g);  // g too goes into the exponent
#pragma unroll 4
                    for (int i = tid; i < count; i += kThreads) {
                        float x[n];
                        unpack<T>(v[i], x);
#pragma unroll
                        for (int j = 0; j < n; ++j) x[j] = pow2(fmaf(x[j], c, -sub));
                        st16(out + i * n, pack<T>(x));
                    }
                } else if (wide) {
#pragma unroll 4
                    for (int i = tid; i < count; i += kThreads) {
                        float x[n];
                        unpack<T>(v[i], x);
#pragma unroll
                        for (int j = 0; j < n; ++j) x[j] = g * q(x[j]);
                        st16(out + i * n, pack<T>(x));
                    }
                } else {
                    for (int i = tid; i < count; i += kThreads) {
                        float x[n];
                        unpack<T>(v[i], x);
#pragma unroll
                        for (int j = 0; j < n; ++j) store_f32(out + i * n + j, zero ? 0.0f : g * q(x[j]));
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + 8 * s);
                bar_group<kThreads>(2);
                if (live) {  // dz at the entries that this CTA's part holds, over what the pass stored there
                    const int32_t *top_i = reinterpret_cast<const int32_t *>(slots + e * 12 * entries);
                    const float *top_p = reinterpret_cast<const float *>(top_i + entries), *top_z = top_p + entries;
                    for (int j = tid; j < p.k; j += kThreads) {
                        const int32_t i = top_i[j];
                        if (i < 0 || i >= p.vocab || !part.holds(i, rank)) continue;  // (a slot that never came holds anything)
                        float sum = top_p[j];
                        if (h.repeated) {
                            sum = 0.0f;
                            bool earlier = false;
                            for (int o = 0; o < p.k; ++o)
                                if (top_i[o] == i) {
                                    earlier |= o < j;
                                    sum += top_p[o];
                                }
                            if (earlier) continue;
                        }
                        store_f32(dz + i, fmaf(-(h.weight * p.inv_tau), sum, zero ? 0.0f : g * q(top_z[j])));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(slot_empty + 8 * e);
            if (++s == S) s = 0, turn ^= 1;
            if (++e == E) e = 0, eturn ^= 1;
        }
    }
    __syncthreads();
    if (exchange) {
        cluster_barrier();  // no CTA leaves while another may write its pair
        // The second group has waited for every pair, unless a wait ran out: the last ones of each barrier may be on their way.
        if (threadIdx.x == 0 && failed)
            for (uint32_t at = 0; at < kMeets && at < exchanged; ++at) {
                int given_up = 0;
                mbar_wait(met + 8 * at, ((exchanged - 1 - at) / kMeets) & 1, &given_up);
            }
    }
    if (threadIdx.x == 0 && failed && p.status) atomicOr(p.status, static_cast<unsigned int>(GAR_STATUS_TIMEOUT));
}

int check(const void *z, int32_t dtype, int64_t rows, int64_t vocab, int64_t ldz, const int32_t *index,
          const float *teacher, int32_t k, float tau, const void *dz, int64_t lddz) {
    if (elem_bytes(dtype) < 0) return fail(GAR_EDTYPE, "unknown dtype %d", dtype);
    if (rows < 0 || rows > 0x7FFFFFFF || vocab < 1 || vocab > 0x7FFFFFFF || k < 1 || k > kMaxTop)
        return fail(GAR_EINVAL, "rows=%lld vocab=%lld k=%d (1 <= k <= %d)", static_cast<long long>(rows),
                    static_cast<long long>(vocab), k, kMaxTop);
    if (!(tau > 0.0f) || !(tau <= 3.0e38f)) return fail(GAR_EINVAL, "tau must be positive and finite");
    if (!(kLog2e * (1.0f / tau) <= 3.4e38f)) return fail(GAR_EINVAL, "tau is too small: log2(e) / tau overflows, and equal logits would give NaN");
    if (rows == 0) return GAR_OK;
    if (!z || !index || !teacher) return fail(GAR_EINVAL, "NULL argument");
    if (ldz < vocab || (dz && lddz < vocab)) return fail(GAR_EINVAL, "a row stride is below the vocabulary");
    if (dz == z && dz && lddz != ldz) return fail(GAR_EINVAL, "dz in place of z needs the same row stride");
    if (!aligned(z, elem_bytes(dtype)) || !aligned(dz, elem_bytes(dtype)) || !aligned(index, 4) || !aligned(teacher, 4))
        return fail(GAR_EALIGN, "misaligned pointer");
    return GAR_OK;
}

template <typename T, int kMode>
int launch_stream(const DistillParams &p, int64_t rows_at_once, size_t shared, cudaStream_t stream) {
    const auto kernel = distill_stream_kernel<T, kMode>;
    // Clusters of 1 << i CTAs that the device holds at one time (its SMs come in groups, so it is fewer than its SMs
    // would make; one more would run after all others), 0: not looked up yet.
    static std::atomic<int> resident[64][4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(GAR_ECUDA, "no current device");
    const unsigned cluster = kMode == kGradOnly ? 1u : 1u << p.log_cluster;
    std::atomic<int> &known = resident[dev & 63][p.log_cluster];
    int clusters = known.load(std::memory_order_relaxed);
    if (clusters == 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes);
        clusters = 1;
        if (e == cudaSuccess && cluster > 1) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(cluster);
            cfg.blockDim = dim3(stream_threads(kMode));
            cfg.dynamicSmemBytes = kSharedBytes;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = cluster;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
        }
        if (e != cudaSuccess || clusters < 1) return fail(GAR_ECUDA, "distill_stream_kernel: %s", cudaGetErrorString(e));
        known.store(clusters, std::memory_order_relaxed);
    }
    // (looked up for one CTA an SM, which is what rows of several CTAs get)
    if (cluster == 1 || clusters > rows_at_once) clusters = static_cast<int>(rows_at_once);
    return launch_early("distill_stream_kernel", kernel, dim3(static_cast<unsigned>(clusters) << p.log_cluster), stream_threads(kMode),
                        shared, cluster, stream, p);
}

template <typename T, bool kSaved, int kHold, int kThreads>
int launch_row(const DistillParams &p, cudaStream_t stream) {
    return launch_early("distill_row_kernel", distill_row_kernel<T, kSaved, kHold, kThreads>, dim3(static_cast<unsigned>(p.rows)),
                        kThreads, 0, 1, stream, p);
}

template <typename T, int kMode>
int launch(DistillParams &p, cudaStream_t stream) {
    const int64_t bytes = static_cast<int64_t>(p.vocab) * sizeof(T);
    const int slot = 12 * ((p.k + 3) & ~3);
    int tables = 32;
    while (tables < 2 * p.k) tables *= 2;
    tables *= 4 * kPrepare;
    p.slots = slot * kMaxSlots <= 24576 ? kMaxSlots : 4;  // eight up to 24 KB
    const int fixed = p.slots * slot + tables;
    // The fewest CTAs a row whose parts fit the stages (one a group works on, and one on its way), and more while
    // there are SMs without a row.
    const auto part = [&](int K) { return (ceil_div(bytes / 16, K) + 1) * 16; };
    const int least = kMode != kGradOnly && 3 * part(kMaxCluster) + fixed <= kSharedBytes ? 3 : 2;
    const auto fits = [&](int K, int room) { return least * part(K) + fixed <= room; };
    int K = 1;
    while (K < kMaxCluster && !fits(K, kSharedBytes)) K *= 2;
    while (K < kMaxCluster && p.rows * K * 2 <= sm_count() && part(K) >= 8192) K *= 2;
    // Rows in registers: up to 16 KB (4096 x 4096 bf16 15.5 us; through shared memory 30; 4096 x 8192 28 and 39), and while
    // every row has an SM to itself, where latency counts, up to 64 KB (8 x 32000 bf16 5.0 us and 6.1; 150 x 16001 fp32 4.8
    // and 10.6; but 8192 x 16384 bf16 133 and 93).  Fewer vectors a thread than eight cost more in barriers than they give.
    constexpr bool kSaved = kMode == kGradOnly;
    if (!fits(K, kSharedBytes)) return launch_row<T, kSaved, 0, 1024>(p, stream);
    if (bytes <= 2048) return launch_row<T, kSaved, 1, 128>(p, stream);
    if (bytes <= 4096) return launch_row<T, kSaved, 2, 128>(p, stream);
    if (bytes <= 8192) return launch_row<T, kSaved, 4, 128>(p, stream);
    if (bytes <= 16384) return launch_row<T, kSaved, 8, 128>(p, stream);
    if (p.rows <= sm_count()) {
        if (bytes <= 32768) return launch_row<T, kSaved, 8, 256>(p, stream);
        if (bytes <= 65536) return launch_row<T, kSaved, 8, 512>(p, stream);
    }
    p.log_cluster = p.log_parts = K == 8 ? 3 : K / 2;
    // The loss alone needs no row whole: a CTA takes a row's parts in turn where there are rows for all SMs (clusters leave
    // SMs free, and each of their CTAs prepares the entries: 2048 x 131072 fp32 with 128 entries 166 us, 195 by clusters).
    // The parts are the fused call's, so the loss is the same bit for bit.
    if (kMode == kLossOnly && p.rows >= sm_count()) p.log_cluster = 0;
    const int cluster = 1 << p.log_cluster;
    p.stage_bytes = static_cast<int32_t>(part(K));
    // two CTAs an SM where two find room for their stages
    const bool two = (kMode == kGradOnly || cluster == 1) && fits(K, two_room(kMode));
    const int room = (two ? two_room(kMode) : kSharedBytes) - fixed;
    p.stages = room / p.stage_bytes < kMaxStages ? room / p.stage_bytes : kMaxStages;
    p.status = device_status();
    int64_t at_once = static_cast<int64_t>(sm_count()) * (two ? 2 : 1) / cluster;
    if (at_once > p.rows) at_once = p.rows;
    return launch_stream<T, kMode>(p, at_once, static_cast<size_t>(p.stages) * p.stage_bytes + fixed, stream);
}

int run(DistillParams &p, int32_t dtype, cudaStream_t stream) {
    if (p.rows == 0) return GAR_OK;
    if (dtype == GAR_F32)
        return p.lse_in ? launch<float, kGradOnly>(p, stream) : p.dz ? launch<float, kFused>(p, stream) : launch<float, kLossOnly>(p, stream);
    return p.lse_in ? launch<uint16_t, kGradOnly>(p, stream)
           : p.dz   ? launch<uint16_t, kFused>(p, stream)
                    : launch<uint16_t, kLossOnly>(p, stream);
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
    p.index = index, p.teacher = teacher, p.weight = weight;
    p.inv_tau = 1.0f / tau;
    p.inv_tau_rest = static_cast<float>(1.0 / static_cast<double>(tau) - static_cast<double>(p.inv_tau));
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
    p.index = index, p.teacher = teacher, p.weight = weight;
    p.inv_tau = 1.0f / tau;
    p.inv_tau_rest = static_cast<float>(1.0 / static_cast<double>(tau) - static_cast<double>(p.inv_tau));
    p.lse_in = lse, p.dz = dz;
    return run(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}
