// experts.cu -- the tokens of P workers sorted by the experts that they chose, and
// back: gar_expert_sort, gar_expert_gather, gar_expert_combine,
// gar_expert_combine_grad, gar_expert_weights, gar_expert_weights_grad.
//
// A pair is one choice of one token, numbered (worker * tokens + token) * k + j.
// Sorting is by counting: the pairs of an expert keep their order, so a pair's
// row is the first row of its expert plus the pairs of that expert ahead of it.
// Every CTA takes a run of pairs; counts by CTA come from a first launch (none
// where one CTA holds all pairs), sums over the CTAs ahead give its first ranks,
// and ranks within it come from comparing 32 pairs at a time.  No atomic decides
// an order, so the rows are the same in every run.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fp8.cuh"
#include "launch.cuh"

namespace gar {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 32;
constexpr int kMaxBlocks = 192;  // of the sort
constexpr int64_t kMaxPairs = 1 << 30;
constexpr unsigned kAll = 0xFFFFFFFFu;

// ---------------------------------------------------------------- the sort
struct SortParams {
    const int32_t *choice[GAR_MAX_WORKERS];
    int32_t *position[GAR_MAX_WORKERS];
    int32_t per_worker;  // pairs of a worker
    int32_t pairs;       // of all
    int32_t per_block;   // a multiple of kThreads
    int32_t experts, align, capacity;
    int64_t rows;
    int32_t *source, *offsets;
    int32_t *counts;     // [blocks][experts]
};

// The expert of pair i, -1 for none.
__device__ __forceinline__ int expert_of(const SortParams &p, int32_t i) {
    const int e = p.choice[i / p.per_worker][i % p.per_worker];
    return e >= 0 && e < p.experts ? e : -1;
}

__global__ void __launch_bounds__(kThreads) expert_count_kernel(const __grid_constant__ SortParams p) {
    __shared__ int32_t of[kMaxExperts];
    for (int e = threadIdx.x; e < p.experts; e += kThreads) of[e] = 0;
    __syncthreads();
    let_next_begin();
    after_previous();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.per_block;
    const int32_t end = static_cast<int32_t>(min(first + p.per_block, static_cast<int64_t>(p.pairs)));
    for (int32_t i = static_cast<int32_t>(first) + threadIdx.x; i < end; i += kThreads) {
        const int e = expert_of(p, i);
        if (e >= 0) atomicAdd(&of[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kThreads) p.counts[static_cast<int64_t>(blockIdx.x) * p.experts + e] = of[e];
}

// Rows of an expert of n pairs, and how many of them hold one.
__device__ __forceinline__ int32_t rows_for(const SortParams &p, int32_t n) {
    return p.capacity > 0 ? p.capacity : (n + p.align - 1) / p.align * p.align;
}

__global__ void __launch_bounds__(kThreads) expert_place_kernel(const __grid_constant__ SortParams p) {
    __shared__ int32_t total[kMaxExperts];   // pairs of each expert
    __shared__ int32_t ahead[kMaxExperts];   // of the CTAs before this one
    __shared__ int32_t start[kMaxExperts];   // first row
    __shared__ int32_t cursor[kWarps][kMaxExperts];
    __shared__ int32_t sums[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = p.experts;
    for (int e = threadIdx.x; e < E; e += kThreads) total[e] = ahead[e] = 0;
    for (int i = threadIdx.x; i < kWarps * E; i += kThreads) cursor[i / E][i % E] = 0;
    __syncthreads();
    let_next_begin();
    after_previous();

    // this CTA's pairs, a run of them to each warp
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * p.per_block;
    const int32_t end = static_cast<int32_t>(min(begin + p.per_block, static_cast<int64_t>(p.pairs)));
    const int32_t run = p.per_block / kWarps, from = static_cast<int32_t>(begin) + warp * run;
    const int32_t to = min(from + run, end);
    for (int32_t i = from + lane; i < to; i += 32) {
        const int e = expert_of(p, i);
        if (e >= 0) atomicAdd(&cursor[warp][e], 1);
    }
    if (gridDim.x > 1) {  // counts of every CTA, an expert by kThreads / E threads
        const int parts = E >= kThreads ? 1 : kThreads / E;
        for (int i = threadIdx.x; i < E * parts; i += kThreads) {
            const int e = i % E, part = i / E;
            int32_t all = 0, before = 0;
            for (int b = part; b < static_cast<int>(gridDim.x); b += parts) {
                const int32_t n = p.counts[static_cast<int64_t>(b) * E + e];
                all += n;
                before += b < static_cast<int>(blockIdx.x) ? n : 0;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&ahead[e], before);
        }
    }
    __syncthreads();
    if (gridDim.x == 1)
        for (int e = threadIdx.x; e < E; e += kThreads) {
            int32_t n = 0;
            for (int w = 0; w < kWarps; ++w) n += cursor[w][e];
            total[e] = n;
        }
    __syncthreads();
    // first rows: a scan over the experts, consecutive ones to each thread
    const int each = (E + kThreads - 1) / kThreads, e0 = min(static_cast<int>(threadIdx.x) * each, E), e1 = min(e0 + each, E);
    int32_t mine = 0;
    for (int e = e0; e < e1; ++e) mine += rows_for(p, total[e]);
    int32_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t v = __shfl_up_sync(kAll, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    int32_t row = scan - mine;
    for (int w = 0; w < warp; ++w) row += sums[w];
    int32_t used = 0;  // rows of all experts
    for (int w = 0; w < kWarps; ++w) used += sums[w];
    for (int e = e0; e < e1; ++e) {
        start[e] = row;
        if (blockIdx.x == 0) p.offsets[e] = row;
        int32_t n = ahead[e];  // ranks that each warp's pairs begin at
        for (int w = 0; w < kWarps; ++w) {
            const int32_t c = cursor[w][e];
            cursor[w][e] = n;
            n += c;
        }
        row += rows_for(p, total[e]);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[E] = used;
    __syncthreads();
    for (int32_t i0 = from; i0 < to; i0 += 32) {
        const int32_t i = i0 + lane;
        const int e = i < to ? expert_of(p, i) : -1;
        const unsigned same = __match_any_sync(kAll, e);
        int32_t at = -1;
        if (e >= 0) {
            const int32_t rank = cursor[warp][e] + __popc(same & ((1u << lane) - 1));
            if (p.capacity == 0 || rank < p.capacity) at = start[e] + rank;
        }
        __syncwarp();
        if (e >= 0 && (same >> lane) == 1u) cursor[warp][e] += __popc(same);  // the last of them
        __syncwarp();
        if (i < to) p.position[i / p.per_worker][i % p.per_worker] = at;
        if (at >= 0) p.source[at] = i;
    }
    // rows without a pair: -1 within an expert's rows, -2 behind the last expert
    for (int e = blockIdx.x; e < E; e += gridDim.x) {
        const int32_t n = rows_for(p, total[e]);
        for (int32_t r = min(total[e], n) + threadIdx.x; r < n; r += kThreads) p.source[start[e] + r] = -1;
    }
    for (int64_t r = used + static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; r < p.rows;
         r += static_cast<int64_t>(gridDim.x) * kThreads)
        p.source[r] = -2;
}

// ------------------------------------------------------- rows there and back
struct MoveParams {
    const void *x[GAR_MAX_WORKERS];        // gather: x; combine: the addend; its gradient: dout
    void *out[GAR_MAX_WORKERS];            // combine: out
    const int32_t *position[GAR_MAX_WORKERS];
    const float *weight[GAR_MAX_WORKERS];
    float *dweight[GAR_MAX_WORKERS];
    const int32_t *source;
    const void *y;                         // the experts' rows read
    void *to;                              // the experts' rows written
    int64_t tokens, items, rows, hidden;   // tokens of a worker; items: P tokens
    int64_t ldx, ldo, ldy, ldt;
    int32_t k;
    int32_t has_weight, has_addend;
};

// V elements of a row, as one load or store of their V * sizeof(T) bytes.
template <typename T, int V>
struct Piece {
    float v[V];
};
template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_piece(const T *p) {
    Piece<T, V> r;
    if constexpr (sizeof(T) * V == 16) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) r.v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) r.v[2 * i] = bf16_lo(w[i]), r.v[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
        static_assert(V == 1);
        r.v[0] = load_f32(p);
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_piece(T *p, const Piece<T, V> &r) {
    if constexpr (sizeof(T) * V == 16) {
        uint32_t w[4];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(r.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(r.v[2 * i], r.v[2 * i + 1]);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        store_f32(p, r.v[0]);
    }
}

// The row of a token's choice `lane`, -1 for none.
__device__ __forceinline__ int32_t row_of(const MoveParams &p, int64_t w, int64_t t, int lane) {
    const int32_t r = lane < p.k ? p.position[w][t * p.k + lane] : -1;
    return r < p.rows ? r : -1;
}

// The experts' rows without a pair set to 0, 32 of them looked at by a warp.
template <typename T, int V>
__device__ __forceinline__ void clear_rows(const MoveParams &p, int64_t r0, int lane) {
    const int64_t r = r0 + lane;
    unsigned empty = __ballot_sync(kAll, r < p.rows && p.source[r < p.rows ? r : 0] == -1);
    const Piece<T, V> zero{};
    while (empty) {
        T *to = static_cast<T *>(p.to) + (r0 + __ffs(empty) - 1) * p.ldt;
        empty &= empty - 1;
        const int64_t whole = p.hidden / V * V;
        for (int64_t h = lane * V; h < whole; h += 32 * V) store_piece<T, V>(to + h, zero);
        for (int64_t h = whole + lane; h < p.hidden; h += 32) store_f32(to + h, 0.0f);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) expert_gather_kernel(const __grid_constant__ MoveParams p) {
    let_next_begin();
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (at >= p.items) {
        clear_rows<T, V>(p, (at - p.items) * 32, lane);
        return;
    }
    const int64_t w = at / p.tokens, t = at % p.tokens;
    const T *x = static_cast<const T *>(p.x[w]) + t * p.ldx;
    const int32_t row = row_of(p, w, t, lane);
    const float weight = p.has_weight && lane < p.k ? p.weight[w][t * p.k + lane] : 1.0f;
    const int64_t whole = p.hidden / V * V;
    for (int64_t h0 = 0; h0 < p.hidden; h0 += 32 * V) {
        const int64_t h = h0 + lane * V;
        const bool in = h < whole;
        Piece<T, V> v{};
        if (in) v = load_piece<T, V>(x + h);
        for (int j = 0; j < p.k; ++j) {
            const int32_t r = __shfl_sync(kAll, row, j);
            const float f = __shfl_sync(kAll, weight, j);
            if (r < 0 || !in) continue;
            Piece<T, V> o = v;
            if (p.has_weight)
#pragma unroll
                for (int i = 0; i < V; ++i) o.v[i] *= f;
            store_piece<T, V>(static_cast<T *>(p.to) + static_cast<int64_t>(r) * p.ldt + h, o);
        }
    }
    for (int j = 0; j < p.k; ++j) {
        const int32_t r = __shfl_sync(kAll, row, j);
        const float f = __shfl_sync(kAll, weight, j);
        if (r >= 0)
            for (int64_t h = whole + lane; h < p.hidden; h += 32)
                store_f32(static_cast<T *>(p.to) + static_cast<int64_t>(r) * p.ldt + h, p.has_weight ? load_f32(x + h) * f : load_f32(x + h));
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) expert_combine_kernel(const __grid_constant__ MoveParams p) {
    let_next_begin();
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (at >= p.items) return;
    const int64_t w = at / p.tokens, t = at % p.tokens;
    const T *add = p.has_addend ? static_cast<const T *>(p.x[w]) + t * p.ldx : nullptr;
    T *out = static_cast<T *>(p.out[w]) + t * p.ldo;
    const int32_t row = row_of(p, w, t, lane);
    const float weight = p.has_weight && lane < p.k ? p.weight[w][t * p.k + lane] : 1.0f;
    const auto take = [&](int64_t h, bool in, auto size) {
        constexpr int N = decltype(size)::value;
        Piece<T, N> sum{};
        for (int j = 0; j < p.k; ++j) {
            const int32_t r = __shfl_sync(kAll, row, j);
            const float f = __shfl_sync(kAll, weight, j);
            if (r < 0 || !in) continue;
            const Piece<T, N> v = load_piece<T, N>(static_cast<const T *>(p.y) + static_cast<int64_t>(r) * p.ldy + h);
#pragma unroll
            for (int i = 0; i < N; ++i) sum.v[i] = fmaf(v.v[i], f, sum.v[i]);
        }
        if (!in) return;
        if (add) {
            const Piece<T, N> a = load_piece<T, N>(add + h);
#pragma unroll
            for (int i = 0; i < N; ++i) sum.v[i] += a.v[i];
        }
        store_piece<T, N>(out + h, sum);
    };
    const int64_t whole = p.hidden / V * V;
    for (int64_t h0 = 0; h0 < whole; h0 += 32 * V) take(h0 + lane * V, h0 + lane * V < whole, std::integral_constant<int, V>{});
    for (int64_t h0 = whole; h0 < p.hidden; h0 += 32) take(h0 + lane, h0 + lane < p.hidden, std::integral_constant<int, 1>{});
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) expert_combine_grad_kernel(const __grid_constant__ MoveParams p) {
    let_next_begin();
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (at >= p.items) {
        clear_rows<T, V>(p, (at - p.items) * 32, lane);
        return;
    }
    const int64_t w = at / p.tokens, t = at % p.tokens;
    const T *dout = static_cast<const T *>(p.x[w]) + t * p.ldx;
    const int32_t row = row_of(p, w, t, lane);
    const float weight = lane < p.k ? p.weight[w][t * p.k + lane] : 0.0f;
    float mine = 0.0f;
    for (int j = 0; j < p.k; ++j) {
        const int32_t r = __shfl_sync(kAll, row, j);
        const float f = __shfl_sync(kAll, weight, j);
        if (r < 0) continue;
        const T *y = static_cast<const T *>(p.y) + static_cast<int64_t>(r) * p.ldy;
        T *to = static_cast<T *>(p.to) + static_cast<int64_t>(r) * p.ldt;
        float dot = 0.0f;
        const auto take = [&](int64_t h, auto size) {
            constexpr int N = decltype(size)::value;
            Piece<T, N> d = load_piece<T, N>(dout + h);
            const Piece<T, N> v = load_piece<T, N>(y + h);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                dot = fmaf(d.v[i], v.v[i], dot);
                d.v[i] *= f;
            }
            store_piece<T, N>(to + h, d);
        };
        const int64_t whole = p.hidden / V * V;
        for (int64_t h = lane * V; h < whole; h += 32 * V) take(h, std::integral_constant<int, V>{});
        for (int64_t h = whole + lane; h < p.hidden; h += 32) take(h, std::integral_constant<int, 1>{});
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
        if (lane == j) mine = dot;
    }
    if (lane < p.k) p.dweight[w][t * p.k + lane] = mine;
}

// ------------------------------------------------ the chosen experts' weights
struct WeightParams {
    const void *z[GAR_MAX_WORKERS];
    void *dz[GAR_MAX_WORKERS];
    const int32_t *choice[GAR_MAX_WORKERS];
    float *weight[GAR_MAX_WORKERS];
    const float *dweight[GAR_MAX_WORKERS];
    int64_t tokens, items, ldz;
    int32_t experts, k, accumulate;
};

// L lanes to a token (L >= k, a power of two), a choice to each.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) expert_weights_kernel(const __grid_constant__ WeightParams p) {
    let_next_begin();
    after_previous();
    const int lane = threadIdx.x & 31, j = lane & (L - 1);
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / L;
    const bool mine = at < p.items && j < p.k;
    const int64_t w = mine ? at / p.tokens : 0, t = mine ? at % p.tokens : 0;
    const int c = mine ? p.choice[w][t * p.k + j] : -1;
    const bool on = c >= 0 && c < p.experts;
    const float z = on ? load_f32(static_cast<const T *>(p.z[w]) + t * p.ldz + c) : -INFINITY;
    float top = z;
    bool nan = z != z;  // the maximum passes over a NaN
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    float e = top == -INFINITY && !nan ? 0.0f : expf(z - top);
    float sum = e;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (mine) p.weight[w][t * p.k + j] = on && e != 0.0f ? e / sum : 0.0f;
}

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) expert_weights_grad_kernel(const __grid_constant__ WeightParams p) {
    let_next_begin();
    after_previous();
    const int lane = threadIdx.x & 31, j = lane & (L - 1);
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * (32 / L);
    const int64_t at = first + lane / L;
    const bool mine = at < p.items && j < p.k;
    const int64_t w = mine ? at / p.tokens : 0, t = mine ? at % p.tokens : 0;
    const int c0 = mine ? p.choice[w][t * p.k + j] : -1;
    const int c = c0 < p.experts ? c0 : -1;
    const float q = c >= 0 ? p.weight[w][t * p.k + j] : 0.0f;
    const float d = c >= 0 ? p.dweight[w][t * p.k + j] : 0.0f;
    float mean = q * d;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) mean += __shfl_xor_sync(kAll, mean, o);
    const float g = q * (d - mean);
    // an expert chosen more than once: the sum, at the first of its lanes
    float sum = 0.0f;
    bool leads = c >= 0;
    for (int i = 0; i < p.k; ++i) {
        const int other = __shfl_sync(kAll, c, i, L);
        const float more = __shfl_sync(kAll, g, i, L);
        if (other == c) {
            sum += more;
            if (i < j) leads = false;
        }
    }
    if (!p.accumulate) {
        for (int i = 0; i < 32 / L; ++i) {
            if (first + i >= p.items) break;
            T *dz = static_cast<T *>(p.dz[(first + i) / p.tokens]) + (first + i) % p.tokens * p.ldz;
            for (int e = lane; e < p.experts; e += 32) store_f32(dz + e, 0.0f);
        }
        __syncwarp();
    }
    if (leads) {
        T *dz = static_cast<T *>(p.dz[w]) + t * p.ldz + c;
        store_f32(dz, p.accumulate ? load_f32(dz) + sum : sum);
    }
}

// ---------------------------------------------------------------------- host
int check_shape(int32_t P, int64_t tokens, int32_t k) {
    if (P < 1 || P > GAR_MAX_WORKERS) return fail(GAR_EINVAL, "P=%d outside 1..%d", P, GAR_MAX_WORKERS);
    if (k < 1 || k > kMaxChoices || tokens < 0 || tokens > kMaxPairs / k / P)
        return fail(GAR_EINVAL, "tokens=%lld k=%d (1..%d; P tokens k up to 2^30)", static_cast<long long>(tokens), k, kMaxChoices);
    return GAR_OK;
}

// Workers' pointers, each present and aligned.
template <typename Out, typename In>
int take_table(Out *to, In *const *from, int32_t P, int alignment, const char *name) {
    if (!from) return fail(GAR_EINVAL, "%s is NULL", name);
    for (int i = 0; i < P; ++i) {
        if (!from[i]) return fail(GAR_EINVAL, "%s has a NULL worker pointer", name);
        if (!aligned(from[i], alignment)) return fail(GAR_EALIGN, "%s has a misaligned worker pointer", name);
        to[i] = from[i];
    }
    return GAR_OK;
}

// Whether all rows start on 16 bytes.
template <typename Ptr>
bool rows_on_16(Ptr *const *rows, int P, int64_t ld, int elem) {
    uint64_t bits = static_cast<uint64_t>(ld) * elem;
    for (int i = 0; i < P; ++i) bits |= reinterpret_cast<uintptr_t>(rows[i]);
    return bits % 16 == 0;
}

int64_t sort_rows(int64_t pairs, int64_t experts, int64_t align, int64_t capacity) {
    return capacity > 0 ? experts * capacity : pairs + experts * (align - 1);
}

int check_rows(const void *y, int64_t ld, int64_t rows, int64_t hidden, int elem, const char *name) {
    if (rows < 0 || rows > 0x7FFFFFFF) return fail(GAR_EINVAL, "rows=%lld", static_cast<long long>(rows));
    if (rows > 0 && (!y || ld < hidden)) return fail(GAR_EINVAL, "%s is NULL or its row stride below the hidden size", name);
    if (!aligned(y, elem)) return fail(GAR_EALIGN, "%s is misaligned", name);
    return GAR_OK;
}

enum { kGather, kCombine, kCombineGrad };
template <typename T, int V>
int launch_move(int which, const MoveParams &p, bool clears, cudaStream_t stream) {
    const int64_t warps = p.items + (clears ? ceil_div(p.rows, int64_t{32}) : 0);
    if (warps == 0) return GAR_OK;
    const dim3 grid(static_cast<unsigned>(ceil_div(warps, int64_t{kWarps})));
    if (which == kGather) return launch_early("expert_gather_kernel", expert_gather_kernel<T, V>, grid, kThreads, 0, 1, stream, p);
    if (which == kCombine) return launch_early("expert_combine_kernel", expert_combine_kernel<T, V>, grid, kThreads, 0, 1, stream, p);
    return launch_early("expert_combine_grad_kernel", expert_combine_grad_kernel<T, V>, grid, kThreads, 0, 1, stream, p);
}
int launch_move_as(int which, int32_t dtype, bool wide, const MoveParams &p, bool clears, cudaStream_t stream) {
    if (dtype == GAR_F32) return wide ? launch_move<float, 4>(which, p, clears, stream) : launch_move<float, 1>(which, p, clears, stream);
    return wide ? launch_move<uint16_t, 8>(which, p, clears, stream) : launch_move<uint16_t, 1>(which, p, clears, stream);
}

template <typename T>
int launch_weights(bool grad, const WeightParams &p, cudaStream_t stream) {
    const auto go = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        const dim3 grid(static_cast<unsigned>(ceil_div(p.items, int64_t{kThreads / L})));
        return grad ? launch_early("expert_weights_grad_kernel", expert_weights_grad_kernel<T, L>, grid, kThreads, 0, 1, stream, p)
                    : launch_early("expert_weights_kernel", expert_weights_kernel<T, L>, grid, kThreads, 0, 1, stream, p);
    };
    if (p.k <= 2) return go(std::integral_constant<int, 2>{});
    if (p.k <= 4) return go(std::integral_constant<int, 4>{});
    if (p.k <= 8) return go(std::integral_constant<int, 8>{});
    if (p.k <= 16) return go(std::integral_constant<int, 16>{});
    return go(std::integral_constant<int, 32>{});
}

}  // namespace
}  // namespace gar

using namespace gar;

extern "C" int64_t gar_expert_rows(int32_t P, int64_t tokens, int32_t k, int32_t experts, int32_t align, int32_t capacity) {
    if (P < 1 || P > GAR_MAX_WORKERS || tokens < 0 || tokens > kMaxPairs / P || k < 1 || k > kMaxChoices || experts < 1 ||
        experts > kMaxExperts || align < 1 || capacity < 0)
        return -1;
    return sort_rows(P * tokens * k, experts, align, capacity);
}

extern "C" size_t gar_expert_workspace_bytes(int32_t P, int64_t tokens, int32_t k, int32_t experts) {
    if (P < 1 || P > GAR_MAX_WORKERS || tokens < 0 || k < 1 || k > kMaxChoices || experts < 1 || experts > kMaxExperts) return 0;
    return static_cast<size_t>(kMaxBlocks) * experts * 4;
}

extern "C" int gar_expert_sort(const int32_t *const *choice, int32_t P, int64_t tokens, int32_t k, int32_t experts, int32_t align,
                               int32_t capacity, int32_t *const *position, int32_t *source, int64_t rows, int32_t *offsets,
                               void *d_workspace, size_t workspace_bytes, gar_stream_t stream_) {
    if (int rc = check_shape(P, tokens, k)) return rc;
    if (experts < 1 || experts > kMaxExperts || align < 1 || capacity < 0 || (capacity > 0 && align != 1))
        return fail(GAR_EINVAL, "experts=%d (1..%d) align=%d (from 1) capacity=%d (from 0, with align 1)", experts, kMaxExperts, align, capacity);
    const int64_t need = sort_rows(P * tokens * k, experts, align, capacity);
    if (rows < need || rows > 0x7FFFFFFF)
        return fail(GAR_EINVAL, "rows=%lld: at least %lld, below 2^31", static_cast<long long>(rows), static_cast<long long>(need));
    if (!offsets || (rows > 0 && !source) || !d_workspace || workspace_bytes < gar_expert_workspace_bytes(P, tokens, k, experts))
        return fail(GAR_EINVAL, "NULL argument, or the workspace is too small");
    if (!aligned(offsets, 4) || !aligned(source, 4) || !aligned(d_workspace, 4)) return fail(GAR_EALIGN, "misaligned pointer");
    SortParams p{};
    if (tokens > 0) {
        if (int rc = take_table(p.choice, choice, P, 4, "choice")) return rc;
        if (int rc = take_table(p.position, position, P, 4, "position")) return rc;
    }
    p.per_worker = static_cast<int32_t>(tokens * k), p.pairs = static_cast<int32_t>(P * tokens * k);
    p.experts = experts, p.align = align, p.capacity = capacity, p.rows = rows;
    p.source = source, p.offsets = offsets, p.counts = static_cast<int32_t *>(d_workspace);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const int64_t most = std::min(sm_count(), kMaxBlocks);
    const int64_t blocks = std::max(std::min(ceil_div(int64_t{p.pairs}, int64_t{2048}), most), int64_t{1});
    p.per_block = static_cast<int32_t>(std::max(ceil_div(ceil_div(int64_t{p.pairs}, blocks), int64_t{kThreads}) * kThreads, int64_t{kThreads}));
    const dim3 grid(static_cast<unsigned>(std::max(ceil_div(int64_t{p.pairs}, int64_t{p.per_block}), int64_t{1})));
    if (grid.x > 1)
        if (int rc = launch_early("expert_count_kernel", expert_count_kernel, grid, kThreads, 0, 1, stream, p)) return rc;
    return launch_early("expert_place_kernel", expert_place_kernel, grid, kThreads, 0, 1, stream, p);
}

extern "C" int gar_expert_gather(const void *const *x, int32_t P, int64_t tokens, int64_t hidden, int64_t ldx, int32_t dtype, int32_t k,
                                 const int32_t *const *position, const int32_t *source, int64_t rows, const float *const *weight,
                                 void *y, int64_t ldy, gar_stream_t stream_) {
    if (int rc = check_shape(P, tokens, k)) return rc;
    const int size = elem_bytes(dtype);
    if (size < 0) return fail(GAR_EDTYPE, "unknown dtype %d", dtype);
    if (hidden < 1 || (tokens > 0 && ldx < hidden)) return fail(GAR_EINVAL, "hidden=%lld, or a row stride below it", static_cast<long long>(hidden));
    if (int rc = check_rows(y, ldy, rows, hidden, size, "y")) return rc;
    if (rows > 0 && !source) return fail(GAR_EINVAL, "source is NULL");
    if (!aligned(source, 4)) return fail(GAR_EALIGN, "source is misaligned");
    MoveParams p{};
    if (tokens > 0) {
        if (int rc = take_table(p.x, x, P, size, "x")) return rc;
        if (int rc = take_table(p.position, position, P, 4, "position")) return rc;
        if (weight)
            if (int rc = take_table(p.weight, weight, P, 4, "weight")) return rc;
    }
    p.source = source, p.to = y;
    p.tokens = tokens, p.items = P * tokens, p.rows = rows, p.hidden = hidden, p.ldx = ldx, p.ldt = ldy, p.k = k;
    p.has_weight = weight != nullptr;
    const bool wide = (tokens == 0 || rows_on_16(p.x, P, ldx, size)) && rows_on_16(&p.to, 1, ldy, size);
    return launch_move_as(kGather, dtype, wide, p, true, reinterpret_cast<cudaStream_t>(stream_));
}

extern "C" int gar_expert_combine(const void *y, int64_t ldy, int64_t rows, int32_t P, int64_t tokens, int64_t hidden, int32_t dtype,
                                  int32_t k, const int32_t *const *position, const float *const *weight, const void *const *addend,
                                  int64_t ld_addend, void *const *out, int64_t ldo, gar_stream_t stream_) {
    if (int rc = check_shape(P, tokens, k)) return rc;
    const int size = elem_bytes(dtype);
    if (size < 0) return fail(GAR_EDTYPE, "unknown dtype %d", dtype);
    if (hidden < 1) return fail(GAR_EINVAL, "hidden=%lld", static_cast<long long>(hidden));
    if (int rc = check_rows(y, ldy, rows, hidden, size, "y")) return rc;
    if (tokens == 0) return GAR_OK;
    if (ldo < hidden || (addend && ld_addend < hidden)) return fail(GAR_EINVAL, "a row stride is below the hidden size");
    MoveParams p{};
    if (int rc = take_table(p.out, out, P, size, "out")) return rc;
    if (int rc = take_table(p.position, position, P, 4, "position")) return rc;
    if (weight)
        if (int rc = take_table(p.weight, weight, P, 4, "weight")) return rc;
    if (addend) {
        if (int rc = take_table(p.x, addend, P, size, "addend")) return rc;
        for (int i = 0; i < P; ++i)
            if (addend[i] == out[i] && ld_addend != ldo) return fail(GAR_EINVAL, "an addend in place of out needs the same row stride");
    }
    p.y = y, p.tokens = tokens, p.items = P * tokens, p.rows = rows, p.hidden = hidden;
    p.ldx = ld_addend, p.ldo = ldo, p.ldy = ldy, p.k = k;
    p.has_weight = weight != nullptr, p.has_addend = addend != nullptr;
    const bool wide = rows_on_16(&p.y, 1, ldy, size) && rows_on_16(p.out, P, ldo, size) && (!addend || rows_on_16(p.x, P, ld_addend, size));
    return launch_move_as(kCombine, dtype, wide, p, false, reinterpret_cast<cudaStream_t>(stream_));
}

extern "C" int gar_expert_combine_grad(const void *const *dout, int64_t ld_dout, const void *y, int64_t ldy, int32_t P, int64_t tokens,
                                       int64_t hidden, int32_t dtype, int32_t k, const int32_t *const *position, const int32_t *source,
                                       int64_t rows, const float *const *weight, void *dy, int64_t lddy, float *const *dweight,
                                       gar_stream_t stream_) {
    if (int rc = check_shape(P, tokens, k)) return rc;
    const int size = elem_bytes(dtype);
    if (size < 0) return fail(GAR_EDTYPE, "unknown dtype %d", dtype);
    if (hidden < 1 || (tokens > 0 && ld_dout < hidden)) return fail(GAR_EINVAL, "hidden=%lld, or a row stride below it", static_cast<long long>(hidden));
    if (int rc = check_rows(y, ldy, rows, hidden, size, "y")) return rc;
    if (int rc = check_rows(dy, lddy, rows, hidden, size, "dy")) return rc;
    if (rows > 0 && !source) return fail(GAR_EINVAL, "source is NULL");
    if (dy == y && dy && ldy != lddy) return fail(GAR_EINVAL, "dy in place of y needs the same row stride");
    if (!aligned(source, 4)) return fail(GAR_EALIGN, "source is misaligned");
    MoveParams p{};
    if (tokens > 0) {
        if (int rc = take_table(p.x, dout, P, size, "dout")) return rc;
        if (int rc = take_table(p.position, position, P, 4, "position")) return rc;
        if (int rc = take_table(p.weight, weight, P, 4, "weight")) return rc;
        if (int rc = take_table(p.dweight, dweight, P, 4, "dweight")) return rc;
    }
    p.source = source, p.y = y, p.to = dy;
    p.tokens = tokens, p.items = P * tokens, p.rows = rows, p.hidden = hidden;
    p.ldx = ld_dout, p.ldy = ldy, p.ldt = lddy, p.k = k, p.has_weight = 1;
    const bool wide = (tokens == 0 || rows_on_16(p.x, P, ld_dout, size)) && rows_on_16(&p.y, 1, ldy, size) && rows_on_16(&p.to, 1, lddy, size);
    return launch_move_as(kCombineGrad, dtype, wide, p, true, reinterpret_cast<cudaStream_t>(stream_));
}

extern "C" int gar_expert_weights(const void *const *z, int32_t P, int64_t tokens, int32_t experts, int64_t ldz, int32_t dtype, int32_t k,
                                  const int32_t *const *choice, float *const *weight, gar_stream_t stream_) {
    if (int rc = check_shape(P, tokens, k)) return rc;
    const int size = elem_bytes(dtype);
    if (size < 0) return fail(GAR_EDTYPE, "unknown dtype %d", dtype);
    if (experts < 1 || experts > kMaxExperts || (tokens > 0 && ldz < experts))
        return fail(GAR_EINVAL, "experts=%d (1..%d), or a row stride below it", experts, kMaxExperts);
    if (tokens == 0) return GAR_OK;
    WeightParams p{};
    if (int rc = take_table(p.z, z, P, size, "z")) return rc;
    if (int rc = take_table(p.choice, choice, P, 4, "choice")) return rc;
    if (int rc = take_table(p.weight, weight, P, 4, "weight")) return rc;
    p.tokens = tokens, p.items = P * tokens, p.ldz = ldz, p.experts = experts, p.k = k;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    return dtype == GAR_F32 ? launch_weights<float>(false, p, stream) : launch_weights<uint16_t>(false, p, stream);
}

extern "C" int gar_expert_weights_grad(const float *const *weight, const float *const *dweight, int32_t P, int64_t tokens, int32_t experts,
                                       int32_t k, const int32_t *const *choice, void *const *dz, int64_t lddz, int32_t dtype,
                                       int32_t accumulate, gar_stream_t stream_) {
    if (int rc = check_shape(P, tokens, k)) return rc;
    const int size = elem_bytes(dtype);
    if (size < 0) return fail(GAR_EDTYPE, "unknown dtype %d", dtype);
    if (experts < 1 || experts > kMaxExperts || (tokens > 0 && lddz < experts))
        return fail(GAR_EINVAL, "experts=%d (1..%d), or a row stride below it", experts, kMaxExperts);
    if (tokens == 0) return GAR_OK;
    WeightParams p{};
    if (int rc = take_table(p.dz, dz, P, size, "dz")) return rc;
    if (int rc = take_table(p.choice, choice, P, 4, "choice")) return rc;
    if (int rc = take_table(p.dweight, dweight, P, 4, "dweight")) return rc;
    if (!weight) return fail(GAR_EINVAL, "weight is NULL");
    for (int i = 0; i < P; ++i) {
        if (!weight[i]) return fail(GAR_EINVAL, "weight has a NULL worker pointer");
        if (!aligned(weight[i], 4)) return fail(GAR_EALIGN, "weight has a misaligned worker pointer");
        p.weight[i] = const_cast<float *>(weight[i]);
    }
    p.tokens = tokens, p.items = P * tokens, p.ldz = lddz, p.experts = experts, p.k = k, p.accumulate = accumulate != 0;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    return dtype == GAR_F32 ? launch_weights<float>(true, p, stream) : launch_weights<uint16_t>(true, p, stream);
}
