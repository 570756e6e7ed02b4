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
// an order, so the rows are the same in every run.  262144 pairs of 256 experts 25 us
// in two launches, 2048 pairs of 64 experts 6 us in one: chains of dependent loads.
//
// Moving rows is bound by HBM: 8 x 4096 tokens to 8 experts each, 4096 bf16, 371 us
// there (6.5 TB/s; each token's row read once), 379 us back (6.4 TB/s), 706 us for the
// gradient of that (6.5 TB/s: dy and dweight from one read of dout and y).  Rows that do
// not start on 16 bytes go element by element: to 4 experts each, 4095 bf16, 399 us there
// (4096: 207), 592 back (212), 565 for the gradient (359).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "fp8.cuh"
#include "launch.cuh"

namespace gar {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kEach = 8;                           // pairs of a lane under way at one time
constexpr int kSortChunk = kSortThreads * kEach;   // pairs that a CTA holds in registers
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
    int32_t per_block;   // a multiple of kSortThreads
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

// kEach pairs of a lane, 32 apart.
__device__ __forceinline__ void experts_of(const SortParams &p, int32_t from, int32_t end, int lane, int (&e)[kEach]) {
#pragma unroll
    for (int m = 0; m < kEach; ++m) {
        const int32_t i = from + m * 32 + lane;
        e[m] = i < end ? expert_of(p, i) : -1;
    }
}

__global__ void __launch_bounds__(kSortThreads) expert_count_kernel(const __grid_constant__ SortParams p) {
    __shared__ int32_t of[kMaxExperts];
    for (int e = threadIdx.x; e < p.experts; e += kSortThreads) of[e] = 0;
    __syncthreads();
    let_next_begin();
    after_previous();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.per_block;
    const int32_t end = static_cast<int32_t>(min(first + p.per_block, static_cast<int64_t>(p.pairs)));
    const int32_t run = p.per_block / kSortWarps, from = static_cast<int32_t>(first) + (threadIdx.x >> 5) * run, to = min(from + run, end);
    for (int32_t at = from; at < to; at += 32 * kEach) {
        int e[kEach];
        experts_of(p, at, to, threadIdx.x & 31, e);
#pragma unroll
        for (int m = 0; m < kEach; ++m)
            if (e[m] >= 0) atomicAdd(&of[e[m]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.experts; e += kSortThreads) p.counts[static_cast<int64_t>(blockIdx.x) * p.experts + e] = of[e];
}

// Rows of an expert of n pairs, and how many of them hold one.
__device__ __forceinline__ int32_t rows_for(const SortParams &p, int32_t n) {
    return p.capacity > 0 ? p.capacity : (n + p.align - 1) / p.align * p.align;
}

__global__ void __launch_bounds__(kSortThreads) expert_place_kernel(const __grid_constant__ SortParams p) {
    extern __shared__ int32_t shared[];
    __shared__ int32_t sums[kSortWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = p.experts;
    int32_t *const total = shared;          // pairs of each expert
    int32_t *const ahead = shared + E;      // of the CTAs before this one
    int32_t *const start = shared + 2 * E;  // first row
    int32_t *const cursor = shared + 3 * E; // [warp][expert]: the next rank
    for (int e = threadIdx.x; e < E; e += kSortThreads) total[e] = ahead[e] = 0;
    for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) cursor[i] = 0;
    __syncthreads();
    let_next_begin();
    after_previous();

    // this CTA's pairs, a run of them to each warp
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * p.per_block;
    const int32_t end = static_cast<int32_t>(min(begin + p.per_block, static_cast<int64_t>(p.pairs)));
    const int32_t run = p.per_block / kSortWarps, from = static_cast<int32_t>(begin) + warp * run;
    const int32_t to = min(from + run, end);
    int of[kEach];  // of the last 256 pairs: all of them, unless a CTA has more than a chunk
    for (int32_t at = from; at < to; at += 32 * kEach) {
        experts_of(p, at, to, lane, of);
#pragma unroll
        for (int m = 0; m < kEach; ++m)
            if (of[m] >= 0) atomicAdd(&cursor[warp * E + of[m]], 1);
    }
    if (gridDim.x > 1) {  // counts of every CTA, an expert by kSortThreads / E threads
        const int parts = E >= kSortThreads ? 1 : kSortThreads / E;
        for (int i = threadIdx.x; i < E * parts; i += kSortThreads) {
            const int e = i % E, part = i / E;
            int32_t all = 0, before = 0;
#pragma unroll 8
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
        for (int e = threadIdx.x; e < E; e += kSortThreads) {
            int32_t n = 0;
            for (int w = 0; w < kSortWarps; ++w) n += cursor[w * E + e];
            total[e] = n;
        }
    __syncthreads();
    // first rows: a scan over the experts, consecutive ones to each thread
    const int each = (E + kSortThreads - 1) / kSortThreads, e0 = min(static_cast<int>(threadIdx.x) * each, E), e1 = min(e0 + each, E);
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
    for (int w = 0; w < kSortWarps; ++w) used += sums[w];
    for (int e = e0; e < e1; ++e) {
        start[e] = row;
        if (blockIdx.x == 0) p.offsets[e] = row;
        int32_t n = ahead[e];  // ranks that each warp's pairs begin at
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t c = cursor[w * E + e];
            cursor[w * E + e] = n;
            n += c;
        }
        row += rows_for(p, total[e]);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[E] = used;
    __syncthreads();
    for (int32_t i0 = from; i0 < to; i0 += 32 * kEach) {
        if (run > 32 * kEach) experts_of(p, i0, to, lane, of);
#pragma unroll
        for (int m = 0; m < kEach; ++m) {
            if (i0 + m * 32 >= to) break;  // all lanes
            const int32_t i = i0 + m * 32 + lane;
            const int e = of[m];
            const unsigned same = __match_any_sync(kAll, e);
            int32_t at = -1;
            if (e >= 0) {
                const int32_t rank = cursor[warp * E + e] + __popc(same & ((1u << lane) - 1));
                if (p.capacity == 0 || rank < p.capacity) at = start[e] + rank;
            }
            __syncwarp();
            if (e >= 0 && (same >> lane) == 1u) cursor[warp * E + e] += __popc(same);  // the last of them
            __syncwarp();
            if (i < to) p.position[i / p.per_worker][i % p.per_worker] = at;
            if (at >= 0) p.source[at] = i;
        }
    }
    // rows without a pair: -1 within an expert's rows (a warp to each), -2 behind the last expert
    if (p.align > 1 || p.capacity > 0)
        for (int e = blockIdx.x * kSortWarps + warp; e < E; e += gridDim.x * kSortWarps) {
            const int32_t end_row = e + 1 < E ? start[e + 1] : used;
            for (int32_t r = start[e] + min(total[e], end_row - start[e]) + lane; r < end_row; r += 32) p.source[r] = -1;
        }
    for (int64_t r = used + static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; r < p.rows;
         r += static_cast<int64_t>(gridDim.x) * kSortThreads)
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
    int64_t segments;                      // of a row
    int32_t k;
    int32_t share;                         // warps of a CTA that share a token: 1, 2, 4 or 8
    int32_t has_weight, has_addend;
};

// V elements of a row as loaded and stored at one time: 16 bytes, or one element.
template <typename T, int V>
struct Piece;
template <>
struct Piece<float, 4> {
    uint4 q;
};
template <>
struct Piece<uint16_t, 8> {
    uint4 q;
};
template <typename T>
struct Piece<T, 1> {
    T q;
};
template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_piece(const T *p) {
    if constexpr (V > 1) return {ld16(p)};
    else return {__ldcs(p)};
}
// The same where `on`, else zero.  Loads that carry their own condition stay ahead of
// their uses: with a branch around each the compiler puts load and use together, one
// row's after the other's (8 rows of 8 KB to each of 32768 tokens 1904 us, 495 with
// one row at a time and more warps).
__device__ __forceinline__ uint4 load16_if(const void *p, bool on) {
    uint4 q;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(q.x), "=&r"(q.y), "=&r"(q.z), "=&r"(q.w)
        : "l"(p), "r"(static_cast<int>(on)));
    return q;
}
__device__ __forceinline__ float load_one_if(const float *p, bool on) {
    float v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.cs.f32 %0, [%1];\n\t}"
                 : "=&f"(v)
                 : "l"(p), "r"(static_cast<int>(on)));
    return v;
}
__device__ __forceinline__ uint16_t load_one_if(const uint16_t *p, bool on) {
    uint16_t v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t@p ld.global.cs.u16 %0, [%1];\n\t}"
                 : "=&h"(v)
                 : "l"(p), "r"(static_cast<int>(on)));
    return v;
}
template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_piece_if(const T *p, bool on) {
    if constexpr (V > 1) return {load16_if(p, on)};
    else return {load_one_if(p, on)};
}
template <typename T, int V>
__device__ __forceinline__ void store_piece(T *p, Piece<T, V> r) {
    if constexpr (V > 1) st16(p, r.q);
    else __stcs(p, r.q);
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Piece<T, V> &r, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = load_f32(&r.q);
    } else {
        const uint32_t w[4] = {r.q.x, r.q.y, r.q.z, r.q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (V == 4) v[i] = __uint_as_float(w[i]);
            else v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ Piece<T, V> pack(const float (&v)[V]) {
    Piece<T, V> r;
    if constexpr (V == 1) store_f32(&r.q, v[0]);
    else if constexpr (V == 4)
        r.q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
        r.q = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    return r;
}

// A row is cut into segments of U pieces of V elements for each lane; `share` warps
// of a CTA take a token's segments in turn, and a lane has all its loads of a segment
// (and of up to J of the token's rows) under way at one time.
__host__ __device__ constexpr int pieces_of(int V, int J) { return V == 1 ? (J >= 8 ? 2 : 4) : (J >= 8 ? 1 : J >= 4 ? 2 : 4); }

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
    const float zero[V] = {};
    while (empty) {
        T *to = static_cast<T *>(p.to) + (r0 + __ffs(empty) - 1) * p.ldt;
        empty &= empty - 1;
        const int64_t whole = p.hidden / V * V;
        for (int64_t h = lane * V; h < whole; h += 32 * V) store_piece<T, V>(to + h, pack<T, V>(zero));
        for (int64_t h = whole + lane; h < p.hidden; h += 32) store_f32(to + h, 0.0f);
    }
}

// A warp's token and segments.
struct Place {
    int64_t w, t, first;
    bool on;
};
__device__ __forceinline__ Place place_of(const MoveParams &p) {
    const int warp = threadIdx.x >> 5;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * (kWarps / p.share) + warp / p.share;
    Place r;
    r.on = at < p.items;
    r.w = r.on ? at / p.tokens : 0, r.t = r.on ? at % p.tokens : 0, r.first = warp % p.share;
    return r;
}
// The CTAs behind the tokens' clear rows.
__device__ __forceinline__ int64_t clearing_cta(const MoveParams &p) {
    return blockIdx.x - (p.items + kWarps / p.share - 1) / (kWarps / p.share);
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) expert_gather_kernel(const __grid_constant__ MoveParams p) {
    let_next_begin();
    after_previous();
    constexpr int U = pieces_of(V, 4);
    const int lane = threadIdx.x & 31;
    if (const int64_t c = clearing_cta(p); c >= 0) {
        clear_rows<T, V>(p, (c * kWarps + (threadIdx.x >> 5)) * 32, lane);
        return;
    }
    const Place at = place_of(p);
    if (!at.on) return;
    const T *x = static_cast<const T *>(p.x[at.w]) + at.t * p.ldx;
    const int32_t row = row_of(p, at.w, at.t, lane);
    const float weight = p.has_weight && lane < p.k ? p.weight[at.w][at.t * p.k + lane] : 1.0f;
    for (int64_t s = at.first; s < p.segments; s += p.share) {
        const int64_t h0 = s * (32 * U * V) + lane * V;
        Piece<T, V> in[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (h0 + u * 32 * V + V <= p.hidden) in[u] = load_piece<T, V>(x + h0 + u * 32 * V);
        for (int j = 0; j < p.k; ++j) {
            const int32_t r = __shfl_sync(kAll, row, j);
            const float f = __shfl_sync(kAll, weight, j);
            if (r < 0) continue;  // all lanes
            T *to = static_cast<T *>(p.to) + r * p.ldt;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t h = h0 + u * 32 * V;
                if (h + V > p.hidden) {  // single elements behind the last whole piece
                    if (V > 1)
                        for (int64_t e = h; e < p.hidden; ++e) store_f32(to + e, p.has_weight ? load_f32(x + e) * f : load_f32(x + e));
                    continue;
                }
                if (p.has_weight) {
                    float v[V];
                    unpack<T, V>(in[u], v);
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] *= f;
                    store_piece<T, V>(to + h, pack<T, V>(v));
                } else {
                    store_piece<T, V>(to + h, in[u]);
                }
            }
        }
    }
}

// J rows of a token at a time (J >= k where k <= 8).
template <typename T, int V, int J>
__global__ void __launch_bounds__(kThreads) expert_combine_kernel(const __grid_constant__ MoveParams p) {
    let_next_begin();
    after_previous();
    constexpr int U = pieces_of(V, J);
    const int lane = threadIdx.x & 31;
    const Place at = place_of(p);
    if (!at.on) return;
    const T *add = p.has_addend ? static_cast<const T *>(p.x[at.w]) + at.t * p.ldx : nullptr;
    T *out = static_cast<T *>(p.out[at.w]) + at.t * p.ldo;
    const T *const y = static_cast<const T *>(p.y);
    const int32_t row = row_of(p, at.w, at.t, lane);
    const float weight = row < 0 ? 0.0f : p.has_weight ? p.weight[at.w][at.t * p.k + lane] : 1.0f;
    for (int64_t s = at.first; s < p.segments; s += p.share) {
        const int64_t h0 = s * (32 * U * V) + lane * V;
        float sum[U][V];
        Piece<T, V> a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] = load_piece_if<T, V>(add + h0 + u * 32 * V, add && h0 + u * 32 * V + V <= p.hidden);
#pragma unroll
            for (int i = 0; i < V; ++i) sum[u][i] = 0.0f;
        }
        for (int j0 = 0; j0 < p.k; j0 += J) {
            Piece<T, V> in[J][U];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int32_t r = __shfl_sync(kAll, row, (j0 + j) & 31);  // lanes behind the choices hold -1
#pragma unroll
                for (int u = 0; u < U; ++u)
                    in[j][u] = load_piece_if<T, V>(y + r * p.ldy + h0 + u * 32 * V, r >= 0 && h0 + u * 32 * V + V <= p.hidden);
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float f = __shfl_sync(kAll, weight, (j0 + j) & 31);  // 0 for a choice without a row
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float v[V];
                    unpack<T, V>(in[j][u], v);
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[u][i] = fmaf(v[i], f, sum[u][i]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t h = h0 + u * 32 * V;
            if (h + V <= p.hidden) {
                if (add) {
                    float v[V];
                    unpack<T, V>(a[u], v);
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[u][i] += v[i];
                }
                store_piece<T, V>(out + h, pack<T, V>(sum[u]));
            } else if (V > 1) {
                for (int64_t e = h; e < p.hidden; ++e) {
                    float v = 0.0f;
                    for (int j = 0; j < p.k; ++j) {
                        const int32_t r = p.position[at.w][at.t * p.k + j];
                        if (r >= 0 && r < p.rows) v = fmaf(load_f32(y + r * p.ldy + e), p.has_weight ? p.weight[at.w][at.t * p.k + j] : 1.0f, v);
                    }
                    store_f32(out + e, add ? v + load_f32(add + e) : v);
                }
            }
        }
    }
}

template <typename T, int V, int J>
__global__ void __launch_bounds__(kThreads) expert_combine_grad_kernel(const __grid_constant__ MoveParams p) {
    __shared__ float dots[kWarps][kMaxChoices];
    let_next_begin();
    after_previous();
    constexpr int U = pieces_of(V, J);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (const int64_t c = clearing_cta(p); c >= 0) {
        clear_rows<T, V>(p, (c * kWarps + warp) * 32, lane);
        return;
    }
    const Place at = place_of(p);
    const T *const y = static_cast<const T *>(p.y);
    T *const to = static_cast<T *>(p.to);
    float mine = 0.0f;  // lane j: the product with row j so far
    if (at.on) {
        const T *dout = static_cast<const T *>(p.x[at.w]) + at.t * p.ldx;
        const int32_t row = row_of(p, at.w, at.t, lane);
        const float weight = lane < p.k ? p.weight[at.w][at.t * p.k + lane] : 0.0f;
        for (int j0 = 0; j0 < p.k; j0 += J) {
            int32_t to_row[J];
            float dot[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                to_row[j] = __shfl_sync(kAll, row, (j0 + j) & 31);  // lanes behind the choices hold -1
                dot[j] = 0.0f;
            }
            for (int64_t s = at.first; s < p.segments; s += p.share) {
                const int64_t h0 = s * (32 * U * V) + lane * V;
                Piece<T, V> d[U], in[J][U];
#pragma unroll
                for (int u = 0; u < U; ++u) d[u] = load_piece_if<T, V>(dout + h0 + u * 32 * V, h0 + u * 32 * V + V <= p.hidden);
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        in[j][u] = load_piece_if<T, V>(y + to_row[j] * p.ldy + h0 + u * 32 * V, to_row[j] >= 0 && h0 + u * 32 * V + V <= p.hidden);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const float f = __shfl_sync(kAll, weight, (j0 + j) & 31);
                    const int32_t r = to_row[j];
                    if (r < 0) continue;  // all lanes
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int64_t h = h0 + u * 32 * V;
                        if (h + V <= p.hidden) {
                            float g[V], v[V];
                            unpack<T, V>(d[u], g);
                            unpack<T, V>(in[j][u], v);
#pragma unroll
                            for (int i = 0; i < V; ++i) {
                                dot[j] = fmaf(g[i], v[i], dot[j]);
                                g[i] *= f;
                            }
                            store_piece<T, V>(to + r * p.ldt + h, pack<T, V>(g));
                        } else if (V > 1) {
                            for (int64_t e = h; e < p.hidden; ++e) {
                                const float g = load_f32(dout + e);
                                dot[j] = fmaf(g, load_f32(y + r * p.ldy + e), dot[j]);
                                store_f32(to + r * p.ldt + e, g * f);
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float v = dot[j];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
                if (lane == j0 + j) mine = v;
            }
        }
    }
    if (p.share > 1) {  // the warps' shares, added in order
        dots[warp][lane] = mine;
        __syncthreads();
        if (warp % p.share != 0) return;
        for (int i = 1; i < p.share; ++i) mine += dots[warp + i][lane];
    }
    if (at.on && lane < p.k) p.dweight[at.w][at.t * p.k + lane] = mine;
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
    int32_t wide;  // dz's rows start on 16 bytes
};

// L lanes to a token (L >= k, a power of two), a choice to each.  Bound by the logits'
// lines of 128 bytes, which DRAM gives whole: 8 of 256 fp32 experts meet two thirds of
// a token's (93 MB for 8 x 16384 tokens, 18.5 us); four tokens of a lane under way at
// one time are no faster.
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
    const bool nan = z != z;  // the maximum passes over a NaN
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    const float e = top == -INFINITY && !nan ? 0.0f : expf(z - top);
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
    // zeros first: they wait for nothing that is read
    if (!p.accumulate) {
        for (int i = 0; i < 32 / L; ++i) {
            if (first + i >= p.items) break;
            T *dz = static_cast<T *>(p.dz[(first + i) / p.tokens]) + (first + i) % p.tokens * p.ldz;
            constexpr int V = 16 / sizeof(T);
            const int whole = p.wide ? p.experts / V * V : 0;
            for (int e = lane * V; e < whole; e += 32 * V) *reinterpret_cast<uint4 *>(dz + e) = make_uint4(0, 0, 0, 0);
            for (int e = whole + lane; e < p.experts; e += 32) store_f32(dz + e, 0.0f);
        }
    }
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
    const unsigned same = __match_any_sync(kAll, c >= 0 ? (lane / L) * kMaxExperts + c : -1 - lane);
    const bool leads = c >= 0 && (same & ((1u << lane) - 1)) == 0;
    float sum = g;
    if (__any_sync(kAll, c >= 0 && same != 1u << lane)) {
        sum = 0.0f;
        for (int i = 0; i < p.k; ++i) {
            const int other = __shfl_sync(kAll, c, i, L);
            const float more = __shfl_sync(kAll, g, i, L);
            if (other == c) sum += more;
        }
    }
    if (!p.accumulate) __syncwarp();
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

// The sort's shared memory at most, told to the runtime once.
int allow_shared() {
    static std::atomic<int> done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(GAR_ECUDA, "no current device");
    if (done[dev & 63].load(std::memory_order_relaxed)) return GAR_OK;
    const cudaError_t e = cudaFuncSetAttribute(expert_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>((3 + kSortWarps) * kMaxExperts * sizeof(int32_t)));
    if (e != cudaSuccess) return fail(GAR_ECUDA, "expert_place_kernel: %s", cudaGetErrorString(e));
    done[dev & 63].store(1, std::memory_order_relaxed);
    return GAR_OK;
}

enum { kGather, kCombine, kCombineGrad };
template <typename T, int V>
int launch_move(int which, MoveParams &p, bool clears, cudaStream_t stream) {
    const auto go = [&](auto rows) {
        constexpr int J = decltype(rows)::value;
        p.segments = ceil_div(p.hidden, int64_t{32 * pieces_of(V, J) * V});
        p.share = 1;
        // few tokens: a warp alone would take a row's segments one after another (4 x 501 x 4 x 1001 fp32, both calls: 82 us with
        // a warp to each, 29 with up to eight); many: a warp reads its token's positions once (8 x 4096 x 4 x 4096 bf16 the
        // gradient 522 us with eight to each, 453 with one)
        while (p.share < kWarps && p.share * 2 <= p.segments && p.items * p.share < sm_count() * int64_t{24}) p.share *= 2;
        const int64_t ctas = ceil_div(p.items, int64_t{kWarps / p.share}) + (clears ? ceil_div(p.rows, int64_t{32 * kWarps}) : 0);
        if (ctas == 0) return static_cast<int>(GAR_OK);
        const dim3 grid(static_cast<unsigned>(ctas));
        if (which == kCombine) return launch_early("expert_combine_kernel", expert_combine_kernel<T, V, J>, grid, kThreads, 0, 1, stream, p);
        if (which == kCombineGrad)
            return launch_early("expert_combine_grad_kernel", expert_combine_grad_kernel<T, V, J>, grid, kThreads, 0, 1, stream, p);
        if constexpr (J == 4) return launch_early("expert_gather_kernel", expert_gather_kernel<T, V>, grid, kThreads, 0, 1, stream, p);
        return static_cast<int>(GAR_OK);
    };
    if (which == kGather) return go(std::integral_constant<int, 4>{});
    if (p.k <= 1) return go(std::integral_constant<int, 1>{});
    if (p.k <= 2) return go(std::integral_constant<int, 2>{});
    if (p.k <= 4) return go(std::integral_constant<int, 4>{});
    return go(std::integral_constant<int, 8>{});
}
int launch_move_as(int which, int32_t dtype, bool wide, MoveParams &p, bool clears, cudaStream_t stream) {
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
    if (P < 1 || P > GAR_MAX_WORKERS || k < 1 || k > kMaxChoices || tokens < 0 || tokens > kMaxPairs / k / P || experts < 1 ||
        experts > kMaxExperts || align < 1 || capacity < 0 || (capacity > 0 && align != 1))
        return -1;
    const int64_t rows = sort_rows(P * tokens * k, experts, align, capacity);
    return rows <= 0x7FFFFFFF ? rows : -1;
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
    // 4096 pairs a CTA, held in registers, as far as the SMs go; one CTA needs no launch for the counts
    const int64_t most = std::min(sm_count(), kMaxBlocks);
    const int64_t blocks = std::max(std::min(ceil_div(int64_t{p.pairs}, int64_t{kSortChunk}), most), int64_t{1});
    p.per_block = static_cast<int32_t>(std::max(ceil_div(ceil_div(int64_t{p.pairs}, blocks), int64_t{kSortThreads}), int64_t{1}) * kSortThreads);
    const dim3 grid(static_cast<unsigned>(std::max(ceil_div(int64_t{p.pairs}, int64_t{p.per_block}), int64_t{1})));
    const size_t shared = static_cast<size_t>(3 + kSortWarps) * experts * sizeof(int32_t);
    if (int rc = allow_shared()) return rc;
    if (grid.x > 1)
        if (int rc = launch_early("expert_count_kernel", expert_count_kernel, grid, kSortThreads, 0, 1, stream, p)) return rc;
    return launch_early("expert_place_kernel", expert_place_kernel, grid, kSortThreads, shared, 1, stream, p);
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
    p.wide = rows_on_16(p.dz, P, lddz, size);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    return dtype == GAR_F32 ? launch_weights<float>(true, p, stream) : launch_weights<uint16_t>(true, p, stream);
}
