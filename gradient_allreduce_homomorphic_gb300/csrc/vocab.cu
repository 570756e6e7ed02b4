// vocab.cu -- softmax cross entropy of a vocabulary layer without its logits:
// gar_vocab_loss, gar_vocab_grad, gar_vocab_grad_with_loss.
//
//   z[t][v] = sum_h x[t][h] w[v][h]              (bf16 operands, fp32 sums)
//   lse[t]  = log sum_v exp z[t][v],  loss[t] = lse[t] - z[t][target[t]]
//   g[t][v] = weight[t] (exp(z[t][v] - lse[t]) - [v = target[t]])
//   dx = g w,   dw = g^T x (+ addend)
//
// The loss is one pass of tensor-core tiles whose epilogue keeps, per row, the
// running maximum and sum of all logits but the target's over a run of vocabulary
// tiles; the runs' pairs are joined by a second, small kernel.  With r the sum's
// logarithm the loss is log(1 + exp(r - z[target])): near 0, where the target has
// almost all of the probability, the rest is a sum of its own and keeps its digits.
// The gradient goes piece by piece of the vocabulary: the piece's logits again, g from
// them in the epilogue (bf16, in the workspace), then the piece's rows of dw and its
// share of dx.  So a loss and its gradient take four products where keeping the logits
// would take three, and no more than a piece of g exists at a time.
//
// g is rounded to bf16 as an operand of the products: of a bf16 gradient that is
// another error of the size of the result's own rounding (dx and a bf16 dw 2.4e-3 from
// the exact ones in the 2-norm, 1.7e-3 of it their own).  An fp32 dw takes g as
// the sum of two bf16 values (16 bits and more of it), a product of twice the
// length, so that its error is what the fp32 sums leave; a caller who asks for them
// (parts) has the same of dx and a bf16 dw, which then are the exact ones rounded but
// for one value in some hundreds.
//
// All products run on one kernel of persistent CTA pairs (cta_group::2): tiles
// of 256 x 256, two accumulators in tensor memory, so that a tile's epilogue
// overlaps the next one's products.  Operands are loaded as they lie: the
// contraction runs along the rows of x and w for the logits, along their
// columns for dw and dx, which the tensor core takes as "MN-major" operands;
// nothing is transposed in memory.
//
// Bound by the tensor cores at the clock that the power limit leaves: 4096 x 16384
// x 4096 the loss 297 us (1850 TFLOP/s, tensor pipe active in 97 % of the cycles,
// SM clock 1.76 GHz of 2.07), logits and g 285, dw 280 (fp32: 612), dx 274 us (92 to 95 %;
// fp32 dw 86); 4096 x 131072 x 4096 loss and gradient 10.2 ms one after another (1720
// TFLOP/s).  With few rows bound by the read of w: the loss of 16 x 131072 x 1024 53 us
// (5.0 TB/s), of 64 x 32000 x 1024 19.1 us, 6 of them the kernel's beginning and end; the
// gradient of 16 x 131072 x 1024 190 us reads w twice (119 us of bytes).  With few chunks a
// tile bound by the exponents: the loss of 4096 x 131072 x 64 214 us, 36 of them products.
#include <algorithm>
#include <atomic>
#include <cfloat>

#include "fp8.cuh"
#include "launch.cuh"
#include "tensorcore.cuh"
#include "tensormap.cuh"

namespace gar {
namespace {

enum { kLoss, kGradient, kWeights, kInputs };
// A gradient with its losses given is a kernel of its own: the load among the exponents costs 32 registers, and the
// bf16 gradient of 4096 x 131072 x 64 without it 831 us instead of 845.  So are the products whose sums are longer than a
// segment: these all go to one accumulator, and the sum of a tile's segments lies in the place of the other.  An
// accumulator is handed back once it is read, and a tile's end is taken from the sum, so that the products wait for
// little more than the reading.
enum { kPlain, kSure, kLong };

constexpr int kTile = 256;    // rows of a pair's tile, and its columns at most
constexpr int kK = 64;        // k per chunk: one swizzled line of bf16
constexpr int kMaxStages = 16;
constexpr int kOperand = 128 * kK * 2;  // bytes of 128 rows of an operand of a stage
constexpr int kThreads = 320;  // warp 0 loads, warp 1 issues products, warps 2-9 epilogue
constexpr int kStaging = 8 * 4096;  // for each epilogue warp a tile of 32 x 64 bf16, two of 32 x 32, or one of 32 x 32 fp32
constexpr int kShared = 224 * 1024, kSmem = 1024 + kShared;
// Chunks that an accumulator adds at most.  The tensor core's additions round toward zero, so that a sum of one sign, or
// one with a large term ahead, is too small by what grows with its length: 3e-5 of it at 8192 k, which logits are held
// to; 1.6e-4 at 32768, beside the 2e-3 of a bf16 result's own rounding (uncut: lse 6e-3 at 2^20 k, a bf16 dw of 4M rows
// 2.6e-2); 3e-6 at 2048, of an fp32 dw (of 4096 rows, random signs, 1.3e-5 in the 2-norm uncut, 3.6e-6 so; at 1024 2.9e-6).
// Longer sums are added up by the epilogue in tensor memory (kLong): an fp32 gradient of 4096 x 131072 x 4096 takes 10.5 ms,
// 10.3 uncut, the loss of 2048 x 32000 x 16384 1220 us, 1160 uncut.  Of two parts of g the low one goes first, while the
// sum is small: its chunks count no more than those of a bf16 result.
template <int kMode, typename T>
constexpr int kSegment = (kMode == kWeights && sizeof(T) == 4 ? 2048 : kMode == kWeights || kMode == kInputs ? 32768 : 8192) / kK;
constexpr int kLowSegment = 32768 / kK;

struct VocabParams {
    int64_t items;       // whole tiles or runs, handed out in order
    int64_t tiles_m;     // tiles along the lanes: rows of x (logits), vocabulary (dw), hidden (dx)
    int64_t tiles_n;     // along the columns: vocabulary (logits), hidden (dw), rows of x (dx)
    int32_t tile_n;      // columns of a tile, a multiple of 32
    // What a stage holds: a_rows rows of operand A in each CTA (in the first alone where `second` is 0) and tile_n / 2 of B.
    // Few rows of x are few rows of A, and more stages: what the tensor core finds in the place of the other rows goes to
    // rows of the result that nobody reads.
    int32_t a_rows, second, stages;
    int32_t runs;        // a run: consecutive column tiles of one item
    int32_t chunks;      // of 64 k, of one part of g
    int32_t parts;       // of g: 1, or 2 along k
    int32_t rest;        // dx: tiles behind the items, whose k is cut
    int32_t splits;      // into as many parts
    int64_t rows, hidden, vocab;
    int64_t first, cols;  // the piece's columns
    const int32_t *target;
    const float *weight, *loss, *lse;  // loss NULL: not given
    float2 *stats;       // [rows][2 runs]: maximum, sum
    float *at_target;    // [rows]
    void *out;           // dw or dx
    const void *addend;
    float *sum;          // dx: sums over the pieces [rows][hidden], where there are several
    float *part;         // dx: sums over parts of k, [splits][rest] tiles of 256 x 256
    int64_t ld_out, ld_addend;
    int32_t last;        // dx: of the last piece
    int32_t by_tma;      // dw: its tiles are stored by TMA
    int32_t by_16;       // dw: it and its addend in pieces of 16 bytes
    // logits of the gradient: x, to be copied to `live` on the way (NULL: not)
    const uint16_t *x;
    uint16_t *live;
    int64_t ldx, ld_live;
    unsigned int *status;
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// Whether a row counts: a weight, and a target of the vocabulary.
__device__ __forceinline__ bool counts(const int32_t *target, const float *weight, int64_t vocab, int64_t t) {
    return target[t] >= 0 && target[t] < vocab && (!weight || weight[t] != 0.0f);
}

// After a wait ran out: the copies into the last `issued` stages before stage
// s have to land before the CTA ends.
__device__ __noinline__ void drain_stages(uint32_t full, uint32_t stages, int issued, uint32_t s, uint32_t turn) {
    for (; issued > 0; --issued) {
        if (s == 0) s = stages, turn ^= 1;
        --s;
        int given_up = 0;
        mbar_wait(full + 8 * s, turn ^ 1, &given_up);
    }
}

// An item: tile m, column tiles n0 .. n1, chunks c0 .. c1.  Runs of 8 tiles of
// rows by all column runs, so that the pairs at work share operands in L2.
// Behind the items come the tiles of dx that would leave pairs without work, cut
// along k: the first parts of all of them, then the second ones, so that the pairs
// at work read the same k.
struct Item {
    int64_t m, run, n0, n1;
    int32_t c0, c1;
    int32_t slot;  // -1: all of k
};
__device__ __forceinline__ void place_item(const VocabParams &p, int64_t i, Item &it) {
    const int64_t per = 8 * static_cast<int64_t>(p.runs), group = i / per, in = i % per;
    const int64_t wide = p.tiles_m - group * 8 < 8 ? p.tiles_m - group * 8 : 8;
    it.m = group * 8 + in % wide;
    it.run = in / wide;
    it.n0 = p.tiles_n * it.run / p.runs, it.n1 = p.tiles_n * (it.run + 1) / p.runs;
}
__device__ __forceinline__ Item item_of(const VocabParams &p, int64_t i) {
    Item it;
    it.c0 = 0, it.c1 = p.chunks * p.parts, it.slot = -1;
    if (i < p.items) {
        place_item(p, i, it);
        return it;
    }
    it.slot = static_cast<int32_t>(i - p.items);
    const int64_t split = it.slot / p.rest;
    place_item(p, p.items + it.slot % p.rest, it);
    const int64_t chunks = static_cast<int64_t>(p.chunks) * p.parts;
    it.c0 = static_cast<int32_t>(chunks * split / p.splits), it.c1 = static_cast<int32_t>(chunks * (split + 1) / p.splits);
    return it;
}

// 32 accumulator columns to rows 0 .. count of d (ld apart), c added where given.
template <typename T, typename C>
__device__ __forceinline__ void store_columns(const float (&v)[32], T *d, int64_t ld, const C *c, int64_t ldc, int count) {
    if (c) {
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = j < count ? load_f32(c + j * ldc) : 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < count) store_f32(d + j * ld, v[j] + x[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < count) store_f32(d + j * ld, v[j]);
    }
}

// A lane's row over an item: its running maximum and sum (loss), or what its
// gradient takes.
struct Row {
    float top, sum, low;       // kLoss: sum + low
    int32_t target;            // -1: the row does not count (gradient), or has none
    float lse, weight;         // kGradient
};

// 32 logits of a row (vocabulary columns col ..) into its running maximum and sum,
// the target's apart.  They never leave registers within a run, and a lane is a row,
// so no lane asks another.
// Exponents are formed from z - maximum, not from z log2(e) in one fma, which would
// lose digits with z.  A run may add thousands of batches, each of them less than half a
// step of a sum that one large term has set: what an addition rounds away is kept (`low`).
__device__ __forceinline__ void take_logits(const VocabParams &p, float (&v)[32], Row &r, int64_t t, int64_t col) {
    if (col + 32 > p.vocab) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (col + j >= p.vocab) v[j] = -INFINITY;
    }
    const int64_t behind = r.target - col;
    const int at = behind >= 0 && behind < 32 ? static_cast<int>(behind) : -1;
    if (__any_sync(0xFFFFFFFFu, at >= 0)) {
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (at == j) z = v[j], v[j] = -INFINITY;
        if (at >= 0) p.at_target[t] = z;
    }
    float m[4] = {r.top, v[0], v[1], v[2]};
#pragma unroll
    for (int j = 3; j < 32; ++j) m[j & 3] = fmaxf(m[j & 3], v[j]);
    const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 32; ++j) s[j & 3] += exp2_fast((v[j] - top) * kLog2e);
    const float batch = (s[0] + s[1]) + (s[2] + s[3]), scale = exp2_fast((r.top - top) * kLog2e), before = __fmul_rn(r.sum, scale);
    const float sum = __fadd_rn(before, batch), added = __fsub_rn(sum, before);
    const float lost = __fadd_rn(__fsub_rn(before, __fsub_rn(sum, added)), __fsub_rn(batch, added));  // exactly: sum + lost = before + batch
    r.low = fmaf(r.low, scale, lost);
    r.top = top, r.sum = sum;
}

// The same logits to g (col counts from the piece's first column), as bf16 pairs:
// to `low` what `high` leaves of an fp32 value.  The target's p - 1 comes from its loss
// where that is given, exp(-loss) - 1: formed from p, it would lose its digits where p is
// near 1, and half a step of lse is as much (a target at 100, lse 100 + 4e-7: nothing left).
template <bool kTwoParts, int kForm>
__device__ __forceinline__ void give_gradient(const VocabParams &p, float (&v)[32], const Row &r, int64_t t, int64_t col,
                                              uint32_t (&high)[16], uint32_t (&low)[16]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = exp2_fast((v[j] - r.lse) * kLog2e);
    const int64_t at = r.target - p.first - col;
    if (__any_sync(0xFFFFFFFFu, at >= 0 && at < 32)) {  // once for a row
        if (kForm == kSure || (kForm == kLong && p.loss)) {
            const float sure = at >= 0 && at < 32 ? expm1f(-p.loss[t]) : 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (at == j) v[j] = sure;
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (at == j) v[j] -= 1.0f;
        }
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= r.weight;
    if (__any_sync(0xFFFFFFFFu, r.target < 0)) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = r.target < 0 ? 0.0f : v[j];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        high[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        if (kTwoParts) low[i] = pack_bf16x2(v[2 * i] - bf16_lo(high[i]), v[2 * i + 1] - bf16_hi(high[i]));
    }
}

// A lane's row of a warp's 32 x 32 tile to shared memory, in the order of the
// 64-byte swizzle (no two lanes of eight in the same banks).
__device__ __forceinline__ void stage_row(uint32_t tile, int lane, const uint32_t (&w)[16]) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(tile + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)), "r"(w[4 * q]),
                     "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                     : "memory");
}

// The same of 32 fp32 values, in the order of the 128-byte swizzle.
__device__ __forceinline__ uint32_t staged(uint32_t tile, int row, int quad) { return tile + row * 128 + ((quad ^ (row & 7)) << 4); }
__device__ __forceinline__ void stage_row(uint32_t tile, int lane, const float (&v)[32]) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(staged(tile, lane, q)), "f"(v[4 * q]), "f"(v[4 * q + 1]),
                     "f"(v[4 * q + 2]), "f"(v[4 * q + 3])
                     : "memory");
}
// A staged tile in pieces of 16 bytes of its rows, an addend's pieces (loaded before
// the tile's sums were there) added to it.
template <typename T>
constexpr int kTilePieces = 32 * 32 * sizeof(T) / 16 / 32;  // of a lane
template <typename T>
__device__ __forceinline__ void load_pieces(uint4 (&x)[kTilePieces<T>], int lane, const T *c, int64_t ldc, int rows, int64_t cols) {
    constexpr int kPerRow = 32 * sizeof(T) / 16, V = 16 / sizeof(T);
#pragma unroll
    for (int q = 0; q < kTilePieces<T>; ++q) {
        const int row = (q * 32 + lane) / kPerRow, e = (q * 32 + lane) % kPerRow * V;
        x[q] = c && row < rows && e < cols ? ld16(c + row * ldc + e) : make_uint4(0, 0, 0, 0);
    }
}
template <typename T>
__device__ __forceinline__ void store_pieces(uint32_t tile, int lane, T *d, int64_t ld, const uint4 (&x)[kTilePieces<T>], int rows, int64_t cols) {
    constexpr int kPerRow = 32 * sizeof(T) / 16, V = 16 / sizeof(T);
#pragma unroll
    for (int q = 0; q < kTilePieces<T>; ++q) {
        const int row = (q * 32 + lane) / kPerRow, e = (q * 32 + lane) % kPerRow * V;
        const uint32_t w[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
        float v[V];
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[4 * i]), "=f"(v[4 * i + 1]), "=f"(v[4 * i + 2]), "=f"(v[4 * i + 3])
                         : "r"(staged(tile, row, e / 4 + i))
                         : "memory");
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (V == 4) o[i] = __float_as_uint(v[i] + __uint_as_float(w[i]));
            else o[i] = pack_bf16x2(v[2 * i] + bf16_lo(w[i]), v[2 * i + 1] + bf16_hi(w[i]));
        }
        if (row < rows && e < cols) *reinterpret_cast<uint4 *>(d + row * ld + e) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}
// A staged tile's rows one after another, a column to each lane: rows that do not
// start on 16 bytes.
template <typename T>
__device__ __forceinline__ void store_rows(uint32_t tile, int lane, T *d, int64_t ld, const T *c, int64_t ldc, int rows, bool on) {
#pragma unroll 1
    for (int i0 = 0; i0 < rows; i0 += 16) {
        float x[16];  // all under way before the first store
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = c && on && i0 + i < rows ? load_f32(c + (i0 + i) * ldc + lane) : 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(staged(tile, i0 + i, lane >> 2) + (lane & 3) * 4) : "memory");
            if (on && i0 + i < rows) store_f32(d + (i0 + i) * ld + lane, c ? v + x[i] : v);
        }
    }
}

// The same of 32 bf16 values, the first (u = 0) or second half of a row of 64.
__device__ __forceinline__ void stage_half_row(uint32_t tile, int lane, int u, const uint32_t (&w)[16]) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(staged(tile, lane, 4 * u + q)), "r"(w[4 * q]), "r"(w[4 * q + 1]),
                     "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                     : "memory");
}

// A row of x to `live`, 0 if it does not count, filled up to whole columns of 64: an
// operand of dw, where a NaN or an infinity in such a row would meet g's zeros.
__device__ __forceinline__ void copy_live_row(const VocabParams &p, int64_t t, int thread, int threads) {
    const bool live = counts(p.target, p.weight, p.vocab, t);
    const uint16_t *from = p.x + t * p.ldx;
    uint16_t *to = p.live + t * p.ld_live;
    const int64_t pieces = live ? p.hidden / 8 : 0;
    for (int64_t i = thread; i < pieces; i += threads) reinterpret_cast<uint4 *>(to)[i] = reinterpret_cast<const uint4 *>(from)[i];
    for (int64_t h = pieces * 8 + thread; h < p.ld_live; h += threads) to[h] = live && h < p.hidden ? from[h] : 0;
}

template <int kMode, typename T, int kForm>
__global__ void __launch_bounds__(kThreads, 1)
    vocab_product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                         const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_d,
                         const __grid_constant__ VocabParams p) {
    constexpr bool kMnA = kMode == kWeights || kMode == kInputs, kMnB = kMode == kWeights;
    // 16 k of a K-major operand are 32 bytes of each line; of an MN-major one two groups of eight lines of 128 bytes
    constexpr uint32_t kStepA = (kMnA ? 2048 : 32) >> 4, kStepB = (kMnB ? 2048 : 32) >> 4;
    // where the accumulator ends that begins at chunk c
    const auto segment_end = [&](int32_t c, int32_t end) {
        if (kForm != kLong) return end;
        int32_t stop = c + kSegment<kMode, T>;
        if (p.parts == 2 && c < p.chunks) stop = p.chunks - c > kLowSegment ? c + kLowSegment : p.chunks + kSegment<kMode, T>;
        return stop < end ? stop : end;
    };
    constexpr uint32_t kBack = kForm == kLong ? 1 : 2;  // accumulators in use
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxStages, acc_full = empty + 8 * kMaxStages, drained = acc_full + 16,
                   done = drained + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_cta_rank();
    const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const int64_t items = p.items + static_cast<int64_t>(p.rest) * p.splits;
    const int tile_n = p.tile_n;
    const uint32_t stages = p.stages, a_bytes = p.a_rows * kK * 2, stage = a_bytes + tile_n * kK;

    let_next_begin();
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kMaxStages; ++i) mbar_init(full + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(drained + 8 * i, 16);  // eight epilogue warps of each CTA
        }
        mbar_init(done, 1);
        failed = 0;
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc<2>(smem_u32(&tmem_slot), 512);
    if (warp == 2 && lane == 0) {  // parameters, not global memory: ahead of the wait
        tma_prefetch_map(&map_a);
        tma_prefetch_map(&map_b);
        if (kMode == kGradient || kMode == kWeights) tma_prefetch_map(&map_c), tma_prefetch_map(&map_d);
    }
    tc_fence_before();
    __syncthreads();
    cluster_barrier();
    tc_fence_after();
    after_previous();
    const uint32_t tmem = tmem_slot;

    if (warp == 0 && lane == 0) {
        const uint32_t lead_full = cluster_map(full, 0);
        uint32_t s = 0, turn = 1;  // the first turn finds every stage free
        int issued = 0;
        bool ok = true;
        for (int64_t i = first; i < items && ok; i += step) {
            const Item it = item_of(p, i);
            const int32_t a = static_cast<int32_t>(it.m * kTile + 128 * rank);
            for (int64_t n = it.n0; n < it.n1 && ok; ++n) {
                const int32_t b = static_cast<int32_t>(n * tile_n + tile_n / 2 * rank);
                for (int32_t c = it.c0; c < it.c1; ++c) {
                    if (!(ok = mbar_wait(empty + 8 * s, turn, &failed))) break;
                    const uint32_t dst = base + s * stage, bar = lead_full + 8 * s;
                    const bool low = (kMode == kWeights || kMode == kInputs) && p.parts == 2 && c < p.chunks;
                    const int32_t k = ((kMode == kWeights || kMode == kInputs) && p.parts == 2 && !low ? c - p.chunks : c) * kK;
                    if (rank == 0) mbar_expect_tx(full + 8 * s, a_bytes * (1 + p.second) + 2 * tile_n * kK);
                    if (kMode == kWeights) {  // the library's own copies: their rows are whole columns of 128 bytes
                        tma_load_columns_pair(dst, low ? &map_c : &map_a, bar, a >> 6, k);
                        tma_load_columns_pair(dst + a_bytes, &map_b, bar, b >> 6, k);
                    } else {
                        if (kMnA) {
                            tma_load_2d_pair(dst, &map_a, bar, a, k);
                            tma_load_2d_pair(dst + kOperand / 2, &map_a, bar, a + 64, k);
                        } else if (rank == 0 || p.second) {
                            tma_load_2d_pair(dst, &map_a, bar, k, a);
                        }
                        tma_load_2d_pair(dst + a_bytes, kMode == kInputs && low ? &map_c : &map_b, bar, k, b);
                    }
                    issued = issued < static_cast<int>(stages) ? issued + 1 : static_cast<int>(stages);
                    if (++s == stages) s = 0, turn ^= 1;
                }
            }
        }
        // both CTAs' copies count on the first one's barriers; the other waits at the cluster barrier below
        if (!ok && rank == 0) drain_stages(full, stages, issued, s, turn);
    } else if (warp == 1 && rank == 0) {
        const uint64_t desc_a = smem_desc(base, kMnA ? kOperand / 2 : 16, 1024, 2);
        const uint64_t desc_b = smem_desc(base + a_bytes, kMnB ? kOperand / 2 : 16, 1024, 2);
        const uint32_t idesc = bf16_idesc(kTile, static_cast<uint32_t>(tile_n), kMnA, kMnB);
        uint32_t s = 0, turn = 0, seq = 0;
        bool ready = false;  // whether the next stage was seen to be full already
        for (int64_t i = first; i < items; i += step) {
            const Item it = item_of(p, i);
            for (int64_t n = it.n0; n < it.n1; ++n) {
                for (int32_t c0 = it.c0; c0 < it.c1; ++seq) {
                    const int32_t c1 = segment_end(c0, it.c1);
                    const uint32_t acc = tmem + (kForm == kLong ? 0 : (seq & 1) * kTile);
                    if (seq >= kBack) mbar_wait_cluster(drained + 8 * ((seq - kBack) & 1), ((seq - kBack) >> 1) & 1, &failed);
                    for (int32_t c = c0; c < c1; ++c) {
                        if (!ready) mbar_wait(full + 8 * s, turn, &failed);
                        tc_fence_after();
                        const uint32_t next = s + 1 == stages ? 0 : s + 1;
                        ready = mbar_test(full + 8 * next, next ? turn : turn ^ 1);
                        if (elect_one()) {
                            const uint64_t da = desc_a + s * (stage >> 4), db = desc_b + s * (stage >> 4);
#pragma unroll
                            for (int k = 0; k < kK / 16; ++k)
                                tc_mma_bf16_pair(acc, da + k * kStepA, db + k * kStepB, idesc, c > c0 || k > 0);
                            tc_commit_pair(empty + 8 * s);
                            if (c == c1 - 1) tc_commit_pair(acc_full + 8 * (seq & 1));
                        }
                        __syncwarp();
                        s = next;
                        if (s == 0) turn ^= 1;
                    }
                    c0 = c1;
                }
            }
        }
        if (elect_one()) tc_commit<2>(done);  // here alone: the other CTA frees its half behind the cluster barrier below
        __syncwarp();
        int given_up = 0;  // a wait of its own limit, for one that ran out elsewhere lets all others pass
        mbar_wait(done, 0, &given_up);
    } else if (warp >= 2) {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t lead_drained = cluster_map(drained, 0);
        const uint32_t staging = base + kShared - kStaging + (warp - 2) * 4096;
        const int batches = tile_n / 32;
        constexpr bool kTwoParts = sizeof(T) == 4;
        // bf16 tiles leave in rows of 128 bytes, 64 columns at a time: TMA takes a row's 64 bytes as long as 128
        const bool wide = !kTwoParts && (kMode == kGradient || (kMode == kWeights && p.by_tma));
        uint32_t seq = 0;
        if (kMode == kGradient && p.live)  // while the first tiles are on their way
            for (int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + warp - 2; t < p.rows; t += static_cast<int64_t>(gridDim.x) * 8)
                copy_live_row(p, t, lane, 32);
        for (int64_t i = first; i < items; i += step) {
            const Item it = item_of(p, i);
            const int64_t lane_at = it.m * kTile + 128 * rank + quarter * 32 + lane;
            Row r{-FLT_MAX, 0.0f, 0.0f, -1, 0.0f, 0.0f};
            if (kMode == kLoss && lane_at < p.rows) r.target = p.target[lane_at];
            if (kMode == kGradient && lane_at < p.rows && counts(p.target, p.weight, p.vocab, lane_at)) {
                r.target = p.target[lane_at];
                r.lse = p.lse[lane_at], r.weight = p.weight ? p.weight[lane_at] : 1.0f;
            }
            // dw: the addend's pieces of batch j of the tile
            uint4 pieces[kTilePieces<T>];
            const auto fetch_pieces = [&](int64_t n, int j) {
                const int64_t row0 = lane_at - lane, left = p.cols - row0, col = n * tile_n + j * 32;
                const T *c = p.addend ? static_cast<const T *>(p.addend) + row0 * p.ld_addend + col : nullptr;
                load_pieces(pieces, lane, c, p.ld_addend, left < 32 ? static_cast<int>(left) : 32, p.hidden - col);
            };
            for (int64_t n = it.n0; n < it.n1; ++n) {
                for (int32_t c0 = it.c0; c0 < it.c1; ++seq) {
                    const int32_t c1 = segment_end(c0, it.c1);
                    const uint32_t buf = seq & 1, so_far = lanes + kTile, from = kForm == kLong ? so_far : lanes + buf * kTile;
                    if (kMode == kWeights && kForm != kLong && p.by_16) fetch_pieces(n, half);
                    mbar_wait(acc_full + 8 * buf, (seq >> 1) & 1, &failed);
                    __syncwarp();
                    tc_fence_after();
                    if (half >= batches) {  // a tile of 32 columns has none for the second warps
                        tc_fence_before();
                        if (lane == 0) mbar_arrive_cluster(lead_drained + 8 * buf);
                    }
                    if (kForm == kLong && half < batches) {  // each column by the warp that takes the whole sum's
#pragma unroll 1
                        for (int u = 0; u < 2; ++u) {  // two batches at a time: registers
                            float v[2][32];
#pragma unroll
                            for (int i = 0; i < 2; ++i) tc_load32(v[i], lanes + (wide ? 2 * half + 4 * u + i : half + 4 * u + 2 * i) * 32);
                            tc_wait_ld();
                            if (u == 1) {
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive_cluster(lead_drained + 8 * buf);
                            }
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t to = so_far + (wide ? 2 * half + 4 * u + i : half + 4 * u + 2 * i) * 32;
                                if (c0 > it.c0) {
                                    float more[32];
                                    tc_load32(more, to);
                                    tc_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 32; ++e) v[i][e] += more[e];
                                }
                                tc_store32(to, v[i]);
                            }
                        }
                        tc_wait_st();
                    }
                    if (kForm == kLong && c1 < it.c1) {
                        c0 = c1;
                        continue;
                    }
                    if (kMode == kWeights && kForm == kLong && p.by_16) fetch_pieces(n, half);  // registers: only now
                    if (wide) {
#pragma unroll 1
                        for (int q = half; q < batches / 2; q += 2) {
                            const int64_t col = n * tile_n + q * 64, row0 = lane_at - lane;
                            const bool on = kMode == kGradient ? row0 < p.rows && col < p.cols : row0 < p.cols && col < p.hidden;  // all lanes
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                __syncwarp();
                                float v[32];
                                tc_load32(v, from + q * 64 + u * 32);
                                tc_wait_ld();
                                if (kForm != kLong && u == 1 && q + 2 >= batches / 2) {
                                    tc_fence_before();
                                    __syncwarp();
                                    if (lane == 0) mbar_arrive_cluster(lead_drained + 8 * buf);
                                }
                                if (!on) continue;
                                uint32_t w[16], none[16];
                                if (kMode == kGradient) {
                                    give_gradient<false, kForm>(p, v, r, lane_at, col + u * 32, w, none);
                                } else {
#pragma unroll
                                    for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
                                }
                                if (u == 0) {  // the tile before has left
                                    if (lane == 0) tma_store_wait_read<0>();
                                    __syncwarp();
                                }
                                stage_half_row(staging, lane, u, w);
                            }
                            if (on) {
                                fence_async_shared();
                                __syncwarp();
                                if (lane == 0) {
                                    tma_store_2d(kMode == kGradient ? &map_c : &map_d, staging, static_cast<int32_t>(col), static_cast<int32_t>(row0));
                                    tma_store_commit();
                                }
                            }
                        }
                    }
#pragma unroll 1
                    for (int j = half; j < batches && !wide; j += 2) {
                        __syncwarp();
                        float v[32];
                        tc_load32(v, from + j * 32);
                        tc_wait_ld();
                        if (kForm != kLong && j + 2 >= batches) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(lead_drained + 8 * buf);
                        }
                        const int64_t col = n * tile_n + j * 32;
                        if (kMode == kLoss) {
                            if (col < p.vocab && lane_at - lane < p.rows) take_logits(p, v, r, lane_at, col);
                        } else if (kMode == kGradient) {
                            if (lane_at - lane >= p.rows || col >= p.cols) continue;  // all lanes: no row, or no column, of theirs
                            uint32_t high[16], low[16];
                            give_gradient<kTwoParts, kForm>(p, v, r, lane_at, col, high, low);
                            if (lane == 0) tma_store_wait_read<0>();
                            __syncwarp();
                            stage_row(staging, lane, high);
                            stage_row(staging + 2048, lane, low);
                            fence_async_shared();
                            __syncwarp();
                            if (lane == 0) {
                                tma_store_2d(&map_c, staging, static_cast<int32_t>(col), static_cast<int32_t>(lane_at));
                                tma_store_2d(&map_d, staging + 2048, static_cast<int32_t>(col), static_cast<int32_t>(lane_at));
                                tma_store_commit();
                            }
                        } else if (kMode == kWeights) {
                            const int64_t row0 = lane_at - lane, left = p.cols - row0;
                            if (left <= 0 || col >= p.hidden) continue;  // all lanes
                            if (p.by_tma) {
                                if (lane == 0) tma_store_wait_read<0>();
                                __syncwarp();
                                stage_row(staging, lane, v);
                                fence_async_shared();
                                __syncwarp();
                                if (lane == 0) {
                                    tma_store_2d(&map_d, staging, static_cast<int32_t>(col), static_cast<int32_t>(row0));
                                    tma_store_commit();
                                }
                            } else if (p.by_16) {
                                stage_row(staging, lane, v);
                                __syncwarp();
                                uint4 mine[kTilePieces<T>];
#pragma unroll
                                for (int q = 0; q < kTilePieces<T>; ++q) mine[q] = pieces[q];
                                if (j + 2 < batches) fetch_pieces(n, j + 2);
                                store_pieces(staging, lane, static_cast<T *>(p.out) + row0 * p.ld_out + col, p.ld_out, mine,
                                             left < 32 ? static_cast<int>(left) : 32, p.hidden - col);
                            } else {
                                stage_row(staging, lane, v);
                                __syncwarp();
                                T *d = static_cast<T *>(p.out) + row0 * p.ld_out + col;
                                const T *c = p.addend ? static_cast<const T *>(p.addend) + row0 * p.ld_addend + col : nullptr;
                                store_rows(staging, lane, d, p.ld_out, c, p.ld_addend, left < 32 ? static_cast<int>(left) : 32,
                                           col + lane < p.hidden);
                            }
                        } else if (const int64_t left = p.rows - col; lane_at < p.hidden && left > 0) {
                            const int count = left < 32 ? static_cast<int>(left) : 32;
                            float *sum = p.sum + col * p.hidden + lane_at;
                            const float *before = p.first > 0 ? sum : nullptr;
                            if (it.slot >= 0)
                                store_columns<float, float>(v, p.part + (static_cast<int64_t>(it.slot) * kTile + j * 32) * kTile + (lane_at & (kTile - 1)),
                                                            kTile, nullptr, 0, count);
                            else if (p.last)
                                store_columns(v, static_cast<uint16_t *>(p.out) + col * p.ld_out + lane_at, p.ld_out, before, p.hidden, count);
                            else
                                store_columns(v, sum, p.hidden, before, p.hidden, count);
                        }
                    }
                    c0 = c1;
                }
            }
            if (kMode == kLoss && lane_at < p.rows)
                p.stats[(lane_at * p.runs + it.run) * 2 + half] = make_float2(r.top, r.sum + r.low);
        }
        if ((kMode == kGradient || kMode == kWeights) && lane == 0) tma_store_wait();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_barrier();
    if (threadIdx.x == 0 && failed && p.status) atomicOr(p.status, static_cast<unsigned int>(GAR_STATUS_TIMEOUT));
    if (warp == 1) tmem_free<2>(tmem, 512);
}

// A row's pairs (maximum, sum) joined, by one warp.
__global__ void __launch_bounds__(256) vocab_join_kernel(const __grid_constant__ VocabParams p, float *loss, float *lse) {
    let_next_begin();
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (t >= p.rows) return;
    if (!counts(p.target, p.weight, p.vocab, t)) {
        if (lane == 0) loss[t] = 0.0f, lse[t] = 0.0f;
        return;
    }
    const float2 *of = p.stats + t * p.runs * 2;
    float top = -FLT_MAX, sum = 0.0f;
    for (int i = lane; i < 2 * p.runs; i += 32) {
        const float2 q = of[i];
        const float m = fmaxf(top, q.x);
        sum = sum * exp2_fast((top - m) * kLog2e) + q.y * exp2_fast((q.x - m) * kLog2e);
        top = m;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, top, o), more = __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float m = fmaxf(top, other);
        sum = sum * exp2_fast((top - m) * kLog2e) + more * exp2_fast((other - m) * kLog2e);
        top = m;
    }
    if (lane == 0) {
        const float z = p.at_target[t], d = (top - z) + logf(sum);
        float of_row = d > 0.0f ? d + log1pf(expf(-d)) : log1pf(expf(d));
        float whole = z >= top ? z + of_row : top + logf(sum + expf(z - top));
        if (!(z < INFINITY)) of_row = whole = z - z;  // NaN
        loss[t] = of_row, lse[t] = whole;
    }
}

// x to `live` alone: the logits take it from there.
__global__ void __launch_bounds__(256) vocab_live_rows_kernel(const __grid_constant__ VocabParams p) {
    let_next_begin();
    after_previous();
    copy_live_row(p, blockIdx.x, threadIdx.x, 256);
}

// The tiles of dx whose k was cut: the parts' sums added in order.  A CTA: four rows
// of x of a tile, four columns to each thread.
__global__ void __launch_bounds__(kTile) vocab_inputs_kernel(const __grid_constant__ VocabParams p) {
    let_next_begin();
    after_previous();
    const int64_t tile = blockIdx.x / (p.tile_n / 4);
    Item it;
    place_item(p, p.items + tile, it);
    const int64_t at = threadIdx.x % 64 * 4, t0 = blockIdx.x % (p.tile_n / 4) * 4 + threadIdx.x / 64;
    const int64_t h = it.m * kTile + at, t = it.n0 * p.tile_n + t0;
    if (h >= p.hidden || t >= p.rows) return;
    const float4 *of = reinterpret_cast<const float4 *>(p.part + (tile * kTile + t0) * kTile + at);
    const int64_t stride = static_cast<int64_t>(p.rest) * kTile * kTile / 4;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int i = 0; i < p.splits; ++i) {
        const float4 a = of[i * stride];
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    }
    float *sum = p.sum + t * p.hidden + h;
    uint16_t *out = static_cast<uint16_t *>(p.out) + t * p.ld_out + h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (h + i >= p.hidden) break;
        if (p.first > 0) v[i] += sum[i];
        if (!p.last) sum[i] = v[i];
        else out[i] = to_bf16(v[i]);
    }
}

// dw where no row is given: the addend, or 0.
template <typename T>
__global__ void __launch_bounds__(256) vocab_no_rows_kernel(const T *addend, int64_t ld_addend, T *dw, int64_t lddw, int64_t vocab, int64_t hidden) {
    let_next_begin();
    after_previous();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < vocab * hidden; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t v = i / hidden, h = i % hidden;
        dw[v * lddw + h] = addend ? addend[v * ld_addend + h] : T(0);
    }
}

// ---------------------------------------------------------------------- host
// Pairs of CTAs that the device holds at one time; looked up once.  < 1: an error, reported.
template <int kMode, typename T, int kForm>
int resident_pairs() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(GAR_ECUDA, "no current device");
    int pairs = known[dev & 63].load(std::memory_order_relaxed);
    if (pairs == 0) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cudaError_t e = cudaFuncSetAttribute(vocab_product_kernel<kMode, T, kForm>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&pairs, vocab_product_kernel<kMode, T, kForm>, &cfg);
        if (e != cudaSuccess || pairs < 1) return fail(GAR_ECUDA, "vocab_product_kernel: %s", cudaGetErrorString(e));
        known[dev & 63].store(pairs, std::memory_order_relaxed);
    }
    return pairs;
}

template <int kMode, typename T, int kForm>
int launch(const VocabParams &p, const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &c, const CUtensorMap &d, cudaStream_t stream) {
    const int resident = resident_pairs<kMode, T, kForm>();
    if (resident < 1) return resident;
    const int64_t pairs = std::min(p.items + static_cast<int64_t>(p.rest) * p.splits, static_cast<int64_t>(resident));
    return launch_early("vocab_product_kernel", vocab_product_kernel<kMode, T, kForm>, dim3(2 * static_cast<unsigned>(pairs)), kThreads, kSmem, 2,
                        stream, a, b, c, d, p);
}

// The product by the kernel that its sums' length and (gradient) the losses ask for.
template <int kMode, typename T>
int launch_form(const VocabParams &p, const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &c, const CUtensorMap &d,
                cudaStream_t stream) {
    const int64_t of_split = ceil_div(static_cast<int64_t>(p.chunks) * p.parts, int64_t{p.splits});
    const int64_t longest = p.items > 0 ? p.chunks : std::min(int64_t{p.chunks}, of_split);
    if (longest > kSegment<kMode, T>) return launch<kMode, T, kLong>(p, a, b, c, d, stream);
    if constexpr (kMode == kGradient)
        if (p.loss) return launch<kMode, T, kSure>(p, a, b, c, d, stream);
    return launch<kMode, T, kPlain>(p, a, b, c, d, stream);
}

// The stages of a product whose first operand has `rows` rows along its summed axis
// (0: lies the other way, always 128).
void lay_out(VocabParams *p, int64_t rows, bool staging) {
    p->a_rows = rows > 0 && rows < 128 ? static_cast<int32_t>(ceil_div(rows, int64_t{8}) * 8) : 128;
    p->second = rows == 0 || rows > 128;
    const int stage = (p->a_rows + p->tile_n / 2) * kK * 2;
    // the last stage's 128 rows of A, as the tensor core reads them, lie in the shared memory too
    p->stages = std::min((kShared - (staging ? kStaging : 0) - std::max(stage, kOperand)) / stage + 1, kMaxStages);
}

int encode(CUtensorMap *map, const void *base, int64_t inner, int64_t outer, int64_t ld, int box_outer) {
    return encode_tile_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, inner, outer, ld * 2, kK, box_outer);
}
int encode_columns(CUtensorMap *map, const void *base, int64_t inner, int64_t outer, int columns) {
    return encode_column_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, inner, outer, inner * 2, columns, kK);
}
// Tiles of 32 rows as the epilogue stores them: of a bf16 matrix, of one of two parts (ld in elements), of fp32.
int encode_store(CUtensorMap *map, const void *base, int64_t inner, int64_t outer, int64_t ld, bool wide) {
    return encode_tile_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, inner, outer, ld * 2, wide ? 64 : 32, 32,
                           wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}
int encode_store_f32(CUtensorMap *map, const void *base, int64_t inner, int64_t outer, int64_t ld) {
    return encode_tile_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, base, inner, outer, ld * 4, 32, 32);
}

// Clocks of a chunk of 64 k at 256 columns, of a tile's beginning and end that its
// neighbours do not hide, and of an item's.  A chunk of fewer columns is held by its
// loads: 128 rows of x and half the columns of w at 63 bytes a clock for each SM; by
// DRAM's 24 where x is a single tile of rows, for then w is read once.
constexpr int64_t kChunkClocks = 520, kTileClocks = 500, kItemClocks = 2500;
int64_t tile_clocks(int64_t chunks, int64_t columns, int64_t tiles_m) {
    return chunks * (tiles_m == 1 ? columns * 27 / 10 : kChunkClocks * (kTile + columns) / (2 * kTile)) + kTileClocks;
}

// Columns of the logits' tiles, and the loss's runs of them: what leaves the pairs
// evenly busy.
struct Split {
    int32_t columns, runs;
};
Split loss_split(int64_t tiles_m, int64_t vocab, int64_t chunks, int64_t pairs) {
    Split best{kTile, 1};
    int64_t least = -1;
    for (int32_t columns = kTile; columns >= 128; columns -= 32) {
        const int64_t tiles = ceil_div(vocab, int64_t{columns});
        for (int64_t rounds = 1; rounds <= 4; ++rounds) {
            const int64_t r = std::max(std::min(tiles, rounds * pairs / tiles_m), int64_t{1});
            const int64_t clocks = ceil_div(tiles_m * r, pairs) * (ceil_div(tiles, r) * tile_clocks(chunks, columns, tiles_m) + kItemClocks);
            if (least < 0 || clocks < least) least = clocks, best = {columns, static_cast<int32_t>(r)};
        }
    }
    return best;
}
int32_t gradient_columns(int64_t tiles_m, int64_t cols, int64_t chunks, int64_t pairs) {
    int32_t best = kTile;
    int64_t least = -1;
    for (int32_t columns = kTile; columns >= 128; columns -= 64) {  // g leaves in tiles of 64 columns
        const int64_t clocks = ceil_div(tiles_m * ceil_div(cols, int64_t{columns}), pairs) * tile_clocks(chunks, columns, tiles_m);
        if (least < 0 || clocks < least) least = clocks, best = columns;
    }
    return best;
}

// dx's tiles over the pairs: whole ones as often as all pairs have one, and the rest
// cut along k where that is sooner than another round (each part costs its beginning,
// the write and the addition of its sums).
struct Rounds {
    int64_t items;
    int32_t rest, splits;
};
constexpr int kMaxParts = 2;  // tiles of partial sums, of each pair
Rounds input_rounds(int64_t tiles, int64_t chunks, int64_t resident) {
    const int64_t rest = tiles % resident;
    int64_t least = chunks * kChunkClocks + kItemClocks, splits = 1;
    for (int64_t s = 2; rest > 0 && s * 4 <= chunks && s * rest <= kMaxParts * resident; ++s) {
        const int64_t clocks = ceil_div(rest * s, resident) * (ceil_div(chunks, s) * kChunkClocks + kItemClocks) + 4000 + s * rest * 150;
        if (clocks < least) least = clocks, splits = s;
    }
    return splits == 1 ? Rounds{tiles, 0, 1} : Rounds{tiles - rest, static_cast<int32_t>(rest), static_cast<int32_t>(splits)};
}

// Of each part of g, at most (or 256 columns).  Every piece ends in a round of few
// pairs and adds to dx's sums: the gradient of 4096 x 131072 x 4096 7.49 ms in pieces of
// 64 MB, 6.80 of 256, 6.81 in one of 1024; of 2048 x 131072 x 1024 1198, 960 and 922 us.
constexpr int64_t kPieceBytes = int64_t{256} << 20;

struct Plan {
    int64_t piece, pieces;   // columns of a piece, a multiple of the tile
    Split split;
    int64_t resident;        // pairs
    int64_t g, x, sum, part, loss, grad;  // bytes
};
int64_t room(int64_t bytes) { return ceil_div(bytes, 256) * 256; }
int64_t live_ld(int64_t hidden) { return ceil_div(hidden, kK) * kK; }

// parts: room for so many of g.
Plan plan_for(int64_t rows, int64_t vocab, int64_t hidden, int64_t parts) {
    Plan p{};
    const int64_t tiles_t = ceil_div(rows, int64_t{kTile});
    p.resident = std::max(sm_count() / 2, 1);
    const int64_t most = std::max(kPieceBytes / (std::max(rows, int64_t{1}) * 2) / kTile, int64_t{1}) * kTile;
    p.pieces = ceil_div(vocab, most);
    p.piece = ceil_div(ceil_div(vocab, p.pieces), int64_t{kTile}) * kTile;
    p.pieces = ceil_div(vocab, p.piece);
    p.split = {kTile, 1};
    if (rows > 0) p.split = loss_split(tiles_t, vocab, ceil_div(hidden, int64_t{kK}), p.resident);
    p.g = room(rows * p.piece * 2);
    p.x = room(rows * live_ld(hidden) * 2);
    p.loss = room(rows * p.split.runs * 16) + room(rows * 4) + p.x;
    p.sum = p.pieces > 1 ? room(rows * hidden * 4) : 0;
    if (rows > 0) {
        const int64_t tile_t = std::min(ceil_div(rows, int64_t{32}) * 32, int64_t{kTile});
        for (const int64_t cols : {std::min(p.piece, vocab), vocab - (p.pieces - 1) * p.piece}) {
            for (int64_t of_dx = 1; of_dx <= parts; ++of_dx) {
                const Rounds r = input_rounds(ceil_div(rows, tile_t) * ceil_div(hidden, int64_t{kTile}), ceil_div(cols, int64_t{kK}) * of_dx, p.resident);
                p.part = std::max(p.part, static_cast<int64_t>(r.rest) * r.splits * kTile * kTile * 4);
            }
        }
    }
    p.grad = p.g * parts + p.x + p.sum + p.part;
    return p;
}

bool sizes_fit(int64_t rows, int64_t vocab, int64_t hidden) {
    return rows >= 0 && vocab >= 1 && hidden >= 1 && rows <= 0x7FFFFFFF - 1024 && vocab <= 0x7FFFFFFF - 1024 && hidden <= (1 << 20);
}

int check(const void *x, int64_t ldx, const void *w, int64_t ldw, const int32_t *target, const float *weight, int64_t rows,
          int64_t vocab, int64_t hidden, int32_t dtype) {
    if (dtype != GAR_BF16) return fail(GAR_EDTYPE, "x and w have to be bf16, not dtype %d", dtype);
    if (!sizes_fit(rows, vocab, hidden))
        return fail(GAR_EINVAL, "rows=%lld vocab=%lld (from 1) hidden=%lld (1..2^20)", static_cast<long long>(rows),
                    static_cast<long long>(vocab), static_cast<long long>(hidden));
    if (rows == 0) return GAR_OK;
    if (!x || !w || !target) return fail(GAR_EINVAL, "x, w or target is NULL");
    if (ldx < hidden || ldw < hidden) return fail(GAR_EINVAL, "a row stride of x or w is below the hidden size");
    if (!aligned(x, 16) || !aligned(w, 16) || ldx % 8 || ldw % 8)
        return fail(GAR_EALIGN, "x, w and their row strides need 16-byte alignment");
    if (!aligned(target, 4) || !aligned(weight, 4)) return fail(GAR_EALIGN, "target or weight is misaligned");
    return GAR_OK;
}

int copy_live_rows(VocabParams p, const uint16_t *x, int64_t ldx, uint16_t *to, cudaStream_t stream) {
    p.x = x, p.ldx = ldx, p.live = to, p.ld_live = live_ld(p.hidden);
    return launch_early("vocab_live_rows_kernel", vocab_live_rows_kernel, dim3(static_cast<unsigned>(p.rows)), 256, 0, 1, stream, p);
}
// Rows of x that do not start on 128 bytes load at half the rate (two lines for each
// one's 128 bytes): copied to such that do where the logits take long enough (loss of
// 1003 x 50001 x 1000 103 us, 78 with the copy's 4; it pays from about 50 GFLOP).
bool copy_pays(const uint16_t *x, int64_t ldx, const VocabParams &p) {
    return (!aligned(x, 128) || ldx % 64) && static_cast<double>(p.rows) * p.vocab * p.hidden > 2.5e10;
}

// dw and the shares of dx of all pieces; T: dw's type; parts: bf16 values that g is taken as, 0: two for an fp32 dw, else one.
template <typename T>
int gradient(const VocabParams &p, const Plan &how, const uint16_t *x, int64_t ldx, const uint16_t *w, int64_t ldw, uint16_t *dx, int64_t lddx,
             const T *addend, int64_t ld_addend, T *dw, int64_t lddw, int parts, uint8_t *workspace, cudaStream_t stream) {
    const int64_t rows = p.rows, vocab = p.vocab, hidden = p.hidden, ld_live = live_ld(hidden);
    const int in_g = sizeof(T) == 4 || parts == 2 ? 2 : 1;
    const auto g = reinterpret_cast<uint16_t *>(workspace), g_low = reinterpret_cast<uint16_t *>(workspace + how.g);
    const auto live = reinterpret_cast<uint16_t *>(workspace + in_g * how.g);
    const auto sum = reinterpret_cast<float *>(workspace + in_g * how.g + how.x);
    const auto part = reinterpret_cast<float *>(workspace + in_g * how.g + how.x + how.sum);
    const int64_t tiles_t = ceil_div(rows, int64_t{kTile}), tiles_h = ceil_div(hidden, int64_t{kTile});
    CUtensorMap rows_k{}, live_mn{}, g_mn{}, low_mn{}, g_to{}, low_to{};
    const bool copied = copy_pays(x, ldx, p);
    const int weights_n = hidden <= 128 ? 128 : kTile;  // columns of dw's tiles: half of 256 would be empty
    if (copied)
        if (int rc = copy_live_rows(p, x, ldx, live, stream)) return rc;
    VocabParams of_rows = p;
    of_rows.tile_n = kTile;
    lay_out(&of_rows, rows, true);
    if (int rc = encode(&rows_k, copied ? live : x, hidden, rows, copied ? ld_live : ldx, of_rows.a_rows)) return rc;
    if (dw) {
        if (int rc = encode_columns(&live_mn, live, ld_live, rows, weights_n / 128)) return rc;
    }
    if (int rc = encode_columns(&g_mn, g, how.piece, rows, 2)) return rc;
    if (int rc = encode_store(&g_to, g, how.piece, rows, how.piece, in_g == 1)) return rc;
    if (in_g == 2) {
        if (int rc = encode_columns(&low_mn, g_low, how.piece, rows, 2)) return rc;
        if (int rc = encode_store(&low_to, g_low, how.piece, rows, how.piece, false)) return rc;
    } else {
        low_mn = g_mn, low_to = g_to;
    }
    for (int64_t first = 0; first < vocab; first += how.piece) {
        const int64_t cols = std::min(how.piece, vocab - first);
        VocabParams q = p;
        q.first = first, q.cols = cols, q.last = first + cols == vocab;
        q.parts = 1, q.rest = 0, q.splits = 1;
        {
            CUtensorMap w_k{};
            q.chunks = static_cast<int32_t>(ceil_div(hidden, int64_t{kK}));
            q.tile_n = gradient_columns(tiles_t, cols, q.chunks, how.resident);
            q.tiles_m = tiles_t, q.tiles_n = ceil_div(cols, int64_t{q.tile_n}), q.runs = static_cast<int32_t>(q.tiles_n);
            q.items = q.tiles_m * q.runs;
            if (int rc = encode(&w_k, w + first * ldw, hidden, cols, ldw, q.tile_n / 2)) return rc;
            lay_out(&q, rows, true);
            if (dw && !copied && first == 0) q.x = x, q.ldx = ldx, q.live = live, q.ld_live = ld_live;
            if (int rc = in_g == 2 ? launch_form<kGradient, float>(q, rows_k, w_k, g_to, low_to, stream)
                                   : launch_form<kGradient, uint16_t>(q, rows_k, w_k, g_to, low_to, stream))
                return rc;
        }
        if (dw) {
            CUtensorMap to{};
            q.tile_n = weights_n;
            q.tiles_m = ceil_div(cols, int64_t{kTile}), q.tiles_n = ceil_div(hidden, int64_t{weights_n}), q.runs = static_cast<int32_t>(q.tiles_n);
            q.chunks = static_cast<int32_t>(ceil_div(rows, int64_t{kK})), q.parts = in_g;
            q.items = q.tiles_m * q.runs;
            q.out = dw + first * lddw, q.ld_out = lddw;
            q.addend = addend ? addend + first * ld_addend : nullptr, q.ld_addend = ld_addend;
            q.by_16 = aligned(q.out, 16) && lddw * sizeof(T) % 16 == 0 && hidden * sizeof(T) % 16 == 0 &&
                      (!addend || (aligned(q.addend, 16) && ld_addend * sizeof(T) % 16 == 0));
            // a tile that ends inside 16 bytes of a row is not TMA's: it writes them whole, past the row's end
            q.by_tma = !addend && aligned(q.out, 16) && lddw * sizeof(T) % 16 == 0 && hidden * sizeof(T) % 16 == 0;
            if (q.by_tma) {
                if (int rc = sizeof(T) == 4 ? encode_store_f32(&to, q.out, hidden, cols, lddw) : encode_store(&to, q.out, hidden, cols, lddw, true))
                    return rc;
            }
            lay_out(&q, 0, true);
            if (int rc = launch_form<kWeights, T>(q, g_mn, live_mn, low_mn, to, stream)) return rc;
        }
        if (dx) {
            CUtensorMap w_mn{}, g_k{}, low_k{};
            q.tile_n = static_cast<int32_t>(std::min(ceil_div(rows, int64_t{32}) * 32, int64_t{kTile}));
            q.tiles_m = tiles_h, q.tiles_n = ceil_div(rows, int64_t{q.tile_n}), q.runs = static_cast<int32_t>(q.tiles_n), q.parts = parts == 2 ? 2 : 1;
            q.chunks = static_cast<int32_t>(ceil_div(cols, int64_t{kK}));
            const Rounds rounds = input_rounds(q.tiles_m * q.tiles_n, static_cast<int64_t>(q.chunks) * q.parts, how.resident);
            q.items = rounds.items, q.rest = rounds.rest, q.splits = rounds.splits;
            q.out = dx, q.ld_out = lddx, q.sum = sum, q.part = part;
            if (int rc = encode(&w_mn, w + first * ldw, hidden, cols, ldw, kK)) return rc;
            if (int rc = encode_tile_map(&g_k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g, cols, rows, how.piece * 2, kK, q.tile_n / 2)) return rc;
            low_k = g_k;
            if (q.parts == 2)
                if (int rc = encode_tile_map(&low_k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g_low, cols, rows, how.piece * 2, kK, q.tile_n / 2)) return rc;
            lay_out(&q, 0, false);
            if (int rc = launch_form<kInputs, uint16_t>(q, w_mn, g_k, low_k, low_k, stream)) return rc;
            if (q.rest > 0)
                if (int rc = launch_early("vocab_inputs_kernel", vocab_inputs_kernel, dim3(static_cast<unsigned>(q.rest * (q.tile_n / 4))), kTile, 0, 1,
                                          stream, q))
                    return rc;
        }
    }
    return GAR_OK;
}

}  // namespace
}  // namespace gar

using namespace gar;

extern "C" size_t gar_vocab_workspace_bytes(int64_t rows, int64_t vocab, int64_t hidden, int32_t dw_type) {
    if (!sizes_fit(rows, vocab, hidden) || elem_bytes(dw_type) < 0) return 0;
    const Plan p = plan_for(rows, vocab, hidden, dw_type == GAR_F32 ? 2 : 1);
    return static_cast<size_t>(std::max(std::max(p.loss, p.grad), int64_t{256}));
}

extern "C" int gar_vocab_loss(const void *x, int64_t ldx, const void *w, int64_t ldw, int32_t dtype, const int32_t *target,
                              const float *weight, int64_t rows, int64_t vocab, int64_t hidden, float *loss, float *lse,
                              void *d_workspace, size_t workspace_bytes, gar_stream_t stream_) {
    if (int rc = check(x, ldx, w, ldw, target, weight, rows, vocab, hidden, dtype)) return rc;
    if (rows == 0) return GAR_OK;
    const Plan how = plan_for(rows, vocab, hidden, 1);
    if (!loss || !lse || !d_workspace || workspace_bytes < static_cast<size_t>(how.loss))
        return fail(GAR_EINVAL, "loss, lse or the workspace is NULL, or the workspace below %lld bytes", static_cast<long long>(how.loss));
    if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(d_workspace, 256)) return fail(GAR_EALIGN, "loss, lse (4 bytes) or the workspace (256) is misaligned");
    VocabParams p{};
    p.rows = rows, p.vocab = vocab, p.hidden = hidden;
    p.target = target, p.weight = weight;
    p.tile_n = how.split.columns;
    p.tiles_m = ceil_div(rows, int64_t{kTile}), p.tiles_n = ceil_div(vocab, int64_t{p.tile_n});
    p.runs = how.split.runs, p.parts = 1, p.splits = 1, p.chunks = static_cast<int32_t>(ceil_div(hidden, int64_t{kK}));
    p.items = p.tiles_m * p.runs;
    p.stats = static_cast<float2 *>(d_workspace);
    p.at_target = reinterpret_cast<float *>(static_cast<uint8_t *>(d_workspace) + room(rows * how.split.runs * 16));
    p.status = device_status();
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const uint16_t *from = static_cast<const uint16_t *>(x);
    if (copy_pays(from, ldx, p)) {
        const auto live = reinterpret_cast<uint16_t *>(reinterpret_cast<uint8_t *>(p.at_target) + room(rows * 4));
        if (int rc = copy_live_rows(p, from, ldx, live, stream)) return rc;
        from = live, ldx = live_ld(hidden);
    }
    CUtensorMap a{}, b{};
    lay_out(&p, rows, false);
    if (int rc = encode(&a, from, hidden, rows, ldx, p.a_rows)) return rc;
    if (int rc = encode(&b, w, hidden, vocab, ldw, p.tile_n / 2)) return rc;
    if (int rc = launch_form<kLoss, float>(p, a, b, b, b, stream)) return rc;
    return launch_early("vocab_join_kernel", vocab_join_kernel, dim3(static_cast<unsigned>(ceil_div(rows, int64_t{8}))), 256, 0, 1, stream, p,
                        loss, lse);
}

namespace {
int vocab_grad(const void *x, int64_t ldx, const void *w, int64_t ldw, int32_t dtype, const int32_t *target, const float *weight,
               int64_t rows, int64_t vocab, int64_t hidden, const float *loss, const float *lse, void *dx, int64_t lddx, const void *addend,
               int64_t ld_addend, void *dw, int64_t lddw, int32_t dw_type, int32_t parts, void *d_workspace, size_t workspace_bytes,
               gar_stream_t stream_) {
    if (int rc = check(x, ldx, w, ldw, target, weight, rows, vocab, hidden, dtype)) return rc;
    const int size = elem_bytes(dw_type);
    if (size < 0) return fail(GAR_EDTYPE, "unknown dtype %d of dw", dw_type);
    if (!dx && !dw) return fail(GAR_EINVAL, "dx and dw are NULL");
    if ((dx && dx == x) || (dw && dw == w)) return fail(GAR_EINVAL, "dx in place of x, or dw in place of w");
    if (addend && !dw) return fail(GAR_EINVAL, "an addend without dw");
    if (dw && (lddw < hidden || (addend && ld_addend < hidden))) return fail(GAR_EINVAL, "a row stride of dw or its addend is below the hidden size");
    if (addend == dw && dw && ld_addend != lddw) return fail(GAR_EINVAL, "an addend in place of dw needs the same row stride");
    if (!aligned(dw, size) || !aligned(addend, size)) return fail(GAR_EALIGN, "dw or its addend is misaligned");
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (rows == 0) {
        if (!dw || (addend == dw)) return GAR_OK;
        const unsigned blocks = static_cast<unsigned>(std::min(ceil_div(vocab * hidden, int64_t{1024}), static_cast<int64_t>(sm_count()) * 8));
        return dw_type == GAR_F32
                   ? launch_early("vocab_no_rows_kernel", vocab_no_rows_kernel<float>, dim3(blocks), 256, 0, 1, stream,
                                  static_cast<const float *>(addend), ld_addend, static_cast<float *>(dw), lddw, vocab, hidden)
                   : launch_early("vocab_no_rows_kernel", vocab_no_rows_kernel<uint16_t>, dim3(blocks), 256, 0, 1, stream,
                                  static_cast<const uint16_t *>(addend), ld_addend, static_cast<uint16_t *>(dw), lddw, vocab, hidden);
    }
    if (dx && lddx < hidden) return fail(GAR_EINVAL, "the row stride of dx is below the hidden size");
    const Plan how = plan_for(rows, vocab, hidden, dw_type == GAR_F32 || parts == 2 ? 2 : 1);
    if (!lse || !d_workspace || workspace_bytes < static_cast<size_t>(how.grad))
        return fail(GAR_EINVAL, "lse or the workspace is NULL, or the workspace below %lld bytes", static_cast<long long>(how.grad));
    if (!aligned(dx, 2) || !aligned(lse, 4) || !aligned(d_workspace, 256)) return fail(GAR_EALIGN, "dx, lse or the workspace (256 bytes) is misaligned");
    VocabParams p{};
    p.rows = rows, p.vocab = vocab, p.hidden = hidden;
    p.target = target, p.weight = weight, p.loss = loss, p.lse = lse;
    p.status = device_status();
    const uint16_t *xh = static_cast<const uint16_t *>(x), *wh = static_cast<const uint16_t *>(w);
    uint16_t *dxh = static_cast<uint16_t *>(dx);
    uint8_t *ws = static_cast<uint8_t *>(d_workspace);
    return dw_type == GAR_F32 ? gradient<float>(p, how, xh, ldx, wh, ldw, dxh, lddx, static_cast<const float *>(addend), ld_addend,
                                                static_cast<float *>(dw), lddw, parts, ws, stream)
                              : gradient<uint16_t>(p, how, xh, ldx, wh, ldw, dxh, lddx, static_cast<const uint16_t *>(addend), ld_addend,
                                                   static_cast<uint16_t *>(dw), lddw, parts, ws, stream);
}
}  // namespace

extern "C" int gar_vocab_grad(const void *x, int64_t ldx, const void *w, int64_t ldw, int32_t dtype, const int32_t *target,
                              const float *weight, int64_t rows, int64_t vocab, int64_t hidden, const float *lse, void *dx, int64_t lddx,
                              const void *addend, int64_t ld_addend, void *dw, int64_t lddw, int32_t dw_type, void *d_workspace,
                              size_t workspace_bytes, gar_stream_t stream) {
    return vocab_grad(x, ldx, w, ldw, dtype, target, weight, rows, vocab, hidden, nullptr, lse, dx, lddx, addend, ld_addend, dw, lddw,
                      dw_type, 0, d_workspace, workspace_bytes, stream);
}

extern "C" int gar_vocab_grad_with_loss(const void *x, int64_t ldx, const void *w, int64_t ldw, int32_t dtype, const int32_t *target,
                                        const float *weight, int64_t rows, int64_t vocab, int64_t hidden, const float *loss,
                                        const float *lse, void *dx, int64_t lddx, const void *addend, int64_t ld_addend, void *dw,
                                        int64_t lddw, int32_t dw_type, int32_t parts, void *d_workspace, size_t workspace_bytes,
                                        gar_stream_t stream) {
    if (parts < 0 || parts > 2 || (parts == 1 && dw && dw_type == GAR_F32))
        return fail(GAR_EINVAL, "parts=%d: 0, 1 (not of an fp32 dw) or 2", parts);
    if (rows > 0 && !loss) return fail(GAR_EINVAL, "loss is NULL");
    if (!aligned(loss, 4)) return fail(GAR_EALIGN, "loss is misaligned");
    return vocab_grad(x, ldx, w, ldw, dtype, target, weight, rows, vocab, hidden, loss, lse, dx, lddx, addend, ld_addend, dw, lddw,
                      dw_type, parts, d_workspace, workspace_bytes, stream);
}
