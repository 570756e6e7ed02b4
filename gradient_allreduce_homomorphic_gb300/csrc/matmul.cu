// matmul.cu -- matrix product of block-scaled 8-bit operands: gar_fp8_matmul.
//
//   D[m][n] = C[m][n] + sum over blocks j of 128 k:
//             2^(sa[m][j] - 127 + sb[n][j] - 127) sum_{k in block j} a[m][k] b[n][k]
//
// on the tensor cores (tcgen05, kind mxf8f6f4: 8-bit operands, power-of-two
// scales applied by the hardware, fp32 accumulators in tensor memory).  The
// hardware's scale covers 32 k; the four 32-k steps of a block take the same
// byte of a row's scale word, and a word's four bytes serve 512 k, so one
// 16-byte-per-lane copy of scales to tensor memory feeds 16 products.
//
// The tile is held transposed: its 128 tensor-memory lanes are columns n of D
// and its columns are rows m, so that a warp's store of one accumulator
// column is 32 consecutive elements of a row of D -- full sectors for any row
// stride and alignment, with no staging -- and few rows of D (a few tokens)
// make a narrow tile (kTM = 32) rather than an empty one.
//
// Warp roles of a CTA: warp 0 loads operand tiles by TMA (128-byte swizzle,
// zero fill past the edges), warp 1 issues scale copies and products, warp 2
// lays the scales out in shared memory, warps 4-7 read the accumulators and
// store.  A grid with fewer tiles than SMs splits k over a cluster of up to 8
// CTAs, whose partial tiles are added through distributed shared memory in
// rank order, so the result does not depend on timing.  Bound by latency (a
// chunk's loads and products follow one another): 16 x 1024 x 2048 8 us and 1003
// x 333 x 1000 to fp32 9 us a call, one after another.
#include <algorithm>
#include <atomic>

#include "fp8.cuh"
#include "launch.cuh"
#include "tensorcore.cuh"
#include "tensormap.cuh"

namespace gar {
namespace {

constexpr int kTN = 128;     // tile rows in tensor memory: columns of D
constexpr int kKC = 128;     // k per chunk: one scale block, one swizzled line
constexpr int kThreads = 256;
// Chunks that an accumulator adds at most, for an fp32 result: the tensor core's additions round toward zero, so its error
// grows with the number of k (measured against 64 bits, of the result: 2.6e-7 at 2048, 8e-7 at 8192 for values of mean 0;
// 1.7e-6 at 8192, 7e-6 at 40000 for values with a mean, whose sums grow all along).
constexpr int kSegment = 64;
constexpr int kScaleBufs = 4;   // of scale words, one for each 512 k, in shared memory; tensor memory has two

struct MatmulParams {
    const uint32_t *sa, *sb;  // scale words [ceil(K / 512)][rows]
    int64_t M, N;
    int32_t chunks;           // of 128 k
    uint32_t idesc;
    void *d;
    const void *c;
    int64_t ldd, ldc;
    int32_t tiles_n;
    int32_t splits;           // CTAs of a cluster along k
    unsigned int *status;
};

template <int TM>
struct Shape {
    static constexpr int kBytesA = kTN * kKC;  // D's columns: the operand b
    static constexpr int kBytesB = TM * kKC;
    static constexpr int kStage = kBytesA + kBytesB;
    static constexpr int kResident = TM == 128 ? 1 : 2;  // CTAs an SM has shared memory for
    static constexpr int kStages = TM == 128 ? 6 : TM == 64 ? 4 : 5;
    static constexpr int kScaleBuf = 512 * 2;            // 128 rows of each operand
    static constexpr int kColumns = TM == 128 ? 256 : TM == 64 ? 128 : 64;
    static constexpr int kSmem = 1024 + kStages * kStage + kScaleBufs * kScaleBuf;
};

// 32 accumulator columns to rows m .. of column n of D, c added where given.
template <typename T>
__device__ __forceinline__ void store32(const float (&v)[32], T *d, int64_t ldd, const T *c, int64_t ldc, int count) {
    if (c) {
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = j < count ? load_f32(c + j * ldc) : 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < count) store_f32(d + j * ldd, v[j] + x[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (j < count) store_f32(d + j * ldd, v[j]);
    }
}

// The sum of kSplits CTAs' partial tiles [m][128], in rank order, to rows m .. of
// D: this CTA's share of the tile's `rows` rows.  A thread has 32 loads of
// distributed shared memory under way.
template <int kSplits, typename T>
__device__ __forceinline__ void add_partials(const MatmulParams &p, uint32_t base, int rank, int64_t m0, int64_t n0, int rows) {
    constexpr int kRows = 8 / kSplits;  // of a warp at a time
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t from[kSplits];
#pragma unroll
    for (int r = 0; r < kSplits; ++r) from[r] = cluster_map(base, r) + lane * 4;
    T *d = static_cast<T *>(p.d) + m0 * p.ldd + n0 + lane;
    const T *c = static_cast<const T *>(p.c) + m0 * p.ldc + n0 + lane;
    for (int j0 = (rank * (kThreads / 32) + warp) * kRows; j0 < rows; j0 += kSplits * (kThreads / 32) * kRows) {
        float v[kRows][4][kSplits];
#pragma unroll
        for (int j = 0; j < kRows; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < kSplits; ++r)  // past the last row it reads what it will not use
                    v[j][i][r] = cluster_load(from[r] + ((j0 + j < rows ? j0 + j : 0) * kTN + 32 * i) * 4);
#pragma unroll
        for (int j = 0; j < kRows; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x = v[j][i][0];
#pragma unroll
                for (int r = 1; r < kSplits; ++r) x += v[j][i][r];
                if (j0 + j < rows && n0 + lane + 32 * i < p.N) {
                    if (p.c) x += load_f32(c + (j0 + j) * p.ldc + 32 * i);
                    store_f32(d + (j0 + j) * p.ldd + 32 * i, x);
                }
            }
    }
}

// The scale words of 128 rows r0 .. of a matrix (its words of one group of four
// blocks at src) to the order that the copy to tensor memory takes, by one warp;
// zero (2^-127, of rows of zeros) past the last row.
__device__ __forceinline__ void copy_scales_async(uint32_t dst, const uint32_t *src, int64_t r0, int64_t rows, int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int64_t r = r0 + 32 * q + lane;
        copy4_async(dst + lane * 16 + q * 4, src + (r < rows ? r : 0), r < rows);
    }
}

// After a wait ran out: the copies into the last `issued` stages before stage
// s (of the pass whose empty parity is turn) have to land before the CTA ends.
__device__ __noinline__ void mbar_drain(uint32_t full, uint32_t stages, int issued, uint32_t s, uint32_t turn) {
    for (; issued > 0; --issued) {
        if (s == 0) s = stages, turn ^= 1;
        --s;
        int given_up = 0;
        mbar_wait(full + 8 * s, turn ^ 1, &given_up);
    }
}

// All products that the issuing warp sent off are done: tensor memory may be
// given back.  A wait of its own limit, for a wait that ran out elsewhere lets all
// others of the CTA pass.
__device__ __forceinline__ void products_done(uint32_t bar) {
    int given_up = 0;
    mbar_wait(bar, 0, &given_up);
}

template <typename T, int TM>
__global__ void __launch_bounds__(kThreads) matmul_kernel(const __grid_constant__ CUtensorMap map_n,
                                                          const __grid_constant__ CUtensorMap map_m,
                                                          const __grid_constant__ MatmulParams p) {
    using S = Shape<TM>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * S::kStages + 2 * kScaleBufs + 1];
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t scales = base + S::kStages * S::kStage;
    const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages, sf_full = empty + 8 * S::kStages,
                   sf_empty = sf_full + 8 * kScaleBufs, done = sf_empty + 8 * kScaleBufs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x % p.splits);
    const int64_t tile = blockIdx.x / p.splits;
    const int64_t n0 = (tile % p.tiles_n) * kTN, m0 = (tile / p.tiles_n) * TM;
    const int c0 = static_cast<int>(static_cast<int64_t>(p.chunks) * rank / p.splits);
    const int c1 = static_cast<int>(static_cast<int64_t>(p.chunks) * (rank + 1) / p.splits);

    let_next_begin();
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * S::kStages + 2 * kScaleBufs + 1; ++i)
            mbar_init(full + 8 * i, i >= 2 * S::kStages && i < 2 * S::kStages + kScaleBufs ? 32 : 1);  // sf_full: a warp's copies
        failed = 0;
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc<1>(smem_u32(&tmem_slot), S::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    after_previous();
    const uint32_t tmem = tmem_slot;
    const uint32_t sf_cols = tmem + TM;  // scale columns: kScaleBufs x (4 + 4)

    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&map_n);
        tma_prefetch_map(&map_m);
        uint32_t s = 0, turn = 1;  // the first turn finds every stage free
        int issued = 0;
        bool ok = true;
        for (int c = c0; c < c1; ++c) {
            if (!(ok = mbar_wait(empty + 8 * s, turn, &failed))) break;
            const uint32_t dst = base + s * S::kStage;
            mbar_expect_tx(full + 8 * s, S::kStage);
            tma_load_2d(dst, &map_n, full + 8 * s, c * kKC, static_cast<int32_t>(n0));
            tma_load_2d(dst + S::kBytesA, &map_m, full + 8 * s, c * kKC, static_cast<int32_t>(m0));
            issued = issued < S::kStages ? issued + 1 : S::kStages;
            if (++s == S::kStages) s = 0, turn ^= 1;
        }
        if (!ok) mbar_drain(full, S::kStages, issued, s, turn);
    } else if (warp == 1) {
        const uint64_t desc = smem_desc(base, 16, 1024, 2);
        uint32_t s = 0, turn = 0, groups = 0, g = 0;
        for (int c = c0; c < c1; ++c) {
            if (c == c0 || (c & 3) == 0) {
                g = groups++;
                const uint32_t b = g % kScaleBufs;
                mbar_wait(sf_full + 8 * b, (g / kScaleBufs) & 1, &failed);
                fence_async_shared();
                if (elect_one())
                    for (int a = 0; a < 2; ++a) tc_copy_scales<1>(sf_cols + (2 * b + a) * 4, scales + b * S::kScaleBuf + 512 * a);
                __syncwarp();
            }
            mbar_wait(full + 8 * s, turn, &failed);
            tc_fence_after();
            if (elect_one()) {
                const uint64_t d = desc + s * (S::kStage >> 4);
                const uint32_t col = sf_cols + (g % kScaleBufs) * 8;
                const uint32_t idesc = p.idesc | mxf8_scale_byte(c & 3);
#pragma unroll
                for (int k = 0; k < kKC / 32; ++k)
                    tc_mma_mxf8<1>(tmem, d + 2 * k, d + (S::kBytesA >> 4) + 2 * k, idesc, col, col + 4, c > c0 || k > 0);
                tc_commit<1>(empty + 8 * s);
                if ((c & 3) == 3 || c == c1 - 1) tc_commit<1>(sf_empty + 8 * (g % kScaleBufs));
            }
            __syncwarp();
            if (++s == S::kStages) s = 0, turn ^= 1;
        }
        if (elect_one()) tc_commit<1>(done);
        __syncwarp();
        products_done(done);
    } else if (warp == 2) {
        const int j0 = c0 >> 2, groups = c0 < c1 ? ((c1 - 1) >> 2) - j0 + 1 : 0;
        for (int g = 0; g < groups; ++g) {
            const uint32_t b = g % kScaleBufs, dst = scales + b * S::kScaleBuf;
            mbar_wait(sf_empty + 8 * b, (g / kScaleBufs + 1) & 1, &failed);
            copy_scales_async(dst, p.sb + static_cast<int64_t>(j0 + g) * p.N, n0, p.N, lane);
            copy_scales_async(dst + 512, p.sa + static_cast<int64_t>(j0 + g) * p.M, m0, p.M, lane);
            copy_async_arrive(sf_full + 8 * b);
        }
        copy_async_wait();
    }
    if (warp >= 4) {
        mbar_wait(done, 0, &failed);
        tc_fence_after();
    }
    __syncwarp();
    const int quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int64_t n = n0 + quarter * 32 + lane;
    const int rows = static_cast<int>(p.M - m0 < TM ? p.M - m0 : TM);
    if (warp >= 4) {
#pragma unroll 1
        for (int j0 = 0; j0 < rows; j0 += 32) {
            float v[32];
            tc_load32(v, lanes + j0);
            tc_wait_ld();
            if (c0 == c1)
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0.0f;
            if (p.splits > 1) {  // every copy into the stages has been used: they hold the partial tile [m][n] now
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((j0 + j) * kTN + quarter * 32 + lane) * 4), "f"(v[j]) : "memory");
            } else if (n < p.N) {
                T *d = static_cast<T *>(p.d) + (m0 + j0) * p.ldd + n;
                const T *c = p.c ? static_cast<const T *>(p.c) + (m0 + j0) * p.ldc + n : nullptr;
                store32<T>(v, d, p.ldd, c, p.ldc, rows - j0 < 32 ? rows - j0 : 32);
            }
        }
    }
    if (p.splits > 1) {
        __syncwarp();
        cluster_barrier();
        if (p.splits == 2) add_partials<2, T>(p, base, rank, m0, n0, rows);
        if (p.splits == 4) add_partials<4, T>(p, base, rank, m0, n0, rows);
        if (p.splits == 8) add_partials<8, T>(p, base, rank, m0, n0, rows);
        cluster_barrier();  // no CTA leaves while another reads its shared memory
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && failed && p.status) atomicOr(p.status, static_cast<unsigned int>(GAR_STATUS_TIMEOUT));
    if (warp == 1) tmem_free<1>(tmem, S::kColumns);
}

// ---------------------------------------------------------------- CTA pairs
// Large products: persistent pairs of CTAs (cta_group::2), each pair computing
// tiles of 256 columns by TM rows of D.  A CTA holds 128 of the tile's columns
// (its tensor-memory lanes) and loads, besides its own 128 rows of b, half of
// the tile's TM rows of a, which both tensor cores then share: at TM = 256,
// 32 KB of operands per CTA and 128 k instead of 48, so shared memory is
// written and read at 64 bytes a clock each rather than 96.
//
// Two accumulators alternate, so the epilogue of a tile overlaps the products
// of the next.  Tensor memory has 512 columns and the scales take 24 of them:
// up to TM = 224 the accumulators lie side by side; at TM = 256 they overlap
// by 32 columns (0..255 and 224..479), which the epilogue reads first and then
// lets the next tile's products start.  TM is chosen so that the tiles fill
// the SMs' last wave (pair_rows below).
//
// With an fp32 result, k is cut into segments of at most kSegment chunks, whose
// sums are added in fp32.
//
// Bound by the tensor cores at the clock that the power limit leaves them:
// 16384 x 4096 x 8192 to fp32 325 us, 3380 TFLOP/s (tensor pipe active in 85 %
// of the cycles, SM clock 1.70 GHz of 2.07), with an fp32 addend 348 us; 4096 x
// 8192 x 2048 to bf16 53 us, 2600 TFLOP/s (65 %: 16 chunks a tile leave its
// beginning and the kernel's, 5.8 us, in sight).
constexpr int kPairThreads = 384;  // warps 0-3 and 4-11 epilogue
constexpr int kPairStages = 6;
constexpr int kPairScaleBuf = 512 * 3;
constexpr int kPairScaleBufs = 8;
constexpr int kPairScaleCols = 480;

struct PairParams {
    MatmulParams mm;
    int64_t tiles_m, tiles;
    int32_t rows;  // TM
    int32_t segments, seg_chunks;
};

__host__ __device__ constexpr int pair_stage(int rows) { return (128 + rows / 2) * kKC; }
constexpr int pair_smem(int rows) { return 1024 + kPairStages * pair_stage(rows) + kPairScaleBufs * kPairScaleBuf; }

// Tiles in the order they are handed out: runs of 8 tiles of rows by all tiles
// of columns, so that the pairs working at one time share operands in L2.
__device__ __forceinline__ void pair_tile(const PairParams &p, int64_t t, int64_t &m0, int64_t &n0) {
    const int64_t per = 8 * static_cast<int64_t>(p.mm.tiles_n), g = t / per, in = t % per;
    const int64_t rows = p.tiles_m - g * 8 < 8 ? p.tiles_m - g * 8 : 8;
    m0 = (g * 8 + in % rows) * p.rows;
    n0 = in / rows * 256;
}

template <typename T>
__global__ void __launch_bounds__(kPairThreads, 1)
    matmul_pair_kernel(const __grid_constant__ CUtensorMap map_n, const __grid_constant__ CUtensorMap map_m,
                       const __grid_constant__ PairParams pp) {
    const MatmulParams &p = pp.mm;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[2 * kPairStages + 3 * kPairScaleBufs + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int failed;
    const uint32_t stage = pair_stage(pp.rows);
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t scales = base + kPairStages * stage;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kPairStages, sf_full = empty + 8 * kPairStages,
                   sf_empty = sf_full + 8 * kPairScaleBufs, acc_full = sf_empty + 8 * kPairScaleBufs,
                   drained = acc_full + 16, sf_here = drained + 16, done = sf_here + 8 * kPairScaleBufs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_cta_rank();
    const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
    const bool overlap = pp.rows == 256;
    const uint32_t acc1 = overlap ? 224 : pp.rows;

    let_next_begin();
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kPairStages; ++i) mbar_init(full + 8 * i, 1);
        for (int i = 0; i < kPairScaleBufs; ++i) {
            mbar_init(sf_here + 8 * i, 32);  // a warp's copies
            mbar_init(sf_full + 8 * i, 2);   // a word from each CTA
            mbar_init(sf_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(drained + 8 * i, 16);  // eight epilogue warps of each CTA
        }
        mbar_init(done, 1);
        failed = 0;
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc<2>(smem_u32(&tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    cluster_barrier();
    tc_fence_after();
    after_previous();
    const uint32_t tmem = tmem_slot;

    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&map_n);
        tma_prefetch_map(&map_m);
        const uint32_t lead_full = cluster_map(full, 0);
        uint32_t s = 0, turn = 1;  // the first turn finds every stage free
        int issued = 0;
        bool ok = true;
        for (int64_t t = first; t < pp.tiles && ok; t += step) {
            int64_t m0, n0;
            pair_tile(pp, t, m0, n0);
            const int32_t yn = static_cast<int32_t>(n0 + 128 * rank), ym = static_cast<int32_t>(m0 + pp.rows / 2 * rank);
            for (int c = 0; c < p.chunks; ++c) {
                if (!(ok = mbar_wait(empty + 8 * s, turn, &failed))) break;
                const uint32_t dst = base + s * stage;
                if (rank == 0) mbar_expect_tx(full + 8 * s, 2 * stage);
                tma_load_2d_pair(dst, &map_n, lead_full + 8 * s, c * kKC, yn);
                tma_load_2d_pair(dst + 128 * kKC, &map_m, lead_full + 8 * s, c * kKC, ym);
                issued = issued < kPairStages ? issued + 1 : kPairStages;
                if (++s == kPairStages) s = 0, turn ^= 1;
            }
        }
        // both CTAs' copies count on the first one's barriers; the other waits at the cluster barrier below
        if (!ok && rank == 0) mbar_drain(full, kPairStages, issued, s, turn);
    } else if (warp == 1 && rank == 0) {
        // Issue of scale copies and products, by one thread: the tensor core takes them in the order of issue, so a
        // copy needs no barrier before the products that use it.  The thread's time per chunk must stay below the
        // products' (512 clocks at TM = 256) and a look at an mbarrier takes about a hundred, so what comes next is
        // looked at before the present products are issued, and waited for only if it was not there.
        uint64_t d = smem_desc(base, 16, 1024, 2);
        const uint64_t d_step = stage >> 4;
        uint32_t s = 0, turn = 0, seq = 0, g = 0;
        const uint32_t lag = overlap ? 1 : 2;
        bool ready = false, sf_ready = false;
        for (int64_t t = first; t < pp.tiles; t += step) {
            for (int c0 = 0; c0 < p.chunks; c0 += pp.seg_chunks, ++seq) {
                const int c1 = min(p.chunks, c0 + pp.seg_chunks);
                const uint32_t acc = tmem + (seq & 1 ? acc1 : 0);
                if (seq >= lag) mbar_wait_cluster(drained + 8 * ((seq - lag) & 1), ((seq - lag) >> 1) & 1, &failed);
                for (int c = c0; c < c1; ++c) {
                    const bool first_of_word = (c & 3) == 0, last_of_word = (c & 3) == 3 || c == p.chunks - 1;
                    const uint32_t col = tmem + kPairScaleCols + (g & 1) * 12;
                    if (first_of_word && !sf_ready) {
                        // scale group g: shared buffer g % 8, tensor-memory buffer g % 2, free once group g - 2 is done
                        mbar_wait_cluster(sf_full + 8 * (g % kPairScaleBufs), (g / kPairScaleBufs) & 1, &failed);
                        if (g >= 2) mbar_wait(sf_empty + 8 * ((g - 2) % kPairScaleBufs), ((g - 2) / kPairScaleBufs) & 1, &failed);
                    }
                    if (!ready) mbar_wait(full + 8 * s, turn, &failed);
                    tc_fence_after();
                    const uint32_t next = s + 1 == kPairStages ? 0 : s + 1;
                    ready = mbar_test(full + 8 * next, next ? turn : turn ^ 1);
                    if (last_of_word) {
                        const uint32_t n = g + 1;
                        sf_ready = mbar_test_cluster(sf_full + 8 * (n % kPairScaleBufs), (n / kPairScaleBufs) & 1) &
                                   (n < 2 || mbar_test(sf_empty + 8 * ((n - 2) % kPairScaleBufs), ((n - 2) / kPairScaleBufs) & 1));
                    }
                    if (elect_one()) {
                        if (first_of_word)
                            for (int a = 0; a < 3; ++a)
                                tc_copy_scales<2>(col + 4 * a, scales + (g % kPairScaleBufs) * kPairScaleBuf + 512 * a);
                        const uint32_t idesc = p.idesc | mxf8_scale_byte(c & 3);
#pragma unroll
                        for (int k = 0; k < kKC / 32; ++k)
                            tc_mma_mxf8<2>(acc, d + 2 * k, d + ((128 * kKC) >> 4) + 2 * k, idesc, col, col + 4, c > c0 || k > 0);
                        tc_commit_pair(empty + 8 * s);
                        if (last_of_word) tc_commit_pair(sf_empty + 8 * (g % kPairScaleBufs));
                        if (c == c1 - 1) tc_commit_pair(acc_full + 8 * (seq & 1));
                    }
                    __syncwarp();
                    g += last_of_word;
                    s = next;
                    if (s == 0) turn ^= 1, d = smem_desc(base, 16, 1024, 2);
                    else d += d_step;
                }
            }
        }
        if (elect_one()) tc_commit<2>(done);  // here alone: the other CTA frees its half behind the cluster barrier below
        __syncwarp();
        products_done(done);
    } else if (warp == 2) {
        const int words = (p.chunks + 3) >> 2;
        uint32_t g = 0;
        for (int64_t t = first; t < pp.tiles; t += step) {
            int64_t m0, n0;
            pair_tile(pp, t, m0, n0);
            for (int j = 0; j < words; ++j, ++g) {
                const uint32_t b = g % kPairScaleBufs, dst = scales + b * kPairScaleBuf;
                const uint32_t *sn = p.sb + static_cast<int64_t>(j) * p.N, *sm = p.sa + static_cast<int64_t>(j) * p.M;
                mbar_wait(sf_empty + 8 * b, (g / kPairScaleBufs + 1) & 1, &failed);
                copy_scales_async(dst, sn, n0 + 128 * rank, p.N, lane);
                copy_scales_async(dst + 512, sm, m0, p.M, lane);
                copy_scales_async(dst + 1024, sm, m0 + 128, p.M, lane);
                copy_async_arrive(sf_here + 8 * b);
            }
        }
        copy_async_wait();
    } else if (warp == 3) {
        // Passes on to the pair's first CTA that a group of scales is here.  Not the copying warp's work: a release to
        // the cluster waits for the thread's own copies under way.
        const uint32_t lead_sf = cluster_map(sf_full, 0);
        const uint32_t words = (p.chunks + 3) >> 2;
        uint32_t g = 0;
        for (int64_t t = first; t < pp.tiles; t += step)
            for (uint32_t j = 0; j < words; ++j, ++g) {
                const uint32_t b = g % kPairScaleBufs;
                mbar_wait(sf_here + 8 * b, (g / kPairScaleBufs) & 1, &failed);
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(lead_sf + 8 * b);
            }
    } else if (warp >= 4) {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t lead_drained = cluster_map(drained, 0);
        const int batches = pp.rows / 32;
        uint32_t seq = 0;
        for (int64_t t = first; t < pp.tiles; t += step) {
            int64_t m0, n0;
            pair_tile(pp, t, m0, n0);
            const int64_t n = n0 + 128 * rank + quarter * 32 + lane, mleft = p.M - m0;
            for (int seg = 0; seg < pp.segments; ++seg, ++seq) {
                const uint32_t buf = seq & 1;
                mbar_wait(acc_full + 8 * buf, (seq >> 1) & 1, &failed);
                __syncwarp();
                tc_fence_after();
                // The halves take alternate batches of 32 columns.  Where the accumulators overlap, the half that
                // holds the shared batch (7 of buffer 0, 0 of buffer 1) starts with it and the other has none.
                const int start = overlap && buf == 0 && half == 1 ? 7 : half;
                bool told = overlap && half == static_cast<int>(buf);
                if (told) {
                    tc_fence_before();
                    if (lane == 0) mbar_arrive_cluster(lead_drained + 8 * buf);
                }
#pragma unroll 1
                for (int i = half; i < batches; i += 2) {
                    int j = start == half ? i : (i == half ? 7 : i - 2);
                    float v[32];
                    tc_load32(v, lanes + (buf ? acc1 : 0) + j * 32);
                    tc_wait_ld();
                    if (!told && (overlap || i + 2 >= batches)) {
                        told = true;
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(lead_drained + 8 * buf);
                    }
                    const int64_t m = m0 + j * 32;
                    const int64_t left = mleft - j * 32;
                    if (n >= p.N || left <= 0) continue;
                    T *d = static_cast<T *>(p.d) + m * p.ldd + n;
                    const T *c = seg > 0 ? d : p.c ? static_cast<const T *>(p.c) + m * p.ldc + n : nullptr;
                    const int64_t ldc = seg > 0 ? p.ldd : p.ldc;
                    store32<T>(v, d, p.ldd, c, ldc, left < 32 ? static_cast<int>(left) : 32);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_barrier();
    if (threadIdx.x == 0 && failed && p.status) atomicOr(p.status, static_cast<unsigned int>(GAR_STATUS_TIMEOUT));
    if (warp == 1) tmem_free<2>(tmem, 512);
}

// Map of the codes [rows, K] (row stride ld bytes) in boxes of `box` rows x 128 bytes.
int encode(CUtensorMap *map, const uint8_t *q, int64_t rows, int64_t K, int64_t ld, int box) {
    return encode_tile_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, K, rows, ld, kKC, box);
}

// Clusters of `splits` CTAs that the device holds at one time (its SMs come in
// groups, so it is fewer than its SMs would make; one more would run after all
// others); looked up once.  < 1: an error, reported.
template <typename T, int TM>
int resident_clusters(int splits) {
    using S = Shape<TM>;
    static std::atomic<int> known[64][4];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(GAR_ECUDA, "no current device");
    std::atomic<int> &slot = known[dev & 63][splits == 8 ? 3 : splits / 2];
    int n = slot.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(static_cast<unsigned>(splits));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = S::kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cudaError_t e = cudaFuncSetAttribute(matmul_kernel<T, TM>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, matmul_kernel<T, TM>, &cfg);
        if (e != cudaSuccess || n < 1) return fail(GAR_ECUDA, "matmul_kernel: %s", cudaGetErrorString(e));
        slot.store(n, std::memory_order_relaxed);
    }
    return n;
}

// A product by CTAs of TM rows: its tiles, the CTAs that split k of each and
// what it takes, in ns, by measurements at M of 16 to 2048, N of 128 to 4096
// and K of 512 to 8192: 3.9 us, 0.33 for a chunk, 1.4 for the exchange of
// partial tiles, and a wave more as often as the CTAs exceed the SMs.  So k is
// split from 12 chunks on, down to four a CTA, as far as all clusters run at
// one time.  Segments (kSegment) are launches of their own, each of which adds
// to the one before's result.
struct Plan {
    int64_t tiles, ns;
    int splits, segments;
};
template <typename T, int TM>
int plan(const MatmulParams &p, Plan *out) {
    out->tiles = ceil_div(p.N, int64_t{kTN}) * ceil_div(p.M, int64_t{TM});
    out->splits = 1;
    int resident = resident_clusters<T, TM>(1);
    if (resident < 1) return resident;
    const int64_t waves = ceil_div(out->tiles, int64_t{resident});
    for (int splits = 2; p.chunks >= 12 && splits <= 8 && p.chunks >= 4 * splits; splits *= 2) {
        const int n = resident_clusters<T, TM>(splits);
        if (n < 1) return n;
        if (out->tiles <= n / Shape<TM>::kResident) out->splits = splits;
    }
    out->segments = sizeof(T) == 2 ? 1 : static_cast<int>(std::max(ceil_div(p.chunks, int64_t{out->splits} * kSegment), int64_t{1}));
    out->ns = out->segments * (3900 + (out->splits > 1 ? 1400 : 0)) + 330 * ceil_div(p.chunks, int64_t{out->splits}) +
              (waves - 1) * (1500 * out->segments + 330 * p.chunks);
    return GAR_OK;
}

// Chunks of each of at most `segments` segments: whole scale words, four chunks each.
int32_t segment_chunks(int32_t chunks, int32_t segments) {
    return static_cast<int32_t>(std::max(ceil_div(ceil_div(chunks, segments), 4) * 4, int64_t{4}));
}

template <typename T, int TM>
int launch(MatmulParams &p, const Plan &how, const uint8_t *a, int64_t lda, const uint8_t *b, int64_t ldb, int64_t K, cudaStream_t stream) {
    using S = Shape<TM>;
    p.tiles_n = static_cast<int32_t>(ceil_div(p.N, int64_t{kTN}));
    p.splits = how.splits;
    if (how.tiles * how.splits > 0x7FFFFFFF) return fail(GAR_EINVAL, "the product has too many tiles");
    p.idesc = p.idesc | mxf8_idesc(0, 0, kTN, TM);
    const int32_t chunks = p.chunks, step = segment_chunks(chunks, how.segments);
    const uint32_t *const sa = p.sa, *const sb = p.sb;
    for (int32_t c0 = 0; c0 == 0 || c0 < chunks; c0 += step) {
        p.chunks = std::min(step, chunks - c0);
        p.sa = sa + p.M * (c0 / 4), p.sb = sb + p.N * (c0 / 4);
        if (c0 > 0) p.c = p.d, p.ldc = p.ldd;
        CUtensorMap map_n{}, map_m{};
        if (K > 0) {
            const int64_t k0 = int64_t{kKC} * c0, k = std::min(int64_t{kKC} * p.chunks, K - k0);
            if (int rc = encode(&map_n, b + k0, p.N, k, ldb, kTN)) return rc;
            if (int rc = encode(&map_m, a + k0, p.M, k, lda, TM)) return rc;
        }
        if (int rc = launch_early("matmul_kernel", matmul_kernel<T, TM>, dim3(static_cast<unsigned>(how.tiles * how.splits)), kThreads,
                                  S::kSmem, static_cast<unsigned>(p.splits), stream, map_n, map_m, p))
            return rc;
    }
    return GAR_OK;
}

// The rows of a pair's tiles: the count that finishes soonest.  In clocks, as
// measured at K = 2048 and 8192 for 192, 224 and 256 rows: a chunk of 128 k
// takes 2 TM + 28, but no less than the issuing thread's 516; a tile begins 500
// after its predecessor's last chunk, 2600 where the accumulators overlap.
int64_t pair_clocks(int rows, int64_t M, int64_t tiles_n, int64_t chunks, int pairs) {
    const int64_t waves = ceil_div(ceil_div(M, int64_t{rows}) * tiles_n, int64_t{pairs});
    return waves * (chunks * std::max(2 * rows + 28, 516) + (rows == 256 ? 2600 : 500));
}
int pair_rows(int64_t M, int64_t tiles_n, int64_t chunks, int pairs) {
    int best = 256;
    for (int rows = 224; rows >= 128; rows -= 32)
        if (pair_clocks(rows, M, tiles_n, chunks, pairs) < pair_clocks(best, M, tiles_n, chunks, pairs)) best = rows;
    return best;
}

template <typename T>
int resident_pairs() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(GAR_ECUDA, "no current device");
    int pairs = known[dev & 63].load(std::memory_order_relaxed);
    if (pairs == 0) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kPairThreads);
        cfg.dynamicSmemBytes = pair_smem(256);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cudaError_t e = cudaFuncSetAttribute(matmul_pair_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, pair_smem(256));
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&pairs, matmul_pair_kernel<T>, &cfg);
        if (e != cudaSuccess || pairs < 1) return fail(GAR_ECUDA, "matmul_pair_kernel: %s", cudaGetErrorString(e));
        known[dev & 63].store(pairs, std::memory_order_relaxed);
    }
    return pairs;
}

template <typename T>
int launch_pair(MatmulParams &mm, int pairs, const uint8_t *a, int64_t lda, const uint8_t *b, int64_t ldb, int64_t K,
                cudaStream_t stream) {
    PairParams p{};
    mm.tiles_n = static_cast<int32_t>(ceil_div(mm.N, int64_t{256}));
    p.rows = pair_rows(mm.M, mm.tiles_n, mm.chunks, pairs);
    mm.idesc |= mxf8_idesc(0, 0, 256, static_cast<uint32_t>(p.rows));
    p.mm = mm;
    p.tiles_m = ceil_div(mm.M, int64_t{p.rows});
    p.tiles = p.tiles_m * mm.tiles_n;
    p.segments = sizeof(T) == 2 ? 1 : static_cast<int32_t>(ceil_div(mm.chunks, kSegment));
    p.seg_chunks = segment_chunks(mm.chunks, p.segments);
    p.segments = static_cast<int32_t>(ceil_div(mm.chunks, p.seg_chunks));
    CUtensorMap map_n{}, map_m{};
    if (int rc = encode(&map_n, b, mm.N, K, ldb, 128)) return rc;
    if (int rc = encode(&map_m, a, mm.M, K, lda, p.rows / 2)) return rc;
    return launch_early("matmul_pair_kernel", matmul_pair_kernel<T>, dim3(2 * static_cast<unsigned>(p.tiles < pairs ? p.tiles : pairs)),
                        kPairThreads, pair_smem(p.rows), 2, stream, map_n, map_m, p);
}

// Small products by single CTAs, large ones by pairs: whichever the measurements
// behind plan() and pair_clocks() say is sooner done (a pair's kernel takes 5.8 us
// beside its tiles).
template <typename T, int TM>
int choose_for(MatmulParams &p, const uint8_t *a, int64_t lda, const uint8_t *b, int64_t ldb, int64_t K, cudaStream_t stream) {
    Plan how;
    if (int rc = plan<T, TM>(p, &how)) return rc;
    if (K > 0) {
        const int pairs = resident_pairs<T>();
        if (pairs < 1) return pairs;
        const int64_t tiles_n = ceil_div(p.N, int64_t{256});
        const int64_t clocks = pair_clocks(pair_rows(p.M, tiles_n, p.chunks, pairs), p.M, tiles_n, p.chunks, pairs);
        if (5800 + clocks * 10 / 19 < how.ns) return launch_pair<T>(p, pairs, a, lda, b, ldb, K, stream);
    }
    return launch<T, TM>(p, how, a, lda, b, ldb, K, stream);
}
template <typename T>
int choose(MatmulParams &p, const uint8_t *a, int64_t lda, const uint8_t *b, int64_t ldb, int64_t K, cudaStream_t stream) {
    if (p.M <= 32) return choose_for<T, 32>(p, a, lda, b, ldb, K, stream);
    if (p.M <= 64) return choose_for<T, 64>(p, a, lda, b, ldb, K, stream);
    return choose_for<T, 128>(p, a, lda, b, ldb, K, stream);
}

int check_operand(const char *name, const uint8_t *q, int64_t ld, int64_t K, const uint8_t *scale, int32_t format) {
    if (format != GAR_F8E4M3 && format != GAR_F8E5M2) return fail(GAR_EDTYPE, "%s: unknown 8-bit format %d", name, format);
    if (K == 0) return GAR_OK;
    if (!q || !scale) return fail(GAR_EINVAL, "%s: codes or scales are NULL", name);
    if (ld < K) return fail(GAR_EINVAL, "%s: row stride %lld < K", name, static_cast<long long>(ld));
    if (!aligned(q, 16) || ld % 16 || !aligned(scale, 4))
        return fail(GAR_EALIGN, "%s: codes and their row stride need 16-byte alignment, scales 4-byte", name);
    return GAR_OK;
}

}  // namespace
}  // namespace gar

using namespace gar;

extern "C" int gar_fp8_matmul(const uint8_t *a, int64_t lda, const uint8_t *a_scale, int32_t a_format, const uint8_t *b,
                              int64_t ldb, const uint8_t *b_scale, int32_t b_format, int64_t M, int64_t N, int64_t K,
                              const void *c, int64_t ldc, void *d, int64_t ldd, int32_t dtype, gar_stream_t stream_) {
    if (M < 0 || N < 0 || K < 0 || M > 0x7FFFFFFF || N > 0x7FFFFFFF || K > 0x7FFFFFFF - 1024)
        return fail(GAR_EINVAL, "M=%lld N=%lld K=%lld", static_cast<long long>(M), static_cast<long long>(N),
                    static_cast<long long>(K));
    if (elem_bytes(dtype) < 0) return fail(GAR_EDTYPE, "unknown dtype %d", dtype);
    if (int rc = check_operand("a", a, lda, M > 0 ? K : 0, a_scale, a_format)) return rc;
    if (int rc = check_operand("b", b, ldb, N > 0 ? K : 0, b_scale, b_format)) return rc;
    if (M == 0 || N == 0) return GAR_OK;
    if (!d || ldd < N || (c && ldc < N)) return fail(GAR_EINVAL, "d is NULL, or a row stride of d or c is below N");
    if (c == d && ldc != ldd) return fail(GAR_EINVAL, "c in place of d needs the same row stride");
    if (!aligned(d, elem_bytes(dtype)) || !aligned(c, elem_bytes(dtype))) return fail(GAR_EALIGN, "d or c is misaligned");
    MatmulParams p{};
    p.sa = reinterpret_cast<const uint32_t *>(a_scale), p.sb = reinterpret_cast<const uint32_t *>(b_scale);
    p.M = M, p.N = N, p.chunks = static_cast<int32_t>(ceil_div(K, int64_t{kKC}));
    p.idesc = mxf8_idesc(b_format == GAR_F8E5M2, a_format == GAR_F8E5M2, 0, 0);  // the tile is transposed
    p.d = d, p.ldd = ldd, p.c = c, p.ldc = ldc;
    p.status = device_status();
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    return dtype == GAR_BF16 ? choose<uint16_t>(p, a, lda, b, ldb, K, stream) : choose<float>(p, a, lda, b, ldb, K, stream);
}
