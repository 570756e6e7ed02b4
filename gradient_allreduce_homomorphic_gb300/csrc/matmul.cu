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
// rank order, so the result does not depend on timing.
#include <atomic>

#include "fp8.cuh"
#include "tensorcore.cuh"

namespace gar {
namespace {

constexpr int kTN = 128;     // tile rows in tensor memory: columns of D
constexpr int kKC = 128;     // k per chunk: one scale block, one swizzled line
constexpr int kThreads = 256;
constexpr int kScaleBufs = 2;

struct MatmulParams {
    const uint32_t *sa, *sb;  // scale words [ceil(K / 512)][rows]
    int64_t M, N;
    int32_t chunks;           // of 128 k
    uint32_t idesc;
    void *d;
    const void *c;
    int64_t ldd, ldc;
    int32_t bf16;
    int32_t tiles_n;
    int32_t splits;           // CTAs of a cluster along k
    unsigned int *status;
};

template <int TM>
struct Shape {
    static constexpr int kBytesA = kTN * kKC;  // D's columns: the operand b
    static constexpr int kBytesB = TM * kKC;
    static constexpr int kStage = kBytesA + kBytesB;
    static constexpr int kStages = TM == 256 ? 4 : TM == 128 ? 6 : 8;
    static constexpr int kAtomsB = TM > 128 ? 2 : 1;
    static constexpr int kScaleBuf = 512 * (1 + kAtomsB);
    static constexpr int kColumns = TM == 256 ? 512 : TM == 128 ? 256 : TM == 64 ? 128 : 64;
    static constexpr int kSmem = 1024 + kStages * kStage + kScaleBufs * kScaleBuf;
};

__device__ __forceinline__ float load_out(const MatmulParams &p, int64_t m, int64_t n) {
    const int64_t i = m * p.ldc + n;
    return p.bf16 ? bf16_one(static_cast<const uint16_t *>(p.c)[i]) : static_cast<const float *>(p.c)[i];
}
__device__ __forceinline__ void store_out(const MatmulParams &p, int64_t m, int64_t n, float v) {
    const int64_t i = m * p.ldd + n;
    if (p.bf16)
        static_cast<uint16_t *>(p.d)[i] = to_bf16(v);
    else
        static_cast<float *>(p.d)[i] = v;
}

template <int TM>
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

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * S::kStages + 2 * kScaleBufs + 1; ++i) mbar_init(full + 8 * i, 1);
        failed = 0;
        mbar_init_fence();
    }
    if (warp == 1) tmem_alloc<1>(smem_u32(&tmem_slot), S::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t sf_cols = tmem + TM;  // scale columns: kScaleBufs x (4 + 4 kAtomsB)
    bool ok = true;

    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&map_n);
        tma_prefetch_map(&map_m);
        int issued = 0;
        for (int c = c0; c < c1; ++c, ++issued) {
            const int s = issued % S::kStages, turn = issued / S::kStages;
            if (turn > 0 && !(ok = mbar_wait(empty + 8 * s, (turn - 1) & 1))) break;
            const uint32_t dst = base + s * S::kStage;
            mbar_expect_tx(full + 8 * s, S::kStage);
            tma_load_2d(dst, &map_n, full + 8 * s, c * kKC, static_cast<int32_t>(n0));
            tma_load_2d(dst + S::kBytesA, &map_m, full + 8 * s, c * kKC, static_cast<int32_t>(m0));
        }
        if (!ok)  // leave no copy in flight
            for (int i = issued > S::kStages ? issued - S::kStages : 0; i < issued; ++i)
                mbar_wait(full + 8 * (i % S::kStages), (i / S::kStages) & 1);
    } else if (warp == 1 && lane == 0) {
        int i = 0, g = -1;
        for (int c = c0; c < c1 && ok; ++c, ++i) {
            const int s = i % S::kStages;
            if (c == c0 || (c & 3) == 0) {
                ++g;
                const int b = g % kScaleBufs;
                if (!(ok = mbar_wait(sf_full + 8 * b, (g / kScaleBufs) & 1))) break;
                tc_fence_after();
                const uint32_t src = scales + b * S::kScaleBuf, col = sf_cols + b * 4 * (1 + S::kAtomsB);
                for (int a = 0; a < 1 + S::kAtomsB; ++a) tc_copy_scales<1>(col + 4 * a, src + 512 * a);
            }
            if (!(ok = mbar_wait(full + 8 * s, (i / S::kStages) & 1))) break;
            tc_fence_after();
            const uint32_t src = base + s * S::kStage;
            const uint32_t col = sf_cols + (g % kScaleBufs) * 4 * (1 + S::kAtomsB);
            const uint32_t idesc = p.idesc | mxf8_scale_byte(c & 3);
#pragma unroll
            for (int k = 0; k < kKC / 32; ++k)
                tc_mma_mxf8<1>(tmem, smem_desc(src + 32 * k, 16, 1024, 2), smem_desc(src + S::kBytesA + 32 * k, 16, 1024, 2),
                               idesc, col, col + 4, i > 0 || k > 0);
            tc_commit(empty + 8 * s);
            if ((c & 3) == 3 || c == c1 - 1) tc_commit(sf_empty + 8 * (g % kScaleBufs));
        }
        tc_commit(done);
    } else if (warp == 2) {
        int g = 0;
        for (int j = c0 >> 2; c0 < c1 && j <= (c1 - 1) >> 2; ++j, ++g) {
            const int b = g % kScaleBufs, turn = g / kScaleBufs;
            if (turn > 0 && !(ok = mbar_wait(sf_empty + 8 * b, (turn - 1) & 1))) break;
            const uint32_t dst = scales + b * S::kScaleBuf + lane * 16;
#pragma unroll
            for (int a = 0; a < 1 + S::kAtomsB; ++a) {
                const uint32_t *src = a == 0 ? p.sb + static_cast<int64_t>(j) * p.N : p.sa + static_cast<int64_t>(j) * p.M;
                const int64_t r0 = a == 0 ? n0 : m0 + (a - 1) * 128, rows = a == 0 ? p.N : p.M;
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t r = r0 + 32 * q + lane;
                    w[q] = r < rows ? __ldg(src + r) : 0x01010101u;
                }
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 512 * a), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                             "r"(w[3])
                             : "memory");
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(sf_full + 8 * b);
        }
    }
    if (warp >= 4) {
        ok = mbar_wait(done, 0);
        tc_fence_after();
    }
    if (!ok) failed = 1;
    __syncwarp();
    const int quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int64_t n = n0 + quarter * 32 + lane;
    const int64_t mleft = p.M - m0;
    if (p.splits == 1) {
        if (warp >= 4) {
#pragma unroll 1
            for (int j0 = 0; j0 < TM && j0 < mleft; j0 += 32) {
                float v[32];
                tc_load32(v, lanes + j0);
                tc_wait_ld();
                if (c0 == c1)
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                if (n < p.N)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j0 + j < mleft) {
                            float x = v[j];
                            if (p.c) x += load_out(p, m0 + j0 + j, n);
                            store_out(p, m0 + j0 + j, n, x);
                        }
            }
        }
    } else {
        // every load of the stages has been consumed: they hold the partial tile [m][n] now
        if (warp >= 4) {
#pragma unroll 1
            for (int j0 = 0; j0 < TM && j0 < mleft; j0 += 32) {
                float v[32];
                tc_load32(v, lanes + j0);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((j0 + j) * kTN + quarter * 32 + lane) * 4),
                                 "f"(c0 == c1 ? 0.0f : v[j])
                                 : "memory");
            }
        }
        cluster_barrier();
        for (int j = rank * (kThreads / kTN) + static_cast<int>(threadIdx.x) / kTN; j < TM && j < mleft;
             j += p.splits * (kThreads / kTN)) {
            const int col = static_cast<int>(threadIdx.x) % kTN;
            const uint32_t at = base + (j * kTN + col) * 4;
            float x = 0.0f;
            for (int r = 0; r < p.splits; ++r) x += cluster_load(cluster_map(at, r));
            if (n0 + col < p.N) {
                if (p.c) x += load_out(p, m0 + j, n0 + col);
                store_out(p, m0 + j, n0 + col, x);
            }
        }
        cluster_barrier();  // no CTA leaves while another reads its shared memory
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && failed && p.status) atomicOr(p.status, static_cast<unsigned int>(GAR_STATUS_TIMEOUT));
    if (warp == 1) tmem_free<1>(tmem, S::kColumns);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::atomic<void *> fn{nullptr};
    void *f = fn.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// Map of the codes [rows, K] (row stride ld bytes) in boxes of `box` rows x 128 bytes.
int encode(CUtensorMap *map, const uint8_t *q, int64_t rows, int64_t K, int64_t ld, int box) {
    EncodeTiled fn = encode_tiled();
    if (!fn) return fail(GAR_ECUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
    const cuuint32_t boxes[2] = {kKC, static_cast<cuuint32_t>(box)};
    const cuuint32_t elem[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(q), dims, strides, boxes, elem,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(GAR_ECUDA, "cuTensorMapEncodeTiled: %d", static_cast<int>(r));
    return GAR_OK;
}

template <int TM>
int launch(MatmulParams &p, const uint8_t *a, int64_t lda, const uint8_t *b, int64_t ldb, int64_t K, cudaStream_t stream) {
    using S = Shape<TM>;
    static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(GAR_ECUDA, "no current device");
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(matmul_kernel<TM>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return fail(GAR_ECUDA, "matmul_kernel: %s", cudaGetErrorString(e));
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    CUtensorMap map_n{}, map_m{};
    if (K > 0) {
        if (int rc = encode(&map_n, b, p.N, K, ldb, kTN)) return rc;
        if (int rc = encode(&map_m, a, p.M, K, lda, TM)) return rc;
    }
    p.tiles_n = static_cast<int32_t>(ceil_div(p.N, kTN));
    const int64_t tiles = p.tiles_n * ceil_div(p.M, int64_t{TM});
    // split k while the cluster's CTAs still find SMs and have two chunks each
    p.splits = 1;
    while (p.splits < 8 && tiles * p.splits * 2 <= sm_count() && p.chunks >= p.splits * 4) p.splits *= 2;
    if (tiles * p.splits > 0x7FFFFFFF) return fail(GAR_EINVAL, "the product has too many tiles");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    p.idesc = p.idesc | mxf8_idesc(0, 0, kTN, TM);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, matmul_kernel<TM>, map_n, map_m, p);
    if (e != cudaSuccess) return fail(GAR_ECUDA, "matmul_kernel: %s", cudaGetErrorString(e));
    return check_launch("matmul_kernel");
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
    p.d = d, p.ldd = ldd, p.c = c, p.ldc = ldc, p.bf16 = dtype == GAR_BF16;
    p.status = device_status();
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (M <= 32) return launch<32>(p, a, lda, b, ldb, K, stream);
    if (M <= 64) return launch<64>(p, a, lda, b, ldb, K, stream);
    if (ceil_div(M, int64_t{256}) * ceil_div(N, int64_t{kTN}) < sm_count())
        return launch<128>(p, a, lda, b, ldb, K, stream);
    return launch<256>(p, a, lda, b, ldb, K, stream);
}
