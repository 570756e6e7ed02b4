// quantize.cu -- block-scaled 8-bit floating point: gar_fp8_quantize.
//
// A block of 128 values (128 consecutive ones along the axis that a product
// will sum over, or a 128 x 128 square) shares the power-of-two scale 2^k,
// k the smallest integer with amax <= FMAX 2^k (amax over the block's finite
// values, FMAX = 448 for e4m3, 57344 for e5m2; both are 1.75 times a power of
// two, so k follows from amax's exponent and one comparison of its
// significand).  Codes are x 2^-k rounded to nearest even: the product with a
// power of two is exact, so this is the only rounding.  A power of two rather
// than amax / FMAX costs at most one binade of the format's 15 (e4m3) or 30
// (e5m2) and nothing in relative precision above its subnormals, and it is
// the scale type that the tensor core applies by itself.
#include "common.cuh"
#include "fp8.cuh"
#include "launch.cuh"

namespace gar {
namespace {

constexpr int kTile = 128;  // rows and columns of one CTA's tile
constexpr int kThreads = 256;

struct QuantizeParams {
    const void *x;
    int64_t rows, cols, ldx;
    uint8_t *q, *qt;          // either may be NULL
    int64_t ldq, ldqt;
    uint8_t *scale, *scale_t;
    int64_t tiles_c;
    int32_t emax;  // 8 (e4m3) or 15 (e5m2): FMAX = 1.75 * 2^emax
    int32_t square, vec;
};

// Biased exponent of the scale from amax's bits: the addition carries into the
// exponent exactly where the significand is above 1.75.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, int emax) {
    const int e = static_cast<int>((amax + 0x1FFFFFu) >> 23) - emax;
    return static_cast<uint32_t>(e < 1 ? 1 : e);
}
// 2^(127 - byte), exact: byte is at most 247.
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

template <bool kE5M2>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    if (kE5M2) {
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    } else {
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    }
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The words that start `bytes` (0 to 14, even) behind the start of w.
template <int kWords>
__device__ __forceinline__ void shift_words(const uint32_t (&w)[kWords + 4], uint32_t bytes, uint32_t (&out)[kWords]) {
    uint32_t a[kWords + 2], b[kWords + 1];
#pragma unroll
    for (int j = 0; j < kWords + 2; ++j) a[j] = bytes & 8 ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < kWords + 1; ++j) b[j] = bytes & 4 ? a[j + 1] : a[j];
#pragma unroll
    for (int j = 0; j < kWords; ++j) out[j] = __funnelshift_r(b[j], b[j + 1], (bytes & 2) * 8);
}

// A thread's 8 rows x 8 columns of x as they are stored, and what both orders
// need of them.  bf16 values stay packed (32 registers rather than 64): their
// absolute values compare as unsigned 16-bit integers, two at a time.
template <typename T>
struct Patch;

template <>
struct Patch<uint16_t> {
    static constexpr uint32_t kInf = 0x7F80u;  // bits of an infinity's absolute value, in 16-bit halves
    uint32_t w[8][4];
    __device__ __forceinline__ void load(int i, const uint16_t *src) {
        const uint4 g = ld16(src);
        w[i][0] = g.x, w[i][1] = g.y, w[i][2] = g.z, w[i][3] = g.w;
    }
    // From any address, by the 16-byte lines that hold the values.
    static constexpr int kLines = 2;
    __device__ __forceinline__ void load_shifted(int i, const uint4 *line, uint32_t bytes) {
        const uint4 g = ld16(line), h = ld16(line + 1);
        const uint32_t x[8] = {g.x, g.y, g.z, g.w, h.x, h.y, h.z, h.w};
        shift_words<4>(x, bytes, w[i]);
    }
    __device__ __forceinline__ void load_some(int i, const uint16_t *src, int64_t left) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = 2 * j < left ? src[2 * j] : 0, hi = 2 * j + 1 < left ? src[2 * j + 1] : 0;
            w[i][j] = lo | (hi << 16);
        }
    }
    __device__ __forceinline__ float value(int i, int j) const {
        return j & 1 ? bf16_hi(w[i][j >> 1]) : bf16_lo(w[i][j >> 1]);
    }
    // Largest absolute values, as fp32 bits: of row i, and of every column (cmax).
    template <bool kSanitize>
    __device__ __forceinline__ uint32_t absw(int i, int j) const {
        uint32_t a = w[i][j] & 0x7FFF7FFFu;
        if (kSanitize) {
            if ((a & 0xFFFFu) >= kInf) a &= 0xFFFF0000u;
            if ((a >> 16) >= kInf) a &= 0xFFFFu;
        }
        return a;
    }
    template <bool kSanitize>
    __device__ __forceinline__ void maxima(uint32_t (&rmax)[8], uint32_t (&cmax)[8]) const {
        uint32_t c[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a = absw<kSanitize>(i, j);
                m = __vmaxu2(m, a);
                c[j] = __vmaxu2(c[j], a);
            }
            rmax[i] = max(m << 16, m & 0xFFFF0000u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) cmax[2 * j] = c[j] << 16, cmax[2 * j + 1] = c[j] & 0xFFFF0000u;
    }
};

template <>
struct Patch<float> {
    uint32_t w[8][8];
    __device__ __forceinline__ void load(int i, const float *src) {
        const uint4 g = ld16(src), h = ld16(src + 4);
        w[i][0] = g.x, w[i][1] = g.y, w[i][2] = g.z, w[i][3] = g.w;
        w[i][4] = h.x, w[i][5] = h.y, w[i][6] = h.z, w[i][7] = h.w;
    }
    static constexpr int kLines = 3;
    __device__ __forceinline__ void load_shifted(int i, const uint4 *line, uint32_t bytes) {
        const uint4 g = ld16(line), h = ld16(line + 1), k = ld16(line + 2);
        const uint32_t x[12] = {g.x, g.y, g.z, g.w, h.x, h.y, h.z, h.w, k.x, k.y, k.z, k.w};
        shift_words<8>(x, bytes, w[i]);
    }
    __device__ __forceinline__ void load_some(int i, const float *src, int64_t left) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = j < left ? __float_as_uint(src[j]) : 0u;
    }
    __device__ __forceinline__ float value(int i, int j) const { return __uint_as_float(w[i][j]); }
    template <bool kSanitize>
    __device__ __forceinline__ void maxima(uint32_t (&rmax)[8], uint32_t (&cmax)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) cmax[j] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t a = w[i][j] & 0x7FFFFFFFu;
                if (kSanitize && a >= 0x7F800000u) a = 0;
                m = max(m, a);
                cmax[j] = max(cmax[j], a);
            }
            rmax[i] = m;
        }
    }
};

// Two bf16 values times two powers of two: exact, or below 2^-126, whose code is 0 either way.
__device__ __forceinline__ uint32_t scale2(uint32_t x, uint32_t f) {
    uint32_t y;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(f));
    return y;
}

// The codes of one tile, both orders.  kBad: the tile has NaN or infinities;
// fma(y, 0, y f) is y f for finite y and NaN else, whose code is the format's NaN.
template <typename T, bool kE5M2, bool kBad>
__device__ __forceinline__ void emit(const QuantizeParams &p, const Patch<T> &v, const uint32_t (&rbyte)[8], const uint32_t (&cbyte)[8],
                                     uint8_t *tile, int64_t tr, int64_t tc, int64_t row0, int64_t col0, int64_t left) {
    const int tid = threadIdx.x, half = tid >> 4, hl = tid & 15;
    const auto scaled = [&](int i, int j, float f) {
        const float y = v.value(i, j);
        return kBad ? __fmaf_rn(y, 0.0f, y * f) : y * f;
    };
    if (p.qt) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (sizeof(T) == 2 && !kBad) {  // two columns at a time, as they are held
                if (j & 1) continue;
                const uint32_t f = pack_bf16x2(inverse_scale(cbyte[j]), inverse_scale(cbyte[j + 1]));
                uint32_t y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = scale2(v.w[i][j >> 1], f);
                *reinterpret_cast<uint2 *>(&tile[(hl * 8 + j) * kTile + ((half ^ hl) << 3)]) =
                    make_uint2(pack4<kE5M2>(bf16_lo(y[0]), bf16_lo(y[1]), bf16_lo(y[2]), bf16_lo(y[3])),
                               pack4<kE5M2>(bf16_lo(y[4]), bf16_lo(y[5]), bf16_lo(y[6]), bf16_lo(y[7])));
                *reinterpret_cast<uint2 *>(&tile[(hl * 8 + j + 1) * kTile + ((half ^ hl) << 3)]) =
                    make_uint2(pack4<kE5M2>(bf16_hi(y[0]), bf16_hi(y[1]), bf16_hi(y[2]), bf16_hi(y[3])),
                               pack4<kE5M2>(bf16_hi(y[4]), bf16_hi(y[5]), bf16_hi(y[6]), bf16_hi(y[7])));
                continue;
            }
            const float f = inverse_scale(cbyte[j]);
            uint2 w;
            w.x = pack4<kE5M2>(scaled(0, j, f), scaled(1, j, f), scaled(2, j, f), scaled(3, j, f));
            w.y = pack4<kE5M2>(scaled(4, j, f), scaled(5, j, f), scaled(6, j, f), scaled(7, j, f));
            *reinterpret_cast<uint2 *>(&tile[(hl * 8 + j) * kTile + ((half ^ hl) << 3)]) = w;
        }
        const int64_t tiles_r = (p.rows + kTile - 1) / kTile;
        if (half == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < left) store_scale(p.scale_t, p.cols, col0 + j, tr, tiles_r, cbyte[j]);
        }
    }
    if (p.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = row0 + i;
            const float f = inverse_scale(rbyte[i]);
            uint2 w;
            if constexpr (sizeof(T) == 2 && !kBad) {
                const uint32_t ff = pack_bf16x2(f, f);
                uint32_t y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = scale2(v.w[i][j], ff);
                w.x = pack4<kE5M2>(bf16_lo(y[0]), bf16_hi(y[0]), bf16_lo(y[1]), bf16_hi(y[1]));
                w.y = pack4<kE5M2>(bf16_lo(y[2]), bf16_hi(y[2]), bf16_lo(y[3]), bf16_hi(y[3]));
            } else {
                w.x = pack4<kE5M2>(scaled(i, 0, f), scaled(i, 1, f), scaled(i, 2, f), scaled(i, 3, f));
                w.y = pack4<kE5M2>(scaled(i, 4, f), scaled(i, 5, f), scaled(i, 6, f), scaled(i, 7, f));
            }
            if (r < p.rows) {
                uint8_t *dst = p.q + r * p.ldq + col0;
                if (left >= 8) {
                    *reinterpret_cast<uint2 *>(dst) = w;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < left) dst[j] = static_cast<uint8_t>((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
                }
                if (hl == 0) store_scale(p.scale, p.rows, r, tc, p.tiles_c, rbyte[i]);
            }
        }
    }
}

// One CTA per 128 x 128 tile, x read once for both orders.  Each half-warp
// owns 8 consecutive rows and each of its lanes 8 consecutive columns, so a
// row's maximum is a shuffle over 16 lanes, a column's is a maximum over the
// thread's 8 rows and then over the 16 half-warps through shared memory, and
// a thread's 8 codes of a column are 8 consecutive bytes of the transposed
// tile.  The transposed tile goes through shared memory; its 8-byte groups
// are exchanged (group h of column c sits at h ^ (c / 8)) so that neither the
// stores nor the loads conflict.  A tile with a NaN or an infinity (one vote
// per tile tells) takes its maxima again without them.
//
// Bound by HBM traffic that a tile's phases (load, maxima, store) leave gaps in;
// the SM's other tiles fill most of them.  16384 x 8192, both orders: bf16 103 us,
// 5.2 TB/s (three CTAs an SM 106 us; 97 us with square blocks, which exchange less);
// fp32 153 us, 5.3 TB/s.  Two orders by two launches would read x twice.
template <typename T, bool kE5M2>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) quantize_kernel(const __grid_constant__ QuantizeParams p) {
    __shared__ uint32_t colmax[16][kTile];
    __shared__ __align__(16) uint8_t tile[kTile * kTile];
    const int tid = threadIdx.x, half = tid >> 4, hl = tid & 15;
    const int64_t tr = blockIdx.x / p.tiles_c, tc = blockIdx.x % p.tiles_c;
    const int64_t row0 = tr * kTile + half * 8, col0 = tc * kTile + hl * 8;
    const T *x = static_cast<const T *>(p.x) + row0 * p.ldx + col0;
    let_next_begin();
    after_previous();
    Patch<T> v;
    const int64_t left = p.cols - col0;
    if (p.vec && row0 + 8 <= p.rows && left >= 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v.load(i, x + i * p.ldx);
    } else {
        // Rows that start anywhere: by whole lines of 16 bytes and shifts where the lines lie within x (8192 x 4095 bf16 42
        // us, fp32 56; 48 and 66 value by value), else value by value.
        const uintptr_t begin = reinterpret_cast<uintptr_t>(p.x);
        const uintptr_t end = begin + static_cast<uintptr_t>((p.rows - 1) * p.ldx + p.cols) * sizeof(T);
        const uintptr_t first = reinterpret_cast<uintptr_t>(x) & ~uintptr_t{15};
        const uintptr_t last = reinterpret_cast<uintptr_t>(x + 7 * p.ldx) & ~uintptr_t{15};
        if (row0 + 8 <= p.rows && left >= 8 && first >= begin && last + 16 * Patch<T>::kLines <= end) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uintptr_t at = reinterpret_cast<uintptr_t>(x + i * p.ldx);
                v.load_shifted(i, reinterpret_cast<const uint4 *>(at & ~uintptr_t{15}), static_cast<uint32_t>(at & 15));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v.load_some(i, x + i * p.ldx, row0 + i < p.rows ? left : 0);
        }
    }
    uint32_t rmax[8], cmax[8];
    v.template maxima<false>(rmax, cmax);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, rmax[i]);
    const bool bad = __syncthreads_or(most >= 0x7F800000u);
    if (bad) v.template maxima<true>(rmax, cmax);
    uint32_t cbyte[8], rbyte[8];
    if (p.square) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, rmax[i]);
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if ((tid & 31) == 0) colmax[0][tid >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) m = max(m, colmax[0][w]);
        const uint32_t b = scale_byte(m, p.emax);
#pragma unroll
        for (int i = 0; i < 8; ++i) rbyte[i] = cbyte[i] = b;
    } else {
        if (p.qt) {
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                *reinterpret_cast<uint4 *>(&colmax[half][hl * 8 + j]) = make_uint4(cmax[j], cmax[j + 1], cmax[j + 2], cmax[j + 3]);
            __syncthreads();
            if (tid < kTile) {
                uint32_t m = 0;
#pragma unroll
                for (int h = 0; h < 16; ++h) m = max(m, colmax[h][tid]);
                colmax[0][tid] = m;  // only this thread reads or writes this column here
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t m = rmax[i];
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            rbyte[i] = scale_byte(m, p.emax);
        }
        if (p.qt) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) cbyte[j] = scale_byte(colmax[0][hl * 8 + j], p.emax);
        }
    }
    if (bad)
        emit<T, kE5M2, true>(p, v, rbyte, cbyte, tile, tr, tc, row0, col0, left);
    else
        emit<T, kE5M2, false>(p, v, rbyte, cbyte, tile, tr, tc, row0, col0, left);
    if (p.qt) {
        __syncthreads();
        const int part = tid & 7;  // 16 bytes of a column: row groups 2 part and 2 part + 1
        const int64_t r = tr * kTile + part * 16;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = k * 32 + (tid >> 3);
            const int64_t cg = tc * kTile + c;
            const int f = c >> 3;
            uint4 g = *reinterpret_cast<const uint4 *>(&tile[c * kTile + (((2 * part) ^ (f & ~1)) << 3)]);
            if (f & 1) g = make_uint4(g.z, g.w, g.x, g.y);
            if (cg >= p.cols || r >= p.rows) continue;
            uint8_t *dst = p.qt + cg * p.ldqt + r;
            if (r + 16 <= p.rows) {
                *reinterpret_cast<uint4 *>(dst) = g;
            } else {
                const uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                for (int b = 0; b < 16; ++b)
                    if (r + b < p.rows) dst[b] = static_cast<uint8_t>(w[b >> 2] >> (8 * (b & 3)));
            }
        }
    }
}

template <typename T>
int launch(const QuantizeParams &p, unsigned blocks, cudaStream_t stream) {
    const auto kernel = p.emax == 15 ? quantize_kernel<T, true> : quantize_kernel<T, false>;
    return launch_early("quantize_kernel", kernel, dim3(blocks), kThreads, 0, 1, stream, p);
}

int check_codes(const char *name, const void *q, int64_t ld, int64_t cols, const void *scale) {
    if (!scale) return fail(GAR_EINVAL, "%s is given without its scales", name);
    if (ld < cols) return fail(GAR_EINVAL, "%s: row stride %lld < %lld columns", name, static_cast<long long>(ld),
                               static_cast<long long>(cols));
    if (!aligned(q, 16) || ld % 16 || !aligned(scale, 4))
        return fail(GAR_EALIGN, "%s: codes and their row stride need 16-byte alignment, scales 4-byte", name);
    return GAR_OK;
}

}  // namespace
}  // namespace gar

using namespace gar;

extern "C" int64_t gar_fp8_scale_bytes(int64_t rows, int64_t cols) {
    return rows < 0 || cols < 0 ? 0 : ceil_div(cols, 512) * rows * 4;
}

extern "C" int gar_fp8_quantize(const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, int32_t format,
                                int32_t square, uint8_t *q, int64_t ldq, uint8_t *scale, uint8_t *qt, int64_t ldqt,
                                uint8_t *scale_t, gar_stream_t stream_) {
    if (rows < 0 || cols < 0 || rows > 0x7FFFFFFF || cols > 0x7FFFFFFF)
        return fail(GAR_EINVAL, "rows=%lld cols=%lld", static_cast<long long>(rows), static_cast<long long>(cols));
    if (elem_bytes(dtype) < 0) return fail(GAR_EDTYPE, "unknown dtype %d", dtype);
    if (format != GAR_F8E4M3 && format != GAR_F8E5M2) return fail(GAR_EDTYPE, "unknown 8-bit format %d", format);
    if (!q && !qt) return fail(GAR_EINVAL, "neither q nor qt is given");
    if (rows == 0 || cols == 0) return GAR_OK;
    if (!x || ldx < cols) return fail(GAR_EINVAL, "x is NULL or its row stride is below its columns");
    if (!aligned(x, elem_bytes(dtype))) return fail(GAR_EALIGN, "x is misaligned");
    if (q)
        if (int rc = check_codes("q", q, ldq, cols, scale)) return rc;
    if (qt)
        if (int rc = check_codes("qt", qt, ldqt, rows, scale_t)) return rc;
    const int64_t tiles_r = ceil_div(rows, kTile), tiles_c = ceil_div(cols, kTile);
    if (tiles_r * tiles_c > 0x7FFFFFFF) return fail(GAR_EINVAL, "the matrix has too many tiles");
    QuantizeParams p{};
    p.x = x, p.rows = rows, p.cols = cols, p.ldx = ldx;
    p.q = q, p.ldq = ldq, p.scale = scale, p.qt = qt, p.ldqt = ldqt, p.scale_t = scale_t;
    p.tiles_c = tiles_c;
    p.emax = format == GAR_F8E5M2 ? 15 : 8;
    p.square = square ? 1 : 0;
    p.vec = aligned(x, 16) && (ldx * elem_bytes(dtype)) % 16 == 0;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const unsigned blocks = static_cast<unsigned>(tiles_r * tiles_c);
    return dtype == GAR_F32 ? launch<float>(p, blocks, stream) : launch<uint16_t>(p, blocks, stream);
}
