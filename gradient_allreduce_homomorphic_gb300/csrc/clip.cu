// clip.cu -- the global norm of many tensors' gradients and clipping by it:
// gar_grad_norm, gar_grad_clip.
//
//   norm[w] = sqrt(sum over the tensors i and elements e of g[w][i][e]^2)
//   c = min(1, max_norm / norm),  out = c g
//
// Two passes: the first leaves one fp64 partial sum per CTA, the second begins in
// every CTA with their sum (in a fixed order, so that every CTA has the same bits)
// and scales.  It goes through the tensors backwards, so that it begins with what
// the first pass has left in L2.  The tables of tensors travel as kernel
// parameters; a long list takes several launches of each pass.
//
// Bound by HBM: the norms of 8 x 45M fp32 values 229 us (6.3 TB/s); by one norm, out
// of place, 482 us (35 for the norm of one worker's, scaling at 6.3 TB/s).  12 small
// tensors 8.8 us a call, the two launches' host time.
//
// Squares are summed sixteen at a time in fp32 before an fp64 addition (fp64 runs
// at 1/64 of the fp32 rate here).  Sixteen whose sum comes near either end of
// fp32's range are squared again in fp64.
#include <algorithm>
#include <cmath>

#include "fp8.cuh"
#include "launch.cuh"

namespace gar {
namespace {

constexpr int kThreads = 256;
// Tiles of 32 KB, 8 loads of a thread under way, handed out round the CTAs: 8 x 45M
// values out of place 484 us; tiles of 16 KB and twice the CTAs 543, two batches of 8
// to a tile 505, runs of tiles to each CTA 550.
constexpr int kVecs = 8;                               // of 16 bytes, of a thread in a tile
constexpr int kCtas = 4;                               // of an SM
constexpr int64_t kTileBytes = kThreads * kVecs * 16;
constexpr int kMaxSums = 2048;                         // partial sums of a worker and launch

template <int NPTR, int NTENSOR>
struct ClipParams {
    int32_t P, count;        // workers, tensors of this launch
    int32_t norms;           // 1 or P
    int32_t sums, launches;  // partial sums of a worker in one launch; launches
    int32_t launch;
    float max_norm;
    double *partial;         // [launches][norms][sums], each written by every call
    float *norm;
    unsigned int *status;
    int64_t tiles;           // of one worker
    struct Tensor {
        int64_t first;  // tile
        int64_t numel : 62;
        int64_t bf16 : 2;
    } tensor[NTENSOR + 1];   // one more, for its first tile
    const void *src[NPTR];   // [tensor][worker]
    void *dst[NPTR];
};
constexpr int kSmallPointers = 96, kSmallTensors = 64, kLargePointers = 1536, kLargeTensors = 320;
// 4 KB of parameters for short lists, else 31: a launch takes the host 1.8 us with the
// one and 2.6 with the other.
using ClipSmall = ClipParams<kSmallPointers, kSmallTensors>;
using ClipLarge = ClipParams<kLargePointers, kLargeTensors>;
static_assert(sizeof(ClipSmall) <= 4096 && sizeof(ClipLarge) <= 32000, "parameters exceed the launch limit");

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
template <typename P>
__device__ __forceinline__ int tensor_of(const P &p, int64_t tile) {
    int lo = 0, hi = p.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.tensor[mid].first <= tile) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The squares of n values (16 or fewer), in fp64.
template <int N>
__device__ __forceinline__ double squares(const float (&x)[N]) {
    constexpr int kChains = N < 4 ? N : 4;
    float s[kChains];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i % kChains] = i < kChains ? x[i] * x[i] : fmaf(x[i], x[i], s[i % kChains]);
    if constexpr (kChains == 4) s[0] = (s[0] + s[1]) + (s[2] + s[3]);
    if (s[0] > 1e-24f && s[0] < 1e38f) return s[0];
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) any |= __float_as_uint(x[i]);
    if ((any & 0x7FFFFFFFu) == 0) return 0.0;
    double d = 0.0;
#pragma unroll 1
    for (int i = 0; i < N; ++i) d += static_cast<double>(x[i]) * x[i];
    return d;
}

template <typename T>
__device__ __forceinline__ void unpack(uint4 q, float *x) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(w[i]);
        else x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
        else w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A tile's elements: [begin, end), the first `head` of tile 0 before the first 16-byte line.
struct Range {
    int64_t begin, body, end;
};
template <typename T>
__device__ __forceinline__ Range tile_range(const T *x, int64_t n, int64_t i) {
    constexpr int64_t kElems = kTileBytes / sizeof(T);
    int64_t head = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T);
    head = min(head, n);
    Range r;
    r.begin = i == 0 ? 0 : head + i * kElems;
    r.body = i == 0 ? head : r.begin;
    r.end = min(head + (i + 1) * kElems, n);
    return r;
}

template <typename T>
__device__ __forceinline__ double tile_squares(const T *x, int64_t n, int64_t i) {
    constexpr int V = 16 / sizeof(T);
    const Range r = tile_range(x, n, i);
    double sum = 0.0;
    if (r.begin >= r.end) return sum;
    const int vecs = static_cast<int>((r.end - r.body) / V);
    const uint4 *from = reinterpret_cast<const uint4 *>(x + r.body);
    uint4 q[kVecs];
    if (vecs == kVecs * kThreads) {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) q[k] = from[k * kThreads + threadIdx.x];
    } else {
#pragma unroll
        for (int k = 0; k < kVecs; ++k) {
            const int at = k * kThreads + threadIdx.x;
            q[k] = at < vecs ? from[at] : make_uint4(0, 0, 0, 0);
        }
    }
    float v[16];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        unpack<T>(q[k], v + (k * V) % 16);
        if ((k + 1) * V % 16 == 0) sum += squares(v);
    }
    const int64_t rest = r.body + vecs * V;
    if (r.begin == r.body && rest == r.end) return sum;  // whole lines alone (fp64 is dear: no additions of nothing)
    float one[1] = {0.0f};
    if (static_cast<int64_t>(threadIdx.x) < r.body - r.begin) one[0] = load_f32(x + r.begin + threadIdx.x);
    sum += squares(one);
    one[0] = 0.0f;
    const int64_t tail = rest + threadIdx.x;
    if (tail < r.end) one[0] = load_f32(x + tail);
    return sum + squares(one);
}

template <typename P>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ P p) {
    __shared__ double of_warp[kThreads / 32];
    let_next_begin();
    after_previous();
    const int w = blockIdx.y;
    double sum = 0.0;
    int i = tensor_of(p, blockIdx.x);
    for (int64_t t = blockIdx.x; t < p.tiles; t += gridDim.x) {
        while (p.tensor[i + 1].first <= t) ++i;
        const void *x = p.src[i * p.P + w];
        const int64_t n = p.tensor[i].numel, at = t - p.tensor[i].first;
        sum += p.tensor[i].bf16 ? tile_squares(static_cast<const uint16_t *>(x), n, at) : tile_squares(static_cast<const float *>(x), n, at);
    }
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int k = 1; k < kThreads / 32; ++k) sum += of_warp[k];
    p.partial[(static_cast<int64_t>(p.launch) * p.norms + w) * p.sums + blockIdx.x] = sum;
}

// Worker w's norm from all partial sums, by one warp: fp64 in every thread of the
// CTAs that scale took longer than the scaling of small tensors.
template <typename P>
__device__ __forceinline__ float norm_of(const P &p, int w) {
    const int lane = threadIdx.x & 31;
    double sum[4] = {0.0, 0.0, 0.0, 0.0};
    for (int l = 0; l < p.launches; ++l) {
        const double *of = p.partial + (static_cast<int64_t>(l) * p.norms + w) * p.sums;
        for (int i = lane; i < p.sums; i += 128)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + 32 * k < p.sums) sum[k] += of[i + 32 * k];
    }
    return static_cast<float>(sqrt(warp_sum((sum[0] + sum[1]) + (sum[2] + sum[3]))));
}

template <typename P>
__global__ void __launch_bounds__(32) grad_norm_final_kernel(const __grid_constant__ P p) {
    let_next_begin();
    after_previous();
    const float norm = norm_of(p, blockIdx.x);
    if (threadIdx.x == 0) p.norm[blockIdx.x] = norm;
}

template <typename T>
__device__ __forceinline__ void scale_tile(const T *x, T *y, int64_t n, int64_t i, float c) {
    constexpr int V = 16 / sizeof(T);
    const Range r = tile_range(x, n, i);
    if (r.begin >= r.end) return;
    // no 16-byte line in common: element by element (one tensor of 45M values, with its norm, fp32 330 us for 94, bf16 268 for 54)
    if ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(y)) & 15) {
        for (int64_t e = r.begin + threadIdx.x; e < r.end; e += kThreads) store_f32(y + e, load_f32(x + e) * c);
        return;
    }
    const int vecs = static_cast<int>((r.end - r.body) / V);
    const uint4 *from = reinterpret_cast<const uint4 *>(x + r.body);
    uint4 *to = reinterpret_cast<uint4 *>(y + r.body);
    uint4 q[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int at = k * kThreads + threadIdx.x;
        if (at < vecs) q[k] = from[at];
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int at = k * kThreads + threadIdx.x;
        if (at >= vecs) continue;
        float v[V];
        unpack<T>(q[k], v);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= c;
        st16(to + at, pack<T>(v));
    }
    if (static_cast<int64_t>(threadIdx.x) < r.body - r.begin) store_f32(y + r.begin + threadIdx.x, load_f32(x + r.begin + threadIdx.x) * c);
    const int64_t tail = r.body + vecs * V + threadIdx.x;
    if (tail < r.end) store_f32(y + tail, load_f32(x + tail) * c);
}

template <typename P>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ P p) {
    __shared__ float scale;
    let_next_begin();
    after_previous();
    const int w = blockIdx.y, of = p.norms == 1 ? 0 : w;
    if (threadIdx.x < 32) {
        const float norm = norm_of(p, of);
        const bool finite = norm < INFINITY;  // false for NaN too
        if (threadIdx.x == 0) {
            scale = finite && norm > p.max_norm ? p.max_norm / norm : 1.0f;
            if (blockIdx.x == 0 && of == w && p.launch == 0) {
                p.norm[w] = norm;
                if (!finite && p.status) atomicOr(p.status, static_cast<unsigned int>(GAR_STATUS_NONFINITE));
            }
        }
    }
    __syncthreads();
    const float c = scale;
    int i = tensor_of(p, p.tiles - 1 - blockIdx.x);
    for (int64_t t = p.tiles - 1 - blockIdx.x; t >= 0; t -= gridDim.x) {
        while (p.tensor[i].first > t) --i;
        const void *x = p.src[i * p.P + w];
        void *y = p.dst[i * p.P + w];
        if (c == 1.0f && x == y) continue;  // stays as it is
        const int64_t n = p.tensor[i].numel, at = t - p.tensor[i].first;
        if (p.tensor[i].bf16) scale_tile(static_cast<const uint16_t *>(x), static_cast<uint16_t *>(y), n, at, c);
        else scale_tile(static_cast<const float *>(x), static_cast<float *>(y), n, at, c);
    }
}

// ---------------------------------------------------------------------- host
int tensors_per_launch(int P, int pointers, int tensors) { return std::max(1, std::min(tensors, pointers / P)); }
bool is_small(int P, int32_t count) { return count <= kSmallTensors && static_cast<int64_t>(P) * count <= kSmallPointers; }
int32_t launches_for(int P, int32_t count) {
    return static_cast<int32_t>(std::max(ceil_div(count, int64_t{tensors_per_launch(P, kLargePointers, kLargeTensors)}), int64_t{1}));
}

template <typename Params>
int run(const void *const *src, void *const *dst, int32_t P, const int64_t *numel, const int32_t *dtype, int32_t count, int32_t norms,
        float max_norm, float *norm, double *partial, bool small, bool scale, cudaStream_t stream) {
    Params p;
    p.norms = norms, p.max_norm = max_norm, p.norm = norm, p.partial = partial, p.status = device_status();
    p.launches = small ? 1 : launches_for(norms, count);
    int64_t tiles = 0;
    for (int32_t i = 0; i < count; ++i) tiles += ceil_div(numel[i] * elem_bytes(dtype[i]), kTileBytes);
    // a CTA to each tile while they are few, else as many as the SMs hold at one time, the workers' together
    const auto ctas = [&](int64_t of_worker, int32_t workers, int64_t few) {
        const int64_t held = std::max(std::min(sm_count() * kCtas, kMaxSums) / workers, 1);
        return static_cast<int32_t>(std::max(of_worker * workers <= few ? of_worker : std::min(of_worker, held), int64_t{1}));
    };
    p.sums = ctas(tiles, norms, kMaxSums);
    const auto fill = [&](int32_t l, int32_t workers, int32_t per_launch) {
        p.launch = l, p.P = workers;
        const int32_t i0 = l * per_launch;
        p.count = std::min(per_launch, count - i0);
        p.tiles = 0;
        for (int32_t i = 0; i < p.count; ++i) {
            p.tensor[i].first = p.tiles;
            p.tensor[i].numel = numel[i0 + i];
            p.tensor[i].bf16 = dtype[i0 + i] == GAR_BF16;
            p.tiles += ceil_div(numel[i0 + i] * elem_bytes(dtype[i0 + i]), kTileBytes);
            for (int w = 0; w < workers; ++w) {
                p.src[i * workers + w] = src[static_cast<int64_t>(w) * count + i0 + i];
                p.dst[i * workers + w] = dst ? dst[static_cast<int64_t>(w) * count + i0 + i] : nullptr;
            }
        }
        p.tensor[p.count].first = p.tiles;
    };
    const auto tensors = [&](int32_t workers) { return small ? std::max(count, 1) : tensors_per_launch(workers, kLargePointers, kLargeTensors); };
    for (int32_t l = 0; l < p.launches; ++l) {
        fill(l, norms, tensors(norms));
        // every launch writes all its sums: a CTA without a tile 0
        if (int rc = launch_early("grad_norm_kernel", grad_norm_kernel<Params>, dim3(static_cast<unsigned>(p.sums), static_cast<unsigned>(norms)),
                                  kThreads, 0, 1, stream, p))
            return rc;
    }
    if (!scale)
        return launch_early("grad_norm_final_kernel", grad_norm_final_kernel<Params>, dim3(static_cast<unsigned>(norms)), 32, 0, 1, stream, p);
    for (int32_t l = (small ? 1 : launches_for(P, count)) - 1; l >= 0; --l) {
        fill(l, P, tensors(P));
        const int32_t blocks = ctas(p.tiles, P, 4 * sm_count() * kCtas);
        if (int rc = launch_early("grad_scale_kernel", grad_scale_kernel<Params>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(P)),
                                  kThreads, 0, 1, stream, p))
            return rc;
    }
    return GAR_OK;
}

int start(const void *const *src, void *const *dst, int32_t P, const int64_t *numel, const int32_t *dtype, int32_t count, int32_t shared,
          float max_norm, float *norm, void *d_workspace, size_t workspace_bytes, bool scale, gar_stream_t stream_) {
    if (P < 1 || P > GAR_MAX_WORKERS) return fail(GAR_EINVAL, "P=%d outside 1..%d", P, GAR_MAX_WORKERS);
    if (count < 0 || (count > 0 && (!src || !numel || !dtype || (scale && !dst)))) return fail(GAR_EINVAL, "count=%d, or a NULL table", count);
    if (!norm || !d_workspace || workspace_bytes < gar_grad_workspace_bytes(P, count))
        return fail(GAR_EINVAL, "norm or the workspace is NULL, or the workspace is too small");
    if (!(max_norm >= 0.0f)) return fail(GAR_EINVAL, "max_norm has to be 0 or more");
    if (!aligned(norm, 4) || !aligned(d_workspace, 8)) return fail(GAR_EALIGN, "norm or the workspace is misaligned");
    for (int32_t i = 0; i < count; ++i) {
        const int size = elem_bytes(dtype[i]);
        if (size < 0) return fail(GAR_EDTYPE, "tensor %d has the unknown dtype %d", i, dtype[i]);
        if (numel[i] < 0 || numel[i] > (int64_t{1} << 60)) return fail(GAR_EINVAL, "tensor %d has %lld elements", i, static_cast<long long>(numel[i]));
        for (int w = 0; w < P && numel[i] > 0; ++w) {
            const int64_t at = static_cast<int64_t>(w) * count + i;
            if (!src[at] || (scale && !dst[at])) return fail(GAR_EINVAL, "worker %d's tensor %d is NULL", w, i);
            if (!aligned(src[at], size) || (scale && !aligned(dst[at], size))) return fail(GAR_EALIGN, "worker %d's tensor %d is misaligned", w, i);
        }
    }
    const int32_t norms = shared || P == 1 ? 1 : P;
    double *partial = static_cast<double *>(d_workspace);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (is_small(P, count))
        return run<ClipSmall>(src, dst, P, numel, dtype, count, norms, max_norm, norm, partial, true, scale, stream);
    return run<ClipLarge>(src, dst, P, numel, dtype, count, norms, max_norm, norm, partial, false, scale, stream);
}

}  // namespace
}  // namespace gar

using namespace gar;

extern "C" size_t gar_grad_workspace_bytes(int32_t P, int32_t count) {
    if (P < 1 || P > GAR_MAX_WORKERS || count < 0) return 0;
    return static_cast<size_t>(launches_for(P, count)) * kMaxSums * sizeof(double);
}

extern "C" int gar_grad_norm(const void *const *src, int32_t P, const int64_t *numel, const int32_t *dtype, int32_t count, float *norm,
                             void *d_workspace, size_t workspace_bytes, gar_stream_t stream) {
    return start(src, nullptr, P, numel, dtype, count, 0, 0.0f, norm, d_workspace, workspace_bytes, false, stream);
}

extern "C" int gar_grad_clip(const void *const *src, void *const *dst, int32_t P, const int64_t *numel, const int32_t *dtype, int32_t count,
                             int32_t shared, float max_norm, float *norm, void *d_workspace, size_t workspace_bytes,
                             gar_stream_t stream) {
    return start(src, dst, P, numel, dtype, count, shared, max_norm, norm, d_workspace, workspace_bytes, true, stream);
}
