// clip.cu -- the 2-norm over all elements of many tensors, and their scaling by
//     c = min(1, max_norm / (norm + 1e-6)),   norm = sqrt(sum g^2).
//
// Two launches: every block sums the squares of its share of the chunks into
// one partial, then every block of the second launch adds all partials (in the
// same order, so in the same bits) and scales its share.  More tensors than one
// launch takes are as many launches of each, with one between that adds the
// partials, once.  Squares are summed in
// fp32 over the 64 bytes that a thread loads at a time and from there on in
// fp64; where such a sum leaves the range in which fp32 squares are sound
// (gradients beyond 1e15 or below 1e-15), its squares are taken again in fp64,
// so the norm is right over the whole range of the types.
//
// Bound by HBM, which the data crosses three times (nothing can be written before
// the last square is known, and little of a large model's gradients stays in
// L2): 294 M fp32 elements take 540 us, 6.5 TB/s of those 3.5 GB; ten tensors of
// 1.8 MB in all take 10 us, two launches' latency.
#include "launch.cuh"
#include "learn.h"
#include "vec.cuh"

#include <algorithm>

namespace kma {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;                                // 16-byte vectors per thread and chunk
constexpr int64_t kChunkBytes = int64_t(kThreads) * kVecs * 16;
// Tensors of a launch, in its parameters: a short list costs the host 0.7 us a
// launch less than a long one.
constexpr int kShortList = 24;
constexpr int kLongList = 256;

template <int MAX>
struct TensorList {
    const void *src[MAX];
    void *dst[MAX];
    int64_t size[MAX];          // elements
    int64_t first_chunk[MAX + 1];
    uint8_t dtype[MAX];
    uint8_t wide[MAX];          // src and dst 16-byte aligned
    int32_t n;
};

// Sum over lane 0 .. 31 in lane 0.
__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v += __shfl_down_sync(kAll, v, off);
    return v;
}

// Sum over the block in thread 0.  The SM adds two fp64 numbers a clock, so one
// warp adds what the others hand it (a few hundred clocks; all warps reducing
// by shuffles, and then each adding the warps' sums, took 5,000).
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double s[kThreads];
    s[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x >= 32)
        return 0.0;
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        t += s[w * 32 + threadIdx.x];
    return warp_sum(t);
}

// Sum of squares of n values held in registers.
template <int N>
__device__ __forceinline__ double squares(const float (&f)[N])
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        s = fmaf(f[i], f[i], s);
    if (s > 1e-30f && s < 1e30f)
        return static_cast<double>(s);
    double d = 0.0;
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        most = fmaxf(most, fabsf(f[i]));
    if (most > 0.0f || s != s)
#pragma unroll
        for (int i = 0; i < N; ++i)
            d += static_cast<double>(f[i]) * static_cast<double>(f[i]);
    return d;
}

// The tensor that chunk c belongs to.
template <int MAX>
__device__ __forceinline__ int tensor_of(const TensorList<MAX> &l, int64_t c)
{
    int lo = 0, hi = l.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.first_chunk[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *p, int64_t n, bool wide)
{
    constexpr int VE = 16 / sizeof(T);
    constexpr int kElems = kThreads * kVecs * VE;
    if (wide && n == kElems) {
        Raw<T, VE> q[kVecs];
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
            q[u] = load_raw<T, VE>(p + (u * kThreads + threadIdx.x) * VE);
        float f[kVecs * VE];
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            float g[VE];
            widen<T, VE>(q[u], g);
#pragma unroll
            for (int v = 0; v < VE; ++v)
                f[u * VE + v] = g[v];
        }
        return squares(f);
    }
    double d = 0.0;
    if (wide) {
        for (int i = threadIdx.x * VE; i + VE <= n; i += kThreads * VE) {
            float g[VE];
            widen<T, VE>(load_raw<T, VE>(p + i), g);
            d += squares(g);
        }
        const int i = static_cast<int>(n / VE * VE) + threadIdx.x;
        if (i < n) {
            const float g[1] = {Elem<T>::up(p[i])};
            d += squares(g);
        }
        return d;
    }
    for (int i = threadIdx.x; i < n; i += kThreads * VE) {
        float g[VE];
#pragma unroll
        for (int v = 0; v < VE; ++v)
            g[v] = i + v * kThreads < n ? Elem<T>::up(p[i + v * kThreads]) : 0.0f;
        d += squares(g);
    }
    return d;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *p, T *o, int64_t n, bool wide, float c)
{
    constexpr int VE = 16 / sizeof(T);
    constexpr int kElems = kThreads * kVecs * VE;
    if (wide && n == kElems) {
        Raw<T, VE> q[kVecs];
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
            q[u] = load_raw<T, VE>(p + (u * kThreads + threadIdx.x) * VE);
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            float g[VE];
            widen<T, VE>(q[u], g);
#pragma unroll
            for (int v = 0; v < VE; ++v)
                g[v] *= c;
            store_raw<T, VE>(o + (u * kThreads + threadIdx.x) * VE, narrow<T, VE>(g));
        }
        return;
    }
    if (wide) {
        for (int i = threadIdx.x * VE; i + VE <= n; i += kThreads * VE) {
            float g[VE];
            widen<T, VE>(load_raw<T, VE>(p + i), g);
#pragma unroll
            for (int v = 0; v < VE; ++v)
                g[v] *= c;
            store_raw<T, VE>(o + i, narrow<T, VE>(g));
        }
        const int i = static_cast<int>(n / VE * VE) + threadIdx.x;
        if (i < n)
            o[i] = Elem<T>::down(Elem<T>::up(p[i]) * c);
        return;
    }
    for (int i = threadIdx.x; i < n; i += kThreads)
        o[i] = Elem<T>::down(Elem<T>::up(p[i]) * c);
}

__device__ __forceinline__ int64_t share_begin(int64_t chunks, int64_t b, int64_t blocks)
{
    return chunks * b / blocks;
}

template <int MAX>
__global__ void __launch_bounds__(kThreads)
    squares_kernel(const __grid_constant__ TensorList<MAX> l, double *__restrict__ partial)
{
    let_next_start();
    wait_for_previous();
    const int64_t chunks = l.first_chunk[l.n];
    const int64_t c1 = share_begin(chunks, blockIdx.x + 1, gridDim.x);
    int64_t c = share_begin(chunks, blockIdx.x, gridDim.x);
    int t = tensor_of(l, c);
    double sum = 0.0;
    for (; c < c1; ++c) {
        while (l.first_chunk[t + 1] <= c)
            ++t;
        const int64_t at = (c - l.first_chunk[t]) * kChunkBytes;
        const bool wide = l.wide[t] != 0;
        if (l.dtype[t] == kFp32) {
            const int64_t i = at / 4;
            sum += chunk_squares(static_cast<const float *>(l.src[t]) + i,
                                 min(l.size[t] - i, kChunkBytes / 4), wide);
        } else {
            const int64_t i = at / 2;
            const int64_t n = min(l.size[t] - i, kChunkBytes / 2);
            if (l.dtype[t] == kBf16)
                sum += chunk_squares(static_cast<const __nv_bfloat16 *>(l.src[t]) + i, n, wide);
            else
                sum += chunk_squares(static_cast<const __half *>(l.src[t]) + i, n, wide);
        }
    }
    const double s = block_sum(sum);
    if (threadIdx.x == 0)
        partial[blockIdx.x] = s;
}

// sqrt of a sum of squares: an fp32 root of the sum scaled by a power of 4 into
// [1, 4), within an fp32 ulp over the range of fp64 (an fp64 root costs the
// scaling kernel half a microsecond).
__device__ __forceinline__ float root(double total)
{
    if (!(total > 0.0) || total > 1e300)
        return static_cast<float>(sqrt(total));   // 0, inf, NaN
    const int half = (((__double2hiint(total) >> 20) & 0x7ff) - 1023) >> 1;
    const double scale = __hiloint2double((1023 - 2 * half) << 20, 0);
    return scalbnf(sqrtf(static_cast<float>(total * scale)), half);
}

// The norm from all partial sums, by one warp; in lane 0.
__device__ __forceinline__ float norm_of(const double *partial, int32_t n)
{
    double v = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += 32)
        v += partial[i];
    return root(warp_sum(v));
}

__global__ void __launch_bounds__(32)
    norm_kernel(const double *partial, int32_t n, float *__restrict__ norm)
{
    wait_for_previous();
    const float f = norm_of(partial, n);
    if (threadIdx.x == 0)
        *norm = f;
}

// partials 0: *norm holds the norm; else it is formed here, and written.
template <int MAX>
__global__ void __launch_bounds__(kThreads)
    scale_kernel(const __grid_constant__ TensorList<MAX> l, const double *partial,
                 int32_t partials, float max_norm, bool in_place, float *norm)
{
    let_next_start();
    wait_for_previous();
    __shared__ float s_coef;
    if (threadIdx.x < 32) {
        const float f = partials == 0 ? *norm : norm_of(partial, partials);
        if (threadIdx.x == 0) {
            const float ratio = max_norm / (f + 1e-6f);
            s_coef = ratio >= 1.0f ? 1.0f : ratio;   // a NaN norm gives NaN
            if (partials != 0 && blockIdx.x == 0)
                *norm = f;
        }
    }
    __syncthreads();
    const float coef = s_coef;
    if (in_place && coef == 1.0f)
        return;
    const int64_t chunks = l.first_chunk[l.n];
    const int64_t c0 = share_begin(chunks, blockIdx.x, gridDim.x);
    int64_t c = share_begin(chunks, blockIdx.x + 1, gridDim.x) - 1;
    if (c < c0)
        return;
    int t = tensor_of(l, c);
    // backwards: what the first launch read last is still in L2
    for (; c >= c0; --c) {
        while (l.first_chunk[t] > c)
            --t;
        const int64_t at = (c - l.first_chunk[t]) * kChunkBytes;
        const bool wide = l.wide[t] != 0;
        if (l.dtype[t] == kFp32) {
            const int64_t i = at / 4;
            chunk_scale(static_cast<const float *>(l.src[t]) + i,
                        static_cast<float *>(l.dst[t]) + i,
                        min(l.size[t] - i, kChunkBytes / 4), wide, coef);
        } else {
            const int64_t i = at / 2;
            const int64_t n = min(l.size[t] - i, kChunkBytes / 2);
            if (l.dtype[t] == kBf16)
                chunk_scale(static_cast<const __nv_bfloat16 *>(l.src[t]) + i,
                            static_cast<__nv_bfloat16 *>(l.dst[t]) + i, n, wide, coef);
            else
                chunk_scale(static_cast<const __half *>(l.src[t]) + i,
                            static_cast<__half *>(l.dst[t]) + i, n, wide, coef);
        }
    }
}

// The next tensors of the call that have elements, from `first` on; returns
// the index of the next one that has, or n.
template <int MAX>
int32_t fill_list(const void *const *src, void *const *dst, const int64_t *sizes,
                  const int32_t *dtypes, int32_t n, int32_t first, TensorList<MAX> *l)
{
    l->n = 0;
    l->first_chunk[0] = 0;
    int32_t i = first;
    for (; i < n && l->n < MAX; ++i) {
        if (sizes[i] == 0)
            continue;
        const int32_t t = l->n++;
        void *d = dst != nullptr ? dst[i] : const_cast<void *>(src[i]);
        l->src[t] = src[i];
        l->dst[t] = d;
        l->size[t] = sizes[i];
        l->dtype[t] = static_cast<uint8_t>(dtypes[i]);
        l->wide[t] = ((reinterpret_cast<uintptr_t>(src[i]) | reinterpret_cast<uintptr_t>(d)) & 15) == 0;
        const int64_t bytes = sizes[i] * dtype_bytes(dtypes[i]);
        l->first_chunk[t + 1] = l->first_chunk[t] + (bytes + kChunkBytes - 1) / kChunkBytes;
    }
    while (i < n && sizes[i] == 0)   // so that no list of a call but its first can be empty
        ++i;
    return i;
}

template <int MAX>
cudaError_t clip_lists(const void *const *grads, void *const *out, const int64_t *sizes,
                       const int32_t *dtypes, int32_t n, bool scale, float max_norm, float *norm,
                       double *partial, int sms, cudaStream_t stream)
{
    auto blocks_of = [&](const TensorList<MAX> &l) {
        return static_cast<unsigned>(std::min<int64_t>(l.first_chunk[l.n], int64_t(sms) * 4));
    };
    TensorList<MAX> l;
    cudaError_t e = cudaSuccess;
    int32_t partials = 0, lists = 0;
    for (int32_t at = 0; at < n && e == cudaSuccess;) {
        at = fill_list(grads, out, sizes, dtypes, n, at, &l);
        if (l.n == 0)
            break;
        const unsigned blocks = blocks_of(l);
        e = launch_after(squares_kernel<MAX>, blocks, kThreads, 0, stream, l, partial + partials);
        partials += static_cast<int32_t>(blocks);
        ++lists;
    }
    if (e == cudaSuccess && (!scale || lists != 1)) {
        e = launch_after(norm_kernel, 1, 32, 0, stream, partial, partials, norm);
        partials = 0;
    }
    if (!scale)
        return e;
    for (int32_t at = 0, i = 0; i < lists && e == cudaSuccess; ++i) {
        if (lists > 1)   // else l still holds the list
            at = fill_list(grads, out, sizes, dtypes, n, at, &l);
        e = launch_after(scale_kernel<MAX>, blocks_of(l), kThreads, 0, stream, l, partial, partials,
                         max_norm, out == nullptr, norm);
    }
    return e;
}

}  // namespace

size_t clip_scratch_bytes(int32_t n, int sms)
{
    const int64_t lists = n <= kShortList ? 1 : (int64_t(n) + kLongList - 1) / kLongList;
    return static_cast<size_t>(lists) * sms * 4 * sizeof(double);
}

cudaError_t launch_clip(const void *const *grads, void *const *out, const int64_t *sizes,
                        const int32_t *dtypes, int32_t n, bool scale, float max_norm, float *norm,
                        double *partial, int sms, cudaStream_t stream)
{
    if (n <= kShortList)
        return clip_lists<kShortList>(grads, out, sizes, dtypes, n, scale, max_norm, norm, partial,
                                      sms, stream);
    return clip_lists<kLongList>(grads, out, sizes, dtypes, n, scale, max_norm, norm, partial, sms,
                                 stream);
}

}  // namespace kma
