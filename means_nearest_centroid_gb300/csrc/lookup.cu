// lookup.cu -- the rows of a table that ids name, weighted and scaled, and the
// gradients of the table and of the weights:
//     out[i]   = scale sum_j w[i][j] table[idx[i][j]]
//     dtable[r] = scale sum over idx[i][j] == r of w[i][j] dout[i]
//     dw[i][j] = scale <dout[i], table[idx[i][j]]>
// (w = 1 without weights; ids outside [0, K) add nothing).  Sums are fp32, each
// output is rounded once.
//
// The gradient of the table sorts the ids by row first (lists.cu).  The sorted
// places are then cut into chunks of a fixed length; a warp sums one slice of
// columns over one chunk in registers and writes a row as soon as its last
// place is passed.  A row that continues past a chunk's end leaves its parts in
// a workspace, and a second launch adds those in chunk order.  Every row of the
// result is written once, by one warp, and the order of every sum follows from
// the sizes alone: the bits do not change from run to run.
#include "internal.h"
#include "vec.cuh"

#include <algorithm>

namespace kma {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ---- lookup ---------------------------------------------------------------

// One thread per VE columns of one output row.
template <typename T, int VE>
__global__ void __launch_bounds__(kThreads)
    lookup_kernel(const T *__restrict__ table, const int32_t *__restrict__ idx,
                  const float *__restrict__ weights, int64_t N, int32_t k, int32_t K, int32_t D,
                  float scale, T *__restrict__ out)
{
    const int32_t vecs = D / VE;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (t >= N * vecs)
        return;
    const int64_t i = t / vecs;
    const int64_t col = (t - i * vecs) * VE;
    float acc[VE] = {};
    for (int32_t j0 = 0; j0 < k; j0 += 8) {
        int32_t r[8];
        Raw<T, VE> q[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            r[u] = j0 + u < k ? __ldg(idx + i * k + j0 + u) : -1;
            if (r[u] >= K)
                r[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (r[u] >= 0)
                q[u] = load_raw<T, VE>(table + static_cast<int64_t>(r[u]) * D + col);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (r[u] >= 0) {
                const float w = weights != nullptr ? __ldg(weights + i * k + j0 + u) : 1.0f;
                float f[VE];
                widen<T, VE>(q[u], f);
#pragma unroll
                for (int v = 0; v < VE; ++v)
                    acc[v] = fmaf(w, f[v], acc[v]);
            }
    }
#pragma unroll
    for (int v = 0; v < VE; ++v)
        acc[v] *= scale;
    store_raw<T, VE>(out + i * D + col, narrow<T, VE>(acc));
}

// ---- gradient of the weights ----------------------------------------------

// One warp per (point, id).
template <typename T, int VE>
__global__ void __launch_bounds__(kThreads)
    dweights_kernel(const T *__restrict__ dout, const T *__restrict__ table,
                    const int32_t *__restrict__ idx, int64_t M, int32_t k, int32_t K, int32_t D,
                    float scale, float *__restrict__ dweights)
{
    const int lane = threadIdx.x & 31;
    const int64_t f = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (f >= M)
        return;
    const int32_t r = __ldg(idx + f);
    float sum = 0.0f;
    if (r >= 0 && r < K) {
        const T *a = dout + f / k * D;
        const T *b = table + static_cast<int64_t>(r) * D;
        for (int c = lane * VE; c < D; c += 32 * VE) {
            float p[VE], q[VE];
            widen<T, VE>(load_raw<T, VE>(a + c), p);
            widen<T, VE>(load_raw<T, VE>(b + c), q);
#pragma unroll
            for (int v = 0; v < VE; ++v)
                sum = fmaf(p[v], q[v], sum);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        sum += __shfl_xor_sync(kAll, sum, off);
    if (lane == 0)
        dweights[f] = sum * scale;
}

// ---- gradient of the table ------------------------------------------------

struct GradArgs {
    const void *dout;
    const float *weights;      // or nullptr
    const int32_t *order;      // sorted places -> flat (point, id) positions
    const int32_t *rows;       // the rows in sorted order
    const int32_t *offsets;    // [K + 1]
    void *dtable;
    float *parts;              // [2][chunks][D]: a chunk's first and last row, unfinished
    int64_t chunks;
    int32_t chunk;             // sorted places per chunk
    int32_t slices;            // column slices of a row
    int64_t sum_blocks;        // blocks that sum; the others zero rows without ids
    int32_t k, K, D;
    int32_t skip;              // a row that takes no gradient, or -1
    float scale;
    bool accumulate;
};

template <typename G, int VE>
__device__ __forceinline__ void put_row(const GradArgs &a, int32_t r, int col,
                                        const float (&acc)[VE])
{
    G *p = static_cast<G *>(a.dtable) + static_cast<int64_t>(r) * a.D + col;
    float f[VE];
#pragma unroll
    for (int v = 0; v < VE; ++v)
        f[v] = acc[v] * a.scale;
    if (r == a.skip) {
        if (a.accumulate)
            return;
#pragma unroll
        for (int v = 0; v < VE; ++v)
            f[v] = 0.0f;
    } else if (a.accumulate) {
        float old[VE];
        widen<G, VE>(load_raw<G, VE>(p), old);
#pragma unroll
        for (int v = 0; v < VE; ++v)
            f[v] += old[v];
    }
    store_raw<G, VE>(p, narrow<G, VE>(f));
}

// T: type of dout, G: of dtable; a warp takes 32 * VE columns.
template <typename T, typename G, int VE>
__global__ void __launch_bounds__(kThreads) segment_kernel(const GradArgs a)
{
    const int lane = threadIdx.x & 31;
    if (blockIdx.x >= a.sum_blocks) {
        // rows that no id names
        const int64_t warps = (static_cast<int64_t>(gridDim.x) - a.sum_blocks) * kWarps;
        for (int64_t r = (static_cast<int64_t>(blockIdx.x) - a.sum_blocks) * kWarps +
                         (threadIdx.x >> 5);
             r < a.K; r += warps) {
            if (__ldg(a.offsets + r) != __ldg(a.offsets + r + 1))
                continue;
            G *p = static_cast<G *>(a.dtable) + r * a.D;
            const float zero[VE] = {};
            for (int c = lane * VE; c < a.D; c += 32 * VE)
                store_raw<G, VE>(p + c, narrow<G, VE>(zero));
        }
        return;
    }
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t chunk = unit / a.slices;
    const int64_t total = __ldg(a.offsets + a.K);
    const int64_t begin = chunk * a.chunk;
    if (chunk >= a.chunks || begin >= total)
        return;
    const int64_t end = min(total, begin + a.chunk);
    const int col = (static_cast<int>(unit - chunk * a.slices) * 32 + lane) * VE;
    const bool in = col < a.D;
    const T *dout = static_cast<const T *>(a.dout) + (in ? col : 0);
    // the row at `begin` began in an earlier chunk / that at `end` goes on
    const bool from_before = begin > 0 && __ldg(a.rows + begin - 1) == __ldg(a.rows + begin);
    const bool goes_on = end < total && __ldg(a.rows + end - 1) == __ldg(a.rows + end);

    float acc[VE] = {};
    int32_t cur = __ldg(a.rows + begin);
    bool first = true;   // cur is the row at `begin`
    auto part = [&](int which) {
        if (in) {
            float *p = a.parts + (which * a.chunks + chunk) * a.D + col;
            store_raw<float, VE>(p, narrow<float, VE>(acc));
        }
    };
    for (int64_t s0 = begin; s0 < end; s0 += 32) {
        // a place per lane
        const int64_t s = s0 + lane;
        int32_t row = -1, point = 0;
        float w = 0.0f;
        if (s < end) {
            const int32_t f = __ldg(a.order + s);
            row = __ldg(a.rows + s);
            point = f / a.k;
            w = a.weights != nullptr ? __ldg(a.weights + f) : 1.0f;
        }
        const int n = static_cast<int>(min(static_cast<int64_t>(32), end - s0));
        for (int u0 = 0; u0 < n; u0 += 8) {
            Raw<T, VE> q[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int32_t i = __shfl_sync(kAll, point, u0 + u);
                if (u0 + u < n && in)
                    q[u] = load_raw<T, VE>(dout + static_cast<int64_t>(i) * a.D);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int32_t r = __shfl_sync(kAll, row, u0 + u);
                const float wu = __shfl_sync(kAll, w, u0 + u);
                if (u0 + u >= n)
                    continue;
                if (r != cur) {
                    if (first && from_before)
                        part(0);
                    else if (in)
                        put_row<G, VE>(a, cur, col, acc);
                    first = false;
                    cur = r;
#pragma unroll
                    for (int v = 0; v < VE; ++v)
                        acc[v] = 0.0f;
                }
                if (in) {
                    float f[VE];
                    widen<T, VE>(q[u], f);
#pragma unroll
                    for (int v = 0; v < VE; ++v)
                        acc[v] = fmaf(wu, f[v], acc[v]);
                }
            }
        }
    }
    if (first && from_before)
        part(0);
    else if (goes_on)
        part(1);
    else if (in)
        put_row<G, VE>(a, cur, col, acc);
}

// Rows that span chunks: the chunk in which such a row begins holds its first
// part as its last row; the following chunks hold the others as their first.
template <typename G, int VE>
__global__ void __launch_bounds__(kThreads) join_kernel(const GradArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t chunk = unit / a.slices;
    const int64_t total = __ldg(a.offsets + a.K);
    const int64_t begin = chunk * a.chunk;
    const int64_t end = begin + a.chunk;
    if (chunk >= a.chunks || end >= total)
        return;
    const int32_t r = __ldg(a.rows + end - 1);
    if (__ldg(a.rows + end) != r || __ldg(a.offsets + r) < begin)
        return;   // ends here, or began in an earlier chunk
    const int64_t last = (static_cast<int64_t>(__ldg(a.offsets + r + 1)) - 1) / a.chunk;
    const int col = (static_cast<int>(unit - chunk * a.slices) * 32 + lane) * VE;
    if (col >= a.D)
        return;
    float acc[VE];
    widen<float, VE>(load_raw<float, VE>(a.parts + (a.chunks + chunk) * a.D + col), acc);
    for (int64_t c0 = chunk + 1; c0 <= last; c0 += 8) {
        Raw<float, VE> q[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (c0 + u <= last)
                q[u] = load_raw<float, VE>(a.parts + (c0 + u) * a.D + col);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (c0 + u <= last) {
                float f[VE];
                widen<float, VE>(q[u], f);
#pragma unroll
                for (int v = 0; v < VE; ++v)
                    acc[v] += f[v];
            }
    }
    put_row<G, VE>(a, r, col, acc);
}

// Elements per vector: the most, up to `most`, that divide D and that every
// pointer's alignment allows for its type.
int vector_elems(int64_t D, int most, std::initializer_list<std::pair<const void *, int>> ptrs)
{
    for (int ve = most; ve > 1; ve >>= 1) {
        bool ok = D % ve == 0;
        for (const auto &p : ptrs)
            if (p.first != nullptr &&
                reinterpret_cast<uintptr_t>(p.first) % std::min(16, ve * p.second) != 0)
                ok = false;
        if (ok)
            return ve;
    }
    return 1;
}

template <typename T, int VE>
cudaError_t lookup_launch(const void *table, const int32_t *idx, const float *weights, int64_t N,
                          int32_t k, int64_t K, int64_t D, float scale, void *out,
                          cudaStream_t stream)
{
    const int64_t blocks = (N * (D / VE) + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidValue;
    lookup_kernel<T, VE><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
        static_cast<const T *>(table), idx, weights, N, k, static_cast<int32_t>(K),
        static_cast<int32_t>(D), scale, static_cast<T *>(out));
    return cudaGetLastError();
}

template <typename T, int VE>
cudaError_t dweights_launch(const void *dout, const void *table, const int32_t *idx, int64_t M,
                            int32_t k, int64_t K, int64_t D, float scale, float *dweights,
                            cudaStream_t stream)
{
    const int64_t blocks = (M + kWarps - 1) / kWarps;
    dweights_kernel<T, VE><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
        static_cast<const T *>(dout), static_cast<const T *>(table), idx, M, k,
        static_cast<int32_t>(K), static_cast<int32_t>(D), scale, dweights);
    return cudaGetLastError();
}

template <typename T, typename G, int VE>
cudaError_t grad_launch(GradArgs a, int sms, cudaStream_t stream)
{
    a.sum_blocks = (a.chunks * a.slices + kWarps - 1) / kWarps;
    int64_t zero_blocks = 0;
    if (!a.accumulate)
        zero_blocks = std::min<int64_t>((a.K + kWarps - 1) / kWarps, int64_t(sms) * 16);
    segment_kernel<T, G, VE>
        <<<static_cast<unsigned>(a.sum_blocks + zero_blocks), kThreads, 0, stream>>>(a);
    if (a.chunks > 1)
        join_kernel<G, VE><<<static_cast<unsigned>(a.sum_blocks), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

// Sorted places per chunk: enough (chunk, slice) units for about 32 warps on
// every SM, in steps of 8 places.
int64_t chunk_places(int64_t M, int64_t slices, int sms)
{
    const int64_t want = (M * slices + int64_t(sms) * 32 - 1) / (int64_t(sms) * 32);
    return std::min<int64_t>(512, std::max<int64_t>(16, (want + 7) / 8 * 8));
}

template <typename T, typename G>
cudaError_t grad_type(GradArgs &a, int ve, int sms, cudaStream_t stream)
{
    switch (ve) {
    case 8:
        if constexpr (sizeof(T) == 2)
            return grad_launch<T, G, 8>(a, sms, stream);
    case 4:
        return grad_launch<T, G, 4>(a, sms, stream);
    case 2:
        return grad_launch<T, G, 2>(a, sms, stream);
    default:
        return grad_launch<T, G, 1>(a, sms, stream);
    }
}

int most_elems(int dtype) { return 16 / dtype_bytes(dtype); }

int grad_elems(const void *dout, int dtype, const void *dtable, int grad_dtype, int64_t D)
{
    return vector_elems(D, most_elems(dtype),
                        {{dout, dtype_bytes(dtype)}, {dtable, dtype_bytes(grad_dtype)}});
}

}  // namespace

#define KMA_BY_VE(CALL, T)                                                                        \
    switch (ve) {                                                                                 \
    case 8:                                                                                       \
        if constexpr (sizeof(T) == 2)                                                             \
            return CALL(T, 8);                                                                    \
    case 4:                                                                                       \
        return CALL(T, 4);                                                                        \
    case 2:                                                                                       \
        return CALL(T, 2);                                                                        \
    default:                                                                                      \
        return CALL(T, 1);                                                                        \
    }

cudaError_t launch_lookup(const void *table, int dtype, int64_t K, int64_t D, const int32_t *idx,
                          const float *weights, int64_t N, int32_t k, float scale, void *out,
                          cudaStream_t stream)
{
    const int es = dtype_bytes(dtype);
    const int ve = vector_elems(D, most_elems(dtype), {{table, es}, {out, es}});
#define KMA_CALL(T, VE)                                                                           \
    (lookup_launch<T, VE>(table, idx, weights, N, k, K, D, scale, out, stream))
    if (dtype == kFp32) {
        KMA_BY_VE(KMA_CALL, float)
    } else if (dtype == kBf16) {
        KMA_BY_VE(KMA_CALL, __nv_bfloat16)
    } else {
        KMA_BY_VE(KMA_CALL, __half)
    }
#undef KMA_CALL
}

cudaError_t launch_dweights(const void *dout, const void *table, int dtype, const int32_t *idx,
                            int64_t M, int32_t k, int64_t K, int64_t D, float scale,
                            float *dweights, cudaStream_t stream)
{
    const int es = dtype_bytes(dtype);
    const int ve = vector_elems(D, most_elems(dtype), {{table, es}, {dout, es}});
#define KMA_CALL(T, VE)                                                                           \
    (dweights_launch<T, VE>(dout, table, idx, M, k, K, D, scale, dweights, stream))
    if (dtype == kFp32) {
        KMA_BY_VE(KMA_CALL, float)
    } else if (dtype == kBf16) {
        KMA_BY_VE(KMA_CALL, __nv_bfloat16)
    } else {
        KMA_BY_VE(KMA_CALL, __half)
    }
#undef KMA_CALL
}
#undef KMA_BY_VE

size_t lookup_grad_parts_bytes(const void *dout, int dtype, const void *dtable, int grad_dtype,
                               int64_t M, int64_t D, int sms)
{
    const int ve = grad_elems(dout, dtype, dtable, grad_dtype, D);
    const int64_t slices = (D + 32 * ve - 1) / (32 * ve);
    const int64_t places = chunk_places(M, slices, sms);
    const int64_t chunks = (M + places - 1) / places;
    return static_cast<size_t>(2 * chunks) * D * 4;
}

cudaError_t launch_lookup_grad(const void *dout, int dtype, const float *weights, int64_t M,
                               int32_t k, int64_t K, int64_t D, float scale, int32_t skip,
                               bool accumulate, const int32_t *order, const int32_t *rows,
                               const int32_t *offsets, float *parts, void *dtable, int grad_dtype,
                               int sms, cudaStream_t stream)
{
    const int ve = grad_elems(dout, dtype, dtable, grad_dtype, D);
    GradArgs a{};
    a.dout = dout;
    a.weights = weights;
    a.order = order;
    a.rows = rows;
    a.offsets = offsets;
    a.dtable = dtable;
    a.parts = parts;
    a.slices = static_cast<int32_t>((D + 32 * ve - 1) / (32 * ve));
    a.chunk = static_cast<int32_t>(chunk_places(M, a.slices, sms));
    a.chunks = (M + a.chunk - 1) / a.chunk;
    a.k = k;
    a.K = static_cast<int32_t>(K);
    a.D = static_cast<int32_t>(D);
    a.skip = skip;
    a.scale = scale;
    a.accumulate = accumulate;
    if (dtype == kFp32)
        return grad_type<float, float>(a, ve, sms, stream);
    if (dtype == kBf16)
        return grad_dtype == kFp32 ? grad_type<__nv_bfloat16, float>(a, ve, sms, stream)
                                   : grad_type<__nv_bfloat16, __nv_bfloat16>(a, ve, sms, stream);
    return grad_dtype == kFp32 ? grad_type<__half, float>(a, ve, sms, stream)
                               : grad_type<__half, __half>(a, ve, sms, stream);
}

}  // namespace kma
