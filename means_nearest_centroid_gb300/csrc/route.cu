// route.cu -- routing: the k rows (experts, codes) of a table that each point
// goes to, and their weights, from the point's logits; and the gradient of the
// logits.
//
// With x = logits[i] widened to fp32, an expert is masked where x is -inf or
// NaN, and the scores of the others are
//     softmax:  s_e = exp(x_e - max x) / sum exp(x - max x)
//     sigmoid:  s_e = 1 / (1 + exp(-x_e))
// (masked: s = 0).  Experts are ordered by x without a bias (the order of s,
// without its rounding and saturation), by the fp32 sum s + b with one; among
// equal keys the lower index comes first.  Each fp32 step is one correctly
// rounded operation or one expf, in a fixed order, so that a row's choice does
// not depend on the batch.
#include "internal.h"
#include "vec.cuh"

#include <algorithm>

namespace kma {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRouteWarps = 8;

// Floats as unsigned numbers of the same order; 0 is below every float.
__device__ __forceinline__ uint32_t ordered(float f)
{
    const uint32_t b = __float_as_uint(f + 0.0f);   // -0 equals +0
    return (b & 0x80000000u) != 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u)
{
    return __uint_as_float((u & 0x80000000u) != 0 ? u & 0x7fffffffu : ~u);
}

// Reductions over the W lanes of a row (all lanes of the warp take part).
template <int W>
__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    if constexpr (W == 32)
        return __reduce_max_sync(kAll, v);
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1)
        v = max(v, __shfl_xor_sync(kAll, v, off));
    return v;
}
template <int W>
__device__ __forceinline__ uint32_t row_min(uint32_t v)
{
    return ~row_max<W>(~v);
}
template <int W>
__device__ __forceinline__ uint32_t row_or(uint32_t v)
{
    if constexpr (W == 32)
        return __reduce_or_sync(kAll, v);
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1)
        v |= __shfl_xor_sync(kAll, v, off);
    return v;
}
template <int W>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1)
        v += __shfl_xor_sync(kAll, v, off);
    return v;
}

__device__ __forceinline__ bool is_masked(float x) { return !(x > -INFINITY); }

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *idx;
    float *weights;
    int64_t N;
    int32_t E, k;
    int32_t groups, topk_groups, group_top;
    int32_t per_group;      // E / groups
    uint32_t group_magic;   // e / per_group == e * group_magic >> 20 for e < 1024
    bool renorm;
    float scale;
};

// One row per W lanes; lane l of them holds experts l, l + W, ... (V of them).
// The k selections are k rounds of a maximum over the row.
template <typename T, int W, int V, bool SIGMOID, bool GROUPS>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a)
{
    constexpr int kRows = 32 / W;        // rows per warp
    constexpr int kSlots = 32 / W;       // selections a lane can hold (k <= 32)
    constexpr int kKeys = W * V + (W * V >> 5);
    __shared__ float s_key[GROUPS ? kRouteWarps * kRows : 1][GROUPS ? kKeys : 1];
    __shared__ float s_group[GROUPS ? kRouteWarps * kRows : 1][GROUPS ? 32 : 1];
    const int lane = threadIdx.x & (W - 1);
    const int local = threadIdx.x / W;
    const int64_t row_any = static_cast<int64_t>(blockIdx.x) * (kRouteWarps * kRows) + local;
    const bool live = row_any < a.N;
    const int64_t row = live ? row_any : a.N - 1;   // spare lanes repeat the last row
    const T *x_row = static_cast<const T *>(a.logits) + row * a.E;

    float x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane + v * W;
        x[v] = e < a.E ? Elem<T>::up(x_row[e]) : -INFINITY;
    }

    // scores (softmax: exp(x - max), normalised by `total` below)
    float part[V];
    float top = 0.0f, total = 1.0f;
    if constexpr (SIGMOID) {
        if (GROUPS || a.bias != nullptr) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                part[v] = is_masked(x[v]) ? 0.0f : sigmoid(x[v]);
        }
    } else {
        uint32_t most = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            most = max(most, is_masked(x[v]) ? 0u : ordered(x[v]));
        top = unordered(row_max<W>(most));
        total = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            part[v] = is_masked(x[v]) ? 0.0f : expf(x[v] - top);
            total += part[v];
        }
        total = row_sum<W>(total);
    }

    // keys: 0 is never selected
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float f = x[v];
        if (a.bias != nullptr) {
            const int e = lane + v * W;
            f = (SIGMOID ? part[v] : part[v] / total) + (e < a.E ? __ldg(a.bias + e) : 0.0f);
        }
        key[v] = is_masked(x[v]) || is_masked(f) ? 0u : ordered(f);
    }

    if constexpr (GROUPS) {
        float *keys = s_key[local];
        float *of_group = s_group[local];
        const bool by_key = a.bias != nullptr || a.group_top == 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane + v * W;
            keys[e + (e >> 5)] =
                key[v] == 0 ? -INFINITY : by_key ? unordered(key[v]) : part[v];
        }
        __syncwarp();
        // lanes_per lanes form one group's key, all groups in one round where they fit
        int lanes_per = W;
        while (lanes_per > 1 && W / lanes_per < a.groups)
            lanes_per >>= 1;
        const int part_of = lane & (lanes_per - 1);
        for (int g0 = 0; g0 < a.groups; g0 += W / lanes_per) {
            const int g = g0 + lane / lanes_per;
            float first = -INFINITY, second = -INFINITY;
            if (g < a.groups)
                for (int m = part_of; m < a.per_group; m += lanes_per) {
                    const int e = g * a.per_group + m;
                    const float f = keys[e + (e >> 5)];
                    second = fmaxf(second, fminf(first, f));
                    first = fmaxf(first, f);
                }
            for (int off = lanes_per >> 1; off > 0; off >>= 1) {
                const float f1 = __shfl_xor_sync(kAll, first, off);
                const float f2 = __shfl_xor_sync(kAll, second, off);
                second = fmaxf(fminf(first, f1), fmaxf(second, f2));
                first = fmaxf(first, f1);
            }
            if (part_of == 0 && g < a.groups)
                of_group[g] = a.group_top == 1 || second == -INFINITY ? first : first + second;
        }
        __syncwarp();
        // a group stays if fewer than topk_groups are ahead of it
        uint32_t stays = 0;
        for (int g = lane; g < a.groups; g += W) {
            const float mine = of_group[g];
            int ahead = 0;
            for (int h = 0; h < a.groups; ++h) {
                const float f = of_group[h];
                ahead += f > mine || (f == mine && h < g);
            }
            if (ahead < a.topk_groups)
                stays |= 1u << g;
        }
        stays = row_or<W>(stays);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t g = (static_cast<uint32_t>(lane + v * W) * a.group_magic) >> 20;
            if (((stays >> (g & 31)) & 1u) == 0)
                key[v] = 0;
        }
    }

    int32_t mine[kSlots];
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
        mine[s] = -1;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0;
        int32_t at = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (key[v] > best) {
                best = key[v];
                at = lane + v * W;
            }
        const uint32_t most = row_max<W>(best);
        const uint32_t e = row_min<W>(best == most ? static_cast<uint32_t>(at) : ~0u);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (e == static_cast<uint32_t>(lane + v * W))
                key[v] = 0;
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            if (j == lane + s * W)
                mine[s] = most != 0 ? static_cast<int32_t>(e) : -1;
    }

    // weights, from the selected logits (just read: in L1)
    float w[kSlots];
    if (a.renorm && !SIGMOID) {
        // the selection's own maximum, so that it never underflows as a whole
        uint32_t most = 0;
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            w[s] = mine[s] >= 0 ? Elem<T>::up(x_row[mine[s]]) : -INFINITY;
            most = max(most, mine[s] >= 0 ? ordered(w[s]) : 0u);
        }
        top = unordered(row_max<W>(most));
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            w[s] = mine[s] >= 0 ? expf(w[s] - top) : 0.0f;
    } else {
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            w[s] = 0.0f;
            if (mine[s] >= 0) {
                const float f = Elem<T>::up(x_row[mine[s]]);
                w[s] = SIGMOID ? sigmoid(f) : expf(f - top);
            }
        }
    }
    if (a.renorm) {
        total = 0.0f;
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            total += w[s];
        total = row_sum<W>(total);
    }
    if (!live)
        return;
    const bool divide = a.renorm || !SIGMOID;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
        const int j = lane + s * W;
        if (j < a.k) {
            float f = w[s];
            if (divide)   // nothing selected, or sigmoids that are all 0: weight 0
                f = mine[s] < 0 || total == 0.0f ? 0.0f : f / total;
            a.idx[row * a.k + j] = mine[s];
            a.weights[row * a.k + j] = f * a.scale;
        }
    }
}

// ---- gradient -------------------------------------------------------------

struct RouteGradArgs {
    const void *logits;
    const int32_t *idx;
    const float *dweights;
    void *dlogits;
    int64_t N;
    int32_t E, k;
    bool renorm;
    float scale;
    int32_t zero_bytes;   // width of the zeroing stores: 16, 8, 4 or 2
};

template <typename Z>
__device__ __forceinline__ void zero_row(void *p, int64_t bytes, int lane)
{
    Z *q = static_cast<Z *>(p);
    const int n = static_cast<int>(bytes / sizeof(Z));
    const Z zero{};
    for (int i = lane; i < n; i += 32)
        q[i] = zero;
}

// One warp per row, lane j < k holds selection j.  The sigmoid and the
// renormalised softmax have a gradient on the selected experts only: the row
// is zeroed with wide stores, then the selected elements are written over (a
// warp's barrier orders the two).  The plain softmax has one on every expert.
//     sigmoid:             scale s_j (1 - s_j) g_j
//     sigmoid, renorm:     scale s_j (1 - s_j) / S (g_j - sum_l s_l g_l / S), S = sum_l s_l
//     softmax (, renorm):  scale p_e (g_e - sum_l p_l g_l), p over all (the selected)
template <typename T, bool SIGMOID>
__global__ void __launch_bounds__(32 * kRouteWarps) route_grad_kernel(const RouteGradArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    if (row >= a.N)
        return;
    const T *x_row = static_cast<const T *>(a.logits) + row * a.E;
    T *out = static_cast<T *>(a.dlogits) + row * a.E;
    int32_t e = lane < a.k ? __ldg(a.idx + row * a.k + lane) : -1;
    float g = 0.0f, x = -INFINITY;
    if (e < 0 || e >= a.E)
        e = -1;
    if (e >= 0) {
        g = __ldg(a.dweights + row * a.k + lane);
        x = Elem<T>::up(x_row[e]);
    }
    const bool on = e >= 0 && !is_masked(x);
    if (!on)
        g = 0.0f;
    float d;
    if (SIGMOID || a.renorm) {
        if (a.zero_bytes == 16)
            zero_row<uint4>(out, static_cast<int64_t>(a.E) * sizeof(T), lane);
        else if (a.zero_bytes == 8)
            zero_row<uint2>(out, static_cast<int64_t>(a.E) * sizeof(T), lane);
        else if (a.zero_bytes == 4)
            zero_row<uint32_t>(out, static_cast<int64_t>(a.E) * sizeof(T), lane);
        else
            zero_row<uint16_t>(out, static_cast<int64_t>(a.E) * sizeof(T), lane);
    }
    if constexpr (SIGMOID) {
        // s and s (1 - s) without cancellation, from t = exp(-|x|)
        const float t = on ? expf(-fabsf(x)) : 0.0f;
        const float s = on ? (x >= 0.0f ? 1.0f : t) / (1.0f + t) : 0.0f;
        const float slope = t / ((1.0f + t) * (1.0f + t));
        if (a.renorm) {
            const float total = row_sum<32>(s);
            const float mean = row_sum<32>(s * g) / total;
            d = total > 0.0f ? slope / total * (g - mean) : 0.0f;
        } else {
            d = slope * g;
        }
    } else {
        float top, total, p;
        if (a.renorm) {
            top = unordered(__reduce_max_sync(kAll, on ? ordered(x) : 0u));
            p = on ? expf(x - top) : 0.0f;
            total = row_sum<32>(p);
        } else {
            uint32_t most = 0;
            for (int i = lane; i < a.E; i += 32) {
                const float f = Elem<T>::up(x_row[i]);
                most = max(most, is_masked(f) ? 0u : ordered(f));
            }
            top = unordered(__reduce_max_sync(kAll, most));
            total = 0.0f;
            for (int i = lane; i < a.E; i += 32) {
                const float f = Elem<T>::up(x_row[i]);
                total += is_masked(f) ? 0.0f : expf(f - top);
            }
            total = row_sum<32>(total);
            p = on ? expf(x - top) : 0.0f;
        }
        p = on ? p / total : 0.0f;
        const float mean = row_sum<32>(p * g);
        d = p * (g - mean);
        if (!a.renorm)
            for (int i = lane; i < a.E; i += 32) {
                const float f = Elem<T>::up(x_row[i]);
                out[i] = Elem<T>::down(
                    is_masked(f) ? 0.0f : -(expf(f - top) / total) * mean * a.scale);
            }
    }
    __syncwarp();
    if (on)
        out[e] = Elem<T>::down(d * a.scale);
}

template <typename T, int W, int V>
cudaError_t route_shape(const RouteArgs &a, bool sigmoid, cudaStream_t stream)
{
    const int rows = kRouteWarps * (32 / W);
    const unsigned blocks = static_cast<unsigned>((a.N + rows - 1) / rows);
    if (sigmoid) {
        if (a.groups > 1)
            route_kernel<T, W, V, true, true><<<blocks, 32 * kRouteWarps, 0, stream>>>(a);
        else
            route_kernel<T, W, V, true, false><<<blocks, 32 * kRouteWarps, 0, stream>>>(a);
    } else {
        if (a.groups > 1)
            route_kernel<T, W, V, false, true><<<blocks, 32 * kRouteWarps, 0, stream>>>(a);
        else
            route_kernel<T, W, V, false, false><<<blocks, 32 * kRouteWarps, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t route_type(const RouteArgs &a, bool sigmoid, cudaStream_t stream)
{
    if (a.E <= 8)
        return route_shape<T, 8, 1>(a, sigmoid, stream);
    if (a.E <= 16)
        return route_shape<T, 8, 2>(a, sigmoid, stream);
    if (a.E <= 32)
        return route_shape<T, 8, 4>(a, sigmoid, stream);
    if (a.E <= 64)
        return route_shape<T, 32, 2>(a, sigmoid, stream);
    if (a.E <= 128)
        return route_shape<T, 32, 4>(a, sigmoid, stream);
    if (a.E <= 256)
        return route_shape<T, 32, 8>(a, sigmoid, stream);
    if (a.E <= 512)
        return route_shape<T, 32, 16>(a, sigmoid, stream);
    return route_shape<T, 32, 32>(a, sigmoid, stream);
}

}  // namespace

cudaError_t launch_route(const void *logits, int dtype, int64_t N, int64_t E, int32_t k,
                         bool sigmoid, const float *bias, int32_t groups, int32_t topk_groups,
                         int32_t group_top, bool renorm, float scale, int32_t *idx,
                         float *weights, cudaStream_t stream)
{
    RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.idx = idx;
    a.weights = weights;
    a.N = N;
    a.E = static_cast<int32_t>(E);
    a.k = k;
    a.groups = topk_groups < groups ? groups : 1;   // all groups stay: no choice to make
    a.topk_groups = topk_groups;
    a.group_top = group_top;
    a.per_group = a.E / groups;
    a.group_magic = (1u << 20) / static_cast<uint32_t>(a.per_group) + 1;
    a.renorm = renorm;
    a.scale = scale;
    switch (dtype) {
    case kFp32:
        return route_type<float>(a, sigmoid, stream);
    case kBf16:
        return route_type<__nv_bfloat16>(a, sigmoid, stream);
    default:
        return route_type<__half>(a, sigmoid, stream);
    }
}

cudaError_t launch_route_grad(const void *logits, int dtype, int64_t N, int64_t E, int32_t k,
                              bool sigmoid, bool renorm, float scale, const int32_t *idx,
                              const float *dweights, void *dlogits, cudaStream_t stream)
{
    RouteGradArgs a{};
    a.logits = logits;
    a.idx = idx;
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.N = N;
    a.E = static_cast<int32_t>(E);
    a.k = k;
    a.renorm = renorm;
    a.scale = scale;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(dlogits) |
                           static_cast<uintptr_t>(E * dtype_bytes(dtype));
    a.zero_bytes = bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2;
    const unsigned blocks = static_cast<unsigned>((N + kRouteWarps - 1) / kRouteWarps);
    const int threads = 32 * kRouteWarps;
    switch (dtype) {
    case kFp32:
        if (sigmoid)
            route_grad_kernel<float, true><<<blocks, threads, 0, stream>>>(a);
        else
            route_grad_kernel<float, false><<<blocks, threads, 0, stream>>>(a);
        break;
    case kBf16:
        if (sigmoid)
            route_grad_kernel<__nv_bfloat16, true><<<blocks, threads, 0, stream>>>(a);
        else
            route_grad_kernel<__nv_bfloat16, false><<<blocks, threads, 0, stream>>>(a);
        break;
    default:
        if (sigmoid)
            route_grad_kernel<__half, true><<<blocks, threads, 0, stream>>>(a);
        else
            route_grad_kernel<__half, false><<<blocks, threads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace kma
