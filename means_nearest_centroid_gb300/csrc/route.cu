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
#include "learn.h"
#include "reciprocal.cuh"
#include "vec.cuh"

#include <algorithm>

namespace kma {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRouteWarps = 8;

// Reductions over the W lanes of a row (all lanes of the warp take part).
// fmaxf's order: a NaN loses to every number.
template <int W>
__device__ __forceinline__ float row_max(float v)
{
    if constexpr (W == 32) {
        float m;
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
        return m;
    }
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1)
        v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
    return v;
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
    int32_t group_lanes;    // lanes per group where each lane's experts are of one group, else 0
    int32_t group_shift;    // its logarithm
    uint32_t group_magic;   // e / per_group == e * group_magic >> 20 for e < 1024
    bool renorm;
    bool wide;              // every lane's experts can be loaded as one vector
    bool bias_wide;         // and their biases
    bool scored;            // the choice needs the scores, not the logits alone
    float scale;
};

// Descending order by Batcher's odd-even merge network (1968): 19, 63 and 191
// compare-exchanges for 8, 16 and 32 values.
template <int V>
__device__ __forceinline__ void sort_down(float (&s)[V])
{
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int k = p; k > 0; k /= 2)
#pragma unroll
            for (int i = 0; i + k < V; ++i)
                if (i >= k % p && ((i - k % p) & k) == 0 && i / (2 * p) == (i + k) / (2 * p)) {
                    const float hi = fmaxf(s[i], s[i + k]);
                    s[i + k] = fminf(s[i], s[i + k]);
                    s[i] = hi;
                }
}

// What an expert with key x counts in its group's sum of scores.  A softmax with
// a +inf logit is NaN there, which maxima pass over: the logit itself, so that
// its group comes first.
template <bool SIGMOID>
__device__ __forceinline__ float group_score(float x, float part)
{
    return x == -INFINITY || (!SIGMOID && x == INFINITY) ? x : part;
}

// The best two of a group's keys, held by several lanes.
struct Best2 {
    float first = -INFINITY, second = -INFINITY;
    __device__ __forceinline__ void add(float f)
    {
        second = fmaxf(second, fminf(first, f));
        first = fmaxf(first, f);
    }
    __device__ __forceinline__ void join(int off)
    {
        const float f1 = __shfl_xor_sync(kAll, first, off);
        const float f2 = __shfl_xor_sync(kAll, second, off);
        second = fmaxf(fminf(first, f1), fmaxf(second, f2));
        first = fmaxf(first, f1);
    }
    __device__ __forceinline__ float key(int32_t top) const
    {
        return top == 1 || second == -INFINITY ? first : first + second;
    }
};

// A row's logits into its W lanes, V experts each: one vector where rows are
// aligned to it, else element by element across the lanes (coalesced) and
// through shared memory (W rows of STRIDE floats).
template <typename T, int W, int V, int STRIDE>
__device__ __forceinline__ void load_row(float (&x)[V], const T *row, int E, bool wide, int lane,
                                         float *shared)
{
    constexpr int VE = V < 8 ? V : 8;
    const int e0 = lane * V;
    if (wide) {
#pragma unroll
        for (int v = 0; v < V; v += VE) {
            float f[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i)
                f[i] = -INFINITY;
            if (e0 + v < E)
                widen<T, VE>(load_raw<T, VE>(row + e0 + v), f);
#pragma unroll
            for (int i = 0; i < VE; ++i)
                x[v + i] = f[i];
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * W + lane;
            x[v] = e < E ? Elem<T>::up(row[e]) : -INFINITY;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * W + lane;
            shared[e / V * STRIDE + e % V] = x[v];
        }
        __syncwarp();
#pragma unroll
        for (int v = 0; v < V; ++v)
            x[v] = shared[lane * STRIDE + v];
        __syncwarp();
    }
}

// One row per W lanes; lane l of them holds the V experts from l V on, so
// that of equal keys the lowest lane's come first.  A key of -inf is never
// selected.  What bounds the kernel is issue: the logits are read once, but a
// score costs an exponential and a reciprocal, and the selection has to order
// k of E keys.  So each lane sorts its V keys once (a network of minima and
// maxima, without indices), and each of the k rounds takes the maximum over
// the lanes' heads and advances the list of the lowest lane that holds it;
// which expert a key belonged to is found once at the end, round j's by lane j,
// from a copy of the keys in shared memory (equal keys of a lane leave it in
// consecutive rounds: the how-manieth is counted).  Measured for 65,536 rows of
// 256 fp32 logits, k = 8, sigmoid, bias, 4 of 8 groups: 45.5 us, 1.6 TB/s (the
// bytes' floor is 10.6 us): 676 warp instructions a row, issue slots 83% busy.
// Rounds over unsorted keys took 94 us; two rows a warp (16 keys a lane) 43 us
// here, but 12% more without bias and groups.
template <typename T, int W, int V, bool SIGMOID, bool GROUPS>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a)
{
    constexpr int kRows = 32 / W;           // rows per warp
    constexpr int kSlots = 32 / W;          // selections a lane can hold (k <= 32)
    constexpr int kPad = V >= 4 ? 4 : 1;    // words after each lane's keys, against bank conflicts
    constexpr int kStride = V + kPad;
    __shared__ alignas(16) float s_key[kRouteWarps * kRows][W * kStride];
    __shared__ float s_group[GROUPS ? kRouteWarps * kRows : 1][GROUPS ? 32 : 1];
    __shared__ int2 s_round[kRouteWarps * kRows][32];
    const int lane = threadIdx.x & (W - 1);
    const int local = threadIdx.x / W;
    const int64_t row_any = static_cast<int64_t>(blockIdx.x) * (kRouteWarps * kRows) + local;
    const bool live = row_any < a.N;
    const int64_t row = live ? row_any : a.N - 1;   // spare lanes repeat the last row
    const T *x_row = static_cast<const T *>(a.logits) + row * a.E;
    const int e0 = lane * V;

    float *keys = s_key[local];
    float x[V];
    load_row<T, W, V, kStride>(x, x_row, a.E, a.wide, lane, keys);

    // scores (softmax: exp(x - max), normalised by `total`); what stands in the
    // places of masked experts is not used
    float part[V];
    float top = 0.0f, total = 1.0f;
    if constexpr (SIGMOID) {
        if (a.scored) {
            float most = 1.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float t = expf(-x[v]);   // formed for all: no branch
                part[v] = 1.0f + (is_masked(x[v]) ? 0.0f : t);
                most = fmaxf(most, part[v]);
            }
            if (__any_sync(kAll, most > 0x1p125f)) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    part[v] = 1.0f / part[v];
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    part[v] = reciprocal(part[v]);
            }
        }
    } else if (a.scored || !a.renorm) {
        float most = -INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v)
            most = fmaxf(most, x[v]);
        top = row_max<W>(most);
        total = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float t = expf(x[v] - top);
            part[v] = is_masked(x[v]) ? 0.0f : t;
            total += part[v];
        }
        total = row_sum<W>(total);
    }

    float key[V];
    if (a.bias != nullptr) {
        float b[V];
        if (a.bias_wide) {
            constexpr int VE = V < 4 ? V : 4;
#pragma unroll
            for (int v = 0; v < V; v += VE) {
                float f[VE] = {};
                if (e0 + v < a.E)
                    widen<float, VE>(load_raw<float, VE>(a.bias + e0 + v), f);
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    b[v + i] = f[i];
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                b[v] = e0 + v < a.E ? __ldg(a.bias + e0 + v) : 0.0f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float f = (SIGMOID ? part[v] : part[v] / total) + b[v];
            key[v] = is_masked(x[v]) ? -INFINITY : fmaxf(f, -INFINITY);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = fmaxf(x[v], -INFINITY);   // NaN is masked as -inf is
    }

    // the lane's keys in descending order
    float sorted[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        sorted[v] = key[v];
    sort_down<V>(sorted);

    if constexpr (GROUPS) {
        float *of_group = s_group[local];
        const bool by_key = a.bias != nullptr || a.group_top == 1;
        if (a.group_lanes > 0) {
            // a lane's experts are of one group: its lanes join theirs directly, then share
            // out the comparisons with the other groups
            Best2 b;
            if (!by_key) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    b.add(group_score<SIGMOID>(key[v], part[v]));
            } else {
                b.first = sorted[0];
                b.second = V > 1 ? sorted[V > 1 ? 1 : 0] : -INFINITY;
            }
#pragma unroll
            for (int off = 1; off < W; off <<= 1)
                if (off < a.group_lanes)
                    b.join(off);
            const float own = b.key(a.group_top);
            const int part_of = lane & (a.group_lanes - 1);
            const int g = lane >> a.group_shift;
            if (part_of == 0 && g < a.groups)
                of_group[g] = own;
            __syncwarp();
            int ahead = 0;
            for (int h = part_of; h < a.groups; h += a.group_lanes) {
                const float f = of_group[h];
                ahead += f > own || (f == own && h < g);
            }
#pragma unroll
            for (int off = 1; off < W; off <<= 1)
                if (off < a.group_lanes)
                    ahead += __shfl_xor_sync(kAll, ahead, off);
            const bool stays = ahead < a.topk_groups;
#pragma unroll
            for (int v = 0; v < V; ++v)
                sorted[v] = stays ? sorted[v] : -INFINITY;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                keys[lane * kStride + v] =
                    by_key ? key[v] : group_score<SIGMOID>(key[v], part[v]);
            __syncwarp();
            // lanes_per lanes form one group's key, all groups in one round where they fit
            int lanes_per = W;
            while (lanes_per > 1 && W / lanes_per < a.groups)
                lanes_per >>= 1;
            const int part_of = lane & (lanes_per - 1);
            for (int g0 = 0; g0 < a.groups; g0 += W / lanes_per) {
                const int g = g0 + lane / lanes_per;
                Best2 b;
                if (g < a.groups)
                    for (int m = part_of; m < a.per_group; m += lanes_per) {
                        const int e = g * a.per_group + m;
                        b.add(keys[e / V * kStride + e % V]);
                    }
                for (int off = lanes_per >> 1; off > 0; off >>= 1)
                    b.join(off);
                if (part_of == 0 && g < a.groups)
                    of_group[g] = b.key(a.group_top);
            }
            __syncwarp();
            // a group stays if fewer than topk_groups are ahead of it
            uint32_t stays = 0;
            for (int g = lane; g < a.groups; g += W) {
                const float own = of_group[g];
                int ahead = 0;
                for (int h = 0; h < a.groups; ++h) {
                    const float f = of_group[h];
                    ahead += f > own || (f == own && h < g);
                }
                if (ahead < a.topk_groups)
                    stays |= 1u << g;
            }
            stays = row_or<W>(stays);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const uint32_t g = (static_cast<uint32_t>(e0 + v) * a.group_magic) >> 20;
                if (((stays >> (g & 31)) & 1u) == 0)
                    key[v] = -INFINITY;
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                sorted[v] = key[v];
            sort_down<V>(sorted);
            __syncwarp();
        }
    }

    int32_t mine[kSlots];
#pragma unroll
    for (int q = 0; q < kSlots; ++q)
        mine[q] = -1;
    // Every key, to find the selected ones in, and each round's key and the lane that gave it
    int2 *rounds = s_round[local];
    if constexpr (V >= 4) {
#pragma unroll
        for (int v = 0; v < V; v += 4)
            *reinterpret_cast<float4 *>(keys + lane * kStride + v) =
                make_float4(key[v], key[v + 1], key[v + 2], key[v + 3]);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            keys[lane * kStride + v] = key[v];
    }
    auto round = [&](int j, int shift) {
        const float most = row_max<W>(sorted[0]);
        const uint32_t holds =
            __ballot_sync(kAll, sorted[0] == most) >> (threadIdx.x & (32 - W));
        const bool gives = lane == __ffs(holds) - 1;   // its row's lanes come first in holds
        if (gives)
            rounds[j] = make_int2(__float_as_int(most), lane);
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < shift)
                sorted[v] = !gives ? sorted[v] : v + 1 < V ? sorted[v + 1] : -INFINITY;
    };
    // round j of k can still look at k - j keys of a lane
    if (a.k <= 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < a.k)
                round(j, 7 - j);
    } else if (V > 8 && a.k <= 16) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j < a.k)
                round(j, 15 - j);
    } else {
        for (int j = 0; j < a.k; ++j)
            round(j, V);
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
        const int j = lane + q * W;
        if (q * W >= a.k || j >= a.k)
            continue;
        const int2 r = rounds[j];
        const float got = __int_as_float(r.x);
        if (got == -INFINITY)
            continue;
        uint32_t equal = 0;   // the lane's keys equal to it
        float own[V];
        if constexpr (V >= 4) {
#pragma unroll
            for (int v = 0; v < V; v += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(keys + r.y * kStride + v);
                own[v] = f.x, own[v + 1] = f.y, own[v + 2] = f.z, own[v + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                own[v] = keys[r.y * kStride + v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            equal |= own[v] == got ? 1u << v : 0u;
        // equal keys of a lane leave it in consecutive rounds
        if ((equal & (equal - 1)) != 0)
            for (int i = j - 1; i >= 0; --i) {
                const int2 before = rounds[i];
                if (__int_as_float(before.x) != got || before.y != r.y)
                    break;
                equal &= equal - 1;
            }
        mine[q] = r.y * V + __ffs(equal) - 1;
    }

    // weights, from the selected logits (just read: in L1)
    float w[kSlots];
#pragma unroll
    for (int q = 0; q < kSlots; ++q)
        w[q] = mine[q] >= 0 ? Elem<T>::up(x_row[mine[q]]) : -INFINITY;
    if (a.renorm && !SIGMOID) {
        // the selection's own maximum, so that it never underflows as a whole
        float most = -INFINITY;
#pragma unroll
        for (int q = 0; q < kSlots; ++q)
            most = fmaxf(most, w[q]);
        top = row_max<W>(most);
    }
#pragma unroll
    for (int q = 0; q < kSlots; ++q)
        if (mine[q] < 0)
            w[q] = 0.0f;
        else
            w[q] = SIGMOID ? sigmoid(w[q]) : expf(w[q] - top);
    if (a.renorm) {
        total = 0.0f;
#pragma unroll
        for (int q = 0; q < kSlots; ++q)
            total += w[q];
        total = row_sum<W>(total);
    }
    if (!live)
        return;
    const bool divide = a.renorm || !SIGMOID;
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
        const int j = lane + q * W;
        if (j < a.k) {
            float f = w[q];
            if (divide)   // nothing selected, or sigmoids that are all 0: weight 0
                f = mine[q] < 0 || total == 0.0f ? 0.0f : f / total;
            a.idx[row * a.k + j] = mine[q];
            a.weights[row * a.k + j] = f * a.scale;
        }
    }
}

// ---- gradient -------------------------------------------------------------
//
//     sigmoid:             scale s_j (1 - s_j) g_j
//     sigmoid, renorm:     scale s_j (1 - s_j) / S (g_j - sum_l s_l g_l / S), S = sum_l s_l
//     softmax (, renorm):  scale p_e (g_e - sum_l p_l g_l), p over all (the selected)
// Bound by the writes of the N E gradients.

struct RouteGradArgs {
    const void *logits;
    const int32_t *idx;
    const float *dweights;
    void *dlogits;
    int64_t N;
    int32_t E, k;
    bool renorm;
    bool wide;            // dense form: as in RouteArgs, for logits and dlogits
    float scale;
};

// Selection j of a row: expert, its logit and its weight's gradient; off where
// the id names no expert or the expert is masked.
template <typename T>
struct Chosen {
    int32_t e;
    float x = -INFINITY, g = 0.0f;
    bool on;
    __device__ __forceinline__ Chosen(const RouteGradArgs &a, int64_t row, int j, bool live)
    {
        e = live && j < a.k ? __ldg(a.idx + row * a.k + j) : -1;
        on = e >= 0 && e < a.E;
        if (on) {
            g = __ldg(a.dweights + row * a.k + j);
            x = Elem<T>::up(static_cast<const T *>(a.logits)[row * a.E + e]);
            on = !is_masked(x);
        }
        if (!on) {
            x = -INFINITY;
            g = 0.0f;
        }
    }
};

// n elements set to 0 by a warp: 16 bytes a lane between the aligned ends.
template <typename T>
__device__ __forceinline__ void zero_span(T *p, int n, int lane)
{
    constexpr int VE = 16 / sizeof(T);
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
    const int head = min(n, off == 0 ? 0 : VE - off);
    const int vecs = (n - head) / VE;
    if (lane < head)
        p[lane] = Elem<T>::down(0.0f);
    uint4 *q = reinterpret_cast<uint4 *>(p + head);
#pragma unroll 8
    for (int i = lane; i < vecs; i += 32)
        q[i] = make_uint4(0u, 0u, 0u, 0u);
    const int rest = head + vecs * VE + lane;
    if (rest < n)
        p[rest] = Elem<T>::down(0.0f);
}

// Gradients on the selected experts only (sigmoid, renormalised softmax): a
// warp zeroes 32 / KW rows with wide stores, which wait for nothing, and forms
// the selected elements meanwhile, lane j of a row's KW lanes selection j;
// they are written over the zeros behind a warp barrier.  65,536 x 256 fp32,
// k = 8: 16.7 us; the 8 logits of a row lie in as many 64-byte DRAM accesses, so
// with them 115 MB move, 6.9 TB/s.  One row a warp, zeroed after the reads: 22.7.
template <typename T, int KW, bool SIGMOID>
__global__ void __launch_bounds__(32 * kRouteWarps) route_grad_sparse_kernel(const RouteGradArgs a)
{
    constexpr int kRows = 32 / KW;
    const int lane = threadIdx.x & 31;
    const int64_t row0 =
        (static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5)) * kRows;
    if (row0 >= a.N)
        return;
    const int64_t row = row0 + lane / KW;
    const bool live = row < a.N;
    T *out = static_cast<T *>(a.dlogits);
    zero_span<T>(out + row0 * a.E,
                 static_cast<int>(min(static_cast<int64_t>(kRows), a.N - row0)) * a.E, lane);
    const Chosen<T> c(a, row, lane & (KW - 1), live);
    float d;
    if constexpr (SIGMOID) {
        // s as the weights have it, 0 below x = -88.7 (and then without a slope); s (1 - s)
        // without cancellation, from t = exp(-|x|)
        const float t = c.on ? expf(-fabsf(c.x)) : 0.0f;
        const float s = c.on ? sigmoid(c.x) : 0.0f;
        const float slope = s > 0.0f ? t / ((1.0f + t) * (1.0f + t)) : 0.0f;
        if (a.renorm) {
            const float total = row_sum<KW>(s);
            const float mean = row_sum<KW>(s * c.g) / total;
            d = total > 0.0f ? slope / total * (c.g - mean) : 0.0f;
        } else {
            d = slope * c.g;
        }
    } else {
        const float top = row_max<KW>(c.x);
        float p = c.on ? expf(c.x - top) : 0.0f;
        const float total = row_sum<KW>(p);
        p = c.on ? p / total : 0.0f;
        d = p * (c.g - row_sum<KW>(p * c.g));
    }
    // an expert that a row names more than once: its first lane takes the sum.  Each lane looks
    // at the half of the others after it (a match over the lanes took 2 us more of 6)
    const int32_t e = c.on ? c.e : -1;
    bool again = false, first = true;
#pragma unroll
    for (int off = 1; off <= KW / 2; ++off)
        again |= __shfl_sync(kAll, e, lane + off, KW) == e;
    if (__any_sync(kAll, again && e >= 0)) {
        float sum = 0.0f;
        for (int j = 0; j < KW; ++j) {
            const float f = __shfl_sync(kAll, d, j, KW);
            if (__shfl_sync(kAll, e, j, KW) == e) {
                sum += f;
                first = first && j >= (lane & (KW - 1));
            }
        }
        d = sum;
    }
    __syncwarp();
    if (c.on && first)
        out[row * a.E + c.e] = Elem<T>::down(d * a.scale);
}

// The softmax over all experts: a gradient on each of them.  Lanes and experts
// as in route_kernel; the row is read once.  65,536 x 256 bf16, k = 8: 31 us, fp32
// 35 (134 MB, 20 at HBM's rate); 30,011 x 72 bf16, k = 6: 9.3 us, of which the
// 10 MB are 1.5.  The rest is latency: a row is read, reduced twice and written by
// one warp, its selected experts marked and written again.  Finding experts named
// twice by a match over the lanes took 39 us for 35, by shuffles 36.9; marking
// before the reductions 37.2.
template <typename T, int W, int V>
__global__ void __launch_bounds__(32 * kRouteWarps) route_grad_dense_kernel(const RouteGradArgs a)
{
    constexpr int kRows = 32 / W;
    constexpr int kSlots = 32 / W;
    constexpr int VE = V < 8 ? V : 8;
    constexpr int kStride = V + (V >= 4 ? 4 : 1);
    __shared__ alignas(16) float s_row[kRouteWarps * kRows][W * kStride];
    float *stage = s_row[threadIdx.x / W];
    const int lane = threadIdx.x & (W - 1);
    const int64_t row_any =
        static_cast<int64_t>(blockIdx.x) * (kRouteWarps * kRows) + threadIdx.x / W;
    const bool live = row_any < a.N;
    const int64_t row = live ? row_any : a.N - 1;
    const T *x_row = static_cast<const T *>(a.logits) + row * a.E;
    T *out = static_cast<T *>(a.dlogits) + row * a.E;
    const int e0 = lane * V;
    float x[V];
    load_row<T, W, V, kStride>(x, x_row, a.E, a.wide, lane, stage);
    float most = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v)
        most = fmaxf(most, x[v]);
    const float top = row_max<W>(most);
    float total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[v] = is_masked(x[v]) ? 0.0f : expf(x[v] - top);
        total += x[v];
    }
    total = row_sum<W>(total);
    float mean = 0.0f, p[kSlots], g[kSlots];
    int32_t e[kSlots];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
        p[s] = g[s] = 0.0f;
        e[s] = -1;
        if (s * W < a.k) {
            const Chosen<T> c(a, row, lane + s * W, live);
            e[s] = c.on ? c.e : -1;
            g[s] = c.g;
            p[s] = c.on ? expf(c.x - top) / total : 0.0f;
            mean += p[s] * g[s];
        }
    }
    mean = row_sum<W>(mean);
    // a row without a single unmasked expert has total 0 and x 0
    const float share = total == 0.0f ? 0.0f : mean / total;
#pragma unroll
    for (int v = 0; v < V; ++v)
        x[v] = -x[v] * share * a.scale;
    if (a.wide) {
#pragma unroll
        for (int v = 0; v < V; v += VE) {
            float f[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i)
                f[i] = x[v + i];
            if (live && e0 + v < a.E)
                store_raw<T, VE>(out + e0 + v, narrow<T, VE>(f));
        }
    } else {   // back through shared memory, so that the stores are coalesced
#pragma unroll
        for (int v = 0; v < V; ++v)
            stage[lane * kStride + v] = x[v];
        __syncwarp();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = v * W + lane;
            if (live && i < a.E)
                out[i] = Elem<T>::down(stage[i / V * kStride + i % V]);
        }
    }
    // an expert that a row names more than once: its first place takes the sum.  Every place
    // marks its expert in shared memory; where another place's mark stands, there are two
    __syncwarp();
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
        if (e[s] >= 0)
            stage[e[s]] = __int_as_float(s * W + lane);
    __syncwarp();
    bool again = false;
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
        if (e[s] >= 0)
            again |= __float_as_int(stage[e[s]]) != s * W + lane;
    if (__any_sync(kAll, again)) {
        float sum[kSlots] = {};
        bool first[kSlots];
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            first[s] = true;
#pragma unroll
        for (int t = 0; t < kSlots; ++t)
            for (int j = 0; j < min(W, a.k - t * W); ++j) {
                const int32_t other = __shfl_sync(kAll, e[t], j, W);
                const float f = __shfl_sync(kAll, g[t], j, W);
#pragma unroll
                for (int s = 0; s < kSlots; ++s)
                    if (other == e[s]) {
                        sum[s] += f;
                        first[s] = first[s] && t * W + j >= s * W + lane;
                    }
            }
#pragma unroll
        for (int s = 0; s < kSlots; ++s) {
            g[s] = sum[s];
            e[s] = first[s] ? e[s] : -1;
        }
    }
    __syncwarp();
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
        if (e[s] >= 0)
            out[e[s]] = Elem<T>::down(p[s] * (g[s] - mean) * a.scale);
}

template <typename T, int W, int V>
cudaError_t route_shape(RouteArgs a, bool sigmoid, cudaStream_t stream)
{
    const uintptr_t vec = std::min<uintptr_t>(16, (V < 8 ? V : 8) * sizeof(T));
    a.wide = a.E % (V < 8 ? V : 8) == 0 && a.E * sizeof(T) % vec == 0 &&
             reinterpret_cast<uintptr_t>(a.logits) % vec == 0;
    a.bias_wide = a.E % (V < 4 ? V : 4) == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
    a.scored = a.bias != nullptr || (a.groups > 1 && a.group_top == 2);
    const int lanes = a.per_group % V == 0 ? a.per_group / V : 0;
    a.group_lanes = lanes > 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    while ((1 << a.group_shift) < a.group_lanes)
        ++a.group_shift;
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
        return route_shape<T, 8, 8>(a, sigmoid, stream);
    if (a.E <= 128)
        return route_shape<T, 16, 8>(a, sigmoid, stream);
    if (a.E <= 256)
        return route_shape<T, 32, 8>(a, sigmoid, stream);
    if (a.E <= 512)
        return route_shape<T, 32, 16>(a, sigmoid, stream);
    return route_shape<T, 32, 32>(a, sigmoid, stream);
}

template <typename T, int W, int V>
cudaError_t dense_shape(RouteGradArgs a, cudaStream_t stream)
{
    const uintptr_t vec = std::min<uintptr_t>(16, (V < 8 ? V : 8) * sizeof(T));
    a.wide = a.E % (V < 8 ? V : 8) == 0 && a.E * sizeof(T) % vec == 0 &&
             (reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits)) %
                     vec == 0;
    const int rows = kRouteWarps * (32 / W);
    route_grad_dense_kernel<T, W, V>
        <<<static_cast<unsigned>((a.N + rows - 1) / rows), 32 * kRouteWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T, int KW>
cudaError_t sparse_shape(const RouteGradArgs &a, bool sigmoid, cudaStream_t stream)
{
    const int rows = kRouteWarps * (32 / KW);
    const unsigned blocks = static_cast<unsigned>((a.N + rows - 1) / rows);
    if (sigmoid)
        route_grad_sparse_kernel<T, KW, true><<<blocks, 32 * kRouteWarps, 0, stream>>>(a);
    else
        route_grad_sparse_kernel<T, KW, false><<<blocks, 32 * kRouteWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t route_grad_type(const RouteGradArgs &a, bool sigmoid, cudaStream_t stream)
{
    if (sigmoid || a.renorm) {
        if (a.k <= 8)
            return sparse_shape<T, 8>(a, sigmoid, stream);
        return a.k <= 16 ? sparse_shape<T, 16>(a, sigmoid, stream)
                         : sparse_shape<T, 32>(a, sigmoid, stream);
    }
    if (a.E <= 8)
        return dense_shape<T, 8, 1>(a, stream);
    if (a.E <= 16)
        return dense_shape<T, 8, 2>(a, stream);
    if (a.E <= 32)
        return dense_shape<T, 8, 4>(a, stream);
    if (a.E <= 64)
        return dense_shape<T, 8, 8>(a, stream);
    if (a.E <= 128)
        return dense_shape<T, 16, 8>(a, stream);
    if (a.E <= 256)
        return dense_shape<T, 32, 8>(a, stream);
    if (a.E <= 512)
        return dense_shape<T, 32, 16>(a, stream);
    return dense_shape<T, 32, 32>(a, stream);
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
    switch (dtype) {
    case kFp32:
        return route_grad_type<float>(a, sigmoid, stream);
    case kBf16:
        return route_grad_type<__nv_bfloat16>(a, sigmoid, stream);
    default:
        return route_grad_type<__half>(a, sigmoid, stream);
    }
}

}  // namespace kma
