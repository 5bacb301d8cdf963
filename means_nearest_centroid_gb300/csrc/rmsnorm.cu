// rmsnorm.cu -- root-mean-square norm of rows, with the residual's addition in
// front and an output in 8 bits behind, and its gradients:
//   t = x + residual (rounded to the rows' type: what is kept is what is normed)
//   rstd = 1 / sqrt(mean(t^2) + eps),   y = t rstd w
//   8 bits: for each block of 128 columns scale = max |y| / 448, codes e4m3(y / scale)
//   g = w dy,  dx = rstd (g - t rstd mean(g t rstd)) + dt,  dw = sum over rows of dy t rstd
//
// Every element crosses HBM once in each direction.  The norm is bound by that (65,536
// x 2,048 bf16, residual added, to 8 bits: 137 us, 6.9 TB/s, DRAM 84% busy).  The
// gradient with the residual's takes 178 us there (6.0 TB/s; 165 in calls on the same
// tensors), of which the partial rows of the weight's are 8; neither DRAM (62% busy) nor
// the issue slots (54%) are full with the 16 warps an SM that its 128 registers allow.
// With single products and elements widened one by one the 165 us were 178.
// Rows at odd addresses are read element by element (30,011 x 777 fp32 gradients 60
// us, 4.7 TB/s; by aligned vectors, ends apart and the weight moved, 110).
// A row lives in the registers of one warp, or of the warps of one block where
// it is longer or where rows are few, so it is read once for its statistics and
// its output alike.  Sums are fp32.  A warp's piece of a row is a whole number
// of 128-column blocks, so the scales need shuffles only.
#include "launch.cuh"
#include "learn.h"
#include "vec.cuh"

#include <cuda_fp8.h>

#include <algorithm>

namespace kma {

namespace {

constexpr float kTop = 448.0f;             // e4m3's largest number
constexpr float kLeast = 7.8886091e-31f;   // 2^-100, under which a block's largest is taken as that

// Column of a thread's vector j: `warps` warps share the row, each warp's
// vectors go in groups that cover whole 128-column blocks.
template <int VE>
__device__ __forceinline__ int column(int j, int warps, int warp, int lane)
{
    constexpr int kGroup = VE >= 4 ? 1 : 4 / VE;
    return (((j / kGroup) * warps + warp) * kGroup + j % kGroup) * 32 * VE + lane * VE;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// The sum over the warps of a block (one row a block); slot: which half of the
// buffer, alternating from call to call.
__device__ __forceinline__ float block_sum(float v, float *buf, int warps, int slot)
{
    v = warp_sum(v);
    if (warps == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        buf[slot * 32 + (threadIdx.x >> 5)] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < warps ? buf[slot * 32 + lane] : 0.0f);
}

template <typename T, int VE>
__device__ __forceinline__ void load_weight(const void *weight, bool fp32, int col, float (&w)[VE])
{
    if (weight == nullptr) {
#pragma unroll
        for (int i = 0; i < VE; ++i)
            w[i] = 1.0f;
    } else if (fp32) {
        const float *p = static_cast<const float *>(weight) + col;
        constexpr int kPart = VE < 4 ? VE : 4;
#pragma unroll
        for (int i = 0; i < VE; i += kPart) {
            float f[kPart];
            widen<float, kPart>(load_raw<float, kPart>(p + i), f);
#pragma unroll
            for (int k = 0; k < kPart; ++k)
                w[i + k] = f[k];
        }
    } else {
        widen<T, VE>(load_raw<T, VE>(static_cast<const T *>(weight) + col), w);
    }
}

template <int VE>
__device__ __forceinline__ void store_codes(uint8_t *p, const float (&v)[VE])
{
    if constexpr (VE == 1) {
        *p = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        __nv_fp8x2_storage_t c[VE / 2];
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
            c[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE,
                                            __NV_E4M3);
        typename RawOf<VE>::type r;
        memcpy(&r, c, sizeof(r));
        *reinterpret_cast<typename RawOf<VE>::type *>(p) = r;
    }
}

struct NormArgs {
    const void *x, *residual, *weight;
    bool weight_fp32;
    int64_t N;
    int32_t D;
    float eps;
    void *total, *out;
    float *scales, *rstd;
};

// NV vectors of VE elements a thread.  warps == 1: a warp a row, four rows a
// block; else one row a block.
template <typename T, bool CODES, int VE, int NV>
__global__ void __launch_bounds__(512) rmsnorm_kernel(const NormArgs a, int warps)
{
    __shared__ float buf[32];
    const int lane = threadIdx.x & 31;
    const int warp = warps == 1 ? 0 : threadIdx.x >> 5;
    const int64_t row =
        warps == 1 ? blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5)
                   : blockIdx.x;
    wait_for_previous();
    let_next_start();
    if (row >= a.N)
        return;   // whole warps; with several warps a row, never
    const int64_t at = row * a.D;
    float t[NV][VE];
    float ss = 0.0f;
    Raw<T, VE> rx[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = column<VE>(j, warps, warp, lane);
        if (col < a.D)
            rx[j] = load_raw<T, VE>(static_cast<const T *>(a.x) + at + col);
    }
    if (a.residual != nullptr) {
        Raw<T, VE> rr[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = column<VE>(j, warps, warp, lane);
            if (col < a.D)
                rr[j] = load_raw<T, VE>(static_cast<const T *>(a.residual) + at + col);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = column<VE>(j, warps, warp, lane);
            if (col < a.D) {
                float u[VE], v[VE];
                widen<T, VE>(rx[j], u);
                widen<T, VE>(rr[j], v);
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    u[i] += v[i];
                rx[j] = narrow<T, VE>(u);
                store_raw<T, VE>(static_cast<T *>(a.total) + at + col, rx[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = column<VE>(j, warps, warp, lane);
        if (col < a.D) {
            widen<T, VE>(rx[j], t[j]);
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i)
                t[j][i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < VE; ++i)
            ss = fmaf(t[j][i], t[j][i], ss);
    }
    ss = block_sum(ss, buf, warps, 0);
    const float rstd = __frcp_rn(__fsqrt_rn(ss / static_cast<float>(a.D) + a.eps));
    if (a.rstd != nullptr && lane == 0 && warp == 0)
        a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = column<VE>(j, warps, warp, lane);
        if (col < a.D) {
            float w[VE];
            load_weight<T, VE>(a.weight, a.weight_fp32, col, w);
#pragma unroll
            for (int i = 0; i < VE; ++i)
                t[j][i] = t[j][i] * rstd * w[i];
            if (!CODES)
                store_raw<T, VE>(static_cast<T *>(a.out) + at + col, narrow<T, VE>(t[j]));
        }
    }
    if constexpr (CODES) {
        constexpr int kGroup = VE >= 4 ? 1 : 4 / VE;    // vectors of a block
        constexpr int kLanes = VE >= 4 ? 128 / VE : 32;   // lanes that share it
        const int blocks = (a.D + 127) / 128;
#pragma unroll
        for (int j = 0; j < NV; j += kGroup) {
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < kGroup; ++k)
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    top = fmaxf(top, fabsf(t[j + k][i]));
#pragma unroll
            for (int d = kLanes / 2; d > 0; d /= 2)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float scale = fmaxf(top, kLeast) / kTop;
            // y / scale, rounded to nearest: the product with the reciprocal, corrected
            // by its residual (Markstein 1990).  A row's values are often exactly
            // between two codes, and the product alone falls on either side.
            const float inverse = __frcp_rn(scale);
            const float back = scale < INFINITY ? scale : 0.0f;
            const int first = column<VE>(j, warps, warp, lane);
            if (lane % kLanes == 0 && first < a.D)
                a.scales[row * blocks + first / 128] = scale;
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                const int col = column<VE>(j + k, warps, warp, lane);
                if (col < a.D) {
                    float q[VE];
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        const float y = t[j + k][i], product = y * inverse;
                        q[i] = fmaf(fmaf(-product, back, y), inverse, product);
                    }
                    store_codes<VE>(static_cast<uint8_t *>(a.out) + at + col, q);
                }
            }
        }
    }
}

struct NormGradArgs {
    const void *dout, *total, *weight, *dtotal;
    bool weight_fp32;
    const float *rstd;
    int64_t N;
    int32_t D;
    void *dx;
    float *parts;   // [groups, D], or NULL
};

// A row's elements in pairs (alone where a vector is one element): two products an
// instruction.
template <int VE>
using Pair = std::remove_reference_t<decltype(Sums<VE>().p[0])>;
template <int VE>
constexpr int kPairs = VE == 1 ? 1 : VE / 2;

__device__ __forceinline__ float both(float v, float) { return v; }
__device__ __forceinline__ uint64_t both(float v, uint64_t) { return pair(v, v); }
__device__ __forceinline__ float times(float a, float b) { return a * b; }
__device__ __forceinline__ uint64_t times(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float fma_of(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ uint64_t fma_of(uint64_t a, uint64_t b, uint64_t c)
{
    fma_pair(c, a, b);
    return c;
}
__device__ __forceinline__ float sum_of(float v) { return v; }
__device__ __forceinline__ float sum_of(uint64_t v)
{
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    return a + b;
}

template <typename T, int VE, int NV>
struct GradRow {
    Raw<T, VE> d[NV], t[NV], s[NV];
    float rstd;
};

// A group of threads (a warp, or the block) takes rows in turn and keeps its
// share of the weight's gradient in registers; one partial row a group.  Where a
// lane holds 16 bytes of a row, the next row is on its way while this one's sum is
// joined, and the weight stays in registers (30,011 x 777 fp32 73 to 60 us, bf16 110
// to 55; with 32 bytes 60,000 x 1,024 fp32 118 to 133, and through shared memory
// 65,536 x 2,048 bf16 165 to 177, so not there).
template <typename T, int VE, int NV>
__global__ void __launch_bounds__(512, VE * NV <= 8 ? 2 : 1)
    rmsnorm_grad_kernel(const NormGradArgs a, int warps, int groups)
{
    __shared__ float buf[64];
    const int lane = threadIdx.x & 31;
    const int warp = warps == 1 ? 0 : threadIdx.x >> 5;
    const int group = warps == 1 ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    wait_for_previous();
    let_next_start();
    if (group >= groups)
        return;   // whole warps
    Sums<VE> dw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        dw[j].zero();
    const float mean = 1.0f / static_cast<float>(a.D);
    constexpr bool kAhead = VE * NV * sizeof(T) <= 16;
    Sums<VE> kept[kAhead ? NV : 1] = {};   // the weight
    const auto load_w = [&](int j, Sums<VE> &w) {
        float f[VE];
        load_weight<T, VE>(a.weight, a.weight_fp32, column<VE>(j, warps, warp, lane), f);
        w.set(f);
    };
    const auto weight_at = [&](int j, Sums<VE> &w) {
        if constexpr (kAhead)
            w = kept[j];
        else
            load_w(j, w);
    };
    const auto load = [](const Raw<T, VE> &r, Sums<VE> &to) {
        float f[VE];
        widen<T, VE>(r, f);
        to.set(f);
    };
    if constexpr (kAhead) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = column<VE>(j, warps, warp, lane);
            if (col < a.D)
                load_w(j, kept[j]);
        }
    }
    const auto load_row = [&](GradRow<T, VE, NV> &r, int64_t row) {
        const int64_t at = row * a.D;
        r.rstd = a.rstd[row];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = column<VE>(j, warps, warp, lane);
            if (col < a.D) {
                r.d[j] = load_raw<T, VE>(static_cast<const T *>(a.dout) + at + col);
                r.t[j] = load_raw<T, VE>(static_cast<const T *>(a.total) + at + col);
                if (a.dtotal != nullptr)
                    r.s[j] = load_raw<T, VE>(static_cast<const T *>(a.dtotal) + at + col);
            }
        }
    };
    GradRow<T, VE, NV> now, next;
    int slot = 0;
    if (kAhead)
        load_row(next, group);
    for (int64_t row = group; row < a.N; row += groups, slot ^= 1) {
        const int64_t at = row * a.D;
        if (kAhead) {
            now = next;
            if (row + groups < a.N)
                load_row(next, row + groups);
        } else {
            load_row(now, row);
        }
        const float rstd = now.rstd;
        const Pair<VE> rr = both(rstd, Pair<VE>{});
        Pair<VE> dots = {};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = column<VE>(j, warps, warp, lane);
            if (col < a.D) {
                Sums<VE> d, t, w;
                load(now.d[j], d);
                load(now.t[j], t);
                weight_at(j, w);
#pragma unroll
                for (int i = 0; i < kPairs<VE>; ++i) {
                    const Pair<VE> n = times(t.p[i], rr);
                    dw[j].p[i] = fma_of(d.p[i], n, dw[j].p[i]);
                    dots = fma_of(times(d.p[i], w.p[i]), n, dots);
                }
            }
        }
        const float c = block_sum(sum_of(dots), buf, warps, slot) * mean;
        const Pair<VE> minus_c = both(-c, Pair<VE>{});
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = column<VE>(j, warps, warp, lane);
            if (col < a.D) {
                Sums<VE> d, t, w, r;
                load(now.d[j], d);
                load(now.t[j], t);
                weight_at(j, w);
                if (a.dtotal != nullptr)
                    load(now.s[j], r);
                else
                    r.zero();
#pragma unroll
                for (int i = 0; i < kPairs<VE>; ++i) {
                    const Pair<VE> g = times(d.p[i], w.p[i]), n = times(t.p[i], rr);
                    r.p[i] = fma_of(fma_of(n, minus_c, g), rr, r.p[i]);
                }
                float o[VE];
                r.get(o);
                store_raw<T, VE>(static_cast<T *>(a.dx) + at + col, narrow<T, VE>(o));
            }
        }
    }
    if (a.parts != nullptr) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = column<VE>(j, warps, warp, lane);
            if (col < a.D) {
                float f[VE];
                dw[j].get(f);
                for (int i = 0; i < VE; ++i)
                    a.parts[static_cast<int64_t>(group) * a.D + col + i] = f[i];
            }
        }
    }
}

// dweight[d] = the sum of the partial rows' column d: 32 columns a block, 32
// warps a column, in an order fixed by the sizes.
__global__ void __launch_bounds__(1024)
    join_parts_kernel(const float *parts, int groups, int D, float *dweight)
{
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float v = 0.0f;
    wait_for_previous();
    if (col < D) {
#pragma unroll 8
        for (int g = warp; g < groups; g += 32)
            v += parts[static_cast<int64_t>(g) * D + col];
    }
    sums[warp][lane] = v;
    __syncthreads();
    v = warp_sum(sums[lane][warp]);
    const int out = blockIdx.x * 32 + warp;
    if (lane == 0 && out < D)
        dweight[out] = v;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int warps_for(int64_t D, int elems)
{
    return static_cast<int>((D + 32 * elems - 1) / (32 * elems));
}

// Vectors a thread: a row in one warp, or in several where it takes more than
// `elems` elements a lane, in up to 16; spread over up to 16 warps where rows
// are few.  (More than 32 elements cost the norm its occupancy: 65,536 x 2,048
// bf16 to 8 bits 64 a lane 190 us, 32 140.  The gradient holds three rows and a
// sum: 32 elements in 16 bits, 8 in fp32, 16,384 x 4,096 of which 141 us, with
// 32 183.)
template <int VE>
int vectors_for(int64_t N, int64_t D, int elems, int sms)
{
    const bool few = N <= 4 * static_cast<int64_t>(sms);
    int nv = VE == 1 ? 4 : 1;
    while (VE * nv < 64) {
        const int warps = warps_for(D, VE * nv);
        if (warps == 1 || (warps <= 16 && (few || VE * nv >= elems)))
            break;
        nv *= VE == 1 ? 4 : 2;
    }
    return nv;
}

template <typename T, bool CODES, int VE, int NV>
cudaError_t run_norm(const NormArgs &a, cudaStream_t s)
{
    const int warps = warps_for(a.D, VE * NV);
    return launch_after(rmsnorm_kernel<T, CODES, VE, NV>,
                        static_cast<unsigned>(warps == 1 ? (a.N + 3) / 4 : a.N),
                        warps == 1 ? 128 : 32 * warps, 0, s, a, warps);
}

template <typename T, bool CODES>
cudaError_t norm_shape(const NormArgs &a, int sms, cudaStream_t s)
{
    constexpr int VE = 16 / sizeof(T);
    const bool wide = a.D % VE == 0 && aligned16(a.x) && aligned16(a.residual) &&
                      aligned16(a.weight) && aligned16(a.total) && aligned16(a.out);
    if (!wide) {
        switch (vectors_for<1>(a.N, a.D, 4, sms)) {
        case 4:
            return run_norm<T, CODES, 1, 4>(a, s);
        case 16:
            return run_norm<T, CODES, 1, 16>(a, s);
        default:
            return run_norm<T, CODES, 1, 64>(a, s);
        }
    }
    switch (vectors_for<VE>(a.N, a.D, 32, sms)) {
    case 1:
        return run_norm<T, CODES, VE, 1>(a, s);
    case 2:
        return run_norm<T, CODES, VE, 2>(a, s);
    case 4:
        return run_norm<T, CODES, VE, 4>(a, s);
    case 8:
        return run_norm<T, CODES, VE, 8>(a, s);
    default:
        return run_norm<T, CODES, VE, 64 / VE>(a, s);
    }
}

template <typename T>
cudaError_t norm_type(const NormArgs &a, bool codes, int sms, cudaStream_t s)
{
    return codes ? norm_shape<T, true>(a, sms, s) : norm_shape<T, false>(a, sms, s);
}

// Row groups of the gradient: as many as are resident at once by their
// registers (64 up to 8 elements a lane), fewer where rows are few.  (65,536 x
// 2,048 bf16: 16 warps an SM 182 us, 12 208, 24, which do not all fit, 215; now 165.)
int grad_groups(int64_t N, int warps, int elems, int sms)
{
    const int resident = elems <= 8 ? 32 : 16;
    return static_cast<int>(
        std::min<int64_t>(N, sms * static_cast<int64_t>(std::max(1, resident / warps))));
}

// The gradient's shape: vectors of ve elements, nv of them a thread, warps of a row,
// groups of rows (and partial rows of the weight's gradient).
struct GradShape {
    int ve, nv, warps, groups;
};

GradShape grad_shape(const NormGradArgs &a, int dtype, int sms)
{
    const int most = 16 / dtype_bytes(dtype);
    const bool wide = a.D % most == 0 && aligned16(a.dout) && aligned16(a.total) &&
                      aligned16(a.weight) && aligned16(a.dtotal) && aligned16(a.dx);
    GradShape g;
    g.ve = wide ? most : 1;
    g.nv = !wide       ? vectors_for<1>(a.N, a.D, 4, sms)
           : most == 4 ? vectors_for<4>(a.N, a.D, 8, sms)
                       : vectors_for<8>(a.N, a.D, 32, sms);
    g.warps = warps_for(a.D, g.ve * g.nv);
    g.groups = grad_groups(a.N, g.warps, g.ve * g.nv, sms);
    return g;
}

template <typename T, int VE, int NV>
cudaError_t run_grad(const NormGradArgs &a, const GradShape &g, cudaStream_t s)
{
    return launch_after(rmsnorm_grad_kernel<T, VE, NV>,
                        g.warps == 1 ? (g.groups + 3) / 4 : g.groups,
                        g.warps == 1 ? 128 : 32 * g.warps, 0, s, a, g.warps, g.groups);
}

template <typename T>
cudaError_t grad_type(const NormGradArgs &a, const GradShape &g, cudaStream_t s)
{
    constexpr int VE = 16 / sizeof(T);
    if (g.ve == 1) {
        switch (g.nv) {
        case 4:
            return run_grad<T, 1, 4>(a, g, s);
        case 16:
            return run_grad<T, 1, 16>(a, g, s);
        default:
            return run_grad<T, 1, 64>(a, g, s);
        }
    }
    switch (g.nv) {
    case 1:
        return run_grad<T, VE, 1>(a, g, s);
    case 2:
        return run_grad<T, VE, 2>(a, g, s);
    case 4:
        return run_grad<T, VE, 4>(a, g, s);
    case 8:
        return run_grad<T, VE, 8>(a, g, s);
    default:
        return run_grad<T, VE, 64 / VE>(a, g, s);
    }
}

}  // namespace

cudaError_t launch_rmsnorm(const void *X, int dtype, int64_t N, int64_t D, const void *residual,
                           const void *weight, int weight_dtype, float eps, void *total, void *out,
                           int out_dtype, float *scales, float *rstd, int sms, cudaStream_t stream)
{
    const NormArgs a{X,   residual, weight, weight_dtype == kFp32, N, static_cast<int32_t>(D), eps,
                     total, out,    scales, rstd};
    const bool codes = out_dtype == kE4m3;
    if (dtype == kFp32)
        return norm_type<float>(a, codes, sms, stream);
    if (dtype == kBf16)
        return norm_type<__nv_bfloat16>(a, codes, sms, stream);
    return norm_type<__half>(a, codes, sms, stream);
}

cudaError_t launch_rmsnorm_grad(const void *dout, int dtype, int64_t N, int64_t D,
                                const void *total, const void *weight, int weight_dtype,
                                const float *rstd, const void *dtotal, void *dX, float *dweight,
                                cudaMemPool_t pool, int sms, cudaStream_t stream)
{
    NormGradArgs a{dout, total, weight, dtotal, weight_dtype == kFp32,
                   rstd, N,     static_cast<int32_t>(D), dX, nullptr};
    const GradShape g = grad_shape(a, dtype, sms);
    Scratch parts(dweight == nullptr ? 0 : static_cast<size_t>(g.groups) * D * sizeof(float), pool,
                  stream);
    if (!parts.ok())
        return cudaErrorMemoryAllocation;
    a.parts = reinterpret_cast<float *>(parts.get());
    cudaError_t e = dtype == kFp32   ? grad_type<float>(a, g, stream)
                    : dtype == kBf16 ? grad_type<__nv_bfloat16>(a, g, stream)
                                     : grad_type<__half>(a, g, stream);
    if (e == cudaSuccess && dweight != nullptr)
        e = launch_after(join_parts_kernel, static_cast<unsigned>((D + 31) / 32), 1024, 0, stream,
                         a.parts, g.groups, static_cast<int>(D), dweight);
    return parts.release() ? e : cudaErrorUnknown;
}

}  // namespace kma
