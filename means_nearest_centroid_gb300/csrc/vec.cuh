// vec.cuh -- vectors of VE elements of a storage type T (float, __nv_bfloat16
// or __half): one raw load or store of VE * sizeof(T) bytes (2 to 32), widened
// to fp32 and rounded back (to nearest even).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

namespace kma {

struct alignas(16) Raw32 {
    uint4 lo, hi;
};
template <int BYTES>
struct RawOf;
template <>
struct RawOf<2> {
    using type = uint16_t;
};
template <>
struct RawOf<4> {
    using type = uint32_t;
};
template <>
struct RawOf<8> {
    using type = uint2;
};
template <>
struct RawOf<16> {
    using type = uint4;
};
template <>
struct RawOf<32> {
    using type = Raw32;
};
template <typename T, int VE>
using Raw = typename RawOf<static_cast<int>(sizeof(T)) * VE>::type;

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static __device__ __forceinline__ float up(float v) { return v; }
    static __device__ __forceinline__ float down(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
    static __device__ __forceinline__ float up(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half down(float v) { return __float2half_rn(v); }
};

template <typename T, int VE>
__device__ __forceinline__ Raw<T, VE> load_raw(const T *p)
{
    return *reinterpret_cast<const Raw<T, VE> *>(p);
}

// Two 16-bit elements of a word at a time, as they lie: one instruction an
// element up, one for both down.
template <typename T, int VE>
__device__ __forceinline__ void widen(const Raw<T, VE> &r, float (&f)[VE])
{
    if constexpr (sizeof(T) == 2 && VE % 2 == 0) {
        uint32_t u[VE / 2];
        memcpy(u, &r, sizeof(r));
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                f[2 * i] = __uint_as_float(u[i] << 16);
                f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            } else {
                __half2 h;
                memcpy(&h, &u[i], sizeof(h));
                const float2 v = __half22float2(h);
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    } else {
        T e[VE];
        memcpy(e, &r, sizeof(r));
#pragma unroll
        for (int i = 0; i < VE; ++i)
            f[i] = Elem<T>::up(e[i]);
    }
}

template <typename T, int VE>
__device__ __forceinline__ Raw<T, VE> narrow(const float (&f)[VE])
{
    Raw<T, VE> r;
    if constexpr (sizeof(T) == 2 && VE % 2 == 0) {
        uint32_t u[VE / 2];
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                memcpy(&u[i], &h, sizeof(h));
            } else {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                memcpy(&u[i], &h, sizeof(h));
            }
        }
        memcpy(&r, u, sizeof(r));
    } else {
        T e[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i)
            e[i] = Elem<T>::down(f[i]);
        memcpy(&r, e, sizeof(r));
    }
    return r;
}

template <typename T, int VE>
__device__ __forceinline__ void store_raw(T *p, const Raw<T, VE> &r)
{
    *reinterpret_cast<Raw<T, VE> *>(p) = r;
}

// Sums of VE elements in fp32, held in pairs: two products an instruction.
template <int VE>
struct Sums {
    static_assert(VE % 2 == 0, "pairs");
    uint64_t p[VE / 2];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
            p[i] = 0;
    }
    __device__ __forceinline__ void set(const float (&f)[VE])
    {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
            asm("mov.b64 %0, {%1, %2};" : "=l"(p[i]) : "f"(f[2 * i]), "f"(f[2 * i + 1]));
    }
    __device__ __forceinline__ void get(float (&f)[VE]) const
    {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
            asm("mov.b64 {%0, %1}, %2;" : "=f"(f[2 * i]), "=f"(f[2 * i + 1]) : "l"(p[i]));
    }
};
template <>
struct Sums<1> {
    float p[1];
    __device__ __forceinline__ void zero() { p[0] = 0.0f; }
    __device__ __forceinline__ void set(const float (&f)[1]) { p[0] = f[0]; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = p[0]; }
};

__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void fma_pair(uint64_t &acc, uint64_t a, uint64_t b)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

// acc += w * q.
template <typename T, int VE>
__device__ __forceinline__ void fma_raw(Sums<VE> &acc, const Raw<T, VE> &q, float w)
{
    float f[VE];
    widen<T, VE>(q, f);
    if constexpr (VE == 1) {
        acc.p[0] = fmaf(w, f[0], acc.p[0]);
    } else {
        const uint64_t ww = pair(w, w);
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
            fma_pair(acc.p[i], pair(f[2 * i], f[2 * i + 1]), ww);
    }
}

// The sum of acc's two elements += <p, q>, p as pairs.
template <typename T, int VE>
__device__ __forceinline__ void dot_raw(Sums<2> &acc, const Sums<VE> &p, const Raw<T, VE> &q)
{
    float f[VE];
    widen<T, VE>(q, f);
    if constexpr (VE == 1) {
        fma_pair(acc.p[0], pair(p.p[0], 0.0f), pair(f[0], 0.0f));
    } else {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
            fma_pair(acc.p[0], p.p[i], pair(f[2 * i], f[2 * i + 1]));
    }
}

}  // namespace kma
