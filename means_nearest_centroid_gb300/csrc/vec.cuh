// vec.cuh -- vectors of VE elements of a storage type T (float, __nv_bfloat16
// or __half): one raw load or store of VE * sizeof(T) bytes (2 to 32), widened
// to fp32 and rounded back (to nearest even).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>

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

template <typename T, int VE>
__device__ __forceinline__ void widen(const Raw<T, VE> &r, float (&f)[VE])
{
    T e[VE];
    memcpy(e, &r, sizeof(r));
#pragma unroll
    for (int i = 0; i < VE; ++i)
        f[i] = Elem<T>::up(e[i]);
}

template <typename T, int VE>
__device__ __forceinline__ Raw<T, VE> narrow(const float (&f)[VE])
{
    T e[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i)
        e[i] = Elem<T>::down(f[i]);
    Raw<T, VE> r;
    memcpy(&r, e, sizeof(r));
    return r;
}

template <typename T, int VE>
__device__ __forceinline__ void store_raw(T *p, const Raw<T, VE> &r)
{
    *reinterpret_cast<Raw<T, VE> *>(p) = r;
}

// acc += w * q, in fp32 (two products an instruction).
template <typename T, int VE>
__device__ __forceinline__ void fma_raw(float (&acc)[VE], const Raw<T, VE> &q, float w)
{
    float f[VE];
    widen<T, VE>(q, f);
    if constexpr (VE == 1) {
        acc[0] = fmaf(w, f[0], acc[0]);
    } else {
#pragma unroll
        for (int i = 0; i < VE; i += 2)
            asm("{\n\t.reg .b64 a, b, c;\n\t"
                "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%0, %1};\n\t"
                "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
                : "+f"(acc[i]), "+f"(acc[i + 1])
                : "f"(f[i]), "f"(f[i + 1]), "f"(w));
    }
}

}  // namespace kma
