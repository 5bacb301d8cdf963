// experts_ptx.cuh -- the PTX wrappers that the experts' products use besides
// those of ptx.cuh: three-dimensional TMA loads, cluster-scope arrivals and waits,
// transposed operand descriptors, 8-bit MMAs.
#pragma once

#include "ptx.cuh"

namespace kma {

// Tile of a three-dimensional tensor into this CTA's shared memory, counted
// on an mbarrier of the CTA pair (cluster address).
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void *map, uint32_t cluster_bar,
                                                 int32_t x, int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void *map, uint32_t cluster_bar,
                                                 int32_t x, int32_t y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y)
        : "memory");
}

// Four rows of a two-dimensional tensor (its map's box is one row high), one
// under another.
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const void *map, uint32_t cluster_bar,
                                                 int32_t x, const int32_t (&row)[4])
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(row[0]), "r"(row[1]),
        "r"(row[2]), "r"(row[3])
        : "memory");
}

// An arrival on an mbarrier of the cluster that publishes this thread's
// shared-memory stores to the CTA that waits.
__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
                 : "memory");
}

// The waiting side of mbar_arrive_release_cluster, for a phase that is known
// to be complete: orders what follows behind it at the cluster's scope.
__device__ __forceinline__ void mbar_acquire_cluster(uint32_t bar, uint32_t parity)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}" ::"r"(bar),
                 "r"(parity)
                 : "memory");
}

// MN-major operand tile, 128-byte swizzle: atoms of 64 16-bit elements along M
// or N by 64 rows of K (128 bytes a row, 8-row groups 1024 bytes apart, the
// stride byte offset); the next 64 elements lie `lbo` bytes on (the leading
// byte offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t lbo)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// 16 lanes x 32 consecutive 32-bit columns: for each 8 columns thread t gets
// columns 2 (t % 4) and the next of lanes t / 4 and t / 4 + 8, in this order.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(r[i]);
}

// Pair MMA of 8-bit floating-point operands (K = 32), fp32 accumulate.
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor but for N (N >> 3 at bit 17): fp32 accumulator, the
// formats of A and B (kind::f16: 0 fp16, 1 bf16; kind::f8f6f4: 0 e4m3), A and B
// MN-major (bits 15, 16), M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc_base(uint32_t format, bool a_mn, bool b_mn, int M)
{
    return (1u << 4) | (format << 7) | (format << 10) | (a_mn ? 1u << 15 : 0u) |
           (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(M >> 4) << 24);
}

}  // namespace kma
