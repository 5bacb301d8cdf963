// experts.cu -- matrix products grouped by expert: every position p of a list
// belongs to the expert e with offsets[e] <= p < offsets[e + 1], and
//   forward    out[p]  = W[e] x_p            (kForward; 16 or 8 bits)
//   rows' grad dx_p    = W[e]^T dy_p         (kRowsGrad)
//   weights'   dW[e]   = sum over p of dy_p x_p^T   (kWeightsGrad)
// with W[e] of F rows and D columns.
//
// All three are one kernel.  A cluster of two CTAs forms a tile of 256 x n
// outputs (n <= 256) by cta_group::2 MMAs: the 256 rows of the tensor-core
// tile are the contiguous axis of the OUTPUT (F, or D for the gradients), its
// columns are the positions (the weights' gradient: F).  So a ragged list costs
// what its positions need, rounded up to 32, instead of a whole tile of 128 or
// 256; and in a step of few points the weights, which are then all that
// counts, are the operand whose 128 rows a CTA streams.
//   operand A (128 rows of 128 bytes a CTA and stage): W[e] K-major (forward)
//     or MN-major (rows' gradient); X MN-major (weights' gradient)
//   operand B (n / 2 rows a CTA): the positions' rows, K-major; for the
//     weights' gradient dY MN-major
// A k-block is 128 bytes: 64 16-bit or 128 8-bit elements of the contraction,
// four MMAs.  Rows named by a list are fetched by the copy engine itself
// (gather4), four to an instruction, a lane each.
//
// Sums: the tensor cores accumulate in fp32 in tensor memory; every kSegment
// k-blocks the consumer warps add what stands there to fp32 registers (rounded
// to nearest), so that long contractions do not run in the tensor core's
// accumulator, which does not round to nearest.  With 8-bit operands a segment
// is one k-block of 128, and is multiplied by the product of its two scales on
// the way; the scale warp forms those products for the tile's columns.
//
// Contraction over positions (weights' gradient): a k-block may end behind the
// list's last position, or name rows that do not exist.  Those rows must be
// zero in both operands (0 * NaN is NaN).  The loading warp then waits for that
// k-block's rows on a barrier of its own, zeroes them in shared memory and
// arrives at the pair's barrier itself.
//
// Schedule: persistent clusters, tiles dealt out in turn; the tiles of expert e
// follow from the lists' lengths (a prefix sum that each CTA forms at its
// start), so that no host code has to know them.
#include "experts_ptx.cuh"
#include "learn.h"
#include "pipeline.cuh"

#include <cuda_fp16.h>

#include <algorithm>

namespace kma {

namespace {

constexpr int kEpilogueWarps = 8;
constexpr int kWarpA = 8, kWarpB = 9, kWarpMma = 10, kWarpScale = 11;
constexpr int kThreads = 32 * 12;
constexpr int kRowsA = 128;                        // rows of A a CTA holds
constexpr int kMaxN = 256;                         // columns of a tile
constexpr uint32_t kPartBytes = kRowsA * 128;      // one operand's k-block in a CTA
constexpr uint32_t kStageBytes = 2 * kPartBytes;
constexpr uint32_t kAtomBytes = 64 * 128;          // MN-major: 64 elements by 64 rows
constexpr int kScaleStages = 8;
constexpr uint32_t kTmemColumns = 2 * kMaxN;       // two accumulators
// 16-bit k-blocks between two additions to registers: 2,048 elements.
constexpr int kSegment = 32;

// Barriers: full and empty of each stage, of the accumulators, of the scales;
// one for each loader's k-blocks with missing rows; the last MMA's.
constexpr int kMaxRing = 8;
constexpr int kFull = 0, kEmpty = kFull + kMaxRing;
constexpr int kAccF = kEmpty + kMaxRing, kAccE = kAccF + 2;
constexpr int kScF = kAccE + 2, kScE = kScF + kScaleStages;
constexpr int kFix = kScE + kScaleStages, kLast = kFix + 2;
constexpr int kBars = kLast + 1;

struct Tile {
    int32_t e, m0, n0, n;      // expert; first row and column; columns (a multiple of 32)
    int32_t lo, hi;            // the expert's positions
    int32_t kblocks;
};

// Shared memory behind the ring: scales, then the lists' starts, ends and the
// tiles before each expert, then barriers.
struct Layout {
    uint32_t ring, scale, lists, bars, end;
};

__host__ __device__ inline Layout layout_of(int stages, int E, bool scaled)
{
    Layout l;
    l.ring = 0;
    l.scale = stages * kStageBytes;
    l.lists = l.scale + (scaled ? kScaleStages * kMaxN * 4u : 0u);
    l.bars = (l.lists + 3u * static_cast<uint32_t>(E + 1) * 4u + 15u) / 16u * 16u;
    l.end = l.bars + kBars * 8u + 16u;
    return l;
}

template <ExpertsKind KIND>
struct Schedule {
    const ExpertsParams &p;
    const int32_t *begin, *end, *before;
    int32_t mblocks, nblocks, total;

    __device__ Schedule(const ExpertsParams &p_, const int32_t *lists) : p(p_)
    {
        begin = lists;
        end = lists + (p.E + 1);
        before = lists + 2 * (p.E + 1);
        mblocks = (p.mdim + 2 * kRowsA - 1) / (2 * kRowsA);
        nblocks = (p.ndim + kMaxN - 1) / kMaxN;
        total = KIND == kWeightsGrad ? p.E * mblocks * nblocks : before[p.E] * mblocks;
    }

    __device__ Tile tile(int t) const
    {
        Tile w;
        const int q = t / mblocks;
        w.m0 = (t - q * mblocks) * 2 * kRowsA;
        if (KIND == kWeightsGrad) {
            w.e = q / nblocks;
            w.n0 = (q - w.e * nblocks) * kMaxN;
            // whole atoms of 64 columns in each CTA
            w.n = min(kMaxN, (p.ndim - w.n0 + 127) / 128 * 128);
            w.lo = begin[w.e];
            w.hi = end[w.e];
            w.kblocks = (w.hi - w.lo + 63) / 64;
            return w;
        }
        int lo = 0, hi = p.E;   // before[lo] <= q < before[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (before[mid] <= q)
                lo = mid;
            else
                hi = mid;
        }
        w.e = lo;
        w.lo = begin[lo];
        w.hi = end[lo];
        // an expert's positions in even parts of at most 256, each a multiple of 32
        const int parts = before[lo + 1] - before[lo];
        w.n = ((w.hi - w.lo + parts - 1) / parts + 31) / 32 * 32;
        w.n0 = w.lo + (q - before[lo]) * w.n;
        w.kblocks = p.kblocks;
        return w;
    }
};

// Starts, ends and tiles before each expert, by one warp.  What the offsets
// hold is clamped to [0, M], an end to its start: no position is out of range,
// whatever they are.
__device__ void form_lists(const ExpertsParams &p, int32_t *lists, int lane)
{
    int32_t *begin = lists, *end = lists + (p.E + 1), *before = lists + 2 * (p.E + 1);
    int done = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < p.E) {
            lo = p.offsets == nullptr ? 0 : min(max(__ldg(p.offsets + e), 0), p.M);
            hi = p.offsets == nullptr ? p.M : min(max(__ldg(p.offsets + e + 1), lo), p.M);
            begin[e] = lo;
            end[e] = hi;
        }
        const int tiles = (hi - lo + kMaxN - 1) / kMaxN;
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int other = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d)
                sum += other;
        }
        if (e < p.E)
            before[e] = done + sum - tiles;
        done += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0)
        before[p.E] = done;
}

// The row of an operand that position `at` stands for; -1: none.
__device__ __forceinline__ int32_t row_of(const RowMap &m, int32_t at, int32_t hi)
{
    if (at >= hi)
        return -1;
    if (m.ids == nullptr)
        return at;
    const int32_t id = __ldg(m.ids + at);
    if (id < 0)
        return -1;
    const int32_t row = m.slots == 1 ? id : id / m.slots;
    return row < m.rows ? row : -1;
}

template <int TYPE>
struct Pack;
template <>
struct Pack<kBf16> {
    static __device__ __forceinline__ uint32_t two(float a, float b)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <>
struct Pack<kFp16> {
    static __device__ __forceinline__ uint32_t two(float a, float b)
    {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};

// 32 columns of a warp's 32 rows: lane l holds element f of the columns' output
// rows, whose index is at lane c for column c (-1: not stored).  Two lanes trade
// so that each stores two neighbouring elements of one row: 64 bytes of a row
// in a warp's store.
template <int TYPE>
__device__ __forceinline__ void store_columns(const float (&v)[32], void *out, int32_t dst,
                                              int32_t f, int32_t mdim, int lane)
{
    const bool odd = lane & 1;
    uint8_t *const base = static_cast<uint8_t *>(out) + 2 * static_cast<int64_t>(f & ~1);
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        const float mine = odd ? v[c + 1] : v[c];
        const float other = __shfl_xor_sync(0xffffffffu, odd ? v[c] : v[c + 1], 1);
        const int32_t row = __shfl_sync(0xffffffffu, dst, c + (lane & 1));
        if (row >= 0 && f < mdim)
            *reinterpret_cast<uint32_t *>(base + 2 * static_cast<int64_t>(row) * mdim) =
                odd ? Pack<TYPE>::two(other, mine) : Pack<TYPE>::two(mine, other);
    }
}
template <>
__device__ __forceinline__ void store_columns<kFp32>(const float (&v)[32], void *out, int32_t dst,
                                                     int32_t f, int32_t mdim, int lane)
{
    float *const base = static_cast<float *>(out) + f;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        const int32_t row = __shfl_sync(0xffffffffu, dst, c);
        if (row >= 0 && f < mdim)
            base[static_cast<int64_t>(row) * mdim] = v[c];
    }
}

template <ExpertsKind KIND, bool E8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    experts_kernel(const __grid_constant__ CUtensorMap amap,
                   const __grid_constant__ CUtensorMap bmap, const ExpertsParams p)
{
    constexpr bool kAMn = KIND != kForward;         // A is MN-major
    constexpr bool kBMn = KIND == kWeightsGrad;
    constexpr bool kFixes = KIND == kWeightsGrad;   // loaders zero missing rows
    constexpr int kSeg = E8 ? 1 : kSegment;
    constexpr int kElems = E8 ? 128 : 64;           // elements of a k-block
    constexpr uint16_t kBoth = 0x3;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const Layout lay = layout_of(p.stages, p.E, E8);
    uint8_t *const sbase = smem_raw + (base - raw);
    int32_t *const lists = reinterpret_cast<int32_t *>(sbase + lay.lists);
    float *const scales = reinterpret_cast<float *>(sbase + lay.scale);
    volatile uint32_t *tmem_slot =
        reinterpret_cast<volatile uint32_t *>(sbase + lay.bars + kBars * 8);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    auto bar = [&](int i) -> uint32_t { return base + lay.bars + 8u * static_cast<uint32_t>(i); };
    auto lead_bar = [&](int i) -> uint32_t { return map_to_rank(bar(i), 0); };
    auto part_a = [&](uint32_t stage) { return base + stage * kStageBytes; };
    auto part_b = [&](uint32_t stage) { return base + stage * kStageBytes + kPartBytes; };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxRing; ++s) {
            // both loaders of the leader, or of both CTAs
            mbar_init(bar(kFull + s), kFixes ? 4 : 2);
            mbar_init(bar(kEmpty + s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar(kAccF + a), 1);
            mbar_init(bar(kAccE + a), 2 * kEpilogueWarps);
            mbar_init(bar(kFix + a), 1);
        }
        for (int s = 0; s < kScaleStages; ++s) {
            mbar_init(bar(kScF + s), 32);
            mbar_init(bar(kScE + s), kEpilogueWarps);
        }
        mbar_init(bar(kLast), 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == kWarpMma) {
        tmem_alloc_pair(smem_addr(const_cast<uint32_t *>(tmem_slot)), kTmemColumns);
        tmem_relinquish_pair();
    } else if (warp == 1) {
        form_lists(p, lists, lane);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers exist before any cross-CTA signal
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const Schedule<KIND> plan(p, lists);
    const int first = static_cast<int>(blockIdx.x >> 1);
    const int step = static_cast<int>(gridDim.x >> 1);
    const uint32_t stages = static_cast<uint32_t>(p.stages);
    // Copies in flight complete on the leader's barriers, out of a CTA's sight:
    // after a wait has run out they get time to land (they take microseconds).
    auto let_copies_land = [&]() {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {
        }
    };

    if (warp == kWarpA || warp == kWarpB) {
        const bool is_a = warp == kWarpA;
        uint32_t stage = 0, phase = 0, fixes = 0;
        bool ok = true;
        if (lane == 0)
            tma_prefetch_desc(is_a ? &amap : &bmap);
        auto next_stage = [&]() {
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        };
        if constexpr (kFixes) {
            // Rows of positions, 64 to a k-block, as atoms of 64 columns:
            // lane l has the four rows 4 (l % 16) .. of atom l / 16.
            const RowMap &map = is_a ? p.a_rows : p.b_rows;
            const void *tmap = is_a ? &amap : &bmap;
            const int four = 4 * (lane & 15), atom = lane >> 4;
            for (int t = first; ok && t < plan.total; t += step) {
                const Tile w = plan.tile(t);
                const int atoms = is_a ? 2 : w.n / 128;
                const int x = (is_a ? w.m0 : w.n0) + static_cast<int>(rank) * 64 * atoms;
                const uint32_t bytes = atoms * kAtomBytes;
                for (int kb = 0; ok && kb < w.kblocks; ++kb, next_stage()) {
                    const int at = w.lo + kb * 64 + four;
                    int32_t row[4];
                    uint32_t gone = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        row[i] = row_of(map, at + i, w.hi);
                        if (row[i] < 0) {
                            gone |= 1u << i;
                            row[i] = 0;   // a row that exists; zeroed below
                        }
                    }
                    const bool fix = __any_sync(0xffffffffu, gone != 0);
                    if (!(ok = wait_warp(bar(kEmpty + stage), phase ^ 1u, abort_flag, p.timeout_ns)))
                        break;
                    const uint32_t dst = is_a ? part_a(stage) : part_b(stage);
                    const uint32_t full = lead_bar(kFull + stage);
                    const uint32_t own_fix = bar(kFix + (is_a ? 0 : 1));
                    if (lane == 0) {
                        if (fix)
                            mbar_arrive_expect_tx(own_fix, bytes);
                        else if (leader)
                            mbar_arrive_expect_tx(bar(kFull + stage), 2 * bytes);
                        else
                            mbar_arrive_cluster(full);
                    }
                    __syncwarp();
                    const uint32_t done = fix ? map_to_rank(own_fix, rank) : full;
                    if (map.ids != nullptr) {
                        if (atom < atoms)
                            tma_gather4_pair(dst + atom * kAtomBytes + four * 128, tmap, done,
                                             x + 64 * atom, row);
                    } else if (lane == 0) {
                        for (int a = 0; a < atoms; ++a)
                            tma_load_2d_pair(dst + a * kAtomBytes, tmap, done, x + 64 * a,
                                             w.lo + kb * 64);
                    }
                    if (fix) {
                        ok = wait_warp(own_fix, fixes & 1u, abort_flag, p.timeout_ns);
                        ++fixes;
                        if (!ok)
                            break;
                        // whole rows: the swizzle moves 16-byte pieces within a row
                        if (atom < atoms) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (gone >> i & 1u)
                                    for (int c = 0; c < 8; ++c)
                                        st_shared_v4_u32(dst + atom * kAtomBytes + (four + i) * 128 +
                                                             16 * c,
                                                         0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive_release_cluster(full);
                    }
                }
            }
        } else if (is_a) {
            // The weights of the tile's 128 rows of this CTA.
            if (lane == 0) {
                for (int t = first; ok && t < plan.total; t += step) {
                    const Tile w = plan.tile(t);
                    const int m = w.m0 + static_cast<int>(rank) * kRowsA;
                    for (int kb = 0; kb < w.kblocks; ++kb, next_stage()) {
                        if (!(ok = wait1(bar(kEmpty + stage), phase ^ 1u, abort_flag, p.timeout_ns)))
                            break;
                        if (leader)
                            mbar_arrive_expect_tx(bar(kFull + stage), 2 * kPartBytes);
                        const uint32_t full = lead_bar(kFull + stage);
                        if (kAMn) {
                            tma_load_3d_pair(part_a(stage), &amap, full, m, kb * 64, w.e);
                            tma_load_3d_pair(part_a(stage) + kAtomBytes, &amap, full, m + 64,
                                             kb * 64, w.e);
                        } else {
                            tma_load_3d_pair(part_a(stage), &amap, full, kb * kElems, m, w.e);
                        }
                    }
                }
            }
        } else {
            // The positions' rows: this CTA's half of the tile's columns.
            for (int t = first; ok && t < plan.total; t += step) {
                const Tile w = plan.tile(t);
                const int half = w.n / 2;
                const int at = w.n0 + static_cast<int>(rank) * half;
                const bool gathers = p.b_rows.ids != nullptr;
                const int boxes = (half + 31) / 32;
                const uint32_t bytes = gathers ? half * 128 : boxes * 4096;
                int32_t row[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)   // a column without a row: any row, not stored or zero
                    row[i] = gathers ? max(row_of(p.b_rows, at + 4 * lane + i, w.hi), 0) : 0;
                for (int kb = 0; kb < w.kblocks; ++kb, next_stage()) {
                    if (!(ok = wait_warp(bar(kEmpty + stage), phase ^ 1u, abort_flag, p.timeout_ns)))
                        break;
                    if (leader && lane == 0)
                        mbar_arrive_expect_tx(bar(kFull + stage), 2 * bytes);
                    const uint32_t full = lead_bar(kFull + stage);
                    if (gathers) {
                        if (4 * lane < half)
                            tma_gather4_pair(part_b(stage) + 512 * lane, &bmap, full, kb * kElems,
                                             row);
                    } else if (lane < boxes) {
                        tma_load_2d_pair(part_b(stage) + 4096 * lane, &bmap, full, kb * kElems,
                                         at + 32 * lane);
                    }
                }
            }
        }
        if (!ok && lane == 0)
            let_copies_land();
        __syncwarp();
    } else if (warp == kWarpMma) {
        if (leader) {
            uint32_t stage = 0, phase = 0, acc = 0;
            bool ok = true, issued = false;
            for (int t = first; ok && t < plan.total; t += step) {
                const Tile w = plan.tile(t);
                const uint32_t idesc = p.idesc | static_cast<uint32_t>(w.n >> 3) << 17;
                for (int k0 = 0; ok && k0 < w.kblocks; k0 += kSeg, ++acc) {
                    const uint32_t as = acc & 1u;
                    if (!(ok = wait_warp(bar(kAccE + as), ((acc >> 1) & 1u) ^ 1u, abort_flag,
                                         p.timeout_ns)))
                        break;
                    tc_fence_after();
                    const uint32_t d = tmem_base + as * kMaxN;
                    const int k1 = min(k0 + kSeg, w.kblocks);
                    for (int kb = k0; kb < k1; ++kb) {
                        if (!(ok = wait_warp(bar(kFull + stage), phase, abort_flag, p.timeout_ns)))
                            break;
                        if (kFixes) {
                            fence_acquire_cluster();
                            fence_proxy_async_smem();
                        }
                        const uint64_t a = kAMn ? sw128_mnmajor_desc(part_a(stage), kAtomBytes)
                                                : sw128_kmajor_desc(part_a(stage));
                        const uint64_t b = kBMn ? sw128_mnmajor_desc(part_b(stage), kAtomBytes)
                                                : sw128_kmajor_desc(part_b(stage));
                        // 32 bytes of K, or 16 rows of it, an MMA
                        constexpr uint32_t kStepA = kAMn ? 128u : 2u, kStepB = kBMn ? 128u : 2u;
                        if (elect_one()) {
#pragma unroll
                            for (uint32_t k = 0; k < 4; ++k) {
                                const uint32_t add = kb != k0 || k != 0;
                                if (E8)
                                    mma_f8_pair(d, a + kStepA * k, b + kStepB * k, idesc, add);
                                else
                                    mma_bf16_pair(d, a + kStepA * k, b + kStepB * k, idesc, add);
                            }
                            mma_commit_pair(bar(kEmpty + stage), kBoth);
                            if (kb == k1 - 1)
                                mma_commit_pair(bar(kAccF + as), kBoth);
                        }
                        __syncwarp();
                        issued = true;
                        if (++stage == stages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
            if (issued) {
                if (elect_one())
                    mma_commit_pair(bar(kLast), 0x1);
                __syncwarp();
                wait_warp(bar(kLast), 0u, abort_flag, kDrainLimitNs, false);
            }
        }
    } else if (warp == kWarpScale) {
        if constexpr (E8) {
            // For each k-block the products of the columns' scales and the
            // scale of this CTA's 128 rows of weights.
            uint32_t n = 0;
            bool ok = true;
            for (int t = first; ok && t < plan.total; t += step) {
                const Tile w = plan.tile(t);
                const int fb = min((w.m0 >> 7) + static_cast<int>(rank), p.fblocks - 1);
                const float *ws =
                    p.wscale + (static_cast<int64_t>(w.e) * p.fblocks + fb) * w.kblocks;
                const float *xs[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    xs[i] = p.xscale + static_cast<int64_t>(max(
                                           row_of(p.b_rows, w.n0 + 32 * i + lane, w.hi), 0)) *
                                           w.kblocks;
                for (int kb = 0; kb < w.kblocks; ++kb, ++n) {
                    const uint32_t s = n % kScaleStages;
                    const float one = __ldg(ws + kb);
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = 32 * i < w.n ? __ldg(xs[i] + kb) * one : 0.0f;
                    if (!(ok = wait_warp(bar(kScE + s), ((n / kScaleStages) & 1u) ^ 1u, abort_flag,
                                         p.timeout_ns)))
                        break;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (32 * i < w.n)
                            scales[s * kMaxN + 32 * i + lane] = v[i];
                    mbar_arrive(bar(kScF + s));
                }
            }
        }
    } else {
        // Consumers: warp q of four holds 32 of the CTA's 128 rows, the two
        // groups of four the lower and the upper 128 columns.
        const int q = warp & 3, group = warp >> 2;
        const int c0 = group * (kMaxN / 2);
        const uint32_t tmem_warp = tmem_base + (static_cast<uint32_t>(q) << 21) + c0;
        if (p.zero_rest) {
            // Rows of no list: before the first and behind the last.
            const int32_t lo = p.E > 0 ? lists[0] : 0, hi = lists[p.E + 1 + p.E - 1];
            const int32_t rest = p.M - (hi - lo);
            const int64_t units = static_cast<int64_t>(p.mdim) * dtype_bytes(p.out_type) / 16;
            for (int64_t r = blockIdx.x * kEpilogueWarps + warp; r < rest;
                 r += gridDim.x * kEpilogueWarps) {
                const int64_t row = r < lo ? r : r - lo + hi;
                uint4 *out = static_cast<uint4 *>(p.out) + row * units;
                for (int64_t i = lane; i < units; i += 32)
                    out[i] = make_uint4(0, 0, 0, 0);
            }
        }
        uint32_t acc = 0, n = 0;
        bool ok = true;
        for (int t = first; ok && t < plan.total; t += step) {
            const Tile w = plan.tile(t);
            const int cols = min(max(w.n - c0, 0), kMaxN / 2);
            float sum[4][32];
            if (E8 || w.kblocks == 0) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        sum[c][i] = 0.0f;
            }
            for (int k0 = 0; k0 < w.kblocks; k0 += kSeg, ++acc) {
                const uint32_t as = acc & 1u;
                const uint32_t s = n % kScaleStages;
                if (E8 && !(ok = wait_warp(bar(kScF + s), (n / kScaleStages) & 1u, abort_flag,
                                           p.timeout_ns)))
                    break;
                if (!(ok = wait_warp(bar(kAccF + as), (acc >> 1) & 1u, abort_flag, p.timeout_ns)))
                    break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (32 * c < cols) {
                        float v[32];
                        tmem_ld_32x32b_x32(tmem_warp + as * kMaxN + 32 * c, v);
                        tmem_wait_ld();
                        if (E8) {
                            const uint32_t sc =
                                base + lay.scale + 4u * (s * kMaxN + c0 + 32 * c);
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 f = ld_shared_v4(sc + 4u * i);
                                fma2(sum[c][i], sum[c][i + 1], v[i], v[i + 1], f.x, f.y, sum[c][i],
                                     sum[c][i + 1]);
                                fma2(sum[c][i + 2], sum[c][i + 3], v[i + 2], v[i + 3], f.z, f.w,
                                     sum[c][i + 2], sum[c][i + 3]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                sum[c][i] = k0 == 0 ? v[i] : sum[c][i] + v[i];
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_cluster(lead_bar(kAccE + as));
                    if (E8)
                        mbar_arrive(bar(kScE + s));
                }
                ++n;
            }
            if (!ok)
                break;
            const int32_t f = w.m0 + static_cast<int>(rank) * kRowsA + 32 * q + lane;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (32 * c >= cols)
                    break;
                const int32_t at = w.n0 + c0 + 32 * c + lane;   // this lane's column
                int32_t dst;
                if (KIND == kWeightsGrad) {
                    dst = at < p.ndim ? w.e * p.ndim + at : -1;
                } else {
                    dst = row_of(p.places, at, w.hi);
                    uint32_t gone = __ballot_sync(
                        0xffffffffu, p.b_rows.ids != nullptr && row_of(p.b_rows, at, w.hi) < 0);
                    if (gone != 0) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (gone >> i & 1u)
                                sum[c][i] = 0.0f;
                    }
                }
                if (p.out_type == kBf16)
                    store_columns<kBf16>(sum[c], p.out, dst, f, p.mdim, lane);
                else if (p.out_type == kFp16)
                    store_columns<kFp16>(sum[c], p.out, dst, f, p.mdim, lane);
                else
                    store_columns<kFp32>(sum[c], p.out, dst, f, p.mdim, lane);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();   // no CTA leaves while its pair can still touch its memory
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemColumns);
    }
}

__global__ void __launch_bounds__(256)
    listed_rows_kernel(const int32_t *offsets, int32_t E, int32_t M, RowMap map, int32_t *row)
{
    const int32_t lo = offsets == nullptr ? 0 : min(max(__ldg(offsets), 0), M);
    const int32_t hi = offsets == nullptr ? M : min(max(__ldg(offsets + E), 0), M);
    for (int64_t at = blockIdx.x * 256 + threadIdx.x; at < M; at += gridDim.x * 256)
        row[at] = at < lo ? -1 : row_of(map, static_cast<int32_t>(at), hi);
}

// Ring depth that fits beside the lists and scales.
int stages_for(int E, bool scaled, size_t smem)
{
    for (int s = kMaxRing; s >= 2; --s)
        if (1024u + layout_of(s, E, scaled).end <= smem)
            return s;
    return 0;
}

template <ExpertsKind KIND, bool E8>
cudaError_t launch(const CUtensorMap &a, const CUtensorMap &b, const ExpertsParams &p, int grid,
                   size_t smem, cudaStream_t stream)
{
    experts_kernel<KIND, E8><<<grid, kThreads, smem, stream>>>(a, b, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t experts_prepare(size_t smem_optin)
{
    const void *kernels[4] = {
        (const void *)experts_kernel<kForward, false>, (const void *)experts_kernel<kForward, true>,
        (const void *)experts_kernel<kRowsGrad, false>,
        (const void *)experts_kernel<kWeightsGrad, false>};
    for (const void *k : kernels) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem_optin));
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

cudaError_t launch_experts(ExpertsKind kind, bool e8, int type, const CUtensorMap &a,
                           const CUtensorMap &b, ExpertsParams p, int sms, size_t smem_optin,
                           cudaStream_t stream)
{
    p.stages = stages_for(p.E, e8, smem_optin);
    if (p.stages == 0)
        return cudaErrorInvalidConfiguration;
    p.idesc = idesc_base(e8 ? 0u : type == kBf16 ? 1u : 0u, kind != kForward, kind == kWeightsGrad,
                         2 * kRowsA);
    const size_t smem = 1024u + layout_of(p.stages, p.E, e8).end;
    // no more clusters than tiles there can be
    const int64_t mblocks = (p.mdim + 2 * kRowsA - 1) / (2 * kRowsA);
    const int64_t tiles =
        kind == kWeightsGrad
            ? mblocks * ((p.ndim + kMaxN - 1) / kMaxN) * p.E
            : mblocks * (std::min<int64_t>(p.E, p.M) + p.M / kMaxN);
    const int grid =
        2 * static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(tiles, sms / 2)));
    switch (kind) {
    case kForward:
        return e8 ? launch<kForward, true>(a, b, p, grid, smem, stream)
                  : launch<kForward, false>(a, b, p, grid, smem, stream);
    case kRowsGrad:
        return launch<kRowsGrad, false>(a, b, p, grid, smem, stream);
    default:
        return launch<kWeightsGrad, false>(a, b, p, grid, smem, stream);
    }
}

cudaError_t launch_listed_rows(const int32_t *offsets, int32_t E, int32_t M, RowMap map,
                               int32_t *row, cudaStream_t stream)
{
    const int blocks = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(M) + 255) / 256, 4096));
    listed_rows_kernel<<<blocks, 256, 0, stream>>>(offsets, E, M, map, row);
    return cudaGetLastError();
}

cudaError_t experts_status_read_and_clear(int *code)
{
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(code, g_status_word, sizeof(int));
    if (e == cudaSuccess && *code != 0)
        e = cudaMemcpyToSymbol(g_status_word, &zero, sizeof(int));
    return e;
}

}  // namespace kma
