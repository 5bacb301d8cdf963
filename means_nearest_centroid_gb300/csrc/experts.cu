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
// counts, are the operand whose 128 rows a CTA streams.  (8 bits with many
// positions are the other way round: experts8_kernel below.)
//   operand A (128 rows of 128 bytes a CTA and stage): W[e] K-major (forward)
//     or MN-major (rows' gradient); X MN-major (weights' gradient)
//   operand B (n / 2 rows a CTA): the positions' rows, K-major; for the
//     weights' gradient dY MN-major
// A k-block is 128 bytes: 64 16-bit or 128 8-bit elements of the contraction,
// four MMAs.
//
// Rows named by ids.  Few positions: the copy engine fetches them (gather4, four
// rows an instruction, a lane each).  That takes it 75 clocks an instruction,
// which many positions cannot wait for (131,072 positions of 2,048: the product
// 1,100 us); nor for copies by threads (cp.async: 18 bytes a clock and SM, 460
// us).  There a pass of its own gathers the rows first (116 us of 463).
//
// Sums: the tensor cores accumulate in fp32 in tensor memory; every kSegment
// k-blocks the consumer warps add what stands there to fp32 registers (rounded
// to nearest), so that long contractions do not run in the tensor core's
// accumulator, which does not round to nearest.  With 8-bit operands a segment
// is one k-block of 128, and is multiplied by the product of its two scales on
// the way; the scale warp forms those products for the tile's columns.
//
// Measured on GB300: 131,072 positions in 64 lists, 2,048 x 1,024 bf16: forward
// 314 us (1,750 TFLOP/s; torch.bmm over equal lists 287-298), rows' gradient 324,
// weights' 316 (fp32: 350).  32,768 in 8 lists, 4,096 x 4,096: 555 (1,980;
// torch.bmm 525-537).  256 lists of 128 of 2,048 x 1,024: 201, bound by HBM (1.27
// GB).  Sixteen points to 8 of 256 experts: 74 us for 428 MB, bound by HBM.
//
// Contraction over positions (weights' gradient): a k-block may end behind the
// list's last position, or hold positions that lack a row.  Those rows must be
// zero in both operands (0 * NaN is NaN).  The copies of such a k-block complete
// on barriers of this CTA; a warp waits for them, zeroes the rows in shared
// memory and passes the k-block on to the pair.
//
// Schedule: persistent clusters, tiles dealt out in turn; the tiles of expert e
// follow from the lists' lengths (a prefix sum that each CTA forms at its
// start), so that no host code has to know them.
#include "experts_ptx.cuh"
#include "launch.cuh"
#include "learn.h"
#include "pipeline.cuh"
#include "vec.cuh"

#include <algorithm>

namespace kma {

namespace {

constexpr int kConsumers = 8;   // warps; then one each for A, B, the MMAs,
constexpr int kWarpA = 8, kWarpB = 9, kWarpMma = 10;   // and the last, scales or fixes
constexpr int kThreads = 32 * 12;
// Registers a thread: the two warpgroups of consumers hold up to 128 sums each,
// the third gives up some of the launch's for them.
constexpr int kConsumerRegs = 208, kOtherRegs = 80;
static_assert(2 * kConsumerRegs + kOtherRegs <= 3 * 168, "the launch's registers");
constexpr int kRowsA = 128;                        // rows of A a CTA holds
constexpr uint32_t kPartA = kRowsA * 128;          // A's k-block in a CTA
constexpr uint32_t kAtomBytes = 64 * 128;          // MN-major: 64 elements by 64 rows
// Scales: a ring of groups of four k-blocks (one hand-over for four segments).
constexpr int kScaleStages = 2, kScaleGroup = 4;
__host__ __device__ constexpr uint32_t scale_bytes(int NT) { return kScaleGroup * NT * 4u; }
constexpr uint32_t kWarpStaging = 2048;            // of a warp of consumers, for its way out
// 16-bit k-blocks between two additions to registers: 2,048 elements, or 512
// positions of a weights' gradient in fp32.
constexpr int kSegment = 32, kSegmentRows = 8;

// Barriers: full and empty of each stage, of the accumulators, of the scales;
// those of each operand's stages while rows are missing; the issuers' last MMAs'.
constexpr int kMaxRing = 10;
constexpr int kFull = 0, kEmpty = kFull + kMaxRing;
constexpr int kAccF = kEmpty + kMaxRing, kAccE = kAccF + 2;
constexpr int kScF = kAccE + 2, kScE = kScF + kScaleStages;
constexpr int kFixA = kScE + kScaleStages, kFixB = kFixA + kMaxRing, kLast = kFixB + kMaxRing;
constexpr int kBars = kLast + 2;

struct Tile {
    int32_t e, m0, n0, n;      // expert; first row and column; columns (a multiple of 32)
    int32_t lo, hi;            // the expert's positions
    int32_t kblocks;
};

// Shared memory behind the ring: the consumers' staging, scales, then the lists'
// starts, ends and the tiles before each expert, then barriers.
struct Layout {
    uint32_t staging, scale, lists, bars, end;
};

__host__ __device__ constexpr uint32_t stage_bytes(int NT) { return kPartA + NT / 2 * 128; }

__host__ __device__ inline Layout layout_of(int NT, int stages, int E, bool scaled)
{
    Layout l;
    l.staging = stages * stage_bytes(NT);
    l.scale = l.staging + kConsumers * kWarpStaging;
    l.lists = l.scale + (scaled ? kScaleStages * scale_bytes(NT) : 0u);
    l.bars = (l.lists + 3u * static_cast<uint32_t>(E + 1) * 4u + 15u) / 16u * 16u;
    l.end = l.bars + kBars * 8u + 16u;
    return l;
}

template <ExpertsKind KIND, int NT>
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
        nblocks = (p.ndim + NT - 1) / NT;
        total = KIND == kWeightsGrad ? p.E * mblocks * nblocks : before[p.E] * mblocks;
    }

    __device__ Tile tile(int t) const
    {
        Tile w;
        const int q = t / mblocks;
        w.m0 = (t - q * mblocks) * 2 * kRowsA;
        if (KIND == kWeightsGrad) {
            w.e = q / nblocks;
            w.n0 = (q - w.e * nblocks) * NT;
            // whole atoms of 64 columns in each CTA
            w.n = min(NT, (p.ndim - w.n0 + 127) / 128 * 128);
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
        // an expert's positions, in units of 32, in parts as even as can be
        const int parts = before[lo + 1] - before[lo], part = q - before[lo];
        const int units = (w.hi - w.lo + 31) / 32;
        const int each = units / parts, more = units - each * parts;
        w.n = 32 * (each + (part < more));
        w.n0 = w.lo + 32 * (part * each + min(part, more));
        w.kblocks = p.kblocks;
        return w;
    }
};

// Starts, ends and tiles before each expert, by one warp.  What the offsets
// hold is clamped to [0, M], and no list starts before the one in front of it
// ends: whatever they are, no position is out of range and the lists have at most
// M positions together, so that the tiles' numbers fit 31 bits.
// A lane takes eight lists of 256, so that their offsets come with one latency
// (32 lists at a time: 2 us more of a product of 256 lists).
template <int NT>
__device__ void form_lists(const ExpertsParams &p, int32_t *lists, int lane)
{
    constexpr int kEach = 8;
    int32_t *begin = lists, *end = lists + (p.E + 1), *before = lists + 2 * (p.E + 1);
    int done = 0, reached = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32 * kEach) {
        const int first = e0 + kEach * lane;
        int at[kEach + 1];   // lists first + i start at at[i], end at at[i + 1]
        bool falls = false;
#pragma unroll
        for (int i = 0; i <= kEach; ++i) {
            const int e = first + i;
            at[i] = e > p.E               ? p.M
                    : p.offsets == nullptr ? (e == 0 ? 0 : p.M)
                                           : min(max(p.offsets[e], 0), p.M);
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            falls |= at[i + 1] < at[i];
        if (__any_sync(0xffffffffu, falls || at[0] < reached)) {
            at[0] = max(at[0], reached);
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                at[i + 1] = max(at[i + 1], at[i]);
            int top = at[kEach];
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int other = __shfl_up_sync(0xffffffffu, top, d);
                if (lane >= d)
                    top = max(top, other);
            }
            top = __shfl_up_sync(0xffffffffu, top, 1);
#pragma unroll
            for (int i = 0; i <= kEach; ++i)
                at[i] = lane == 0 ? at[i] : max(at[i], top);
        }
        reached = __shfl_sync(0xffffffffu, at[kEach], 31);
        int tiles = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            tiles += first + i < p.E ? (at[i + 1] - at[i] + NT - 1) / NT : 0;
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int other = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d)
                sum += other;
        }
        int here = done + sum - tiles;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int e = first + i;
            if (e < p.E) {
                begin[e] = at[i];
                end[e] = at[i + 1];
                before[e] = here;
                here += (at[i + 1] - at[i] + NT - 1) / NT;
            }
        }
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
    const int32_t id = m.ids[at];
    if (id < 0)
        return -1;
    const int32_t row = m.slots == 1 ? id : id / m.slots;
    return row < m.rows ? row : -1;
}

__device__ __forceinline__ void zero16(uint32_t addr) { st_shared_v4_u32(addr, 0, 0, 0, 0); }

// Weights' gradient: whether a position adds nothing.
__device__ __forceinline__ bool missing(const ExpertsParams &p, int32_t at, int32_t hi)
{
    return row_of(p.from, at, hi) < 0 || row_of(p.placed, at, hi) < 0;
}

// After a wait has run out: no warp of the CTA issues copies any more (one thread calls
// this behind the block's barrier), but some may be in flight, and they complete on the
// leader's barriers, whose phases need both CTAs' copies of a stage and may never end.
// They get as long as the bound that ran out, from 1 ms to the teardown's limit, before
// either CTA leaves.  (All CTAs' rings are 48 MB at most, 8 us at HBM's rate.)
__device__ __forceinline__ void let_copies_land(uint64_t bound_ns)
{
    const uint64_t limit = min(max(bound_ns, uint64_t(1000000)), kDrainLimitNs);
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < limit) {
    }
}

// Waits for a stage's operands (a whole warp).  Where threads of either CTA may
// have written them, the wait acquires at the cluster's scope.
__device__ __forceinline__ bool wait_operands(uint32_t bar, uint32_t parity, bool threads_write,
                                              volatile uint32_t *abort_flag, uint64_t limit_ns)
{
    if (!wait_warp(bar, parity, abort_flag, limit_ns))
        return false;
    if (threads_write)
        mbar_acquire_cluster(bar, parity);   // complete already: returns at once
    return true;
}

// A warp's sums: 32 rows (elements of an output row) by COLS columns (output
// rows).  Lane l holds, for each half of 16 rows and each 8 columns, rows l / 4
// and l / 4 + 8 of columns 2 (l % 4) and the next: v[0], v[1] and v[2], v[3].
template <int COLS>
struct Frags {
    float v[COLS / 8][2][4];
};

// 8 x 8 16-bit matrices out of such fragments to shared memory, transposed:
// lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void store_matrices(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                               uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

template <typename O>
__device__ __forceinline__ uint32_t pack_two(float a, float b)
{
    const O two[2] = {Elem<O>::down(a), Elem<O>::down(b)};
    uint32_t r;
    memcpy(&r, two, 4);
    return r;
}

// 32 columns of a warp's fragments become rows of the output by way of the warp's
// own shared memory: 64 bytes of 32 rows (fp32: 128 bytes of 16, twice), whose
// 16-byte pieces are moved about so that no two lanes meet in a bank, and which
// go out a row to four lanes (fp32: eight).  No warp waits for another: with four
// warps meeting over runs of 256 bytes the weights' gradient of 256 lists of 128,
// whose stores take longer than its product, took 285 us (here 259; fp32 440, 384).
// dst: lane c has column c's row of the output; -1: none, -2 - row: a row of zeros.
template <typename O>
__device__ __forceinline__ void store_columns(const float (*v)[2][4], uint8_t *stage, int32_t dst,
                                              void *out, int32_t f, int32_t mdim, int lane)
{
    constexpr int kCols = sizeof(O) == 2 ? 32 : 16;   // at a time
    constexpr int kPieces = 2 * sizeof(O);            // of 16 bytes in a row's 32 elements
    const int piece = lane % kPieces;
    const bool inside = f + piece * (16 / static_cast<int>(sizeof(O))) < mdim;
    uint8_t *const to =
        static_cast<uint8_t *>(out) + f * static_cast<int64_t>(sizeof(O)) + 16 * piece;
    const int64_t pitch = static_cast<int64_t>(mdim) * sizeof(O);
    auto at = [&](int col, int p) {
        return stage + col * (32 * sizeof(O)) +
               16 * (p ^ (sizeof(O) == 2 ? col >> 1 & 3 : col & 7));
    };
#pragma unroll
    for (int c = 0; c < 32; c += kCols) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kCols / 8; ++j) {
            const float(&w)[2][4] = v[c / 8 + j];
            if constexpr (sizeof(O) == 2) {
                store_matrices(smem_addr(at(8 * j + (lane & 7), lane >> 3)),
                               pack_two<O>(w[0][0], w[0][1]), pack_two<O>(w[0][2], w[0][3]),
                               pack_two<O>(w[1][0], w[1][1]), pack_two<O>(w[1][2], w[1][3]));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = 16 * (i >> 2) + 8 * (i >> 1 & 1) + (lane >> 2);
                    *reinterpret_cast<float *>(at(8 * j + 2 * (lane & 3) + (i & 1), row >> 2) +
                                               4 * (row & 3)) = w[i >> 2][i & 3];
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kCols; i += 32 / kPieces) {
            const int col = i + lane / kPieces;
            const int32_t d = __shfl_sync(0xffffffffu, dst, c + col);
            uint4 w = *reinterpret_cast<const uint4 *>(at(col, piece));
            if (d < -1)
                w = make_uint4(0, 0, 0, 0);
            const int32_t row = d < -1 ? -2 - d : d;
            if (row >= 0 && inside)
                *reinterpret_cast<uint4 *>(to + row * pitch) = w;
        }
    }
}

// Zeros in the rows of no list, before the first and behind the last: one of
// `of` warps' share.
__device__ __forceinline__ void zero_rows(const ExpertsParams &p, const int32_t *lists,
                                          int64_t warp, int64_t of, int lane)
{
    const int32_t lo = lists[0], hi = lists[p.E + 1 + p.E - 1];
    const int32_t rest = p.M - (hi - lo);
    const int64_t units = static_cast<int64_t>(p.mdim) * dtype_bytes(p.out_type) / 16;
    for (int64_t r = warp; r < rest; r += of) {
        const int64_t row = r < lo ? r : r - lo + hi;
        uint4 *out = static_cast<uint4 *>(p.out) + row * units;
        for (int64_t i = lane; i < units; i += 32)
            out[i] = make_uint4(0, 0, 0, 0);
    }
}

template <ExpertsKind KIND, bool E8, int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    experts_kernel(const __grid_constant__ CUtensorMap amap,
                   const __grid_constant__ CUtensorMap bmap, const ExpertsParams p)
{
    constexpr bool kAMn = KIND != kForward;         // A is MN-major
    constexpr bool kBMn = KIND == kWeightsGrad;
    constexpr bool kFixes = KIND == kWeightsGrad;   // missing rows are zeroed
    const int kSeg = E8 ? 1 : p.segment;            // k-blocks between additions
    constexpr int kElems = E8 ? 128 : 64;           // elements of a k-block
    constexpr bool kGathers = KIND == kForward && NT == 64;
    constexpr uint32_t kStageBytes = stage_bytes(NT);
    constexpr int kGroupCols = NT / 2;              // columns of a group of consumers
    constexpr uint32_t kTmemColumns = 2 * NT;       // two accumulators
    constexpr uint16_t kBoth = 0x3;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const Layout lay = layout_of(NT, p.stages, p.E, E8);
    uint8_t *const sbase = smem_raw + (base - raw);
    int32_t *const lists = reinterpret_cast<int32_t *>(sbase + lay.lists);
    volatile uint32_t *tmem_slot =
        reinterpret_cast<volatile uint32_t *>(sbase + lay.bars + kBars * 8);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    auto bar = [&](int i) -> uint32_t { return base + lay.bars + 8u * static_cast<uint32_t>(i); };
    auto lead_bar = [&](int i) -> uint32_t { return map_to_rank(bar(i), 0); };
    // Bounded waits on barrier i, of a warp and of one thread.
    auto wait = [&](int i, uint32_t parity) {
        return wait_warp(bar(i), parity, abort_flag, p.timeout_ns);
    };
    auto wait_one = [&](int i, uint32_t parity) {
        return wait1(bar(i), parity, abort_flag, p.timeout_ns);
    };
    auto part_a = [&](uint32_t stage) { return base + stage * kStageBytes; };
    auto part_b = [&](uint32_t stage) { return base + stage * kStageBytes + kPartA; };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const bool gathers = kGathers && p.b_rows.ids != nullptr;

    if (threadIdx.x == 32) {
        tma_prefetch_desc(&amap);
        tma_prefetch_desc(&bmap);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxRing; ++s) {
            // the leader's loaders; both CTAs' where rows may be missing
            mbar_init(bar(kFull + s), kFixes ? 4 : 2);
            mbar_init(bar(kEmpty + s), 1);
            mbar_init(bar(kFixA + s), 1);
            mbar_init(bar(kFixB + s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar(kAccF + a), 1);
            mbar_init(bar(kAccE + a), 2 * kConsumers);
        }
        mbar_init(bar(kLast), 1);
        for (int s = 0; s < kScaleStages; ++s) {
            mbar_init(bar(kScF + s), 1);
            mbar_init(bar(kScE + s), kConsumers);
        }
        *abort_flag = 0u;
        fence_mbar_init();
    }
    wait_for_previous();
    let_next_start();   // all blocks of this launch are resident: the next one may set itself up
    if (warp == kWarpMma) {
        tmem_alloc_pair(smem_addr(const_cast<uint32_t *>(tmem_slot)), kTmemColumns);
        tmem_relinquish_pair();
    } else if (warp == 1) {
        form_lists<NT>(p, lists, lane);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers exist before any cross-CTA signal
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const Schedule<KIND, NT> plan(p, lists);
    const int first = static_cast<int>(blockIdx.x >> 1);
    const int step = static_cast<int>(gridDim.x >> 1);
    const uint32_t stages = static_cast<uint32_t>(p.stages);

    if (warp >= kConsumers) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kWarpA || warp == kWarpB) {
            const bool is_a = warp == kWarpA;
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            auto next_stage = [&]() {
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            };
            if constexpr (kFixes) {
                // Rows of positions, 64 to a k-block, as atoms of 64 columns.
                const void *tmap = is_a ? &amap : &bmap;
                const bool holes = p.holes != nullptr && *p.holes != 0;
                for (int t = first; ok && t < plan.total; t += step) {
                    const Tile w = plan.tile(t);
                    const int atoms = is_a ? 2 : w.n / 128;
                    const int x = (is_a ? w.m0 : w.n0) + static_cast<int>(rank) * 64 * atoms;
                    const uint32_t bytes = atoms * kAtomBytes;
                    for (int kb = 0; ok && kb < w.kblocks; ++kb, next_stage()) {
                        const int at = w.lo + kb * 64;
                        const bool fix = at + 64 > w.hi || holes;
                        if (!(ok = wait(kEmpty + stage, phase ^ 1u)))
                            break;
                        const uint32_t dst = is_a ? part_a(stage) : part_b(stage);
                        const uint32_t full = lead_bar(kFull + stage);
                        const uint32_t own = bar((is_a ? kFixA : kFixB) + stage);
                        if (lane == 0) {
                            if (fix)   // the fixing warp goes on from here
                                mbar_arrive_expect_tx(own, bytes);
                            else if (leader)
                                mbar_arrive_expect_tx(bar(kFull + stage), 2 * bytes);
                            else
                                mbar_arrive_cluster(full);
                            const uint32_t done = fix ? map_to_rank(own, rank) : full;
                            for (int a = 0; a < atoms; ++a)
                                tma_load_2d_pair(dst + a * kAtomBytes, tmap, done, x + 64 * a, at);
                        }
                        __syncwarp();
                    }
                }
            } else if (is_a) {
                // The weights of the tile's 128 rows of this CTA.
                if (lane == 0) {
                    for (int t = first; ok && t < plan.total; t += step) {
                        const Tile w = plan.tile(t);
                        const int m = w.m0 + static_cast<int>(rank) * kRowsA;
                        for (int kb = 0; kb < w.kblocks; ++kb, next_stage()) {
                            if (!(ok = wait_one(kEmpty + stage, phase ^ 1u)))
                                break;
                            if (leader)
                                mbar_arrive_expect_tx(bar(kFull + stage), 2 * kPartA);
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
                    const int boxes = (half + 31) / 32;
                    const uint32_t bytes = gathers ? half * 128 : boxes * 4096;
                    int32_t row[4];
                    if (kGathers) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)   // none: any row, the column is not used
                            row[i] = !gathers ? 0
                                              : max(row_of(p.b_rows, at + 4 * lane + i, w.hi), 0);
                    }
                    for (int kb = 0; kb < w.kblocks; ++kb, next_stage()) {
                        if (!(ok = wait(kEmpty + stage, phase ^ 1u)))
                            break;
                        if (leader && lane == 0)
                            mbar_arrive_expect_tx(bar(kFull + stage), 2 * bytes);
                        const uint32_t full = lead_bar(kFull + stage);
                        if (gathers) {
                            if (4 * lane < half)
                                tma_gather4_pair(part_b(stage) + 512 * lane, &bmap, full,
                                                 kb * kElems, row);
                        } else if (lane < boxes) {
                            tma_load_2d_pair(part_b(stage) + 4096 * lane, &bmap, full, kb * kElems,
                                             at + 32 * lane);
                        }
                    }
                }
            }
            __syncwarp();
        } else if (warp == kWarpMma) {
            if (leader) {
                uint32_t stage = 0, phase = 0, acc = 0;
                bool ok = true, issued = false;
                auto next_stage = [&]() {
                    if (++stage == stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                };
                for (int t = first; ok && t < plan.total; t += step) {
                    const Tile w = plan.tile(t);
                    const uint32_t idesc = p.idesc | static_cast<uint32_t>(w.n >> 3) << 17;
                    for (int k0 = 0; ok && k0 < w.kblocks; k0 += kSeg, ++acc) {
                        const uint32_t as = acc & 1u;
                        if (!(ok = wait(kAccE + as, ((acc >> 1) & 1u) ^ 1u)))
                            break;
                        tc_fence_after();
                        const uint32_t d = tmem_base + as * NT;
                        const int k1 = min(k0 + kSeg, w.kblocks);
                        for (int kb = k0; kb < k1; ++kb, next_stage()) {
                            if (!(ok = wait_operands(bar(kFull + stage), phase, kFixes, abort_flag,
                                                     p.timeout_ns)))
                                break;
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
                                        mma_bf16_pair(d, a + kStepA * k, b + kStepB * k, idesc,
                                                      add);
                                }
                                mma_commit_pair(bar(kEmpty + stage), kBoth);
                                if (kb == k1 - 1)
                                    mma_commit_pair(bar(kAccF + as), kBoth);
                            }
                            __syncwarp();
                            issued = true;
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
        } else {
            if constexpr (kFixes) {
                // K-blocks with missing rows: once both operands have landed here the
                // rows are zeroed and the pair's barrier gets both loaders' arrivals.
                // (The loaders themselves go on: waiting for such a block, the last of
                // most tiles, they fell behind by 1.5 us a tile.)
                const bool holes = p.holes != nullptr && *p.holes != 0;
                uint32_t stage = 0, used = 0;   // bit s: parity of stage s's next such block
                bool ok = true;
                for (int t = first; ok && t < plan.total; t += step) {
                    const Tile w = plan.tile(t);
                    const int atoms_b = w.n / 128;
                    for (int kb = 0; kb < w.kblocks; ++kb) {
                        const int at = w.lo + kb * 64;
                        if (at + 64 > w.hi || holes) {
                            if (!(ok = wait(kFixA + stage, used >> stage & 1u) &&
                                       wait(kFixB + stage, used >> stage & 1u)))
                                break;
                            used ^= 1u << stage;
                            // lane l: whether positions l and 32 + l are missing
                            const uint32_t gone[2] = {
                                __ballot_sync(0xffffffffu, missing(p, at + lane, w.hi)),
                                __ballot_sync(0xffffffffu, missing(p, at + 32 + lane, w.hi))};
                            // whole rows: the swizzle moves 16-byte pieces within a row
                            for (int i = lane; i < 64 * 8; i += 32)
                                if (gone[i >> 8] >> (i >> 3 & 31) & 1u) {
                                    for (int a = 0; a < 2; ++a)
                                        zero16(part_a(stage) + a * kAtomBytes + 16 * i);
                                    for (int a = 0; a < atoms_b; ++a)
                                        zero16(part_b(stage) + a * kAtomBytes + 16 * i);
                                }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane < 2)
                                mbar_arrive_release_cluster(lead_bar(kFull + stage));
                        }
                        if (++stage == stages)
                            stage = 0;
                    }
                }
            }
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
                    constexpr int kPer = NT / 32;   // columns a lane
                    int32_t row[kPer];
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        row[i] = max(row_of(p.from, w.n0 + 32 * i + lane, w.hi), 0);
                    for (int k0 = 0; k0 < w.kblocks; k0 += kScaleGroup, ++n) {
                        const uint32_t s = n % kScaleStages;
                        float *const to = reinterpret_cast<float *>(sbase + lay.scale +
                                                                    s * scale_bytes(NT));
                        float v[kScaleGroup][kPer], one[kScaleGroup];
#pragma unroll
                        for (int j = 0; j < kScaleGroup; ++j) {
                            const int kb = min(k0 + j, w.kblocks - 1);
                            one[j] = ws[kb];
#pragma unroll
                            for (int i = 0; i < kPer; ++i)
                                v[j][i] =
                                    p.xscale[static_cast<int64_t>(row[i]) * w.kblocks + kb];
                        }
                        if (!(ok = wait(kScE + s, ((n / kScaleStages) & 1u) ^ 1u)))
                            break;
#pragma unroll
                        for (int j = 0; j < kScaleGroup; ++j)
#pragma unroll
                            for (int i = 0; i < kPer; ++i)
                                to[j * NT + 32 * i + lane] = v[j][i] * one[j];
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar(kScF + s));
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
        // Consumers: warp q of four holds 32 of the CTA's 128 rows, the two
        // groups of four the lower and the upper half of the columns.
        const int q = warp & 3, group = warp >> 2;
        const int c0 = group * kGroupCols;
        const uint32_t tmem_warp = tmem_base + (static_cast<uint32_t>(q) << 21) + c0;
        if (p.zero_rest)
            zero_rows(p, lists, blockIdx.x * kConsumers + warp, gridDim.x * kConsumers, lane);
        uint8_t *const staging = sbase + lay.staging + warp * kWarpStaging;
        uint32_t acc = 0, n = 0;
        bool ok = true;
        for (int t = first; ok && t < plan.total; t += step) {
            const Tile w = plan.tile(t);
            const int cols = min(max(w.n - c0, 0), kGroupCols);
            int32_t dst[kGroupCols / 32];   // of columns 32 i + lane
#pragma unroll
            for (int i = 0; i < kGroupCols / 32; ++i) {
                const int32_t at = w.n0 + c0 + 32 * i + lane;
                if (KIND == kWeightsGrad) {
                    dst[i] = at < p.ndim ? w.e * p.ndim + at : -1;
                } else {
                    dst[i] = row_of(p.places, at, w.hi);
                    if (dst[i] >= 0 && row_of(p.from, at, w.hi) < 0)
                        dst[i] = -2 - dst[i];
                }
            }
            Frags<kGroupCols> sum;
#pragma unroll
            for (int i = 0; i < kGroupCols; ++i)
                sum.v[i / 8][i / 4 % 2][i % 4] = 0.0f;
            for (int k0 = 0; k0 < w.kblocks; k0 += kSeg, ++acc) {
                const uint32_t as = acc & 1u;
                const uint32_t s = n % kScaleStages;
                if (E8 && k0 % kScaleGroup == 0 &&
                    !(ok = wait(kScF + s, (n / kScaleStages) & 1u)))
                    break;
                const float *const scales =
                    reinterpret_cast<const float *>(sbase + lay.scale + s * scale_bytes(NT)) +
                    k0 % kScaleGroup * NT;
                const bool last = k0 % kScaleGroup == kScaleGroup - 1 || k0 == w.kblocks - 1;
                if (!(ok = wait(kAccF + as, (acc >> 1) & 1u)))
                    break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kGroupCols; c += 32) {
                    if (c < cols) {
                        float2 f[4];
                        if constexpr (E8) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                f[j] = *reinterpret_cast<const float2 *>(
                                    scales + c0 + c + 8 * j + 2 * (lane & 3));
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float v[16];
                            tmem_ld_16x256b_x4(tmem_warp + (h << 20) + as * NT + c, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float &to = sum.v[c / 8 + i / 4][h][i % 4];
                                if constexpr (E8)
                                    to = fmaf(v[i], i & 1 ? f[i / 4].y : f[i / 4].x, to);
                                else
                                    to += v[i];
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_cluster(lead_bar(kAccE + as));
                    if (E8 && last)
                        mbar_arrive(bar(kScE + s));
                }
                n += last;
            }
            if (!ok)
                break;
            const int32_t f = w.m0 + static_cast<int>(rank) * kRowsA + 32 * q;
#pragma unroll
            for (int i = 0; i < kGroupCols / 32; ++i) {
                if (32 * i < cols) {
                    const float(*const v)[2][4] = sum.v + 4 * i;
                    if (p.out_type == kBf16)
                        store_columns<__nv_bfloat16>(v, staging, dst[i], p.out, f, p.mdim, lane);
                    else if (p.out_type == kFp16)
                        store_columns<__half>(v, staging, dst[i], p.out, f, p.mdim, lane);
                    else
                        store_columns<float>(v, staging, dst[i], p.out, f, p.mdim, lane);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag)
        let_copies_land(p.timeout_ns);
    cluster_sync();   // no CTA leaves while its pair can still touch its memory
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemColumns);
    }
}

// ---- 8 bits, many positions -------------------------------------------------
//
// Here a tile's rows are positions (256 of a list) and its columns elements of
// the output (256).  A thread of the consumers then holds one position's row, so
// that a segment's scale is one number a thread, which it loads itself: the sums
// cost one FMA an element and nothing else.  (With positions as columns each
// element needs its column's scale out of shared memory, and the rest of a
// segment's hand-over does not hide that: 32,768 positions in 8 lists, 4,096 x
// 4,096, took 700 us, here 518, 2,120 TFLOP/s.)  What bounds it: a k-block takes
// 1,140 clocks, of which its MMAs are 512; the rest is taken for the loads of the
// accumulator, which the MMAs would not overlap (a tile of 128 columns takes 730, which
// gives 320 clocks for a segment's hand-over and 3.2 a column, where the MMAs take 2).  As
// long: two CTAs with MMAs and hand-overs of their own and the weights multicast
// (537 us), scales loaded four k-blocks at a time (558), 64 columns in flight a
// warp (605).  Slower: 128 columns and four accumulators (667).  Lists are rounded
// up to 256, so only products of many positions an expert come here.

constexpr int kLoad8 = 8, kIssue8 = 9;   // warps behind the 8 of consumers; two issue

struct Tile8 {
    int32_t e, m0, n0, n, hi;
};

struct Layout8 {
    uint32_t staging, lists, bars, end;
};

__host__ __device__ inline Layout8 layout8_of(int stages, int E)
{
    Layout8 l;
    l.staging = stages * stage_bytes(256);
    l.lists = l.staging + kConsumers * kWarpStaging;
    l.bars = (l.lists + 3u * static_cast<uint32_t>(E + 1) * 4u + 15u) / 16u * 16u;
    l.end = l.bars + kBars * 8u + 16u;
    return l;
}

// A warp's rows (lane l: row l's next 64 bytes, as four pieces) to shared
// memory and from there to the output, four lanes to a row.
__device__ __forceinline__ void store_rows(uint8_t *stage, const uint4 (&v)[4], uint8_t *out,
                                           int64_t pitch, int32_t dst, int32_t bytes, int lane)
{
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 4; ++p)
        *reinterpret_cast<uint4 *>(stage + lane * 64 + 16 * (p ^ (lane >> 1 & 3))) = v[p];
    __syncwarp();
    const int piece = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 2);
        const int32_t d = __shfl_sync(0xffffffffu, dst, row);
        if (d >= 0 && 16 * piece < bytes)
            *reinterpret_cast<uint4 *>(out + d * pitch + 16 * piece) =
                *reinterpret_cast<const uint4 *>(stage + row * 64 + 16 * (piece ^ (row >> 1 & 3)));
    }
}

template <typename O>
__device__ __forceinline__ void store_sums(const float (&sum)[128], uint8_t *stage, void *out,
                                           int32_t mdim, int32_t f, int32_t dst, bool zero,
                                           int lane)
{
    constexpr int kCols = 64 / sizeof(O);
    const int64_t pitch = static_cast<int64_t>(mdim) * sizeof(O);
#pragma unroll
    for (int c = 0; c < 128; c += kCols) {
        uint4 v[4];
        if constexpr (sizeof(O) == 2) {
#pragma unroll
            for (int p = 0; p < 4; ++p)
                v[p] = make_uint4(pack_two<O>(sum[c + 8 * p], sum[c + 8 * p + 1]),
                                  pack_two<O>(sum[c + 8 * p + 2], sum[c + 8 * p + 3]),
                                  pack_two<O>(sum[c + 8 * p + 4], sum[c + 8 * p + 5]),
                                  pack_two<O>(sum[c + 8 * p + 6], sum[c + 8 * p + 7]));
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p)
                v[p] = make_uint4(
                    __float_as_uint(sum[c + 4 * p]), __float_as_uint(sum[c + 4 * p + 1]),
                    __float_as_uint(sum[c + 4 * p + 2]), __float_as_uint(sum[c + 4 * p + 3]));
        }
        if (zero) {
#pragma unroll
            for (int p = 0; p < 4; ++p)
                v[p] = make_uint4(0, 0, 0, 0);
        }
        const int32_t left = mdim - (f + c);
        if (left <= 0)   // the same for the whole warp
            break;
        store_rows(stage, v, static_cast<uint8_t *>(out) + (f + c) * sizeof(O), pitch, dst,
                   min(64, left * static_cast<int>(sizeof(O))), lane);
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    experts8_kernel(const __grid_constant__ CUtensorMap amap,
                    const __grid_constant__ CUtensorMap bmap, const ExpertsParams p)
{
    constexpr uint32_t kStageBytes = stage_bytes(256);
    constexpr uint16_t kBoth = 0x3;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const Layout8 lay = layout8_of(p.stages, p.E);
    uint8_t *const sbase = smem_raw + (base - raw);
    int32_t *const lists = reinterpret_cast<int32_t *>(sbase + lay.lists);
    volatile uint32_t *tmem_slot =
        reinterpret_cast<volatile uint32_t *>(sbase + lay.bars + kBars * 8);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    auto bar = [&](int i) -> uint32_t { return base + lay.bars + 8u * static_cast<uint32_t>(i); };
    auto lead_bar = [&](int i) -> uint32_t { return map_to_rank(bar(i), 0); };
    // Bounded waits on barrier i, of a warp and of one thread.
    auto wait = [&](int i, uint32_t parity) {
        return wait_warp(bar(i), parity, abort_flag, p.timeout_ns);
    };
    auto wait_one = [&](int i, uint32_t parity) {
        return wait1(bar(i), parity, abort_flag, p.timeout_ns);
    };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;

    if (threadIdx.x == 32) {
        tma_prefetch_desc(&amap);
        tma_prefetch_desc(&bmap);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxRing; ++s) {
            mbar_init(bar(kFull + s), 1);
            mbar_init(bar(kEmpty + s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar(kAccF + a), 1);
            mbar_init(bar(kAccE + a), 2 * kConsumers);
            mbar_init(bar(kLast + a), 1);
        }
        *abort_flag = 0u;
        fence_mbar_init();
    }
    wait_for_previous();
    let_next_start();   // all blocks of this launch are resident: the next one may set itself up
    if (warp == kLoad8) {
        tmem_alloc_pair(smem_addr(const_cast<uint32_t *>(tmem_slot)), 512);
        tmem_relinquish_pair();
    } else if (warp == 1) {
        form_lists<256>(p, lists, lane);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers exist before any cross-CTA signal
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int32_t *const begin = lists, *const end = lists + (p.E + 1),
                        *const before = lists + 2 * (p.E + 1);
    const int nblocks = (p.mdim + 255) / 256;
    const int total = before[p.E] * nblocks;
    const int first = static_cast<int>(blockIdx.x >> 1);
    const int step = static_cast<int>(gridDim.x >> 1);
    const uint32_t stages = static_cast<uint32_t>(p.stages);
    auto tile = [&](int t) -> Tile8 {
        const int q = t / nblocks;
        int lo = 0, hi = p.E;   // before[lo] <= q < before[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (before[mid] <= q)
                lo = mid;
            else
                hi = mid;
        }
        Tile8 w;
        w.e = lo;
        w.m0 = begin[lo] + (q - before[lo]) * 256;
        w.hi = end[lo];
        w.n0 = (t - q * nblocks) * 256;
        w.n = min(256, (p.mdim - w.n0 + 31) / 32 * 32);
        return w;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        auto next_stage = [&]() {
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        };
        if (warp == kLoad8) {
            if (lane == 0) {
                for (int t = first; ok && t < total; t += step) {
                    const Tile8 w = tile(t);
                    const int m = w.m0 + static_cast<int>(rank) * kRowsA;
                    const int n = w.n0 + static_cast<int>(rank) * (w.n / 2);
                    for (int kb = 0; kb < p.kblocks; ++kb, next_stage()) {
                        if (!(ok = wait_one(kEmpty + stage, phase ^ 1u)))
                            break;
                        if (leader)
                            mbar_arrive_expect_tx(bar(kFull + stage), 2 * kStageBytes);
                        const uint32_t full = lead_bar(kFull + stage);
                        const uint32_t to = base + stage * kStageBytes;
                        tma_load_2d_pair(to, &amap, full, kb * 128, m);
                        tma_load_3d_pair(to + kPartA, &bmap, full, kb * 128, n, w.e);
                    }
                }
            }
            __syncwarp();
        } else if (leader && (warp == kIssue8 || warp == kIssue8 + 1)) {
            // One warp for each accumulator: a segment has a hand-over at both ends.
            const uint32_t me = static_cast<uint32_t>(warp - kIssue8);
            uint32_t acc = 0;
            bool issued = false;
            for (int t = first; ok && t < total; t += step) {
                const Tile8 w = tile(t);
                const uint32_t idesc = p.idesc | static_cast<uint32_t>(w.n >> 3) << 17;
                for (int kb = 0; kb < p.kblocks; ++kb, ++acc, next_stage()) {
                    if ((acc & 1u) != me)
                        continue;
                    if (!(ok = wait(kAccE + me, ((acc >> 1) & 1u) ^ 1u) &&
                               wait(kFull + stage, phase)))
                        break;
                    tc_fence_after();
                    const uint64_t a = sw128_kmajor_desc(base + stage * kStageBytes);
                    const uint64_t b = sw128_kmajor_desc(base + stage * kStageBytes + kPartA);
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k)
                            mma_f8_pair(tmem_base + me * 256, a + 2u * k, b + 2u * k, idesc,
                                        k != 0);
                        mma_commit_pair(bar(kEmpty + stage), kBoth);
                        mma_commit_pair(bar(kAccF + me), kBoth);
                    }
                    __syncwarp();
                    issued = true;
                }
            }
            if (issued) {
                if (elect_one())
                    mma_commit_pair(bar(kLast + me), 0x1);
                __syncwarp();
                wait_warp(bar(kLast + me), 0u, abort_flag, kDrainLimitNs, false);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
        const int q = warp & 3, group = warp >> 2;
        const uint32_t tmem_warp =
            tmem_base + (static_cast<uint32_t>(q) << 21) + static_cast<uint32_t>(group) * 128u;
        uint8_t *const staging = sbase + lay.staging + warp * kWarpStaging;
        if (p.zero_rest)
            zero_rows(p, lists, blockIdx.x * kConsumers + warp, gridDim.x * kConsumers, lane);
        uint32_t acc = 0;
        bool ok = true;
        for (int t = first; ok && t < total; t += step) {
            const Tile8 w = tile(t);
            const int at = w.m0 + static_cast<int>(rank) * kRowsA + 32 * q + lane;
            const int32_t row = row_of(p.from, at, w.hi);
            const int32_t dst = row_of(p.places, at, w.hi);
            const int f0 = w.n0 + 128 * group;
            const int cols = min(128, w.n - 128 * group);   // may be none
            const float *const xs = p.xscale + static_cast<int64_t>(max(row, 0)) * p.kblocks;
            const float *const ws =
                p.wscale +
                (static_cast<int64_t>(w.e) * p.fblocks + min(f0 >> 7, p.fblocks - 1)) * p.kblocks;
            float sum[128];
#pragma unroll
            for (int i = 0; i < 128; ++i)
                sum[i] = 0.0f;
            float x_next = *xs, w_next = *ws;
            for (int kb = 0; kb < p.kblocks; ++kb, ++acc) {
                const float scale = x_next * w_next;
                if (kb + 1 < p.kblocks) {
                    x_next = xs[kb + 1];
                    w_next = ws[kb + 1];
                }
                const uint32_t as = acc & 1u;
                if (!(ok = wait(kAccF + as, (acc >> 1) & 1u)))
                    break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    if (c < cols) {
                        float v[32];
                        tmem_ld_32x32b_x32(tmem_warp + as * 256 + c, v);
                        tmem_wait_ld();
                        if (c + 32 >= cols) {   // the last: the accumulator may be written again
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive_cluster(lead_bar(kAccE + as));
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            sum[c + i] = fmaf(v[i], scale, sum[c + i]);
                    }
                }
                if (cols <= 0 && lane == 0)
                    mbar_arrive_cluster(lead_bar(kAccE + as));
            }
            if (!ok)
                break;
            if (cols <= 0)
                continue;
            if (p.out_type == kBf16)
                store_sums<__nv_bfloat16>(sum, staging, p.out, p.mdim, f0, dst, row < 0, lane);
            else if (p.out_type == kFp16)
                store_sums<__half>(sum, staging, p.out, p.mdim, f0, dst, row < 0, lane);
            else
                store_sums<float>(sum, staging, p.out, p.mdim, f0, dst, row < 0, lane);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag)
        let_copies_land(p.timeout_ns);
    cluster_sync();   // no CTA leaves while its pair can still touch its memory
    if (warp == kLoad8) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

__global__ void __launch_bounds__(256)
    listed_rows_kernel(const int32_t *offsets, int32_t E, int32_t M, RowMap map, int32_t *row,
                       int32_t *zero)
{
    wait_for_previous();
    if (zero != nullptr && blockIdx.x == 0 && threadIdx.x == 0)
        *zero = 0;
    const int32_t lo = offsets == nullptr ? 0 : min(max(offsets[0], 0), M);
    const int32_t hi = offsets == nullptr ? M : min(max(offsets[E], 0), M);
    for (int64_t at = blockIdx.x * 256 + threadIdx.x; at < M; at += gridDim.x * 256)
        row[at] = at < lo ? -1 : row_of(map, static_cast<int32_t>(at), hi);
}

// Rows in the lists' order: to[p] = the row that map names for position p,
// zeros where there is none in map or in also (*holes is then set, if given).
// A power of two of lanes a row, up to four 16-byte pieces in flight a lane.
// Bound by HBM, for the most part by what it writes (131,072 rows of 4,096 bytes of a
// matrix of 16,384: 118 us for 604 MB, DRAM 79% busy, L2 46%; bulk copies through shared
// memory 147); streaming stores leave the matrix in L2 (with plain ones 129).
__global__ void __launch_bounds__(256)
    gather_rows_kernel(const int32_t *offsets, int32_t E, int32_t M, RowMap map, RowMap also,
                       const uint4 *from, int32_t units, int32_t lanes, uint4 *to, int32_t *holes)
{
    wait_for_previous();
    let_next_start();
    const int32_t lo = offsets == nullptr ? 0 : min(max(offsets[0], 0), M);
    const int32_t hi = offsets == nullptr ? M : min(max(offsets[E], 0), M);
    const int32_t mine = threadIdx.x & (lanes - 1);
    const int32_t rows = 256 / lanes;
    const int64_t at = blockIdx.x * static_cast<int64_t>(rows) + threadIdx.x / lanes;
    if (at < M) {
        const int32_t p = static_cast<int32_t>(at);
        int32_t row = -1;
        if (p >= lo && p < hi) {
            row = row_of(map, p, hi);
            if (row_of(also, p, hi) < 0)
                row = -1;
            if (row < 0 && holes != nullptr && mine == 0)
                *holes = 1;
        }
        const uint4 *const src = from + static_cast<int64_t>(row) * units;
        uint4 *const dst = to + at * units;
        int32_t u = mine;
        if (row >= 0) {
            for (; u + 3 * lanes < units; u += 4 * lanes) {
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[k] = src[u + k * lanes];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    __stcs(dst + u + k * lanes, v[k]);
            }
        }
        for (; u < units; u += lanes)
            dst[u] = row >= 0 ? src[u] : make_uint4(0, 0, 0, 0);
    }
}

// Ring depth that fits beside the lists and scales.
int stages_for(int NT, int E, bool scaled, size_t smem)
{
    for (int s = kMaxRing; s >= 2; --s)
        if (1024u + layout_of(NT, s, E, scaled).end <= smem)
            return s;
    return 0;
}

template <ExpertsKind KIND, bool E8, int NT>
cudaError_t launch(const CUtensorMap &a, const CUtensorMap &b, ExpertsParams p, int sms,
                   size_t smem_optin, cudaStream_t stream)
{
    p.stages = stages_for(NT, p.E, E8, smem_optin);
    if (p.stages == 0)
        return cudaErrorInvalidConfiguration;
    const size_t smem = 1024u + layout_of(NT, p.stages, p.E, E8).end;
    // no more clusters than tiles there can be
    const int64_t mblocks = (p.mdim + 2 * kRowsA - 1) / (2 * kRowsA);
    const int64_t tiles = KIND == kWeightsGrad
                              ? mblocks * ((p.ndim + NT - 1) / NT) * p.E
                              : mblocks * (std::min<int64_t>(p.E, p.M) + p.M / NT);
    const int grid =
        2 * static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(tiles, sms / 2)));
    return launch_after(experts_kernel<KIND, E8, NT>, grid, kThreads, smem, stream, a, b, p);
}

cudaError_t launch8(const CUtensorMap &a, const CUtensorMap &b, ExpertsParams p, int sms,
                    size_t smem_optin, cudaStream_t stream)
{
    p.stages = 0;
    for (int s = kMaxRing; s >= 2 && p.stages == 0; --s)
        if (1024u + layout8_of(s, p.E).end <= smem_optin)
            p.stages = s;
    if (p.stages == 0)
        return cudaErrorInvalidConfiguration;
    p.idesc = idesc_base(0u, false, false, 2 * kRowsA);
    const int64_t tiles =
        (std::min<int64_t>(p.E, p.M) + p.M / 256) * ((p.mdim + 255) / 256);
    const int grid = 2 * static_cast<int>(std::min<int64_t>(tiles, sms / 2));
    return launch_after(experts8_kernel, grid, kThreads, 1024u + layout8_of(p.stages, p.E).end,
                        stream, a, b, p);
}

}  // namespace

cudaError_t experts_prepare(size_t smem_optin)
{
    const void *kernels[] = {(const void *)experts_kernel<kForward, false, 64>,
                             (const void *)experts_kernel<kForward, false, 256>,
                             (const void *)experts_kernel<kForward, true, 64>,
                             (const void *)experts8_kernel,
                             (const void *)experts_kernel<kRowsGrad, false, 64>,
                             (const void *)experts_kernel<kRowsGrad, false, 256>,
                             (const void *)experts_kernel<kWeightsGrad, false, 256>};
    for (const void *k : kernels) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem_optin));
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

// Rows by ids, 64 lists of 32 / 64 positions of 2,048 in 16 bits, 1,024 columns:
// narrow tiles 50 / 63 us, wide ones behind a pass that gathers the rows 55 / 60.
// In 8 bits, 64 / 96 positions: narrow 40 / 58, positions as rows 52 / 54 (256
// lists: 131 / 212 and 171 / 180).  The rule knows the mean length only: 8,192 positions
// of 256 lists take 186 us by narrow and 187 by wide tiles where all lists have some, but
// 135 and 72 on 64 of them, 105 and 35 on one (8 bits 115 and 166, 86 and 62, 66 and 34).
bool experts_few(int64_t M, int64_t E, bool e8) { return M <= (e8 ? 64 : 32) * E; }

cudaError_t launch_experts(ExpertsKind kind, bool e8, int type, const CUtensorMap &a,
                           const CUtensorMap &b, ExpertsParams p, int sms, size_t smem_optin,
                           cudaStream_t stream)
{
    p.idesc = idesc_base(e8 ? 0u : type == kBf16 ? 1u : 0u, kind != kForward, kind == kWeightsGrad,
                         2 * kRowsA);
    p.segment = kind == kWeightsGrad && p.out_type == kFp32 ? kSegmentRows : kSegment;
    const bool few = experts_few(p.M, p.E, e8);
    switch (kind) {
    case kForward:
        if (e8)
            return few ? launch<kForward, true, 64>(a, b, p, sms, smem_optin, stream)
                       : launch8(b, a, p, sms, smem_optin, stream);
        return few ? launch<kForward, false, 64>(a, b, p, sms, smem_optin, stream)
                   : launch<kForward, false, 256>(a, b, p, sms, smem_optin, stream);
    case kRowsGrad:
        return few ? launch<kRowsGrad, false, 64>(a, b, p, sms, smem_optin, stream)
                   : launch<kRowsGrad, false, 256>(a, b, p, sms, smem_optin, stream);
    default:
        return launch<kWeightsGrad, false, 256>(a, b, p, sms, smem_optin, stream);
    }
}

cudaError_t launch_listed_rows(const int32_t *offsets, int32_t E, int32_t M, RowMap map,
                               int32_t *row, int32_t *zero, cudaStream_t stream)
{
    const int blocks =
        static_cast<int>(std::min<int64_t>((static_cast<int64_t>(M) + 255) / 256, 4096));
    return launch_after(listed_rows_kernel, blocks, 256, 0, stream, offsets, E, M, map, row, zero);
}

cudaError_t launch_gather_rows(const int32_t *offsets, int32_t E, int32_t M, RowMap map,
                               RowMap also, const void *from, int64_t pitch, void *to,
                               int32_t *holes, cudaStream_t stream)
{
    const int32_t units = static_cast<int32_t>(pitch / 16);
    int32_t lanes = 32;
    while (lanes > 1 && lanes / 2 >= units)
        lanes /= 2;
    const int64_t blocks = (static_cast<int64_t>(M) * lanes + 255) / 256;
    return launch_after(gather_rows_kernel, static_cast<unsigned>(blocks), 256, 0, stream, offsets,
                        E, M, map, also, static_cast<const uint4 *>(from), units, lanes,
                        static_cast<uint4 *>(to), holes);
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
