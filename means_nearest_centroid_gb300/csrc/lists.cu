// lists.cu -- inverted lists: the positions of idx[0, M) grouped by the row
// that they name, each group in ascending order (a stable sort), with ids
// outside [0, K) left out; offsets[r] is where row r's group begins.
//
// A radix sort of (row, position) pairs from the lowest digit up.  Each of up
// to two blocks an SM owns one contiguous share of the pairs, so the order within a
// digit is: earlier blocks first, then the block's own items in order.  Per digit
//   count:    block b counts its items -> H[b][digit];
//   scatter:  block b sums H[b'][digit] over the blocks b' before it and over
//             all blocks, scans the digits, and takes its items in tiles: ranks
//             them (a warp's equal digits by votes, warps by their counts in
//             shared memory), orders the tile by digit in shared memory, and
//             writes it out in runs of consecutive places.
// The two launches cost less than one whose blocks count the next digit for
// each other with atomics (2^20 ids of 4,096 rows: 31 us a scatter with atomics
// and without the ordered tile, about 12 as it is).  Each launch of a sort may
// start while the one before it ends.  2^20 ids of 4,096 rows take 32 us in five
// launches, of which the ids' and lists' 8.4 MB are 1.3: every scatter block's
// chain of loads, votes, scans and barriers (issue slots 47% busy) bounds it, not
// memory.  Up to kClusterMax items are one launch of a cluster of eight blocks that
// exchange counts and pairs through each other's shared memory, and up to
// kOneBlockMax one of one block (512 ids of 256 rows: 3 us).  Nothing depends on
// timing: the result is unique.
//
// offsets are found by a search in the sorted rows within the row's last digit,
// eight ways at a step: a third of bisection's dependent loads.
#include "launch.cuh"
#include "learn.h"

#include <cooperative_groups.h>

#include <algorithm>

namespace kma {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDigitBits = 10;
constexpr int kBlocksPerSm = 2;            // of kThreads
constexpr int64_t kOneBlockMax = 2048;     // that many ids of 256 / 4,096 rows: 4.4 / 8.9 us by one block, 5.8 / 10.1 by eight
constexpr int64_t kOneOffsetsMax = 8192;   // rows whose offsets the one block finds itself
constexpr int kOneBits = 8;                // digit of the one-block sort
constexpr int kClusterBlocks = 8;
constexpr int kClusterThreads = 1024;
constexpr int kClusterItems = 2;           // a thread
constexpr int64_t kClusterMax = int64_t(kClusterBlocks) * kClusterThreads * kClusterItems;
constexpr int kOneBins = 1 << kOneBits;

// Exclusive scan over the block of one value per thread; *total: the sum.
// warp_sums: WARPS + 1 values.
template <int WARPS>
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t *warp_sums, int32_t *total)
{
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    int32_t incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int32_t t = __shfl_up_sync(kAll, incl, off);
        if (lane >= off)
            incl += t;
    }
    if (lane == 31)
        warp_sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int32_t w = lane < WARPS ? warp_sums[lane] : 0;
        int32_t wi = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t t = __shfl_up_sync(kAll, wi, off);
            if (lane >= off)
                wi += t;
        }
        if (lane < WARPS)
            warp_sums[lane] = wi - w;
        if (lane == 31)
            warp_sums[WARPS] = wi;
    }
    __syncthreads();
    const int32_t out = incl - v + warp_sums[warp];
    *total = warp_sums[WARPS];
    __syncthreads();
    return out;
}

// Rank of the lane's item among the items of its digit seen so far by this
// warp; `counts` (the warp's own bins) takes the new ones.  d < 0: no item.
// Equal digits are found bit by bit, by votes.
__device__ __forceinline__ int32_t warp_rank(int32_t d, int bits, uint16_t *counts, int lane)
{
    const uint32_t valid = __ballot_sync(kAll, d >= 0);
    uint32_t same = d >= 0 ? valid : ~valid;
#pragma unroll
    for (int b = 0; b < kMaxDigitBits; ++b) {
        if (b >= bits)
            break;
        const bool one = (d & (1 << b)) != 0;
        const uint32_t ones = __ballot_sync(kAll, one);
        same &= one ? ones : ~ones;
    }
    const uint32_t below = same & ((1u << lane) - 1u);
    int32_t base = 0;
    if (d >= 0 && below == 0) {
        base = counts[d];
        counts[d] = static_cast<uint16_t>(base + __popc(same));
    }
    base = __shfl_sync(kAll, base, __ffs(same) - 1);
    __syncwarp();
    return base + __popc(below);
}

// Memory that the sort's scatter launches zero besides: blocks past a launch's
// own write a share of it while those wait for their loads.  16 MiB a launch
// (what it hides whole), more where that is not enough.
struct Fill {
    uint8_t *p;
    int64_t bytes;     // 0: none
    int32_t part, parts;
    __host__ __device__ __forceinline__ bool any() const { return bytes > 0 && part < parts; }
};

__device__ __forceinline__ void fill_zero(const Fill &f, int64_t block, int64_t blocks)
{
    const int64_t head = min(f.bytes, static_cast<int64_t>(-reinterpret_cast<uintptr_t>(f.p) & 15));
    uint4 *body = reinterpret_cast<uint4 *>(f.p + head);
    const int64_t units = (f.bytes - head) >> 4;
    const int64_t end = units * (f.part + 1) / f.parts;
#pragma unroll 4
    for (int64_t i = units * f.part / f.parts + block * blockDim.x + threadIdx.x; i < end;
         i += blocks * blockDim.x)
        body[i] = make_uint4(0u, 0u, 0u, 0u);
    if (f.part == 0 && block == 0) {   // the ends, fewer than 16 bytes each, of 2-byte elements
        uint16_t *ends = reinterpret_cast<uint16_t *>(f.p);
        const int t = static_cast<int>(threadIdx.x);
        if (t < 8 && 2 * t < head)
            ends[t] = 0;
        const int64_t tail = head + units * 16 + 2 * t;
        if (t < 8 && tail < f.bytes)
            ends[tail >> 1] = 0;
    }
}

struct SortArgs {
    const int32_t *rows_in;   // first pass: idx, and the position is the index
    const int32_t *pos_in;
    int32_t *rows_out;        // last pass: may be nullptr
    int32_t *pos_out;
    int32_t *offsets;         // of a one-digit sort, else nullptr
    int32_t *hist;            // H[block][bins] of this digit
    int32_t *total;           // number of valid ids: set by the first pass
    int32_t *starts;          // last pass: [bins + 1] where each digit's items start, or nullptr
    int64_t M;
    int64_t share;            // items per block
    int32_t K;
    int32_t shift, bins;      // this digit: (row >> shift) & (bins - 1)
    int32_t blocks;
    bool last;
    Fill fill;
};

template <bool FIRST>
__global__ void __launch_bounds__(kThreads) lists_count_kernel(const SortArgs a)
{
    extern __shared__ int32_t smem[];
    let_next_start();
    for (int d = threadIdx.x; d < a.bins; d += kThreads)
        smem[d] = 0;
    __syncthreads();
    wait_for_previous();
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.share;
    const int64_t end = min(FIRST ? a.M : static_cast<int64_t>(*a.total), begin + a.share);
#pragma unroll 4
    for (int64_t i = begin + threadIdx.x; i < end; i += kThreads) {
        const int32_t r = a.rows_in[i];
        if (!FIRST || (r >= 0 && r < a.K))
            atomicAdd(smem + ((r >> a.shift) & (a.bins - 1)), 1);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.bins; d += kThreads)
        a.hist[static_cast<int64_t>(blockIdx.x) * a.bins + d] = smem[d];
}

// Shared memory of a scatter block: the places of each digit, its start in
// the tile, the tile's pairs, the warps' counts.
size_t scatter_smem(int bins, int items)
{
    return static_cast<size_t>(bins) * 8 + static_cast<size_t>(kThreads) * items * 8 +
           static_cast<size_t>(kWarps) * bins * 2;
}

template <int ITEMS, bool FIRST>
__global__ void __launch_bounds__(kThreads) lists_scatter_kernel(const SortArgs a)
{
    extern __shared__ int32_t smem[];
    constexpr int kTile = kThreads * ITEMS;
    int32_t *place = smem;                // [bins] next place of each digit, this block
    int32_t *start = place + a.bins;      // [bins] its first item in the ordered tile
    int32_t *t_row = start + a.bins;      // [kTile]
    int32_t *t_pos = t_row + kTile;       // [kTile]
    uint16_t *counts = reinterpret_cast<uint16_t *>(t_pos + kTile);   // [kWarps][bins]
    __shared__ int32_t warp_sums[kWarps + 1];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    let_next_start();
    if (blockIdx.x >= a.blocks) {
        wait_for_previous();
        fill_zero(a.fill, blockIdx.x - a.blocks, gridDim.x - a.blocks);
        return;
    }
    for (int d = threadIdx.x; d < 2 * a.bins; d += kThreads)
        smem[d] = 0;
    __syncthreads();
    wait_for_previous();

    // places: all smaller digits, then this digit in earlier blocks; the
    // threads share out the blocks' counts of a digit (integer sums)
    if (a.bins >= 4) {
        // four digits a thread, so that a load covers 16 bytes
        const int quads = a.bins >> 2;
        const int lanes = kThreads / quads;   // at least 2
        const int d = (threadIdx.x & (quads - 1)) << 2;
        int4 all = make_int4(0, 0, 0, 0), before = all;
#pragma unroll 8
        for (int b = threadIdx.x / quads; b < a.blocks; b += lanes) {
            const int4 n = *reinterpret_cast<const int4 *>(a.hist + static_cast<int64_t>(b) * a.bins + d);
            const int m = b < static_cast<int>(blockIdx.x) ? -1 : 0;
            all.x += n.x, all.y += n.y, all.z += n.z, all.w += n.w;
            before.x += n.x & m, before.y += n.y & m, before.z += n.z & m, before.w += n.w & m;
        }
        atomicAdd(start + d, all.x), atomicAdd(start + d + 1, all.y);
        atomicAdd(start + d + 2, all.z), atomicAdd(start + d + 3, all.w);
        atomicAdd(place + d, before.x), atomicAdd(place + d + 1, before.y);
        atomicAdd(place + d + 2, before.z), atomicAdd(place + d + 3, before.w);
    } else {
        for (int t = threadIdx.x; t < a.bins * a.blocks; t += kThreads) {
            const int b = t / a.bins, d = t % a.bins;
            const int32_t n = a.hist[t];
            atomicAdd(start + d, n);
            if (b < static_cast<int>(blockIdx.x))
                atomicAdd(place + d, n);
        }
    }
    __syncthreads();
    int32_t total = 0;
    for (int d0 = 0; d0 < a.bins; d0 += kThreads) {
        const int d = d0 + threadIdx.x;
        int32_t sum;
        const int32_t first =
            total + block_scan<kWarps>(d < a.bins ? start[d] : 0, warp_sums, &sum);
        total += sum;
        if (d < a.bins) {
            place[d] += first;
            if (a.offsets != nullptr && blockIdx.x == 0 && d < a.K)
                a.offsets[d] = first;
            if (a.starts != nullptr && blockIdx.x == 0)
                a.starts[d] = first;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (FIRST)
            *a.total = total;
        if (a.starts != nullptr)
            a.starts[a.bins] = total;
        if (a.offsets != nullptr)
            a.offsets[a.K] = total;
    }

    const int bits = 31 - __clz(a.bins);
    const int64_t limit = FIRST ? a.M : total;
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.share;
    const int64_t end = min(limit, begin + a.share);
    for (int64_t t0 = begin; t0 < end; t0 += kTile) {
        uint32_t *words = reinterpret_cast<uint32_t *>(counts);
        for (int c = threadIdx.x; c < (kWarps * a.bins) >> 1; c += kThreads)
            words[c] = 0;
        int32_t row[ITEMS], pos[ITEMS], rank[ITEMS];
        const int64_t w0 = t0 + static_cast<int64_t>(warp) * (32 * ITEMS) + lane;
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            const int64_t i = w0 + u * 32;
            row[u] = -1;
            pos[u] = static_cast<int32_t>(i);
            if (i < end) {
                const int32_t r = a.rows_in[i];
                row[u] = !FIRST || (r >= 0 && r < a.K) ? r : -1;
                if (!FIRST)
                    pos[u] = a.pos_in[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            const int32_t d = row[u] < 0 ? -1 : (row[u] >> a.shift) & (a.bins - 1);
            rank[u] = warp_rank(d, bits, counts + warp * a.bins, lane);
        }
        __syncthreads();
        // per digit: where its items, and each warp's of them, start in the ordered tile
        int32_t in_tile = 0;
        for (int d0 = 0; d0 < a.bins; d0 += kThreads) {
            const int d = d0 + threadIdx.x;
            int32_t n = 0;
            if (d < a.bins)
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const uint16_t c = counts[w * a.bins + d];
                    counts[w * a.bins + d] = static_cast<uint16_t>(n);
                    n += c;
                }
            int32_t sum;
            const int32_t first = in_tile + block_scan<kWarps>(n, warp_sums, &sum);
            in_tile += sum;
            if (d < a.bins) {
                start[d] = first;
                place[d] -= first;   // so that an item's place is this plus its number in the tile
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < ITEMS; ++u)
            if (row[u] >= 0) {
                const int32_t d = (row[u] >> a.shift) & (a.bins - 1);
                const int to = start[d] + counts[warp * a.bins + d] + rank[u];
                t_row[to] = row[u];
                t_pos[to] = pos[u];
            }
        __syncthreads();
#pragma unroll 4
        for (int t = threadIdx.x; t < in_tile; t += kThreads) {
            const int32_t r = t_row[t];
            const uint32_t to = place[(r >> a.shift) & (a.bins - 1)] + t;
            a.pos_out[to] = t_pos[t];
            if (a.rows_out != nullptr)
                a.rows_out[to] = r;
        }
        __syncthreads();
        // place: past this tile's items of the digit, no longer less its start
        for (int d = threadIdx.x; d < a.bins; d += kThreads)
            place[d] += d + 1 < a.bins ? start[d + 1] : in_tile;
        __syncthreads();
    }
    // places that no valid id takes
    if (a.last)
        for (int64_t i = max(begin, static_cast<int64_t>(total)) + threadIdx.x;
             i < min(a.M, begin + a.share); i += kThreads)
            a.pos_out[i] = -1;
}

// Up to THREADS * ITEMS items: every digit by one block, the pairs in shared
// memory.  The first digit's pass drops ids outside [0, K).
template <int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS)
    lists_one_block_kernel(const int32_t *idx, int32_t M, int32_t K, int32_t bits,
                           int32_t *__restrict__ order, int32_t *__restrict__ rows,
                           int32_t *__restrict__ offsets, int32_t *__restrict__ total, Fill fill)
{
    constexpr int kW = THREADS / 32;
    constexpr int kMax = THREADS * ITEMS;
    static_assert(THREADS >= kOneBins, "a thread per digit");
    __shared__ int32_t s_row[kMax];
    __shared__ uint16_t s_pos[kMax];
    __shared__ uint16_t counts[kW][kOneBins];
    __shared__ int32_t warp_sums[kW + 1];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    let_next_start();
    wait_for_previous();
    if (blockIdx.x > 0) {
        fill_zero(fill, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    int32_t n = M;   // items of this pass
    for (int shift = 0; shift == 0 || shift < bits; shift += kOneBits) {
        const int items = (n + THREADS - 1) / THREADS;   // per thread, <= ITEMS
        for (int c = threadIdx.x; c < kW * kOneBins / 2; c += THREADS)
            reinterpret_cast<uint32_t *>(&counts[0][0])[c] = 0;
        int32_t row[ITEMS], pos[ITEMS], rank[ITEMS];
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            const int i = warp * (32 * items) + u * 32 + lane;
            row[u] = -1;
            pos[u] = i;
            if (u < items && i < n) {
                if (shift == 0) {
                    const int32_t r = idx[i];
                    row[u] = r >= 0 && r < K ? r : -1;
                } else {
                    row[u] = s_row[i];
                    pos[u] = s_pos[i];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < ITEMS; ++u)
            if (u < items)
                rank[u] = warp_rank(row[u] < 0 ? -1 : (row[u] >> shift) & (kOneBins - 1),
                                    min(kOneBits, bits - shift), counts[warp], lane);
        __syncthreads();
        int32_t mine = 0;
        if (threadIdx.x < kOneBins)
#pragma unroll
            for (int w = 0; w < kW; ++w)
                mine += counts[w][threadIdx.x];
        int32_t run = block_scan<kW>(mine, warp_sums, &n);
        if (threadIdx.x < kOneBins) {
            if (bits <= kOneBits && offsets != nullptr && threadIdx.x < K)
                offsets[threadIdx.x] = run;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const int32_t c = counts[w][threadIdx.x];
                counts[w][threadIdx.x] = static_cast<uint16_t>(run);
                run += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < ITEMS; ++u)
            if (u < items && row[u] >= 0) {
                const int to = counts[warp][(row[u] >> shift) & (kOneBins - 1)] + rank[u];
                s_row[to] = row[u];
                s_pos[to] = static_cast<uint16_t>(pos[u]);
            }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < M; i += THREADS) {
        order[i] = i < n ? s_pos[i] : -1;
        if (rows != nullptr && i < n)
            rows[i] = s_row[i];
    }
    if (total != nullptr && threadIdx.x == 0)
        *total = n;
    if (offsets == nullptr)
        return;
    if (threadIdx.x == 0)
        offsets[K] = n;
    if (bits <= kOneBits)
        return;
    // K <= kOneOffsetsMax: the first place whose row is at least r
    for (int r = threadIdx.x; r < K; r += THREADS) {
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_row[mid] < r)
                lo = mid + 1;
            else
                hi = mid;
        }
        offsets[r] = lo;
    }
}

// ---- up to kClusterMax items: one cluster ------------------------------------

struct ClusterArgs {
    const int32_t *idx;
    int32_t *order;
    int32_t *rows;       // or nullptr
    int32_t *offsets;    // of a one-digit sort, else nullptr
    int32_t *starts;     // of the last of several digits, else nullptr
    int32_t *total;
    int32_t M, K;
    int32_t passes;
    int32_t bits[4], shift[4];
    Fill fill;
};

// Shared memory of a block: its share of the pairs, the warps' counts, and the
// digits' counts and places.
constexpr int kClusterSmem = kClusterThreads * kClusterItems * 8 +
                             (kClusterThreads / 32) * (2 << kMaxDigitBits) + (8 << kMaxDigitBits);

// Block b owns the places [b share, (b + 1) share) of every pass; a thread holds
// two of its block's pairs in registers while they are placed.  Two cluster
// barriers a digit: after the first the blocks read each other's counts (and all
// have read their pairs), after the second the pairs are in their places.
// Clusters after the first fill.  16,384 ids of 131,072 rows take 15 us (with the
// search for the offsets) where the launches of the larger sorts took 22 to 24;
// with four pairs a thread 30,000 ids of 16,384 rows took 19 for 22, but the
// gradients that zero a table besides got 3 us slower.
__global__ void __cluster_dims__(kClusterBlocks, 1, 1) __launch_bounds__(kClusterThreads)
    lists_cluster_kernel(const ClusterArgs a)
{
    namespace cg = cooperative_groups;
    constexpr int kW = kClusterThreads / 32;
    constexpr int ITEMS = kClusterItems;
    constexpr int kShare = kClusterThreads * ITEMS;
    constexpr int kBins = 1 << kMaxDigitBits;
    extern __shared__ __align__(16) uint8_t cluster_smem[];
    int2 *pairs = reinterpret_cast<int2 *>(cluster_smem);                        // [kShare] row, position
    uint16_t *counts = reinterpret_cast<uint16_t *>(pairs + kShare);     // [kW][bins]
    int32_t *hist = reinterpret_cast<int32_t *>(counts + kW * kBins);    // [bins] of this block
    int32_t *place = hist + kBins;                                       // [bins]
    __shared__ int32_t warp_sums[kW + 1];
    let_next_start();
    wait_for_previous();
    if (blockIdx.x >= kClusterBlocks) {
        fill_zero(a.fill, blockIdx.x - kClusterBlocks, gridDim.x - kClusterBlocks);
        return;
    }
    cg::cluster_group cluster = cg::this_cluster();
    const int block = static_cast<int>(blockIdx.x);
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    int2 item[ITEMS];
    int32_t rank[ITEMS];
    int n = a.M;   // pairs of this pass
    for (int pass = 0; pass < a.passes; ++pass) {
        const int bits = a.bits[pass], shift = a.shift[pass], bins = 1 << bits;
        for (int c = threadIdx.x; c < kW * bins / 2; c += kClusterThreads)
            reinterpret_cast<uint32_t *>(counts)[c] = 0;
        const int mine = min(kShare, max(0, n - block * kShare));
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            const int i = warp * (32 * ITEMS) + u * 32 + lane;
            item[u] = make_int2(-1, block * kShare + i);
            if (i < mine) {
                if (pass > 0) {
                    item[u] = pairs[i];
                } else {
                    const int32_t r = a.idx[block * kShare + i];
                    if (r >= 0 && r < a.K)
                        item[u].x = r;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < ITEMS; ++u)
            rank[u] = warp_rank(item[u].x < 0 ? -1 : (item[u].x >> shift) & (bins - 1), bits,
                                counts + warp * bins, lane);
        __syncthreads();
        const int d = threadIdx.x;   // a digit a thread
        if (d < bins) {
            int32_t run = 0;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const uint16_t c = counts[w * bins + d];
                counts[w * bins + d] = static_cast<uint16_t>(run);
                run += c;
            }
            hist[d] = run;
        }
        cluster.sync();
        int32_t all = 0, before = 0;
        if (d < bins)
#pragma unroll
            for (int b = 0; b < kClusterBlocks; ++b) {
                const int32_t c = cluster.map_shared_rank(hist, b)[d];
                all += c;
                before += b < block ? c : 0;
            }
        const int32_t first = block_scan<kW>(all, warp_sums, &n);
        if (d < bins) {
            place[d] = first + before;
            if (block == 0 && a.offsets != nullptr && d < a.K)
                a.offsets[d] = first;
            if (block == 0 && a.starts != nullptr && pass == a.passes - 1)
                a.starts[d] = first;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < ITEMS; ++u)
            if (item[u].x >= 0) {
                const int32_t e = (item[u].x >> shift) & (bins - 1);
                const int to = place[e] + counts[warp * bins + e] + rank[u];
                cluster.map_shared_rank(pairs, to / kShare)[to % kShare] = item[u];
            }
        cluster.sync();
    }
    if (block == 0 && threadIdx.x == 0) {
        *a.total = n;
        if (a.offsets != nullptr)
            a.offsets[a.K] = n;
        if (a.starts != nullptr)
            a.starts[1 << a.bits[a.passes - 1]] = n;
    }
    for (int i = threadIdx.x; i < kShare; i += kClusterThreads) {
        const int p = block * kShare + i;
        if (p < n) {
            const int2 rp = pairs[i];
            a.order[p] = rp.y;
            if (a.rows != nullptr)
                a.rows[p] = rp.x;
        } else if (p < a.M) {
            a.order[p] = -1;
        }
    }
}

// offsets[r] for r in [0, K]: the number of sorted rows below r.  starts: where
// the rows with each value of r >> shift start (nullptr: only their number,
// *total).
__global__ void __launch_bounds__(128)
    lists_offsets_kernel(const int32_t *rows, const int32_t *total, const int32_t *starts,
                         int32_t shift, int32_t K, int32_t *__restrict__ offsets)
{
    let_next_start();
    wait_for_previous();
    const uint32_t r = blockIdx.x * 128u + threadIdx.x;   // K < 2^31
    if (r > static_cast<uint32_t>(K))
        return;
    // the answer is in [lo, lo + n]
    int32_t lo = 0, n;
    if (starts != nullptr && r < static_cast<uint32_t>(K)) {
        lo = starts[r >> shift];
        n = starts[(r >> shift) + 1] - lo;
    } else {
        n = *total;
    }
    if (r == static_cast<uint32_t>(K)) {
        offsets[r] = n;
        return;
    }
    while (n > 0) {
        // seven probes cut the range into eight; count those below r
        const int32_t step = (n >> 3) + ((n & 7) != 0);
        int32_t below = 0;
#pragma unroll
        for (int q = 1; q < 8; ++q) {
            const int32_t at = q * step - 1;
            below += at < n && rows[lo + at] < static_cast<int32_t>(r);
        }
        lo += below * step;
        n -= below * step;
        if (below < 7)
            n = min(step - 1, n);
    }
    offsets[r] = lo;
}

struct SortPlan {
    int passes;
    int32_t bits[4], shift[4];
    int items;      // per thread and tile: 2, 4 or 8
    int blocks;
    int64_t share;
};

int row_bits(int64_t K)
{
    int bits = 0;
    while ((int64_t(1) << bits) < K)
        ++bits;
    return bits;
}

// The digits of a row id, as many bits each as evenly as they divide.
int digits(int64_t K, int most, int32_t *bits, int32_t *shift)
{
    const int all = row_bits(K);
    const int passes = std::max(1, (all + most - 1) / most);
    int at = 0;
    for (int i = 0; i < passes; ++i) {
        bits[i] = (all - at + (passes - i) - 1) / (passes - i);
        shift[i] = at;
        at += bits[i];
    }
    return passes;
}

SortPlan sort_plan(int64_t M, int64_t K, int sms)
{
    const int64_t most = int64_t(sms) * kBlocksPerSm;
    SortPlan p{};
    p.passes = digits(K, kMaxDigitBits, p.bits, p.shift);
    // the smallest tiles of which every block has one, else large ones in turn
    p.items = 8;
    for (int items = 4; items >= 2; items >>= 1)
        if (M <= most * kThreads * items)
            p.items = items;
    const int64_t tile = int64_t(kThreads) * p.items;
    const int64_t tiles = (M + tile - 1) / tile;
    const int64_t per = (tiles + most - 1) / most;
    p.share = per * tile;
    p.blocks = static_cast<int>((M + p.share - 1) / p.share);
    return p;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

int32_t fill_parts(size_t bytes, int32_t launches)
{
    return static_cast<int32_t>(
        std::min<size_t>((bytes + (size_t(16) << 20) - 1) >> 24, static_cast<size_t>(launches)));
}

// Blocks of `threads` threads that fill a share: 16 KiB or more each, at most
// as many as the SMs hold.
unsigned fill_blocks(const Fill &f, int threads, int sms)
{
    if (!f.any())
        return 0;
    return static_cast<unsigned>(
        std::min<int64_t>(f.bytes / f.parts / 16384 + 1, int64_t(sms) * 2048 / threads));
}

cudaError_t launch_offsets(const int32_t *rows, const int32_t *total, const int32_t *starts,
                           int32_t shift, int64_t K, int32_t *offsets, cudaStream_t stream)
{
    return launch_after(lists_offsets_kernel, static_cast<unsigned>(K / 128 + 1), 128, 0, stream,
                        rows, total, starts, shift, K, offsets);
}

template <bool FIRST>
cudaError_t sort_pass(SortArgs &a, int items, int sms, cudaStream_t stream)
{
    const cudaError_t e = launch_after(lists_count_kernel<FIRST>, static_cast<unsigned>(a.blocks),
                                       kThreads, static_cast<size_t>(a.bins) * 4, stream, a);
    if (e != cudaSuccess)
        return e;
    const unsigned blocks = static_cast<unsigned>(a.blocks) + fill_blocks(a.fill, kThreads, sms);
    const size_t smem = scatter_smem(a.bins, items);
    switch (items) {
    case 2:
        return launch_after(lists_scatter_kernel<2, FIRST>, blocks, kThreads, smem, stream, a);
    case 4:
        return launch_after(lists_scatter_kernel<4, FIRST>, blocks, kThreads, smem, stream, a);
    default:
        return launch_after(lists_scatter_kernel<8, FIRST>, blocks, kThreads, smem, stream, a);
    }
}

}  // namespace

cudaError_t lists_prepare()
{
    const int smem = static_cast<int>(scatter_smem(1 << kMaxDigitBits, 8));
    for (auto *f : {lists_scatter_kernel<2, false>, lists_scatter_kernel<2, true>,
                    lists_scatter_kernel<4, false>, lists_scatter_kernel<4, true>,
                    lists_scatter_kernel<8, false>, lists_scatter_kernel<8, true>}) {
        const cudaError_t e =
            cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return e;
    }
    return cudaFuncSetAttribute(lists_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kClusterSmem);
}

size_t lists_scratch_bytes(int64_t M, int64_t K, int sms)
{
    if (M <= kOneBlockMax)
        return K <= kOneOffsetsMax ? 0 : 16 + static_cast<size_t>(M) * 4;
    if (M <= kClusterMax)   // total, the last digit's starts, the sorted rows
        return 16 + up16((size_t(4) << kMaxDigitBits) + 4) + up16(static_cast<size_t>(M) * 4);
    const SortPlan p = sort_plan(M, K, sms);
    // total, the digits' counts, two sets of pairs (the second set's rows may
    // stand in for the sorted rows)
    size_t n = 16;
    for (int i = 0; i < p.passes; ++i)
        n += up16((size_t(4) << p.bits[i]) * p.blocks);
    n += up16((size_t(4) << p.bits[p.passes - 1]) + 4);   // the last digit's starts
    const size_t sets = p.passes == 1 ? 0 : p.passes == 2 ? 1 : 2;
    return n + sets * 2 * up16(static_cast<size_t>(M) * 4) + up16(static_cast<size_t>(M) * 4);
}

cudaError_t launch_lists(const int32_t *idx, int64_t M, int64_t K, int32_t *order, int32_t *rows,
                         int32_t *offsets, int32_t *total, void *scratch, void *zero,
                         size_t zero_bytes, int sms, cudaStream_t stream)
{
    cudaError_t e = cudaSuccess;
    Fill fill{static_cast<uint8_t *>(zero), static_cast<int64_t>(zero_bytes), 0, 1};
    if (M <= kOneBlockMax) {
        const bool search = offsets != nullptr && K > kOneOffsetsMax;   // in a launch of its own
        int32_t *own = search ? nullptr : offsets;
        if (search && total == nullptr)
            total = static_cast<int32_t *>(scratch);
        if (search && rows == nullptr)
            rows = static_cast<int32_t *>(scratch) + 4;
        fill.parts = fill_parts(zero_bytes, 1);
        if (M <= 1024)
            e = launch_after(lists_one_block_kernel<256, 4>, 1 + fill_blocks(fill, 256, sms), 256,
                             0, stream, idx, M, K, row_bits(K), order, rows,
                             own, total, fill);
        else
            e = launch_after(lists_one_block_kernel<1024, 2>, 1 + fill_blocks(fill, 1024, sms), 1024,
                             0, stream, idx, M, K, row_bits(K), order, rows,
                             own, total, fill);
        if (e == cudaSuccess && search)
            e = launch_offsets(rows, total, nullptr, 0, K, offsets, stream);
        return e;
    }
    if (M <= kClusterMax) {
        ClusterArgs a{};
        a.passes = digits(K, kMaxDigitBits, a.bits, a.shift);
        a.idx = idx;
        a.order = order;
        uint8_t *at = static_cast<uint8_t *>(scratch);
        a.total = total != nullptr ? total : reinterpret_cast<int32_t *>(at);
        if (a.passes == 1 || offsets == nullptr) {
            a.offsets = offsets;
            a.rows = rows;
        } else {
            a.starts = reinterpret_cast<int32_t *>(at + 16);
            a.rows = rows != nullptr
                         ? rows
                         : reinterpret_cast<int32_t *>(at + 16 + up16((size_t(4) << kMaxDigitBits) + 4));
        }
        a.M = static_cast<int32_t>(M);
        a.K = static_cast<int32_t>(K);
        fill.parts = fill_parts(zero_bytes, 1);
        a.fill = fill;
        // clusters that fill: on four fifths of the SMs (120 blocks of GB300's 152), so that they
        // run at once with the one that sorts
        const unsigned most = std::max<unsigned>(
            kClusterBlocks, static_cast<unsigned>(sms) * 4 / 5 / kClusterBlocks * kClusterBlocks);
        const unsigned blocks =
            kClusterBlocks +
            (std::min(fill_blocks(fill, kClusterThreads, sms), most) + kClusterBlocks - 1) /
                kClusterBlocks * kClusterBlocks;
        e = launch_after(lists_cluster_kernel, blocks, kClusterThreads, kClusterSmem, stream, a);
        if (e == cudaSuccess && a.starts != nullptr)
            e = launch_offsets(a.rows, a.total, a.starts, a.shift[a.passes - 1], K, offsets, stream);
        return e;
    }
    const SortPlan p = sort_plan(M, K, sms);
    const size_t ids = up16(static_cast<size_t>(M) * 4);
    uint8_t *at = static_cast<uint8_t *>(scratch);
    if (total == nullptr)
        total = reinterpret_cast<int32_t *>(at);
    at += 16;
    int32_t *hist[4] = {};
    for (int i = 0; i < p.passes; ++i) {
        hist[i] = reinterpret_cast<int32_t *>(at);
        at += up16((size_t(4) << p.bits[i]) * p.blocks);
    }
    int32_t *starts = reinterpret_cast<int32_t *>(at);
    at += up16((size_t(4) << p.bits[p.passes - 1]) + 4);
    int32_t *sorted = rows;
    if (sorted == nullptr && p.passes > 1 && offsets != nullptr)
        sorted = reinterpret_cast<int32_t *>(at);   // searched for the offsets
    at += ids;
    int32_t *set[2][2] = {};   // rows, positions
    for (int i = 0; i < std::min(p.passes - 1, 2); ++i)
        for (int j = 0; j < 2; ++j) {
            set[i][j] = reinterpret_cast<int32_t *>(at);
            at += ids;
        }
    fill.parts = fill_parts(zero_bytes, p.passes);
    for (int i = 0; i < p.passes && e == cudaSuccess; ++i) {
        SortArgs a{};
        a.fill = fill;
        a.fill.part = i;
        a.last = i == p.passes - 1;
        a.rows_in = i == 0 ? idx : set[(i - 1) & 1][0];
        a.pos_in = i == 0 ? nullptr : set[(i - 1) & 1][1];
        a.rows_out = a.last ? sorted : set[i & 1][0];
        a.pos_out = a.last ? order : set[i & 1][1];
        a.offsets = p.passes == 1 ? offsets : nullptr;
        a.hist = hist[i];
        a.total = total;
        a.starts = a.last ? starts : nullptr;
        a.M = M;
        a.share = p.share;
        a.K = static_cast<int32_t>(K);
        a.shift = p.shift[i];
        a.bins = 1 << p.bits[i];
        a.blocks = p.blocks;
        e = i == 0 ? sort_pass<true>(a, p.items, sms, stream)
                   : sort_pass<false>(a, p.items, sms, stream);
    }
    if (e == cudaSuccess && p.passes > 1 && offsets != nullptr)
        e = launch_offsets(sorted, total, starts, p.shift[p.passes - 1], K, offsets, stream);
    return e;
}

}  // namespace kma
