// lists.cu -- inverted lists: the positions of idx[0, M) grouped by the row
// that they name, each group in ascending order (a stable sort), with ids
// outside [0, K) left out; offsets[r] is where row r's group begins.
//
// A radix sort from the lowest digit up, of (row, position) pairs.  Each of up
// to 152 blocks owns one contiguous share of the pairs, so the order within a
// digit is: earlier blocks first, then the block's own items in order.
//   count:    block b counts its items by the first digit -> H0[b][digit]
//   scatter:  block b sums H[b'][digit] over the blocks b' before it and over
//             all blocks, scans the digits, ranks its items (a warp's equal
//             digits by match, warps by a per-warp count in shared memory) and
//             writes them; it also counts the next digit for the block that
//             will own the written place (integer atomics: any order gives the
//             same counts).
// So a sort of P digits is 1 + P launches, and up to kOneBlockMax items are one
// launch of one block.  Nothing depends on timing: the result is unique.
#include "internal.h"

#include <algorithm>

namespace kma {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDigitBits = 10;
constexpr int kMaxBins = 1 << kMaxDigitBits;
constexpr int kMaxBlocks = 152;
constexpr int64_t kOneBlockMax = 4096;
constexpr int64_t kOneOffsetsMax = 8192;   // rows whose offsets the one block finds itself
constexpr int kOneThreads = 1024;
constexpr int kOneWarps = kOneThreads / 32;
constexpr int kOneItems = static_cast<int>(kOneBlockMax) / kOneThreads;
constexpr int kOneBits = 6;   // digit of the one-block sort
constexpr int kOneBins = 1 << kOneBits;

// Exclusive scan over the block of one value per thread; *total: the sum.
// warp_sums: blockDim.x / 32 + 1 values.
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
__device__ __forceinline__ int32_t warp_rank(int32_t d, int32_t *counts, int lane)
{
    const uint32_t same = __match_any_sync(kAll, d);
    const uint32_t below = same & ((1u << lane) - 1u);
    int32_t base = 0;
    if (d >= 0 && below == 0) {
        base = counts[d];
        counts[d] = base + __popc(same);
    }
    base = __shfl_sync(kAll, base, __ffs(same) - 1);
    __syncwarp();
    return base + __popc(below);
}

struct SortArgs {
    const int32_t *idx;     // first pass: the rows, position = index
    const int2 *in;         // later passes: (row, position)
    int2 *out;              // all but the last pass
    int32_t *order;         // last pass
    int32_t *rows;          // last pass, or nullptr: the rows in sorted order
    int32_t *offsets;       // last pass of a one-digit sort, else nullptr
    const int32_t *hist;    // H[block][bins] of this digit
    int32_t *next_hist;     // of the next digit, or nullptr
    int32_t *total;         // valid ids: written by the first pass, read by later ones
    int64_t M;
    int64_t share;          // items per block
    int32_t K;
    int32_t shift, bins;    // this digit: (row >> shift) & (bins - 1)
    int32_t next_shift, next_bins;
    int32_t blocks;
};

// H[b][d] of the first digit; the later digits' counts are zeroed.
__global__ void __launch_bounds__(kThreads)
    lists_count_kernel(const int32_t *__restrict__ idx, int64_t M, int64_t share, int32_t K,
                       int32_t bins, int32_t *__restrict__ hist, int32_t *__restrict__ later,
                       int64_t n_later)
{
    __shared__ int32_t h[kMaxBins];
    for (int d = threadIdx.x; d < bins; d += kThreads)
        h[d] = 0;
    for (int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; d < n_later;
         d += static_cast<int64_t>(gridDim.x) * kThreads)
        later[d] = 0;
    __syncthreads();
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * share;
    const int64_t end = min(M, begin + share);
    for (int64_t i = begin + threadIdx.x; i < end; i += kThreads) {
        const int32_t r = __ldg(idx + i);
        if (r >= 0 && r < K)
            atomicAdd(h + (r & (bins - 1)), 1);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += kThreads)
        hist[static_cast<int64_t>(blockIdx.x) * bins + d] = h[d];
}

template <int ITEMS, bool FIRST>
__global__ void __launch_bounds__(kThreads) lists_scatter_kernel(const SortArgs a)
{
    extern __shared__ int32_t smem[];
    int32_t *base = smem;                    // [bins] next place of each digit, this block
    int32_t *counts = smem + a.bins;         // [kWarps][bins] of one tile
    __shared__ int32_t warp_sums[kWarps + 1];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;

    // places: all smaller digits, then this digit in earlier blocks; the
    // threads share out the blocks' counts of a digit (integer sums)
    int32_t *all = counts, *before = counts + a.bins;
    for (int d = threadIdx.x; d < 2 * a.bins; d += kThreads)
        counts[d] = 0;
    __syncthreads();
    const int lanes = max(1, kThreads / a.bins);   // threads per digit
    for (int t = threadIdx.x; t < a.bins * lanes; t += kThreads) {
        const int d = t & (a.bins - 1);
        int32_t n_all = 0, n_before = 0;
#pragma unroll 8
        for (int b = t / a.bins; b < a.blocks; b += lanes) {
            const int32_t n = __ldg(a.hist + static_cast<int64_t>(b) * a.bins + d);
            n_all += n;
            n_before += b < static_cast<int>(blockIdx.x) ? n : 0;
        }
        atomicAdd(all + d, n_all);
        atomicAdd(before + d, n_before);
    }
    __syncthreads();
    int32_t carry = 0;
    for (int d0 = 0; d0 < a.bins; d0 += kThreads) {
        const int d = d0 + threadIdx.x;
        int32_t sum;
        const int32_t first =
            carry + block_scan<kWarps>(d < a.bins ? all[d] : 0, warp_sums, &sum);
        carry += sum;
        if (d < a.bins) {
            base[d] = first + before[d];
            if (a.offsets != nullptr && blockIdx.x == 0 && d < a.K)
                a.offsets[d] = first;
        }
    }
    __syncthreads();   // counts is reused below
    const int32_t total = carry;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (FIRST && a.total != nullptr)
            *a.total = total;
        if (a.offsets != nullptr)
            a.offsets[a.K] = total;
    }

    const int64_t limit = FIRST ? a.M : total;
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * a.share;
    const int64_t end = min(limit, begin + a.share);
    for (int64_t t0 = begin; t0 < end; t0 += kThreads * ITEMS) {
        for (int c = threadIdx.x; c < kWarps * a.bins; c += kThreads)
            counts[c] = 0;
        __syncthreads();
        int32_t row[ITEMS], pos[ITEMS], rank[ITEMS];
        const int64_t w0 = t0 + static_cast<int64_t>(warp) * (32 * ITEMS) + lane;
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            const int64_t i = w0 + u * 32;
            row[u] = -1;
            pos[u] = static_cast<int32_t>(i);
            if (i < end) {
                if constexpr (FIRST) {
                    const int32_t r = __ldg(a.idx + i);
                    row[u] = r >= 0 && r < a.K ? r : -1;
                } else {
                    const int2 rp = __ldg(a.in + i);
                    row[u] = rp.x;
                    pos[u] = rp.y;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < ITEMS; ++u) {
            const int32_t d = row[u] < 0 ? -1 : (row[u] >> a.shift) & (a.bins - 1);
            rank[u] = warp_rank(d, counts + warp * a.bins, lane);
        }
        __syncthreads();
        // per digit: the warps' starts
        for (int d = threadIdx.x; d < a.bins; d += kThreads) {
            int32_t run = base[d];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int32_t n = counts[w * a.bins + d];
                counts[w * a.bins + d] = run;
                run += n;
            }
            base[d] = run;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < ITEMS; ++u)
            if (row[u] >= 0) {
                const int32_t d = (row[u] >> a.shift) & (a.bins - 1);
                const int32_t to = counts[warp * a.bins + d] + rank[u];
                if (a.next_hist != nullptr) {
                    a.out[to] = make_int2(row[u], pos[u]);
                    const uint32_t owner = static_cast<uint32_t>(to) / static_cast<uint32_t>(a.share);
                    atomicAdd(a.next_hist + static_cast<int64_t>(owner) * a.next_bins +
                                  ((row[u] >> a.next_shift) & (a.next_bins - 1)),
                              1);
                } else {
                    a.order[to] = pos[u];
                    if (a.rows != nullptr)
                        a.rows[to] = row[u];
                }
            }
        __syncthreads();
    }
    // places that no valid id takes
    if (a.next_hist == nullptr)
        for (int64_t i = max(begin, static_cast<int64_t>(total)) + threadIdx.x;
             i < min(a.M, begin + a.share); i += kThreads)
            a.order[i] = -1;
}

// Up to kOneBlockMax items: every digit by one block, the pairs in shared
// memory.  Ids outside [0, K) carry the row K, sort last and become -1.
__global__ void __launch_bounds__(kOneThreads)
    lists_one_block_kernel(const int32_t *__restrict__ idx, int32_t M, int32_t K, int32_t bits,
                           int32_t *__restrict__ order, int32_t *__restrict__ rows,
                           int32_t *__restrict__ offsets, int32_t *__restrict__ total)
{
    __shared__ int32_t s_row[kOneBlockMax];
    __shared__ uint16_t s_pos[kOneBlockMax];
    __shared__ int32_t counts[kOneWarps][kOneBins];
    __shared__ int32_t warp_sums[kOneWarps + 1];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int items = (M + kOneThreads - 1) / kOneThreads;   // per thread, <= kOneItems
    int32_t row[kOneItems], pos[kOneItems], rank[kOneItems];
#pragma unroll
    for (int u = 0; u < kOneItems; ++u) {
        const int i = warp * (32 * items) + u * 32 + lane;
        const bool in = u < items && i < M;
        pos[u] = i;
        row[u] = -1;
        if (in) {
            const int32_t r = __ldg(idx + i);
            row[u] = r >= 0 && r < K ? r : K;
        }
    }
    for (int shift = 0; shift < bits; shift += kOneBits) {
        for (int c = threadIdx.x; c < kOneWarps * kOneBins; c += kOneThreads)
            (&counts[0][0])[c] = 0;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kOneItems; ++u)
            if (u < items) {
                const int32_t d = row[u] < 0 ? -1 : (row[u] >> shift) & (kOneBins - 1);
                rank[u] = warp_rank(d, counts[warp], lane);
            }
        __syncthreads();
        int32_t all = 0;
        if (threadIdx.x < kOneBins)
#pragma unroll
            for (int w = 0; w < kOneWarps; ++w)
                all += counts[w][threadIdx.x];
        int32_t sum;
        int32_t run = block_scan<kOneWarps>(all, warp_sums, &sum);
        if (threadIdx.x < kOneBins)
#pragma unroll
            for (int w = 0; w < kOneWarps; ++w) {
                const int32_t n = counts[w][threadIdx.x];
                counts[w][threadIdx.x] = run;
                run += n;
            }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kOneItems; ++u)
            if (u < items && row[u] >= 0) {
                const int to = counts[warp][(row[u] >> shift) & (kOneBins - 1)] + rank[u];
                s_row[to] = row[u];
                s_pos[to] = static_cast<uint16_t>(pos[u]);
            }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kOneItems; ++u) {
            const int i = warp * (32 * items) + u * 32 + lane;
            if (u < items && i < M) {
                row[u] = s_row[i];
                pos[u] = s_pos[i];
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kOneItems; ++u) {
        const int i = warp * (32 * items) + u * 32 + lane;
        if (u < items && i < M) {
            order[i] = row[u] < K ? pos[u] : -1;
            if (rows != nullptr)
                rows[i] = row[u];
            s_row[i] = row[u];
        }
    }
    __syncthreads();
    // offsets[r]: the first place whose row is at least r (K <= kOneOffsetsMax;
    // else only their number, for the offsets' own launch)
    const int32_t most = offsets != nullptr ? K : threadIdx.x == 0 ? K : -1;
    for (int32_t r = offsets != nullptr ? threadIdx.x : K; r <= most; r += kOneThreads) {
        int lo = 0, hi = M;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_row[mid] < r)
                lo = mid + 1;
            else
                hi = mid;
        }
        if (offsets != nullptr)
            offsets[r] = lo;
        else
            *total = lo;
        if (r == K)
            break;   // no step past the largest row
    }
}

// offsets[r] for r in [0, K] by bisection in the sorted rows.
__global__ void __launch_bounds__(256)
    lists_offsets_kernel(const int32_t *__restrict__ rows, const int32_t *__restrict__ total,
                         int32_t K, int32_t *__restrict__ offsets)
{
    const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (r > K)
        return;
    int32_t lo = 0, hi = *total;
    while (lo < hi) {
        const int32_t mid = lo + ((hi - lo) >> 1);
        if (__ldg(rows + mid) < r)
            lo = mid + 1;
        else
            hi = mid;
    }
    offsets[r] = lo;
}

struct SortPlan {
    int passes;
    int bits[4], shift[4];
    int items;      // per thread and tile: 2 or 8
    int blocks;
    int64_t share;
};

SortPlan sort_plan(int64_t M, int64_t K)
{
    SortPlan p{};
    int bits = 0;
    while ((int64_t(1) << bits) < K)
        ++bits;
    p.passes = std::max(1, (bits + kMaxDigitBits - 1) / kMaxDigitBits);
    int at = 0;
    for (int i = 0; i < p.passes; ++i) {
        p.bits[i] = (bits - at + (p.passes - i) - 1) / (p.passes - i);
        p.shift[i] = at;
        at += p.bits[i];
    }
    p.items = M <= int64_t(kMaxBlocks) * kThreads * 2 ? 2 : 8;
    const int64_t tile = int64_t(kThreads) * p.items;
    const int64_t tiles = (M + tile - 1) / tile;
    const int64_t per = (tiles + kMaxBlocks - 1) / kMaxBlocks;
    p.share = per * tile;
    p.blocks = static_cast<int>((M + p.share - 1) / p.share);
    return p;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

void launch_offsets(const int32_t *rows, const int32_t *total, int64_t K, int32_t *offsets,
                    cudaStream_t stream)
{
    const int64_t blocks = (K + 1 + 255) / 256;
    lists_offsets_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        rows, total, static_cast<int32_t>(K), offsets);
}

template <bool FIRST>
void scatter(const SortArgs &a, int items, cudaStream_t stream)
{
    const size_t smem = static_cast<size_t>(kWarps + 1) * a.bins * 4;
    if (items == 2)
        lists_scatter_kernel<2, FIRST><<<a.blocks, kThreads, smem, stream>>>(a);
    else
        lists_scatter_kernel<8, FIRST><<<a.blocks, kThreads, smem, stream>>>(a);
}

}  // namespace

cudaError_t lists_prepare()
{
    const int smem = (kWarps + 1) * kMaxBins * 4;
    for (auto *f : {lists_scatter_kernel<2, false>, lists_scatter_kernel<2, true>,
                    lists_scatter_kernel<8, false>, lists_scatter_kernel<8, true>}) {
        const cudaError_t e =
            cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

size_t lists_scratch_bytes(int64_t M, int64_t K)
{
    if (M <= kOneBlockMax)
        return K <= kOneOffsetsMax ? 0 : 16 + static_cast<size_t>(M) * 4;
    const SortPlan p = sort_plan(M, K);
    size_t n = 16;   // total
    for (int i = 0; i < p.passes; ++i)
        n += up16((size_t(4) << p.bits[i]) * p.blocks);
    if (p.passes > 1)
        n += static_cast<size_t>(std::min(p.passes - 1, 2)) * up16(static_cast<size_t>(M) * 8) +
             up16(static_cast<size_t>(M) * 4);
    return n;
}

cudaError_t launch_lists(const int32_t *idx, int64_t M, int64_t K, int32_t *order, int32_t *rows,
                         int32_t *offsets, void *scratch, cudaStream_t stream)
{
    if (M <= kOneBlockMax) {
        int bits = 0;
        while ((int64_t(1) << bits) <= K)   // rows 0 to K
            ++bits;
        const bool own = K <= kOneOffsetsMax;
        int32_t *total = static_cast<int32_t *>(scratch);
        if (!own && rows == nullptr)
            rows = total + 4;
        lists_one_block_kernel<<<1, kOneThreads, 0, stream>>>(
            idx, static_cast<int32_t>(M), static_cast<int32_t>(K), bits, order, rows,
            own ? offsets : nullptr, total);
        if (!own)
            launch_offsets(rows, total, K, offsets, stream);
        return cudaGetLastError();
    }
    const SortPlan p = sort_plan(M, K);
    uint8_t *at = static_cast<uint8_t *>(scratch);
    int32_t *total = reinterpret_cast<int32_t *>(at);
    at += 16;
    int32_t *hist[4] = {};
    int64_t later = 0;   // counters of the later digits, one piece of memory
    for (int i = 0; i < p.passes; ++i) {
        hist[i] = reinterpret_cast<int32_t *>(at);
        at += up16((size_t(4) << p.bits[i]) * p.blocks);
        if (i > 0)
            later += up16((size_t(4) << p.bits[i]) * p.blocks) / 4;
    }
    int2 *pairs[2] = {};
    int32_t *sorted = rows;
    if (p.passes > 1) {
        for (int i = 0; i < std::min(p.passes - 1, 2); ++i) {
            pairs[i] = reinterpret_cast<int2 *>(at);
            at += up16(static_cast<size_t>(M) * 8);
        }
        if (sorted == nullptr)
            sorted = reinterpret_cast<int32_t *>(at);
    }
    lists_count_kernel<<<p.blocks, kThreads, 0, stream>>>(
        idx, M, p.share, static_cast<int32_t>(K), 1 << p.bits[0], hist[0], hist[1], later);
    for (int i = 0; i < p.passes; ++i) {
        const bool last = i == p.passes - 1;
        SortArgs a{};
        a.idx = idx;
        a.in = i > 0 ? pairs[(i - 1) & 1] : nullptr;
        a.out = last ? nullptr : pairs[i & 1];
        a.order = order;
        a.rows = sorted;
        a.offsets = p.passes == 1 ? offsets : nullptr;
        a.hist = hist[i];
        a.next_hist = last ? nullptr : hist[i + 1];
        a.total = total;
        a.M = M;
        a.share = p.share;
        a.K = static_cast<int32_t>(K);
        a.shift = p.shift[i];
        a.bins = 1 << p.bits[i];
        a.next_shift = last ? 0 : p.shift[i + 1];
        a.next_bins = last ? 1 : 1 << p.bits[i + 1];
        a.blocks = p.blocks;
        if (i == 0)
            scatter<true>(a, p.items, stream);
        else
            scatter<false>(a, p.items, stream);
    }
    if (p.passes > 1)
        launch_offsets(sorted, total, K, offsets, stream);
    return cudaGetLastError();
}

}  // namespace kma
