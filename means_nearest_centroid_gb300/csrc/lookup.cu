// lookup.cu -- the rows of a table that ids name, weighted and scaled, and the
// gradients of the table and of the weights:
//     out[i]   = scale sum_j w[i][j] table[idx[i][j]]
//     dtable[r] = scale sum over idx[i][j] == r of w[i][j] dout[i]
//     dw[i][j] = scale <dout[i], table[idx[i][j]]>
// (w = 1 without weights; ids outside [0, K) add nothing).  Sums are fp32, each
// output is rounded once.
//
// The gradient of the table sorts the ids by row first (lists.cu).  The sorted
// places are then cut into chunks of a fixed length; a group of lanes sums one
// slice of columns over one chunk in registers and writes a row as soon as its
// last place is passed.  A row that continues past a chunk's end leaves its
// parts in a workspace, and a second launch adds those in chunk order.  Every
// row that ids name is written once, by one group, and the order of every sum
// follows from the sizes alone: the bits do not change from run to run.  The
// whole table is zeroed by the sort's launches, which leave HBM idle: for 131,072
// rows of 2,048 (1.07 GB, 140 us) that hides the sort: the gradient of 16,384
// tokens takes 191 us, where blocks that zeroed the rows without ids after the
// same sort took 42 us longer.
#include "launch.cuh"
#include "learn.h"
#include "vec.cuh"

#include <algorithm>
#include <initializer_list>
#include <utility>

namespace kma {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kThreads = 256;

// ---- lookup ---------------------------------------------------------------

struct LookupArgs {
    const void *table;
    const int32_t *idx;
    const float *weights;
    void *out;
    int64_t N;
    int32_t K, D;
    int32_t vecs;          // vectors per row
    int32_t rows;          // rows of a block side by side
    uint32_t magic;        // t / vecs == t * magic >> 16 for t < 256
    float scale;
};

// A block takes rows side by side where several fit its threads, else one and
// a piece of 256 vectors of it (blockIdx.y); the thread's vector and row.
__device__ __forceinline__ bool lookup_place(const LookupArgs &a, int &row, int &vec)
{
    row = static_cast<int>((threadIdx.x * a.magic) >> 16);
    vec = static_cast<int>(threadIdx.x) - row * a.vecs;
    if (a.vecs > kThreads) {
        row = 0;
        vec = static_cast<int>(blockIdx.y) * kThreads + threadIdx.x;
    }
    return row < a.rows && vec < a.vecs;
}

// One id a point: a copy, U points a thread in flight.  Bound by HBM: 16,384
// rows of 2,048 bf16 take 22.7 us, 5.9 TB/s (floor 20).
template <typename T, int VE, int U>
__global__ void __launch_bounds__(kThreads) lookup_one_kernel(const LookupArgs a)
{
    int r0, vec;
    if (!lookup_place(a, r0, vec))
        return;
    const T *table = static_cast<const T *>(a.table) + static_cast<int64_t>(vec) * VE;
    T *out = static_cast<T *>(a.out) + static_cast<int64_t>(vec) * VE;
    int64_t i[U];
    int32_t r[U];
    Raw<T, VE> q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        i[u] = (static_cast<int64_t>(blockIdx.x) * U + u) * a.rows + r0;
        r[u] = i[u] < a.N ? __ldg(a.idx + i[u]) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (r[u] >= 0 && r[u] < a.K)
            q[u] = load_raw<T, VE>(table + static_cast<int64_t>(r[u]) * a.D);
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (i[u] < a.N) {
            float acc[VE] = {};
            if (r[u] >= 0 && r[u] < a.K) {
                widen<T, VE>(q[u], acc);
                const float w = a.weights != nullptr ? __ldg(a.weights + i[u]) : 1.0f;
#pragma unroll
                for (int v = 0; v < VE; ++v)
                    acc[v] *= w;
            }
#pragma unroll
            for (int v = 0; v < VE; ++v)
                acc[v] *= a.scale;
            store_raw<T, VE>(out + i[u] * a.D, narrow<T, VE>(acc));
        }
}

// The same for rows of an odd number of 2-byte elements, or at odd offsets: a
// thread writes an aligned 16-byte vector of its output row (at the row's ends
// some elements of one), gathered from aligned words of the table's row; where
// the two rows' offsets differ by an odd number of elements, words are joined in
// pairs.  16,384 rows of 2,047 bf16: 39 us (2,048: 23); an element a thread 56,
// a word of two elements a thread 66.
template <typename T>
__global__ void __launch_bounds__(kThreads) lookup_odd_kernel(const LookupArgs a)
{
    static_assert(sizeof(T) == 2, "two elements a word");
    constexpr int VE = 8;
    int r0, vec;
    if (!lookup_place(a, r0, vec))
        return;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * a.rows + r0;
    if (i >= a.N)
        return;
    T *out = static_cast<T *>(a.out) + i * a.D;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(out) & 15) / 2;
    const int e0 = vec * VE - off, begin = max(e0, 0), end = min(e0 + VE, a.D);
    if (begin >= end)
        return;
    const int32_t r = __ldg(a.idx + i);
    const bool there = static_cast<uint32_t>(r) < static_cast<uint32_t>(a.K);
    const float w = there && a.weights != nullptr ? __ldg(a.weights + i) : 1.0f;
    const T *table = static_cast<const T *>(a.table);
    const T *row = table + static_cast<int64_t>(there ? r : 0) * a.D;
    const T *from = row + e0;
    const bool odd = (reinterpret_cast<uintptr_t>(from) & 3) != 0;
    // an odd start reads one element more at either end, which has to be the table's
    if (end - begin < VE ||
        (odd && (from == table || from + VE == table + static_cast<int64_t>(a.K) * a.D))) {
        for (int e = begin; e < end; ++e)
            out[e] = Elem<T>::down(there ? Elem<T>::up(row[e]) * w * a.scale : 0.0f);
        return;
    }
    uint32_t q[4] = {0u, 0u, 0u, 0u};
    if (there) {
        if (!odd) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                q[u] = __ldg(reinterpret_cast<const uint32_t *>(from) + u);
        } else {
            const uint32_t *words = reinterpret_cast<const uint32_t *>(from - 1);
            uint32_t p[5];
#pragma unroll
            for (int u = 0; u < 5; ++u)
                p[u] = __ldg(words + u);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                q[u] = __funnelshift_r(p[u], p[u + 1], 16);
        }
    }
    float f[VE];
    Raw<T, VE> raw;
    memcpy(&raw, q, 16);
    widen<T, VE>(raw, f);
#pragma unroll
    for (int v = 0; v < VE; ++v)
        f[v] = f[v] * w * a.scale;
    store_raw<T, VE>(out + e0, narrow<T, VE>(f));
}

// ---- groups of lanes over columns -------------------------------------------
//
// What sums rows works in groups of LG lanes (8, 16 or 32, for rows of up to 64,
// 128 or more columns), each lane holding 8 columns as NV vectors of VE, so
// that narrow or oddly aligned rows cost the same bookkeeping per id as wide ones.

constexpr int kLaneCols = 8;

template <int VE, int LG>
struct Columns {
    static constexpr int kVectors = kLaneCols / VE;
    static constexpr int kSlice = LG * kLaneCols;   // columns of a group
    __device__ static __forceinline__ int at(int slice, int lane, int v)
    {
        return slice * kSlice + v * LG * VE + lane * VE;
    }
    // A lane's vectors of a row, from its first one on (fixed distances, so that a row costs
    // one address); zeros past D, or where the row is not there.
    template <typename T>
    __device__ static __forceinline__ void read(Raw<T, VE> (&q)[kVectors], const T *first,
                                                const bool (&in)[kVectors], bool there)
    {
#pragma unroll
        for (int v = 0; v < kVectors; ++v) {
            q[v] = Raw<T, VE>{};
            if (there && in[v])
                q[v] = load_raw<T, VE>(first + v * LG * VE);
        }
    }
};

// ---- lookup of several ids --------------------------------------------------

struct GatherArgs {
    const void *table;
    const int32_t *idx;
    const float *weights;
    void *out;
    int64_t N;
    int32_t k, K, D;
    int32_t slices;
    float scale;
};

// A group of lanes per point and slice of columns; lane u reads id u of eight,
// U rows are in flight.  Bound by the rows' way from L2 (268 MB for 65,536
// points of 8 ids in a table of 8 MB: 27 us, 10 TB/s); 20,011 points of 7 ids and
// 255 columns, at 2-byte boundaries, 16.5 with the call.  Groups that went through several
// points and read the next ids early, and rows copied asynchronously into shared
// memory, were 0 to 50% slower.
template <typename T, int VE, int LG, int U>
__global__ void __launch_bounds__(kThreads) lookup_many_kernel(const GatherArgs a)
{
    using C = Columns<VE, LG>;
    constexpr int NV = C::kVectors;
    const int lane = threadIdx.x & (LG - 1);
    const int64_t unit =
        static_cast<int64_t>(blockIdx.x) * (kThreads / LG) + threadIdx.x / LG;
    const bool live = unit < a.N * a.slices;
    const int64_t i = live ? unit / a.slices : a.N - 1;
    const int slice = live ? static_cast<int>(unit - i * a.slices) : 0;
    const T *table = static_cast<const T *>(a.table);
    const int col = C::at(slice, lane, 0);
    bool in[NV];
    Sums<VE> acc[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        in[v] = C::at(slice, lane, v) < a.D;
        acc[v].zero();
    }
    for (int32_t j0 = 0; j0 < a.k; j0 += 8) {
        const int32_t j = j0 + (lane & 7);
        int32_t r = -1;
        float w = 0.0f;   // an id of no row adds nothing, whatever its weight
        if (j < a.k) {
            r = __ldg(a.idx + i * a.k + j);
            if (static_cast<uint32_t>(r) >= static_cast<uint32_t>(a.K))
                r = -1;
            else
                w = a.weights != nullptr ? __ldg(a.weights + i * a.k + j) : 1.0f;
        }
#pragma unroll
        for (int u0 = 0; u0 < 8; u0 += U) {
            if (j0 + u0 >= a.k)
                break;
            Raw<T, VE> q[U][NV];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t ru = __shfl_sync(kAll, r, u0 + u, LG);
                C::template read<T>(q[u], table + static_cast<int64_t>(ru) * a.D + col, in, ru >= 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float wu = __shfl_sync(kAll, w, u0 + u, LG);
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    fma_raw<T, VE>(acc[v], q[u][v], wu);
            }
        }
    }
    T *out = static_cast<T *>(a.out) + i * a.D + col;
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (live && in[v]) {
            float f[VE];
            acc[v].get(f);
#pragma unroll
            for (int e = 0; e < VE; ++e)
                f[e] *= a.scale;
            store_raw<T, VE>(out + v * LG * VE, narrow<T, VE>(f));
        }
}

// Adds U values over a group's lanes together: after the step of distance d a
// lane holds the values whose numbers' bits its own lane's bits picked, half as
// many each time (for 8 values and 32 lanes 9 exchanges, not 40).  Returns the
// number of the value that sum[0] then holds; lanes with lane % (LG / U) == 0
// hold each once.
template <int U, int LG>
__device__ __forceinline__ int add_over_lanes(float (&sum)[U], int lane)
{
    int j = 0;
#pragma unroll
    for (int half = U / 2, off = LG / 2; half > 0; half >>= 1, off >>= 1) {
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int u = 0; u < half; ++u) {
            const float give = up ? sum[u] : sum[u + half];
            const float keep = up ? sum[u + half] : sum[u];
            sum[u] = keep + __shfl_xor_sync(kAll, give, off);
        }
        j += up ? half : 0;
    }
#pragma unroll
    for (int off = LG / U / 2; off > 0; off >>= 1)
        sum[0] += __shfl_xor_sync(kAll, sum[0], off);
    return j;
}

// ---- gradient of the weights ----------------------------------------------

struct DweightsArgs {
    const void *dout, *table;
    const int32_t *idx;
    float *dweights;
    int64_t N;
    int32_t k, K, D;
    float scale;
};

// For rows of more than one slice, or without a gradient of the table.  A group
// of lanes per point: its gradient is held in registers while the rows of its
// ids pass, eight in flight.  Bound by the gather of N k rows from L2.
template <typename T, int VE, int LG>
__global__ void __launch_bounds__(kThreads, 2) dweights_kernel(const DweightsArgs a)
{
    using C = Columns<VE, LG>;
    constexpr int NV = C::kVectors;
    constexpr int U = sizeof(T) == 2 ? 8 : 4;   // rows in flight
    const int lane = threadIdx.x & (LG - 1);
    const int64_t groups = static_cast<int64_t>(gridDim.x) * (kThreads / LG);
    const T *table = static_cast<const T *>(a.table);
    const int slices = (a.D + C::kSlice - 1) / C::kSlice;
    int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / LG) + threadIdx.x / LG;
    int32_t j0 = 0;
    auto read = [&](int64_t at, int32_t j) {   // lane u: id u of the eight, -1 for none
        const int32_t mine = j + (lane & 7);
        const int32_t r = at < a.N && mine < a.k ? __ldg(a.idx + at * a.k + mine) : -1;
        return static_cast<uint32_t>(r) < static_cast<uint32_t>(a.K) ? r : -1;
    };
    int32_t next = read(i, 0);
    // the groups of a warp go through as many points each, the last ones idle
    while (__any_sync(kAll, i < a.N)) {
        const int32_t ids = next;
        const int64_t at = i;
        const int32_t at_j = j0;
        j0 += 8;
        if (j0 >= a.k) {
            j0 = 0;
            i += groups;
        }
        next = read(i, j0);
        const T *dout = static_cast<const T *>(a.dout) + (at < a.N ? at : 0) * a.D;
        Sums<2> two[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            two[u].zero();
        for (int s = 0; s < slices; ++s) {
            const int col = C::at(s, lane, 0);
            bool in[NV];
            Sums<VE> p[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v)
                in[v] = C::at(s, lane, v) < a.D;
            Raw<T, VE> d[NV];
            C::template read<T>(d, dout + col, in, true);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float f[VE];
                widen<T, VE>(d[v], f);
                p[v].set(f);
            }
#pragma unroll
            for (int u0 = 0; u0 < 8; u0 += U) {
                Raw<T, VE> q[U][NV];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int32_t r = __shfl_sync(kAll, ids, u0 + u, LG);
                    C::template read<T>(q[u], table + static_cast<int64_t>(r) * a.D + col, in,
                                        r >= 0);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        dot_raw<T, VE>(two[u0 + u], p[v], q[u][v]);
            }
        }
        float sum[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            float f[2];
            two[u].get(f);
            sum[u] = f[0] + f[1];
        }
        const int j = add_over_lanes<8, LG>(sum, lane);
        // an id of no row counts 0, whatever dout holds
        const bool there = __shfl_sync(kAll, ids, j, LG) >= 0;
        if (at < a.N && (lane & (LG / 8 - 1)) == 0 && at_j + j < a.k)
            a.dweights[at * a.k + at_j + j] = there ? sum[0] * a.scale : 0.0f;
    }
}

// ---- gradient of the table ------------------------------------------------

struct GradArgs {
    const void *dout;
    const float *weights;      // or nullptr
    const int32_t *idx;        // of the points, for dweights
    const void *table;
    float *dweights;           // formed on the way, or nullptr
    const int32_t *order;      // sorted places -> flat (point, id) positions
    const int32_t *rows;       // the rows in sorted order
    const int32_t *total;      // sorted places
    void *dtable;
    float *parts;              // [2][chunks][D]: a chunk's first and last row, unfinished
    int64_t M;                 // ids
    int64_t chunks;
    int32_t chunk;             // sorted places per chunk, a multiple of 8
    int32_t slices;            // column slices of a row
    int32_t k, K, D;
    int32_t pitch;             // elements from a row of dtable to the next
    int32_t skip;              // a row that takes no gradient, or -1
    float scale;
    bool accumulate;
};

template <typename G, int VE>
__device__ __forceinline__ void put(const GradArgs &a, int32_t r, int col, const float (&acc)[VE])
{
    G *p = static_cast<G *>(a.dtable) + static_cast<int64_t>(r) * a.pitch + col;
    float f[VE];
#pragma unroll
    for (int v = 0; v < VE; ++v)
        f[v] = acc[v] * a.scale;
    if (r == a.skip) {
        if (a.accumulate)
            return;
#pragma unroll
        for (int v = 0; v < VE; ++v)
            f[v] = 0.0f;
    } else if (a.accumulate) {
        float old[VE];
        widen<G, VE>(load_raw<G, VE>(p), old);
#pragma unroll
        for (int v = 0; v < VE; ++v)
            f[v] += old[v];
    }
    store_raw<G, VE>(p, narrow<G, VE>(f));
}

// T: type of dout, G: of dtable.  DW (one slice): a place's weight's gradient is
// formed on the way, from the row of the table that its group holds meanwhile;
// the four sums of a batch are added over the lanes together.  For 30,011 points
// of 8 ids, 250 columns of bf16 and 16,384 rows it takes 32 us: the gathered
// rows come from L2 (131 MB), at 84 warp instructions each, and the 24 warps that
// 80 registers allow wait for them.  An address per vector instead of one per row
// cost 23 instructions more (40 us); the two gathers in kernels of their own 57 us
// on that footing.  Whole gradients of nine shapes: eight rows in flight at 16
// warps 7% faster to 7% slower (58.7 to 60.7 us here), 32 warps of 64 registers up
// to 16% slower (68), chunks for 48 warps up to 7%, ids and table rows read ahead
// of their use 0 to 5%.
template <typename T, typename G, int VE, int LG, bool DW>
__global__ void __launch_bounds__(kThreads, VE == 1 ? 2 : 3) segment_kernel(const GradArgs a)
{
    using C = Columns<VE, LG>;
    constexpr int NV = C::kVectors;
    constexpr int U = 4;   // rows in flight
    let_next_start();
    wait_for_previous();
    if constexpr (DW) {
        // ids of no row, which are not among the sorted places
        const int64_t threads = static_cast<int64_t>(gridDim.x) * kThreads;
        for (int64_t f = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; f < a.M;
             f += threads)
            if (static_cast<uint32_t>(a.idx[f]) >= static_cast<uint32_t>(a.K))
                a.dweights[f] = 0.0f;
    }
    const int lane = threadIdx.x & (LG - 1);
    const int64_t unit =
        static_cast<int64_t>(blockIdx.x) * (kThreads / LG) + threadIdx.x / LG;
    const int64_t chunk = unit / a.slices;
    const int slice = static_cast<int>(unit - chunk * a.slices);
    const int64_t total = *a.total;
    const int64_t begin = chunk * a.chunk;
    const bool live = chunk < a.chunks && begin < total;   // else: no place of its own
    const int64_t end = live ? min(total, begin + a.chunk) : begin;
    const T *dout = static_cast<const T *>(a.dout);
    // the row at `begin` began in an earlier chunk / that at `end` goes on
    const bool from_before = live && begin > 0 && a.rows[begin - 1] == a.rows[begin];
    const bool goes_on = live && end < total && a.rows[end - 1] == a.rows[end];

    const int col = C::at(slice, lane, 0);
    bool in[NV];
    Sums<VE> acc[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        in[v] = C::at(slice, lane, v) < a.D;
        acc[v].zero();
    }
    int32_t cur = live ? a.rows[begin] : -1;
    bool first = true;   // cur is the row at `begin`
    Sums<VE> t_row[DW ? NV : 1];   // the table's row cur, 0 past D
    auto read_row = [&]() {
        if constexpr (DW) {
            Raw<T, VE> t[NV];
            C::template read<T>(
                t, static_cast<const T *>(a.table) + static_cast<int64_t>(cur) * a.D + col, in, true);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float f[VE];
                widen<T, VE>(t[v], f);
                t_row[v].set(f);
            }
        }
    };
    if (DW && live)
        read_row();
    // the row summed so far: written, or left as the chunk's first (0) or last (1) part
    auto finish = [&](int which) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float f[VE];
            acc[v].get(f);
            if (in[v]) {
                if (which < 0)
                    put<G, VE>(a, cur, col + v * LG * VE, f);
                else
                    store_raw<float, VE>(
                        a.parts + (which * a.chunks + chunk) * a.D + col + v * LG * VE,
                        narrow<float, VE>(f));
            }
        }
    };
    for (int32_t s0 = 0; s0 < a.chunk; s0 += LG) {
        // a place per lane; the groups of a warp go through their chunks in step
        const int64_t s = begin + s0 + lane;
        int32_t row = -1, point = 0, f = -1;
        float w = 0.0f;
        if (s0 + lane < a.chunk && s < end) {
            f = a.order[s];
            row = a.rows[s];
            point = a.k == 1 ? f : f / a.k;
            w = a.weights != nullptr ? a.weights[f] : 1.0f;
        }
        const int n = min(LG, a.chunk - s0);
        for (int u0 = 0; u0 < n; u0 += U) {
            // every group of the warp has U places here, or some have fewer, or none any
            const bool whole = __all_sync(kAll, begin + s0 + u0 + U <= end);
            if (!whole && !__any_sync(kAll, begin + s0 + u0 < end))
                break;
            Raw<T, VE> q[U][NV];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t i = __shfl_sync(kAll, point, u0 + u, LG);
                C::template read<T>(q[u], dout + static_cast<int64_t>(i) * a.D + col, in,
                                    whole || begin + s0 + u0 + u < end);
            }
            Sums<2> two[DW ? U : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t r = __shfl_sync(kAll, row, u0 + u, LG);
                const float wu = __shfl_sync(kAll, w, u0 + u, LG);
                if (r != cur && r >= 0) {
                    finish(first && from_before ? 0 : -1);
                    first = false;
                    cur = r;
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        acc[v].zero();
                    if constexpr (DW)
                        read_row();
                }
                if constexpr (DW)
                    two[u].zero();
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    fma_raw<T, VE>(acc[v], q[u][v], wu);
                    if constexpr (DW)
                        dot_raw<T, VE>(two[u], t_row[v], q[u][v]);
                }
            }
            if constexpr (DW) {
                float sum[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float h[2];
                    two[u].get(h);
                    sum[u] = h[0] + h[1];
                }
                const int j = add_over_lanes<U, LG>(sum, lane);
                const int32_t to = __shfl_sync(kAll, f, u0 + j, LG);
                if (to >= 0 && (lane & (LG / U - 1)) == 0)
                    a.dweights[to] = sum[0] * a.scale;
            }
        }
    }
    if (live)
        finish(first && from_before ? 0 : goes_on ? 1 : -1);
}

// Rows that span chunks: the chunk in which such a row begins holds its first
// part as its last row; the following chunks hold the others as their first,
// the last of them found from the sorted rows at the chunks' starts.  A few us
// after the sums above, of dependent loads.
template <typename G, int VE, int LG>
__global__ void __launch_bounds__(kThreads) join_kernel(const GradArgs a)
{
    using C = Columns<VE, LG>;
    wait_for_previous();
    const int lane = threadIdx.x & (LG - 1);
    const int64_t unit =
        static_cast<int64_t>(blockIdx.x) * (kThreads / LG) + threadIdx.x / LG;
    const int64_t chunk = unit / a.slices;
    const int slice = static_cast<int>(unit - chunk * a.slices);
    const int64_t total = *a.total;
    const int64_t begin = chunk * a.chunk;
    const int64_t end = begin + a.chunk;
    if (chunk >= a.chunks || end >= total)
        return;
    const int32_t r = a.rows[end - 1];
    if (a.rows[end] != r || (begin > 0 && a.rows[begin] == r && a.rows[begin - 1] == r))
        return;   // ends here, or began in an earlier chunk
    // the last chunk that begins with the row: its lanes look at as many chunks at a time
    const uint32_t group = LG == 32 ? kAll : ((1u << LG) - 1u) << (threadIdx.x & (32 - LG));
    int64_t last = chunk + 1;
    for (;;) {
        const int64_t c = last + 1 + lane;
        const bool on = c < a.chunks && c * a.chunk < total && a.rows[c * a.chunk] == r;
        const int ahead = __popc(__ballot_sync(group, on) & group);
        last += ahead;   // the rows are sorted: those that are on come first
        if (ahead < LG)
            break;
    }
#pragma unroll 1
    for (int v = 0; v < C::kVectors; ++v) {
        const int col = C::at(slice, lane, v);
        if (col >= a.D)
            return;
        float acc[VE];
        widen<float, VE>(load_raw<float, VE>(a.parts + (a.chunks + chunk) * a.D + col), acc);
        for (int64_t c0 = chunk + 1; c0 <= last; c0 += 8) {
            Raw<float, VE> q[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (c0 + u <= last)
                    q[u] = load_raw<float, VE>(a.parts + (c0 + u) * a.D + col);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (c0 + u <= last) {
                    float f[VE];
                    widen<float, VE>(q[u], f);
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        acc[e] += f[e];
                }
        }
        put<G, VE>(a, r, col, acc);
    }
}

// ---- choices --------------------------------------------------------------

// Elements per vector: the most, up to 16 bytes of the input type, that
// divide D and that every pointer's alignment allows for its type.
int vector_elems(int64_t D, int most, std::initializer_list<std::pair<const void *, int>> ptrs)
{
    for (int ve = most; ve > 1; ve >>= 1) {
        bool ok = D % ve == 0;
        for (const auto &p : ptrs)
            if (p.first != nullptr &&
                reinterpret_cast<uintptr_t>(p.first) % std::min(16, ve * p.second) != 0)
                ok = false;
        if (ok)
            return ve;
    }
    return 1;
}

int most_elems(int dtype) { return 16 / dtype_bytes(dtype); }

// Calls f with an integral constant of ve (8 only for 16-bit types).
template <typename T, typename F>
cudaError_t by_elems(int ve, F f)
{
    if constexpr (sizeof(T) == 2)
        if (ve == 8)
            return f(std::integral_constant<int, 8>{});
    if (ve >= 4)
        return f(std::integral_constant<int, 4>{});
    if (ve == 2)
        return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1>{});
}

template <typename F>
cudaError_t by_type(int dtype, F f)
{
    if (dtype == kFp32)
        return f(float{});
    if (dtype == kBf16)
        return f(__nv_bfloat16{});
    return f(__half{});
}

int lane_group(int64_t D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

template <typename F>
cudaError_t by_group(int64_t D, F f)
{
    switch (lane_group(D)) {
    case 8:
        return f(std::integral_constant<int, 8>{});
    case 16:
        return f(std::integral_constant<int, 16>{});
    default:
        return f(std::integral_constant<int, 32>{});
    }
}

int64_t column_slices(int64_t D)
{
    const int64_t cols = lane_group(D) * kLaneCols;
    return (D + cols - 1) / cols;
}

// Sorted places per chunk: enough (chunk, slice) units for the 24 warps that an
// SM holds, in steps of 8 places, at most 512.
int64_t chunk_places(int64_t M, int64_t D, int sms)
{
    if (M <= 32)
        return 32;   // one chunk: no row spans two, and no second launch
    const int64_t groups = int64_t(sms) * 24 * (32 / lane_group(D));
    const int64_t want = (M * column_slices(D) + groups - 1) / groups;
    return std::min<int64_t>(512, std::max<int64_t>(16, (want + 7) / 8 * 8));
}

template <typename T, typename G, int VE, bool DW = false>
cudaError_t segments_launch(const GradArgs &a, cudaStream_t stream)
{
    return by_group(a.D, [&](auto LG) {
        constexpr int kGroup = decltype(LG)::value, kUnits = kThreads / kGroup;
        const int64_t want = (a.chunks * a.slices + kUnits - 1) / kUnits;
        if (want > 0x7fffffff)
            return cudaErrorInvalidValue;
        const unsigned blocks = static_cast<unsigned>(want);
        cudaError_t e =
            launch_after(segment_kernel<T, G, VE, kGroup, DW>, blocks, kThreads, 0, stream, a);
        if (e == cudaSuccess && a.chunks > 1)
            e = launch_after(join_kernel<G, VE, kGroup>, blocks, kThreads, 0, stream, a);
        return e;
    });
}

template <typename T, typename G>
cudaError_t grad_launch(const GradArgs &a, int ve, cudaStream_t stream)
{
    return by_elems<T>(ve, [&](auto VE) {
        constexpr int kElems = decltype(VE)::value;
        return a.dweights != nullptr ? segments_launch<T, G, kElems, true>(a, stream)
                                     : segments_launch<T, G, kElems>(a, stream);
    });
}

// What does not depend on the entry point: rows of D elements, as far apart.
GradArgs grad_args(const void *dout, int64_t M, int64_t D, const int32_t *order,
                   const int32_t *rows, const int32_t *total, float *parts, void *dtable, int sms)
{
    GradArgs a{};
    a.dout = dout;
    a.order = order;
    a.rows = rows;
    a.total = total;
    a.dtable = dtable;
    a.parts = parts;
    a.M = M;
    a.slices = static_cast<int32_t>(column_slices(D));
    a.chunk = static_cast<int32_t>(chunk_places(M, D, sms));
    a.chunks = (M + a.chunk - 1) / a.chunk;
    a.D = a.pitch = static_cast<int32_t>(D);
    return a;
}

}  // namespace

cudaError_t launch_lookup(const void *table, int dtype, int64_t K, int64_t D, const int32_t *idx,
                          const float *weights, int64_t N, int32_t k, float scale, void *out,
                          int sms, cudaStream_t stream)
{
    const int es = dtype_bytes(dtype);
    const int ve = vector_elems(D, most_elems(dtype), {{table, es}, {out, es}});
    if (k > 1) {
        GatherArgs a{};
        a.table = table;
        a.idx = idx;
        a.weights = weights;
        a.out = out;
        a.N = N;
        a.k = k;
        a.K = static_cast<int32_t>(K);
        a.D = static_cast<int32_t>(D);
        a.slices = static_cast<int32_t>(column_slices(D));
        a.scale = scale;
        return by_type(dtype, [&](auto t) {
            using T = decltype(t);
            return by_elems<T>(ve, [&](auto VE) {
                return by_group(D, [&](auto LG) {
                    constexpr int kUnits = kThreads / decltype(LG)::value;
                    const int64_t blocks = (N * a.slices + kUnits - 1) / kUnits;
                    if (blocks > 0x7fffffff)
                        return cudaErrorInvalidValue;
                    // rows in flight: as many as ids, within the registers
                    constexpr int kMost = decltype(VE)::value * sizeof(T) >= 8 ? 8 : 4;
                    const unsigned grid = static_cast<unsigned>(blocks);
                    if (k <= 2)
                        lookup_many_kernel<T, decltype(VE)::value, decltype(LG)::value, 2>
                            <<<grid, kThreads, 0, stream>>>(a);
                    else if (k <= 4)
                        lookup_many_kernel<T, decltype(VE)::value, decltype(LG)::value, 4>
                            <<<grid, kThreads, 0, stream>>>(a);
                    else
                        lookup_many_kernel<T, decltype(VE)::value, decltype(LG)::value, kMost>
                            <<<grid, kThreads, 0, stream>>>(a);
                    return cudaGetLastError();
                });
            });
        });
    }
    LookupArgs a{};
    a.table = table;
    a.idx = idx;
    a.weights = weights;
    a.out = out;
    a.N = N;
    a.K = static_cast<int32_t>(K);
    a.D = static_cast<int32_t>(D);
    const bool odd = ve * es == 2 && D >= 32;   // shorter rows: an element a thread
    a.vecs = static_cast<int32_t>(odd ? (D + 7) / 8 + 1 : D / ve);
    a.rows = a.vecs <= kThreads ? kThreads / a.vecs : 1;
    a.magic = (65536u + a.vecs - 1) / static_cast<uint32_t>(a.vecs);
    a.scale = scale;
    const unsigned pieces = static_cast<unsigned>((a.vecs + kThreads - 1) / kThreads);
    const int64_t blocks = (N + a.rows - 1) / a.rows;
    // four points a thread once that still gives every SM eight blocks
    const bool four = blocks * pieces >= int64_t(sms) * 32;
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        const dim3 fours(static_cast<unsigned>((blocks + 3) / 4), pieces);
        const dim3 ones(static_cast<unsigned>(blocks), pieces);
        if constexpr (sizeof(T) == 2)
            if (odd) {
                lookup_odd_kernel<T><<<ones, kThreads, 0, stream>>>(a);
                return cudaGetLastError();
            }
        return by_elems<T>(ve, [&](auto VE) {
            if (four)
                lookup_one_kernel<T, decltype(VE)::value, 4><<<fours, kThreads, 0, stream>>>(a);
            else
                lookup_one_kernel<T, decltype(VE)::value, 1><<<ones, kThreads, 0, stream>>>(a);
            return cudaGetLastError();
        });
    });
}

cudaError_t launch_dweights(const void *dout, const void *table, int dtype, const int32_t *idx,
                            int64_t N, int32_t k, int64_t K, int64_t D, float scale,
                            float *dweights, int sms, cudaStream_t stream)
{
    const int es = dtype_bytes(dtype);
    const int ve = vector_elems(D, most_elems(dtype), {{table, es}, {dout, es}});
    DweightsArgs a{dout, table, idx, dweights, N, k, static_cast<int32_t>(K),
                   static_cast<int32_t>(D), scale};
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        return by_elems<T>(ve, [&](auto VE) {
            return by_group(D, [&](auto LG) {
                constexpr int kUnits = kThreads / decltype(LG)::value;
                // the blocks that fit the SMs at once go through the points
                const int64_t blocks = std::min<int64_t>((N + kUnits - 1) / kUnits, sms * 2);
                dweights_kernel<T, decltype(VE)::value, decltype(LG)::value>
                    <<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a);
                return cudaGetLastError();
            });
        });
    });
}

size_t lookup_grad_parts_bytes(int64_t M, int64_t D, int sms)
{
    const int64_t places = chunk_places(M, D, sms);
    const int64_t chunks = (M + places - 1) / places;
    return static_cast<size_t>(2 * chunks) * D * 4;
}

bool dweights_with_dtable(int64_t D) { return column_slices(D) == 1; }

cudaError_t launch_lookup_grad(const void *dout, int dtype, const int32_t *idx,
                               const float *weights, const void *table, int64_t M, int32_t k,
                               int64_t K, int64_t D, float scale, int32_t skip, bool accumulate,
                               const int32_t *order, const int32_t *rows, const int32_t *total,
                               float *parts, void *dtable, int grad_dtype, float *dweights,
                               int sms, cudaStream_t stream)
{
    const int ve = vector_elems(
        D, most_elems(dtype),
        {{dout, dtype_bytes(dtype)},
         {dweights != nullptr ? table : nullptr, dtype_bytes(dtype)},
         {dtable, dtype_bytes(grad_dtype)}});
    GradArgs a = grad_args(dout, M, D, order, rows, total, parts, dtable, sms);
    a.weights = weights;
    a.idx = idx;
    a.table = table;
    a.dweights = dweights;
    a.k = k;
    a.K = static_cast<int32_t>(K);
    a.skip = skip;
    a.scale = scale;
    a.accumulate = accumulate;
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        if (grad_dtype == kFp32)
            return grad_launch<T, float>(a, ve, stream);
        return grad_launch<T, T>(a, ve, stream);
    });
}

cudaError_t launch_sum_rows(const float *from, int64_t M, int64_t D, const int32_t *order,
                            const int32_t *rows, const int32_t *total, float *parts, void *out,
                            int dtype, int64_t pitch, int sms, cudaStream_t stream)
{
    GradArgs a = grad_args(from, M, D, order, rows, total, parts, out, sms);
    a.k = 1;
    a.pitch = static_cast<int32_t>(pitch);
    a.skip = -1;
    a.scale = 1.0f;
    return dtype == kBf16 ? segments_launch<float, __nv_bfloat16, 4>(a, stream)
                          : segments_launch<float, __half, 4>(a, stream);
}

}  // namespace kma
