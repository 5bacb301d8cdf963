// learn.h -- declarations of the learned assignments' translation units, and of
// the host helpers that api.cu shares with learn_api.cu.  (internal.h is one of
// the assignment kernels' sources, to which none of this belongs.)
#pragma once

#include "internal.h"

namespace kma {

// ---- host helpers (api.cu) -------------------------------------------------

// The current device's stream-ordered pool and number of SMs; a kmassign status.
int library_device(cudaMemPool_t *pool, int *sms);

// Every non-NULL pointer must be device (or managed) memory of one device,
// which is made current; KMASSIGN_ERR_NOT_DEVICE otherwise.
int check_device_ptrs(const void *const *ptrs, int n);

// Largest dynamic shared memory of a block on the current device (library_device's), and the bound
// on every pipeline wait.
int library_smem(size_t *bytes);
uint64_t wait_timeout_ns();

// A tensor map of rank 2 or 3 (dims, innermost first; strides[i]: bytes from one index of dims[i + 1]
// to the next), 128-byte swizzle, zeros outside; false if the driver refuses it.
bool encode_tiled(CUtensorMap *map, CUtensorMapDataType type, const void *ptr, int rank,
                  const uint64_t *dims, const uint64_t *strides, const uint32_t *box);

// One stream-ordered allocation from the library's pool, released (in stream
// order) when it goes out of scope.
class Scratch {
public:
    Scratch(size_t bytes, cudaMemPool_t pool, cudaStream_t stream) : stream_(stream)
    {
        if (bytes > 0 && cudaMallocFromPoolAsync(&p_, bytes, pool, stream) != cudaSuccess) {
            cudaGetLastError();
            p_ = nullptr;
            ok_ = false;
        }
    }
    ~Scratch() { release(); }
    bool ok() const { return ok_; }
    uint8_t *get() const { return static_cast<uint8_t *>(p_); }
    bool release()
    {
        void *p = p_;
        p_ = nullptr;
        return p == nullptr || cudaFreeAsync(p, stream_) == cudaSuccess;
    }
    Scratch(const Scratch &) = delete;
    Scratch &operator=(const Scratch &) = delete;

private:
    cudaStream_t stream_;
    void *p_ = nullptr;
    bool ok_ = true;
};

// Puts back the calling thread's current device when an entry point returns
// (check_device_ptrs makes the pointers' device current for the launches;
// the caller's own notion of its current device must not change).
class DeviceRestore {
public:
    DeviceRestore()
    {
        if (cudaGetDevice(&dev_) != cudaSuccess) {
            cudaGetLastError();
            dev_ = -1;
        }
    }
    ~DeviceRestore()
    {
        int cur = -1;
        if (dev_ >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != dev_)
            cudaSetDevice(dev_);
    }
    DeviceRestore(const DeviceRestore &) = delete;
    DeviceRestore &operator=(const DeviceRestore &) = delete;

private:
    int dev_ = -1;
};

// ---- routing, row lookup, inverted lists, gradient clipping ----------------

// Element types (the KMASSIGN_FP32, _BF16, _FP16 of kmassign.h).
constexpr int kFp32 = 0, kBf16 = 1, kFp16 = 2;
constexpr int kE4m3 = 3;   // KMASSIGN_E4M3: the experts' products and the norm's output only
__host__ __device__ inline int dtype_bytes(int dtype) { return dtype == kFp32 ? 4 : 2; }

cudaError_t launch_route(const void *logits, int dtype, int64_t N, int64_t E, int32_t k,
                         bool sigmoid, const float *bias, int32_t groups, int32_t topk_groups,
                         int32_t group_top, bool renorm, float scale, int32_t *idx,
                         float *weights, cudaStream_t stream);
cudaError_t launch_route_grad(const void *logits, int dtype, int64_t N, int64_t E, int32_t k,
                              bool sigmoid, bool renorm, float scale, const int32_t *idx,
                              const float *dweights, void *dlogits, cudaStream_t stream);
// Shared-memory attributes of the sort's kernels, once per device.
cudaError_t lists_prepare();
// The stable sort of the positions [0, M) by row: order, the sorted rows (may
// be NULL), offsets[K + 1] and the number of valid ids, total (either may be
// NULL, not both); scratch (16-byte aligned) of lists_scratch_bytes.  Places
// past offsets[K] hold -1 in order and nothing in particular in rows.
// zero_bytes (even) at zero are zeroed besides.
size_t lists_scratch_bytes(int64_t M, int64_t K, int sms);
cudaError_t launch_lists(const int32_t *idx, int64_t M, int64_t K, int32_t *order, int32_t *rows,
                         int32_t *offsets, int32_t *total, void *scratch, void *zero,
                         size_t zero_bytes, int sms, cudaStream_t stream);
cudaError_t launch_lookup(const void *table, int dtype, int64_t K, int64_t D, const int32_t *idx,
                          const float *weights, int64_t N, int32_t k, float scale, void *out,
                          int sms, cudaStream_t stream);
cudaError_t launch_dweights(const void *dout, const void *table, int dtype, const int32_t *idx,
                            int64_t N, int32_t k, int64_t K, int64_t D, float scale,
                            float *dweights, int sms, cudaStream_t stream);
// The gradient of the table from the sorted ids (launch_lists with rows);
// parts: 16-byte aligned workspace of lookup_grad_parts_bytes.
size_t lookup_grad_parts_bytes(int64_t M, int64_t D, int sms);
cudaError_t launch_lookup_grad(const void *dout, int dtype, const int32_t *idx,
                               const float *weights, const void *table, int64_t M, int32_t k,
                               int64_t K, int64_t D, float scale, int32_t skip, bool accumulate,
                               const int32_t *order, const int32_t *rows, const int32_t *total,
                               float *parts, void *dtable, int grad_dtype, float *dweights,
                               int sms, cudaStream_t stream);
// out[r] = the sum of from's rows (fp32 [M, D]) that are sorted to r, rounded once
// to dtype (16 bits); out's rows are pitch elements apart.  D and pitch are multiples
// of 4, from and out 16-byte aligned; order, rows, total, parts as above.
cudaError_t launch_sum_rows(const float *from, int64_t M, int64_t D, const int32_t *order,
                            const int32_t *rows, const int32_t *total, float *parts, void *out,
                            int dtype, int64_t pitch, int sms, cudaStream_t stream);
// Whether launch_lookup_grad can form dweights (else NULL there, and
// launch_dweights).
bool dweights_with_dtable(int64_t D);
// The norm over n tensors, and with `scale` their scaling into out (NULL: in
// place); partial: workspace of clip_scratch_bytes.
size_t clip_scratch_bytes(int32_t n, int sms);
cudaError_t launch_clip(const void *const *grads, void *const *out, const int64_t *sizes,
                        const int32_t *dtypes, int32_t n, bool scale, float max_norm, float *norm,
                        double *partial, int sms, cudaStream_t stream);

// ---- products grouped by expert, root-mean-square norm ----------------------

// The row that a list position stands for: ids[p] / slots, or p where ids is
// NULL; none where that is outside [0, rows).
struct RowMap {
    const int32_t *ids;
    int32_t slots, rows;
};

enum ExpertsKind { kForward, kRowsGrad, kWeightsGrad };

struct ExpertsParams {
    const int32_t *offsets;   // [E + 1]; NULL: one list of all M positions
    int32_t E, M;
    int32_t mdim;             // the outputs' contiguous extent (F; gradients: D)
    int32_t ndim;             // weights' gradient: F
    int32_t kblocks;          // 128-byte blocks of the contraction (not the weights' gradient)
    RowMap b_rows;            // rows of X, where the product gathers them itself (few positions)
    RowMap from;              // rows of X (and of xscale), of dY for the rows' gradient: a
                              // position without one has a product of zeros
    RowMap placed;            // weights' gradient: rows of dY; a position that lacks either row
    const int32_t *holes;     // adds nothing.  Whether there is one (NULL: none)
    RowMap places;            // rows of the output (forward, rows' gradient)
    bool zero_rest;           // rows of no list are written 0
    void *out;
    int32_t out_type;
    const float *xscale, *wscale;   // 8 bits: [rows, kblocks], [E, fblocks, kblocks]
    int32_t fblocks;
    // set by launch_experts: depth of the ring, k-blocks between additions to registers, MMA shape
    int32_t stages, segment;
    uint32_t idesc;
    uint64_t timeout_ns;
};

// Shared-memory attributes, once per device.
cudaError_t experts_prepare(size_t smem_optin);
// Boxes of the operands' tensor maps (rows of 128 bytes): A as [E][F][D], 128
// rows K-major (forward) or 64 MN-major, X 64 rows; B 32 rows (the weights'
// gradient 64), or one where b_rows has ids.
constexpr uint32_t kExpertsBoxA = 128, kExpertsBoxMn = 64, kExpertsBoxB = 32;
// Whether lists of M positions are short on average: the product then has
// tiles for few columns, and gathers rows itself.
bool experts_few(int64_t M, int64_t E, bool e8);
cudaError_t launch_experts(ExpertsKind kind, bool e8, int type, const CUtensorMap &a,
                           const CUtensorMap &b, ExpertsParams p, int sms, size_t smem_optin,
                           cudaStream_t stream);
cudaError_t experts_status_read_and_clear(int *code);
// row[p] = the row that map names for positions of a list, -1 for the others;
// *zero = 0 (may be NULL).
cudaError_t launch_listed_rows(const int32_t *offsets, int32_t E, int32_t M, RowMap map,
                               int32_t *row, int32_t *zero, cudaStream_t stream);
// to[p] = the row (pitch bytes, a multiple of 16) that map names for positions
// of a list, zeros for the others and where also names none; *holes (may be
// NULL) is set to 1 if a position of a list gets zeros.
cudaError_t launch_gather_rows(const int32_t *offsets, int32_t E, int32_t M, RowMap map,
                               RowMap also, const void *from, int64_t pitch, void *to,
                               int32_t *holes, cudaStream_t stream);

cudaError_t launch_rmsnorm(const void *X, int dtype, int64_t N, int64_t D, const void *residual,
                           const void *weight, int weight_dtype, float eps, void *total, void *out,
                           int out_dtype, float *scales, float *rstd, int sms,
                           cudaStream_t stream);
// The weight's partial sums are an allocation of its own from the pool, if dweight is given.
cudaError_t launch_rmsnorm_grad(const void *dout, int dtype, int64_t N, int64_t D,
                                const void *total, const void *weight, int weight_dtype,
                                const float *rstd, const void *dtotal, void *dX, float *dweight,
                                cudaMemPool_t pool, int sms, cudaStream_t stream);

}  // namespace kma
