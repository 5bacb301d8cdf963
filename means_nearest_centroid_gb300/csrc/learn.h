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
inline int dtype_bytes(int dtype) { return dtype == kFp32 ? 4 : 2; }

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
// Whether launch_lookup_grad can form dweights (else NULL there, and
// launch_dweights).
bool dweights_with_dtable(int64_t D);
// The norm over n tensors, and with `scale` their scaling into out (NULL: in
// place); partial: workspace of clip_scratch_bytes.
size_t clip_scratch_bytes(int32_t n, int sms);
cudaError_t launch_clip(const void *const *grads, void *const *out, const int64_t *sizes,
                        const int32_t *dtypes, int32_t n, bool scale, float max_norm, float *norm,
                        double *partial, int sms, cudaStream_t stream);

}  // namespace kma
