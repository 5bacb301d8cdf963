// learn_api.cu -- the C ABI of routing, row lookup, inverted lists and gradient
// clipping: argument checks, temporaries and launches.  No arithmetic of the
// operators lives here.
#include "kmassign.h"
#include "learn.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>
#include <new>
#include <vector>

namespace {

using kma::check_device_ptrs;
using kma::DeviceRestore;

constexpr int64_t kLimit = int64_t(1) << 31;
constexpr int64_t kMaxDim = 65536;        // D of a table
constexpr int32_t kMaxTensors = 1 << 20;  // of one clipping call

bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

bool known_type(int dtype) { return dtype >= KMASSIGN_FP32 && dtype <= KMASSIGN_FP16; }

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

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

int done(cudaError_t e) { return e == cudaSuccess ? KMASSIGN_OK : KMASSIGN_ERR_CUDA; }

int check_route(int dtype, int64_t N, int64_t E, int32_t k, int32_t score, float scale)
{
    if (N < 0 || N >= kLimit || E < 1 || E > KMASSIGN_ROUTE_MAX)
        return KMASSIGN_ERR_SHAPE;
    if (!known_type(dtype) || k < 1 || k > std::min<int64_t>(E, KMASSIGN_TOPK_MAX) ||
        (score != KMASSIGN_SOFTMAX && score != KMASSIGN_SIGMOID) || !std::isfinite(scale))
        return KMASSIGN_ERR_ARG;
    return N * k >= kLimit ? KMASSIGN_ERR_SHAPE : KMASSIGN_OK;
}

int check_table(int dtype, int64_t N, int64_t k, int64_t K, int64_t D, float scale)
{
    if (N < 0 || N >= kLimit || K < 1 || K >= kLimit || k < 1 || k >= kLimit || N * k >= kLimit)
        return KMASSIGN_ERR_SHAPE;
    if (D < 1 || D > kMaxDim)
        return KMASSIGN_ERR_UNSUPPORTED_D;
    if (!known_type(dtype) || !std::isfinite(scale))
        return KMASSIGN_ERR_ARG;
    return KMASSIGN_OK;
}

int run_clip(const void *const *grads, void *const *out, const int64_t *sizes,
             const int32_t *dtypes, int32_t n, bool scale, float max_norm, float *norm,
             cudaStream_t stream)
{
    if (n < 0 || n > kMaxTensors)
        return KMASSIGN_ERR_SHAPE;
    if (scale && !(max_norm >= 0.0f))
        return KMASSIGN_ERR_ARG;
    if (norm == nullptr || (n > 0 && (grads == nullptr || sizes == nullptr || dtypes == nullptr)))
        return KMASSIGN_ERR_NULL;
    if (!aligned(norm, 4))
        return KMASSIGN_ERR_ALIGN;
    for (int32_t i = 0; i < n; ++i) {
        if (!known_type(dtypes[i]))
            return KMASSIGN_ERR_ARG;
        if (sizes[i] < 0 || sizes[i] > (int64_t(1) << 48))
            return KMASSIGN_ERR_SHAPE;
        if (sizes[i] == 0)
            continue;
        const uintptr_t es = static_cast<uintptr_t>(kma::dtype_bytes(dtypes[i]));
        if (grads[i] == nullptr || (out != nullptr && out[i] == nullptr))
            return KMASSIGN_ERR_NULL;
        if (!aligned(grads[i], es) || (out != nullptr && !aligned(out[i], es)))
            return KMASSIGN_ERR_ALIGN;
    }
    // every pointer of a tensor with elements, and norm, on one device
    std::vector<const void *> ptrs;
    try {
        ptrs.reserve(2 * static_cast<size_t>(n) + 1);
    } catch (const std::bad_alloc &) {
        return KMASSIGN_ERR_CUDA;
    }
    ptrs.push_back(norm);
    for (int32_t i = 0; i < n; ++i)
        if (sizes[i] > 0) {
            ptrs.push_back(grads[i]);
            if (out != nullptr)
                ptrs.push_back(out[i]);
        }
    int rc = check_device_ptrs(ptrs.data(), static_cast<int>(ptrs.size()));
    if (rc != KMASSIGN_OK)
        return rc;
    cudaMemPool_t pool;
    int sms;
    if ((rc = kma::library_device(&pool, &sms)) != KMASSIGN_OK)
        return rc;
    Scratch scratch(kma::clip_scratch_bytes(n, sms), pool, stream);
    if (!scratch.ok())
        return KMASSIGN_ERR_CUDA;
    rc = done(kma::launch_clip(grads, out, sizes, dtypes, n, scale, max_norm, norm,
                               reinterpret_cast<double *>(scratch.get()), sms, stream));
    return scratch.release() ? rc : KMASSIGN_ERR_CUDA;
}

}  // namespace

extern "C" {

int kmassign_route(const void *logits, int32_t dtype, int64_t N, int64_t E, int32_t k,
                   int32_t score, const float *bias, int32_t groups, int32_t topk_groups,
                   int32_t group_top, int32_t renorm, float scale, int32_t *idx, float *weights,
                   void *stream)
{
    DeviceRestore restore;
    int rc = check_route(dtype, N, E, k, score, scale);
    if (rc != KMASSIGN_OK)
        return rc;
    if (groups < 1 || groups > 32 || E % groups != 0 || topk_groups < 1 || topk_groups > groups ||
        (group_top != 1 && group_top != 2) || k > topk_groups * (E / groups) ||
        (renorm != 0 && renorm != 1))
        return KMASSIGN_ERR_ARG;
    if (N == 0)
        return KMASSIGN_OK;
    if (logits == nullptr || idx == nullptr || weights == nullptr)
        return KMASSIGN_ERR_NULL;
    if (!aligned(logits, kma::dtype_bytes(dtype)) || !aligned(bias, 4) || !aligned(idx, 4) ||
        !aligned(weights, 4))
        return KMASSIGN_ERR_ALIGN;
    const void *ptrs[4] = {logits, bias, idx, weights};
    if ((rc = check_device_ptrs(ptrs, 4)) != KMASSIGN_OK)
        return rc;
    return done(kma::launch_route(logits, dtype, N, E, k, score == KMASSIGN_SIGMOID, bias, groups,
                                  topk_groups, group_top, renorm != 0, scale, idx, weights,
                                  static_cast<cudaStream_t>(stream)));
}

int kmassign_route_grad(const void *logits, int32_t dtype, int64_t N, int64_t E, int32_t k,
                        int32_t score, int32_t renorm, float scale, const int32_t *idx,
                        const float *dweights, void *dlogits, void *stream)
{
    DeviceRestore restore;
    int rc = check_route(dtype, N, E, k, score, scale);
    if (rc != KMASSIGN_OK)
        return rc;
    if (renorm != 0 && renorm != 1)
        return KMASSIGN_ERR_ARG;
    if (N == 0)
        return KMASSIGN_OK;
    if (logits == nullptr || idx == nullptr || dweights == nullptr || dlogits == nullptr)
        return KMASSIGN_ERR_NULL;
    const uintptr_t es = static_cast<uintptr_t>(kma::dtype_bytes(dtype));
    if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(idx, 4) || !aligned(dweights, 4))
        return KMASSIGN_ERR_ALIGN;
    const void *ptrs[4] = {logits, idx, dweights, dlogits};
    if ((rc = check_device_ptrs(ptrs, 4)) != KMASSIGN_OK)
        return rc;
    return done(kma::launch_route_grad(logits, dtype, N, E, k, score == KMASSIGN_SIGMOID,
                                       renorm != 0, scale, idx, dweights, dlogits,
                                       static_cast<cudaStream_t>(stream)));
}

int kmassign_lists(const int32_t *idx, int64_t M, int64_t K, int32_t *order, int32_t *offsets,
                   void *stream)
{
    DeviceRestore restore;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M < 0 || M >= kLimit || K < 1 || K >= kLimit)
        return KMASSIGN_ERR_SHAPE;
    if ((M > 0 && (idx == nullptr || order == nullptr)) || offsets == nullptr)
        return KMASSIGN_ERR_NULL;
    if (!aligned(idx, 4) || !aligned(order, 4) || !aligned(offsets, 4))
        return KMASSIGN_ERR_ALIGN;
    const void *ptrs[3] = {idx, order, offsets};
    int rc = check_device_ptrs(ptrs, 3);
    if (rc != KMASSIGN_OK)
        return rc;
    cudaMemPool_t pool;
    int sms;
    if ((rc = kma::library_device(&pool, &sms)) != KMASSIGN_OK)
        return rc;
    Scratch scratch(kma::lists_scratch_bytes(M, K, sms), pool, s);
    if (!scratch.ok())
        return KMASSIGN_ERR_CUDA;
    rc = done(kma::launch_lists(idx, M, K, order, nullptr, offsets, nullptr, scratch.get(), nullptr,
                                0, sms, s));
    return scratch.release() ? rc : KMASSIGN_ERR_CUDA;
}

int kmassign_lookup(const void *table, int32_t dtype, int64_t K, int64_t D, const int32_t *idx,
                    const float *weights, int64_t N, int32_t k, float scale, void *out,
                    void *stream)
{
    DeviceRestore restore;
    int rc = check_table(dtype, N, k, K, D, scale);
    if (rc != KMASSIGN_OK)
        return rc;
    if (N == 0)
        return KMASSIGN_OK;
    if (table == nullptr || idx == nullptr || out == nullptr)
        return KMASSIGN_ERR_NULL;
    const uintptr_t es = static_cast<uintptr_t>(kma::dtype_bytes(dtype));
    if (!aligned(table, es) || !aligned(out, es) || !aligned(idx, 4) || !aligned(weights, 4))
        return KMASSIGN_ERR_ALIGN;
    const void *ptrs[4] = {table, idx, weights, out};
    if ((rc = check_device_ptrs(ptrs, 4)) != KMASSIGN_OK)
        return rc;
    cudaMemPool_t pool;
    int sms;
    if ((rc = kma::library_device(&pool, &sms)) != KMASSIGN_OK)
        return rc;
    return done(kma::launch_lookup(table, dtype, K, D, idx, weights, N, k, scale, out, sms,
                                   static_cast<cudaStream_t>(stream)));
}

int kmassign_lookup_grad(const void *dout, int32_t dtype, const int32_t *idx, const float *weights,
                         const void *table, int64_t N, int32_t k, int64_t K, int64_t D,
                         float scale, int32_t padding, int32_t accumulate, void *dtable,
                         int32_t grad_dtype, float *dweights, void *stream)
{
    DeviceRestore restore;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int rc = check_table(dtype, N, k, K, D, scale);
    if (rc != KMASSIGN_OK)
        return rc;
    if ((accumulate != 0 && accumulate != 1) ||
        (grad_dtype != KMASSIGN_FP32 && grad_dtype != dtype))
        return KMASSIGN_ERR_ARG;
    if ((N > 0 && (dout == nullptr || idx == nullptr)) || (dtable == nullptr && dweights == nullptr))
        return KMASSIGN_ERR_NULL;
    if (N > 0 && dweights != nullptr && table == nullptr)
        return KMASSIGN_ERR_NULL;
    const uintptr_t es = static_cast<uintptr_t>(kma::dtype_bytes(dtype));
    if (!aligned(dout, es) || !aligned(table, es) || !aligned(idx, 4) || !aligned(weights, 4) ||
        !aligned(dtable, kma::dtype_bytes(grad_dtype)) || !aligned(dweights, 4))
        return KMASSIGN_ERR_ALIGN;
    const void *ptrs[6] = {dout, idx, weights, table, dtable, dweights};
    if ((rc = check_device_ptrs(ptrs, 6)) != KMASSIGN_OK)
        return rc;
    const int64_t M = N * k;
    cudaMemPool_t pool;
    int sms;
    if ((rc = kma::library_device(&pool, &sms)) != KMASSIGN_OK)
        return rc;
    const bool both = dtable != nullptr && dweights != nullptr && kma::dweights_with_dtable(D);
    if (dweights != nullptr && N > 0 && !both &&
        kma::launch_dweights(dout, table, dtype, idx, N, k, K, D, scale, dweights, sms, s) !=
            cudaSuccess)
        return KMASSIGN_ERR_CUDA;
    if (dtable == nullptr || (N == 0 && accumulate))
        return KMASSIGN_OK;
    // one allocation: order, sorted rows, their number, the sort's scratch, row parts
    const size_t ids = up16(static_cast<size_t>(M) * 4);
    const size_t sort = up16(kma::lists_scratch_bytes(M, K, sms));
    Scratch scratch(2 * ids + 16 + sort + kma::lookup_grad_parts_bytes(M, D, sms), pool, s);
    if (!scratch.ok())
        return KMASSIGN_ERR_CUDA;
    uint8_t *p = scratch.get();
    int32_t *order = reinterpret_cast<int32_t *>(p);
    int32_t *rows = reinterpret_cast<int32_t *>(p + ids);
    int32_t *total = reinterpret_cast<int32_t *>(p + 2 * ids);
    p += 2 * ids + 16;
    cudaError_t e = kma::launch_lists(
        idx, M, K, order, rows, nullptr, total, p, accumulate ? nullptr : dtable,
        accumulate ? 0 : static_cast<size_t>(K) * D * kma::dtype_bytes(grad_dtype), sms, s);
    if (e == cudaSuccess && M > 0)
        e = kma::launch_lookup_grad(dout, dtype, idx, weights, table, M, k, K, D, scale, padding,
                                    accumulate != 0, order, rows, total,
                                    reinterpret_cast<float *>(p + sort), dtable, grad_dtype,
                                    both ? dweights : nullptr, sms, s);
    rc = done(e);
    return scratch.release() ? rc : KMASSIGN_ERR_CUDA;
}

int kmassign_grad_norm(const void *const *grads, const int64_t *sizes, const int32_t *dtypes,
                       int32_t n, float *norm, void *stream)
{
    DeviceRestore restore;
    return run_clip(grads, nullptr, sizes, dtypes, n, false, 0.0f, norm,
                    static_cast<cudaStream_t>(stream));
}

int kmassign_clip(const void *const *grads, void *const *out, const int64_t *sizes,
                  const int32_t *dtypes, int32_t n, float max_norm, float *norm, void *stream)
{
    DeviceRestore restore;
    return run_clip(grads, out, sizes, dtypes, n, true, max_norm, norm,
                    static_cast<cudaStream_t>(stream));
}

}  // extern "C"
