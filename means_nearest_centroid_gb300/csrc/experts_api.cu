// experts_api.cu -- the C ABI of the experts' products and of the
// root-mean-square norm: argument checks, tensor maps, temporaries and
// launches.  No arithmetic of the operators lives here.
#include "kmassign.h"
#include "learn.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

namespace {

using kma::check_device_ptrs;
using kma::DeviceRestore;
using kma::ExpertsParams;
using kma::RowMap;
using kma::Scratch;

constexpr int64_t kLimit = int64_t(1) << 31;
constexpr int64_t kMaxDim = 65536;
constexpr int64_t kMaxNormDim = 32768;

bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

int done(cudaError_t e) { return e == cudaSuccess ? KMASSIGN_OK : KMASSIGN_ERR_CUDA; }

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

bool half_type(int32_t t) { return t == KMASSIGN_BF16 || t == KMASSIGN_FP16; }
bool known_type(int32_t t) { return t >= KMASSIGN_FP32 && t <= KMASSIGN_FP16; }

CUtensorMapDataType map_type(int32_t t)
{
    return t == KMASSIGN_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
           : t == KMASSIGN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// Rows of `cols` elements, in boxes of 128 bytes by `box` rows.
bool rows_map(CUtensorMap *m, int32_t type, const void *p, int64_t rows, int64_t cols, uint32_t box)
{
    const uint64_t es = type == KMASSIGN_E4M3 ? 1 : 2;
    const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
    const uint64_t strides[1] = {dims[0] * es};
    const uint32_t boxes[2] = {static_cast<uint32_t>(128 / es), box};
    return kma::encode_tiled(m, map_type(type), p, 2, dims, strides, boxes);
}

// W as [E][F][D], or the first `cols` of its rows' D elements.
bool weights_map(CUtensorMap *m, int32_t type, const void *p, int64_t E, int64_t F, int64_t D,
                 int64_t cols, uint32_t box)
{
    const uint64_t es = type == KMASSIGN_E4M3 ? 1 : 2;
    const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(F),
                              static_cast<uint64_t>(E)};
    const uint64_t strides[2] = {static_cast<uint64_t>(D) * es,
                                 static_cast<uint64_t>(D) * dims[1] * es};
    const uint32_t boxes[3] = {static_cast<uint32_t>(128 / es), box, 1};
    return kma::encode_tiled(m, map_type(type), p, 3, dims, strides, boxes);
}

struct Shape {
    int64_t R, D, E, F, M, out_rows;
    int32_t slots;
};

int check_shape(const Shape &s, int32_t type, const int32_t *offsets, const int32_t *rows,
                const int32_t *places)
{
    if (s.R < 0 || s.R >= kLimit || s.M < 0 || s.M >= kLimit / 2 || s.out_rows < 0 ||
        s.out_rows >= kLimit || s.E < 1 || s.E > KMASSIGN_EXPERTS_MAX || s.slots < 1 ||
        (rows == nullptr && (s.M > s.R || (s.M > 0 && s.slots != 1))) ||
        (places == nullptr && s.M > s.out_rows) || (offsets == nullptr && s.E != 1))
        return KMASSIGN_ERR_SHAPE;
    const int64_t step = type == KMASSIGN_E4M3 ? 16 : 8;
    if (s.D < step || s.D > kMaxDim || s.D % step != 0 || s.F < 8 || s.F > kMaxDim || s.F % 8 != 0)
        return KMASSIGN_ERR_UNSUPPORTED_D;
    return KMASSIGN_OK;
}

bool ids_aligned(const int32_t *offsets, const int32_t *rows, const int32_t *places)
{
    return aligned(offsets, 4) && aligned(rows, 4) && aligned(places, 4);
}

struct Device {
    cudaMemPool_t pool;
    int sms;
    size_t smem;
    int get()
    {
        const int rc = kma::library_device(&pool, &sms);
        return rc != KMASSIGN_OK ? rc : kma::library_smem(&smem);
    }
};

ExpertsParams params_of(const Shape &s, const int32_t *offsets)
{
    ExpertsParams p = {};
    p.offsets = offsets;
    p.E = static_cast<int32_t>(s.E);
    p.M = static_cast<int32_t>(s.M);
    p.timeout_ns = kma::wait_timeout_ns();
    return p;
}

// How many columns of the rows' gradients are formed in fp32 at a time where they are
// summed by row: all where they take half of the GiB that the pool keeps, else half, which
// take the room of X's 16-bit rows.  (15,009 positions of 1,000: both gradients 133 us, in
// halves 154; 131,072 of 2,048, 1 GiB: 1,137 back to back but 1,286 alone, for the pool
// then maps memory in every call, in halves 1,164 and 1,210; of 7,168: 3,200 and 5,100,
// 3,070 and 3,745.)
int64_t sum_columns(int64_t M, int64_t D)
{
    constexpr int64_t kRoom = int64_t(1) << 29;
    return M * D * 4 <= kRoom ? D : std::min(D, (D + 511) / 512 * 256);
}

RowMap map_of(const int32_t *ids, int32_t slots, int64_t rows)
{
    return RowMap{ids, slots, static_cast<int32_t>(rows)};
}

}  // namespace

extern "C" {

int kmassign_experts(const void *X, int32_t dtype, int64_t R, int64_t D, const void *W, int64_t E,
                     int64_t F, const float *xscale, const float *wscale, const int32_t *offsets,
                     int64_t M, const int32_t *rows, int32_t slots, const int32_t *places,
                     void *out, int32_t out_dtype, int64_t out_rows, void *stream)
{
    DeviceRestore restore;
    const bool e8 = dtype == KMASSIGN_E4M3;
    if ((!e8 && !half_type(dtype)) || !known_type(out_dtype) ||
        (!e8 && out_dtype != KMASSIGN_FP32 && out_dtype != dtype) ||
        (!e8 && (xscale != nullptr || wscale != nullptr)))
        return KMASSIGN_ERR_ARG;
    const Shape s{R, D, E, F, M, out_rows, slots};
    int rc = check_shape(s, dtype, offsets, rows, places);
    if (rc != KMASSIGN_OK)
        return rc;
    if (M == 0 || out_rows == 0)
        return KMASSIGN_OK;
    if (R == 0 && places != nullptr)
        return KMASSIGN_ERR_SHAPE;
    if ((R > 0 && X == nullptr) || W == nullptr || out == nullptr ||
        (e8 && ((R > 0 && xscale == nullptr) || wscale == nullptr)))
        return KMASSIGN_ERR_NULL;
    if (!aligned(X, 16) || !aligned(W, 16) || !aligned(out, 16) || !aligned(xscale, 4) ||
        !aligned(wscale, 4) || !ids_aligned(offsets, rows, places))
        return KMASSIGN_ERR_ALIGN;
    const void *ptrs[8] = {X, W, out, xscale, wscale, offsets, rows, places};
    if ((rc = check_device_ptrs(ptrs, 8)) != KMASSIGN_OK)
        return rc;
    Device dev;
    if ((rc = dev.get()) != KMASSIGN_OK)
        return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (R == 0) {
        // every position names a row that is not there: zeros
        return done(cudaMemsetAsync(out, 0, static_cast<size_t>(M) * F * kma::dtype_bytes(out_dtype),
                                    st));
    }
    // Many positions: their rows first come into the lists' order, by a pass of
    // its own, and are then loaded in whole boxes.
    const int64_t pitch = D * (e8 ? 1 : 2);
    const bool few = kma::experts_few(M, E, e8);
    // 8 bits and many: positions are the tile's rows
    const uint32_t box = e8 && !few ? kma::kExpertsBoxA : kma::kExpertsBoxB;
    const int32_t kblocks = static_cast<int32_t>((pitch + 127) / 128);
    Scratch sorted(rows != nullptr && !few ? static_cast<size_t>(M * pitch) : 0, dev.pool, st);
    if (!sorted.ok())
        return KMASSIGN_ERR_CUDA;
    const RowMap from = map_of(rows, slots, R);
    const bool gathers = rows != nullptr && few;
    CUtensorMap a, b;
    if (!weights_map(&a, dtype, W, E, F, D, D, kma::kExpertsBoxA) ||
        (sorted.get() != nullptr ? !rows_map(&b, dtype, sorted.get(), M, D, box)
                                 : !rows_map(&b, dtype, X, R, D, gathers ? 1 : box)))
        return KMASSIGN_ERR_CUDA;
    ExpertsParams p = params_of(s, offsets);
    p.mdim = static_cast<int32_t>(F);
    p.kblocks = kblocks;
    p.fblocks = static_cast<int32_t>((F + 127) / 128);
    p.b_rows = gathers ? from : map_of(nullptr, 1, M);
    p.from = from;
    p.places = map_of(places, 1, out_rows);
    p.zero_rest = places == nullptr;
    p.out = out;
    p.out_type = out_dtype;
    p.xscale = xscale;
    p.wscale = wscale;
    cudaError_t e = cudaSuccess;
    if (sorted.get() != nullptr)
        e = kma::launch_gather_rows(offsets, p.E, p.M, from, map_of(nullptr, 1, M), X, pitch,
                                    sorted.get(), nullptr, st);
    if (e == cudaSuccess)
        e = kma::launch_experts(kma::kForward, e8, dtype, a, b, p, dev.sms, dev.smem, st);
    rc = done(e);
    return sorted.release() ? rc : KMASSIGN_ERR_CUDA;
}

int kmassign_experts_grad(const void *dout, int32_t dtype, int64_t out_rows, int64_t F,
                          const void *X, int64_t R, int64_t D, const void *W, int64_t E,
                          const int32_t *offsets, int64_t M, const int32_t *rows, int32_t slots,
                          const int32_t *places, void *dX, void *dW, int32_t dw_dtype, void *stream)
{
    DeviceRestore restore;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!half_type(dtype) || (dw_dtype != KMASSIGN_FP32 && dw_dtype != dtype))
        return KMASSIGN_ERR_ARG;
    const Shape s{R, D, E, F, M, out_rows, slots};
    int rc = check_shape(s, dtype, offsets, rows, places);
    if (rc != KMASSIGN_OK)
        return rc;
    if (dX == nullptr && dW == nullptr)
        return KMASSIGN_ERR_NULL;
    const bool work = M > 0 && R > 0 && out_rows > 0;   // a position can have a row on either side
    if (work && (dout == nullptr || (dX != nullptr && W == nullptr) ||
                 (dW != nullptr && X == nullptr)))
        return KMASSIGN_ERR_NULL;
    if (!aligned(dout, 16) || !aligned(X, 16) || !aligned(W, 16) || !aligned(dX, 16) ||
        !aligned(dW, 16) || !ids_aligned(offsets, rows, places))
        return KMASSIGN_ERR_ALIGN;
    const void *ptrs[8] = {dout, X, W, dX, dW, offsets, rows, places};
    if ((rc = check_device_ptrs(ptrs, 8)) != KMASSIGN_OK)
        return rc;
    Device dev;
    if ((rc = dev.get()) != KMASSIGN_OK)
        return rc;
    const size_t dw_bytes = static_cast<size_t>(E) * F * D * kma::dtype_bytes(dw_dtype);
    if (!work) {
        if (dX != nullptr && R > 0 &&
            cudaMemsetAsync(dX, 0, static_cast<size_t>(R) * D * 2, st) != cudaSuccess)
            return KMASSIGN_ERR_CUDA;
        return dW == nullptr ? KMASSIGN_OK : done(cudaMemsetAsync(dW, 0, dw_bytes, st));
    }
    // Rows that ids name come into the lists' order first.  Without row ids
    // position p's gradient is row p's; with them the rows' gradients are formed
    // position by position, in fp32, and summed by row like those of a lookup
    // (sorted, no atomics), so many columns at a time.
    const RowMap from = map_of(rows, slots, R), placed = map_of(places, 1, out_rows);
    const bool sum = dX != nullptr && rows != nullptr;
    const int64_t cols = sum_columns(M, D), rest = D - (D - 1) / cols * cols;
    const size_t ids = sum ? up16(static_cast<size_t>(M) * 4) : 0;
    const size_t sort = sum ? up16(kma::lists_scratch_bytes(M, R, dev.sms)) : 0;
    const size_t parts = sum ? up16(std::max(kma::lookup_grad_parts_bytes(M, cols, dev.sms),
                                             kma::lookup_grad_parts_bytes(M, rest, dev.sms)))
                             : 0;
    // X's rows, and later the rows' gradients
    const size_t each = std::max(rows != nullptr && dW != nullptr ? static_cast<size_t>(M) * D * 2 : 0,
                                 sum ? static_cast<size_t>(M) * cols * 4 : 0);
    const size_t dys = places != nullptr ? static_cast<size_t>(M) * F * 2 : 0;
    const bool gathers = rows != nullptr || places != nullptr;
    Scratch scratch(each + dys + (gathers ? 16 : 0) + 3 * ids + (sum ? 16 : 0) + sort + parts,
                    dev.pool, st);
    if (!scratch.ok())
        return KMASSIGN_ERR_CUDA;
    uint8_t *q = scratch.get();
    uint8_t *const by_position = q, *const dy_sorted = q + each;
    q += each + dys;
    int32_t *holes = nullptr;
    const void *const dy = places != nullptr ? dy_sorted : dout;
    const int64_t dy_rows = places != nullptr ? M : out_rows;
    cudaError_t e = cudaSuccess;
    if (gathers) {
        holes = reinterpret_cast<int32_t *>(q);
        q += 16;
        // a position whose place is missing has a gradient of zeros: it may be summed
        if (sum)
            e = kma::launch_listed_rows(offsets, static_cast<int32_t>(E), static_cast<int32_t>(M),
                                        from, reinterpret_cast<int32_t *>(q), holes, st);
        else if (dW != nullptr)
            e = cudaMemsetAsync(holes, 0, 4, st);
    }
    if (e == cudaSuccess && places != nullptr)
        e = kma::launch_gather_rows(offsets, static_cast<int32_t>(E), static_cast<int32_t>(M),
                                    placed, from, dout, 2 * F, dy_sorted, holes, st);
    ExpertsParams p = params_of(s, offsets);
    p.mdim = static_cast<int32_t>(D);
    p.b_rows = p.places = map_of(nullptr, 1, M);
    p.from = from;
    p.placed = placed;
    CUtensorMap a, b;
    if (e == cudaSuccess && dW != nullptr) {
        if (e == cudaSuccess && rows != nullptr)
            e = kma::launch_gather_rows(offsets, p.E, p.M, from, placed, X, 2 * D, by_position,
                                        holes, st);
        if (!rows_map(&a, dtype, rows != nullptr ? by_position : X, rows != nullptr ? M : R, D,
                      kma::kExpertsBoxMn) ||
            !rows_map(&b, dtype, dy, dy_rows, F, kma::kExpertsBoxMn))
            return KMASSIGN_ERR_CUDA;
        p.holes = holes;
        p.ndim = static_cast<int32_t>(F);
        p.out = dW;
        p.out_type = dw_dtype;
        if (e == cudaSuccess)
            e = kma::launch_experts(kma::kWeightsGrad, false, dtype, a, b, p, dev.sms, dev.smem, st);
    }
    int32_t *const row = reinterpret_cast<int32_t *>(q);
    int32_t *const order = reinterpret_cast<int32_t *>(q + ids);
    int32_t *const sorted = reinterpret_cast<int32_t *>(q + 2 * ids);
    int32_t *const total = reinterpret_cast<int32_t *>(q + 3 * ids);
    uint8_t *const space = q + 3 * ids + 16;
    if (e == cudaSuccess && sum)
        e = kma::launch_lists(row, M, R, order, sorted, nullptr, total, space, dX,
                              static_cast<size_t>(R) * D * 2, dev.sms, st);
    const int64_t width = sum ? cols : D;
    for (int64_t d = 0; e == cudaSuccess && dX != nullptr && d < D; d += width) {
        const int64_t n = std::min(width, D - d);
        if (!weights_map(&a, dtype, static_cast<const uint8_t *>(W) + 2 * d, E, F, D, n,
                         kma::kExpertsBoxMn) ||
            !rows_map(&b, dtype, dy, dy_rows, F, kma::kExpertsBoxB))
            return KMASSIGN_ERR_CUDA;
        p.mdim = static_cast<int32_t>(n);
        p.kblocks = static_cast<int32_t>((F + 63) / 64);
        p.from = placed;
        p.zero_rest = !sum;
        p.out = sum ? by_position : dX;
        p.out_type = sum ? KMASSIGN_FP32 : dtype;
        e = kma::launch_experts(kma::kRowsGrad, false, dtype, a, b, p, dev.sms, dev.smem, st);
        if (e == cudaSuccess && sum)
            e = kma::launch_sum_rows(reinterpret_cast<const float *>(by_position), M, n, order,
                                     sorted, total, reinterpret_cast<float *>(space + sort),
                                     static_cast<uint8_t *>(dX) + 2 * d, dtype, D, dev.sms, st);
    }
    if (e == cudaSuccess && dX != nullptr && rows == nullptr && R > M)
        e = cudaMemsetAsync(static_cast<uint8_t *>(dX) + static_cast<size_t>(M) * D * 2, 0,
                            static_cast<size_t>(R - M) * D * 2, st);
    rc = done(e);
    return scratch.release() ? rc : KMASSIGN_ERR_CUDA;
}

int kmassign_rmsnorm(const void *X, int32_t dtype, int64_t N, int64_t D, const void *residual,
                     const void *weight, int32_t weight_dtype, float eps, void *total, void *out,
                     int32_t out_dtype, float *scales, float *rstd, void *stream)
{
    DeviceRestore restore;
    if (N < 0 || N >= kLimit)
        return KMASSIGN_ERR_SHAPE;
    if (D < 1 || D > kMaxNormDim)
        return KMASSIGN_ERR_UNSUPPORTED_D;
    if (!known_type(dtype) || (out_dtype != dtype && out_dtype != KMASSIGN_E4M3) ||
        (weight_dtype != KMASSIGN_FP32 && weight_dtype != dtype) || !(eps >= 0.0f) ||
        !std::isfinite(eps))
        return KMASSIGN_ERR_ARG;
    if (N == 0)
        return KMASSIGN_OK;
    if (X == nullptr || out == nullptr || (residual != nullptr && total == nullptr) ||
        (out_dtype == KMASSIGN_E4M3 && scales == nullptr))
        return KMASSIGN_ERR_NULL;
    const uintptr_t es = static_cast<uintptr_t>(kma::dtype_bytes(dtype));
    if (!aligned(X, es) || !aligned(residual, es) || !aligned(total, es) ||
        !aligned(weight, static_cast<uintptr_t>(kma::dtype_bytes(weight_dtype))) ||
        (out_dtype == dtype && !aligned(out, es)) || !aligned(scales, 4) || !aligned(rstd, 4))
        return KMASSIGN_ERR_ALIGN;
    const void *ptrs[7] = {X, residual, weight, total, out, scales, rstd};
    int rc = check_device_ptrs(ptrs, 7);
    if (rc != KMASSIGN_OK)
        return rc;
    cudaMemPool_t pool;
    int sms;
    if ((rc = kma::library_device(&pool, &sms)) != KMASSIGN_OK)
        return rc;
    return done(kma::launch_rmsnorm(X, dtype, N, D, residual, weight, weight_dtype, eps, total, out,
                                    out_dtype, scales, rstd, sms,
                                    static_cast<cudaStream_t>(stream)));
}

int kmassign_rmsnorm_grad(const void *dout, int32_t dtype, int64_t N, int64_t D, const void *total,
                          const void *weight, int32_t weight_dtype, const float *rstd,
                          const void *dtotal, void *dX, float *dweight, void *stream)
{
    DeviceRestore restore;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N < 0 || N >= kLimit)
        return KMASSIGN_ERR_SHAPE;
    if (D < 1 || D > kMaxNormDim)
        return KMASSIGN_ERR_UNSUPPORTED_D;
    if (!known_type(dtype) || (weight_dtype != KMASSIGN_FP32 && weight_dtype != dtype))
        return KMASSIGN_ERR_ARG;
    if (N > 0 && (dout == nullptr || total == nullptr || rstd == nullptr || dX == nullptr))
        return KMASSIGN_ERR_NULL;
    const uintptr_t es = static_cast<uintptr_t>(kma::dtype_bytes(dtype));
    if (!aligned(dout, es) || !aligned(total, es) || !aligned(dtotal, es) || !aligned(dX, es) ||
        !aligned(weight, static_cast<uintptr_t>(kma::dtype_bytes(weight_dtype))) ||
        !aligned(rstd, 4) || !aligned(dweight, 4))
        return KMASSIGN_ERR_ALIGN;
    if (N == 0 && dweight == nullptr)
        return KMASSIGN_OK;
    const void *ptrs[7] = {dout, total, weight, rstd, dtotal, dX, dweight};
    int rc = check_device_ptrs(ptrs, 7);
    if (rc != KMASSIGN_OK)
        return rc;
    if (N == 0)
        return done(cudaMemsetAsync(dweight, 0, static_cast<size_t>(D) * 4, st));
    cudaMemPool_t pool;
    int sms;
    if ((rc = kma::library_device(&pool, &sms)) != KMASSIGN_OK)
        return rc;
    return done(kma::launch_rmsnorm_grad(dout, dtype, N, D, total, weight, weight_dtype, rstd,
                                         dtotal, dX, dweight, pool, sms, st));
}

}  // extern "C"
