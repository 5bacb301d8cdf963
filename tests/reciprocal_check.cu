// Compares reciprocal(y) with the quotient 1.0f / y, bit by bit, for all 2^23
// significands of the exponent e: the number that differ is added to *count.
#include "reciprocal.cuh"

#include <cuda_runtime.h>

__global__ void compare(int e, unsigned *count)
{
    const unsigned m = blockIdx.x * blockDim.x + threadIdx.x;
    if (m >= 1u << 23)
        return;
    const float y = __uint_as_float(static_cast<unsigned>(127 + e) << 23 | m);
    if (__float_as_uint(kma::reciprocal(y)) != __float_as_uint(1.0f / y))
        atomicAdd(count, 1u);
}

extern "C" int reciprocal_check(int e, void *count)
{
    if (e < 0 || e > 124)
        return -1;
    compare<<<(1 << 23) / 256, 256>>>(e, static_cast<unsigned *>(count));
    return static_cast<int>(cudaGetLastError());
}
