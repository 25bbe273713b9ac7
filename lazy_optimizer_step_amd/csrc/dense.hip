// dense.hip - the validation shared by the dense operators.
#include "dense.hpp"

namespace spopt {

template <class T>
__global__ __launch_bounds__(256) void k_check_finite(const T* x, int64_t rows, int64_t cols,
                                                      int64_t stride, uint32_t* status) {
    bool bad = false;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += 256) bad |= !finite_f((float)x[r * stride + c]);
    if (bad) atomicOr(status, (uint32_t)kStatusNonFinite);
}

int launch_check_finite(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride,
                        uint32_t* status, hipStream_t s) {
    const unsigned grid = (unsigned)(rows < 4096 ? rows : 4096);
    if (dtype == SPOPT_DTYPE_F32)
        k_check_finite<<<grid, 256, 0, s>>>((const float*)x, rows, cols, stride, status);
    else if (dtype == SPOPT_DTYPE_BF16)
        k_check_finite<<<grid, 256, 0, s>>>((const __bf16*)x, rows, cols, stride, status);
    else
        k_check_finite<<<grid, 256, 0, s>>>((const _Float16*)x, rows, cols, stride, status);
    SPOPT_LAUNCHED();
    return SPOPT_OK;
}

}  // namespace spopt
