// dense.hpp - what the dense operators' sources share.
#pragma once

#include "common.hpp"
#include "dense_ops.h"

namespace spopt {

inline size_t dtype_bytes(int32_t dtype) { return dtype == SPOPT_DTYPE_F32 ? 4 : 2; }

// Sets kStatusNonFinite where a rows x cols array (row stride in elements)
// holds a NaN or an infinity.
int launch_check_finite(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride,
                        uint32_t* status, hipStream_t s);

}  // namespace spopt
