// Device helpers of the row operators (routing.hip, residual.hip, checkpoint.hip, weight_grad.hip).
#pragma once

#include "common.h"

namespace mpnn {

using bf16 = __bf16;

// Values are read to and computed in fp32 and rounded once, to nearest even, when stored.
template <class T> __device__ __forceinline__ float to_f32(T v) { return (float)v; }
template <class T> __device__ __forceinline__ T from_f32(float v) { return (T)v; }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

}  // namespace mpnn
