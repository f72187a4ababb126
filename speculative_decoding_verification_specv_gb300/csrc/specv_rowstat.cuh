// specv_rowstat.cuh -- row statistics with a weighted sum, shared by the
// log-probability and the distillation kernels.
//
// A row's softmax statistics are (m, S) = (max_v z_v, sum_v e^{z_v - m}); the
// entropy and the divergences need one more sum of the form
// T = sum_v e^{z_v - m} t_v, taken in the same pass.  All sums are fp32, formed
// per thread and merged in a fixed order, so equal inputs give equal outputs.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "specv_device.cuh"

namespace specv {

// Differences z - m are held above this where they are multiplied by e^{z - m}
// (which is 0 there): a masked entry then adds 0 * kFarBelow and not 0 * -inf.
constexpr float kFarBelow = -1e4f;

// Where row (b, n) of a [B][N][V] view with element strides (sb, sn, 1) begins.
__device__ __forceinline__ int64_t row_offset(int64_t r, int N, int64_t sb, int64_t sn) {
  const int64_t b = r / N;
  return b * sb + (r - b * N) * sn;
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fffffff); }

}  // namespace specv
