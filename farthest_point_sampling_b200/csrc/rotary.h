// Launcher of the multi-axis rotary position kernel (rotary.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/fpstok.h"

namespace fpstok {

struct RotaryCall {
  const void* x;
  void* y;
  int dtype;  // FPS_DTYPE_*
  int64_t T;
  int H, D;
  int64_t x_token, x_head, y_token, y_head;  // strides in elements
  const float* positions;                    // [T, axes], rows position_stride floats apart
  int64_t position_stride;
  int inverse;
};

cudaError_t launch_rotary(const RotaryCall& c, const fps_rotary_table& table, cudaStream_t s);

}  // namespace fpstok
