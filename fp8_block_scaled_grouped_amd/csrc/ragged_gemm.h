// Products grouped by expert over ragged row segments, 16-bit operands: the
// argument block of ragged_gemm.hip's kernel.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe355 {

// What a launch of the ragged kernels computes for expert e's rows [lo, hi) (from `offsets`):
//   kRaggedFwd    y[r, n]     = sum_k x[r, k] w[e, n, k]
//   kRaggedDgrad  dx[r, k]    = sum_n dy[r, n] w[e, n, k]
//   kRaggedWgrad  dw[e, n, k] = sum_{r in [lo, hi)} dy[r, n] x[r, k]
enum RaggedOp : int { kRaggedFwd = 0, kRaggedDgrad = 1, kRaggedWgrad = 2 };

struct RaggedArgs {
  const uint16_t* a;       // fwd: x [R, K]; dgrad, wgrad: dy [R, N]
  const uint16_t* b;       // fwd, dgrad: w [E, N, K]; wgrad: x [R, K]
  void* c;                 // fwd: y [R, N]; dgrad: dx [R, K]; wgrad: dw [E, N, K]
  const int32_t* offsets;  // [E + 1] on the device
  int64_t lda, ldb, ldc;   // row strides in elements
  int R, E, N, K;
};

}  // namespace moe355
