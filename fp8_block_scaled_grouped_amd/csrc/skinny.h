// Linear layers with few rows, weights streamed once: 4-bit weights with group scales
// or 16-bit weights, one matrix or one per expert (skinny.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe355 {

struct SkinnyArgs {
  const uint16_t* x;       // [R, K] bf16 or fp16 bits, row stride ldx (elements)
  const uint8_t* w;        // [E, N, K]: 4-bit codes (K / 2 bytes a row) or 16-bit values
  const void* scale;       // 4-bit: [E, N, G] fp32 or E8M0 bytes, G = ceil(K / group)
  const int32_t* offsets;  // [E + 1] on the device: expert e has rows [offsets[e], offsets[e + 1]); NULL: one matrix
  uint16_t* c;             // [R, N], the type of x, row stride ldc
  int64_t ldx, ldc;
  int R, E, N, K;
  int splits;              // runs of K whose fp32 partial sums are added by a second launch (1: none)
  float* part;             // [splits, R, N], when splits > 1
};

// Weights of a launch: 16-bit, or 4-bit with groups of 32, 64 or 128 and fp32 or E8M0 scales.
enum SkinnyWeights : int { kW16 = 0, kFp4 = 1, kFp4E8M0 = 2 };

// Runs of K that launch_skinny wants for one matrix (fp32 partial sums [runs, M, N] when above 1).
int skinny_splits(int M, int N, int K);

// Checks nothing (the entry points do); MOE355_* status.
int launch_skinny(const SkinnyArgs& g, int weights, int group, int fp16, hipStream_t stream);

}  // namespace moe355
