// 16-bit MFMA operands and products (gfx950).
#pragma once

#include "device_common.h"

namespace moe355 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// D = A(16x32) * B(32x16) + C, bf16 or fp16 operands, fp32 result.  Lane l holds row/column
// l % 16 and k slots [8 (l / 16), 8 (l / 16) + 8); output element (4 (l / 16) + i, l % 16) in c[i].
template <bool F16>
__device__ __forceinline__ v4f mfma16x16x32(const s16x8& a, const s16x8& b, const v4f& c) {
  if constexpr (F16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
}

// Eight e2m1 codes (4 bits each, lowest first) -> eight bf16 or fp16 values times 2^(scale's
// exponent); every code is exact in both types, and so is the product in bf16 up to a scale of 2^125 (6 x 2^126
// and more become infinities).
template <bool F16>
__device__ __forceinline__ s16x8 e2m1x8(uint32_t codes, float scale) {
  u32x4 r;
  if constexpr (F16) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3));
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  }
  return __builtin_bit_cast(s16x8, r);
}

// Eight e2m1 codes -> eight bf16 values times a power of two from 2^-129 to 2^125, or NaN: exact too, subnormal
// values (multiples of 2^-130) among them.
__device__ __forceinline__ s16x8 e2m1x8_times(uint32_t codes, float scale) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3)};
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __float_as_uint(v[i][0] * scale) >> 16 | (__float_as_uint(v[i][1] * scale) & 0xffff0000u);
  return __builtin_bit_cast(s16x8, r);
}

constexpr uint32_t kPastEnd = 0x80000000u;  // a lane offset beyond every descriptor's length

// Buffer descriptor of at most 2^31 - 16 bytes (none for a negative count, which as an unsigned
// length would check nothing) for dma16_buf; lane offsets from `bytes` on read zeros.
__device__ __forceinline__ u32x4 dma_buffer(const void* base, int64_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v),
               (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32)) & 0xffffu,
               (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)min(max(bytes, (int64_t)0), (int64_t)0x7ffffff0)), 0x00020000u};
}

// LDS-DMA through a buffer descriptor: lane l moves 16 bytes from base + off to
// LDS[m0 + 16 l]; off at or past the descriptor's length writes zeros.  Completion is
// counted with vm_wait.
__device__ __forceinline__ void dma16_buf(u32x4 rsrc, uint32_t off, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(rsrc), "s"(m0)
               : "memory");
}

// fp32 value of an E8M0 scale code, 2^(code - 127) or NaN for 255: the conversion of the e4m3
// code of 1.0 under that scale, which also gets the subnormal 2^-127 right.
__device__ __forceinline__ float e8m0_to_f32(uint32_t code) {
  return __builtin_amdgcn_cvt_scalef32_f32_fp8(0x38, __uint_as_float(code << 23), 0);
}

// Segment [lo, hi) of expert e, kept inside [0, R] whatever the offsets hold.
__device__ __forceinline__ void segment(const int32_t* offsets, int R, int e, int& lo, int& hi) {
  lo = min(max(offsets[e], 0), R);
  hi = min(max(offsets[e + 1], lo), R);
}

}  // namespace moe355
