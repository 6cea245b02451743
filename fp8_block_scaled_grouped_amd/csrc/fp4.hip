// 4-bit (OCP e2m1) weights with group scales: packing, unpacking, and the entry points of
// the linear layers on them.
//
//   amax over a group of 32, 64 or 128 along k (the last group of a row may be shorter)
//   fp32 scale: s = fl32(amax / 6), 1 for an all-zero group; E8M0: s = 2^(floor(log2 amax) - 2),
//   the exponent kept in [-127, 127], 1 for an all-zero group
//   code = nearest e2m1 of fl32(w / s), ties to the even code, saturating at +-6, sign kept
#include <algorithm>
#include <type_traits>

#include "device_common.h"
#include "frag16.h"
#include "host_common.h"
#include "skinny.h"

namespace moe355 {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 22;  // of a launch: larger tensors take more turns of its loop
constexpr int64_t kMaxLd = 1 << 21;  // a pass's rows stay within 2^31 bytes
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <bool F16>
__device__ __forceinline__ void widen8(const u32x4& v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F16) {
      const uint32_t pair = v[i];  // a copy: a bit cast of a vector's element takes element 0
      const f16x2 h = __builtin_bit_cast(f16x2, pair);
      f[2 * i] = (float)h[0];
      f[2 * i + 1] = (float)h[1];
    } else {
      f[2 * i] = bf16_to_f32(v[i] & 0xffffu);
      f[2 * i + 1] = bf16_to_f32(v[i] >> 16);
    }
  }
}

// fl32(w / s) by r = fl32(1 / s): with q = fl(w r) the remainder w - q s is exact, and fl(q + r (w - q s))
// is the correctly rounded quotient (P. Markstein, IBM J. Res. Dev. 34, 1990); 3 operations where the
// division takes about 10.  Scales so small or large that a step could leave the normal range divide.
__device__ __forceinline__ float quotient(float w, float s, float r, bool plain) {
  if (plain) return w / s;
  const float q = w * r;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, w), r, q), w);  // -0 stays -0
}

// 8 values a lane; GROUP / 8 lanes own a group.  FLAT: rows of whole groups, one after the other, as one
// row (no division to find their place).  Bound by memory: 2 K bytes in, K / 2 and the scales out a row;
// 131072 x 7168 takes 0.42 ms with E8M0 scales of 32 (5.7 TB/s; 0.43 to 0.46 between other calls), 0.50 with fp32
// scales of 128 (4.8 TB/s).
template <bool F16, bool E8M0, int GROUP, bool FLAT>
__global__ __launch_bounds__(kThreads) void fp4_quant_kernel(const uint16_t* __restrict__ w, int64_t ld_w, int64_t rows,
                                                             int64_t K, int64_t G, uint8_t* __restrict__ q,
                                                             void* scale) {
  constexpr int L = GROUP / 8;
  const int sub = threadIdx.x % L;
  const int64_t step = (int64_t)gridDim.x * (kThreads / L);
  for (int64_t gi = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L; gi < rows * G; gi += step) {  // groups stay whole
    const int64_t row = FLAT ? 0 : gi / G;
    const int64_t k = (gi - row * G) * GROUP + sub * 8;
    const bool live = FLAT || k < K;
    const u32x4 v = live ? *reinterpret_cast<const u32x4*>(w + row * ld_w + k) : u32x4{0, 0, 0, 0};
    float f[8];
    widen8<F16>(v, f);
    float amax = 0.0f;
    int bad = 0;  // a NaN or an infinity in the group: its scale becomes NaN
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      amax = fmaxf(amax, fabsf(f[i]));
      bad |= !(fabsf(f[i]) <= 3.4028234e38f);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      amax = fmaxf(amax, __shfl_xor(amax, o, kWave));
      bad |= __shfl_xor(bad, o, kWave);
    }
    float y[8];
    if constexpr (E8M0) {
      int ex = amax == 0.0f ? 0 : min(max(__builtin_amdgcn_frexp_expf(amax) - 3, -127), 127);
      if (bad) ex = 128;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_ldexpf(f[i], -ex);  // exact where it decides a code
      if (sub == 0) reinterpret_cast<uint8_t*>(scale)[gi] = (uint8_t)(ex + 127);
    } else {
      const float s = bad ? __uint_as_float(0x7fc00000u) : amax == 0.0f ? 1.0f : amax / 6.0f, r = 1.0f / s;
      const bool plain = !(s >= 0x1p-60f && s <= 0x1p60f);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = quotient(f[i], s, r, plain);
      if (sub == 0) reinterpret_cast<float*>(scale)[gi] = s;
    }
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], 1.0f, 3);
    if (live) *reinterpret_cast<uint32_t*>(q + row * (K / 2) + k / 2) = c;
  }
}

// 8 values a lane; FLAT as above.  131072 x 7168: 0.52 ms (4.6 TB/s), bound by the 16-bit stores.
template <bool F16, bool E8M0, bool FLAT>
__global__ __launch_bounds__(kThreads) void fp4_dequant_kernel(const uint8_t* __restrict__ q, const void* scale,
                                                               int64_t rows, int64_t K, int shift, int64_t G,
                                                               uint16_t* __restrict__ w, int64_t ld_w) {
  const int64_t C = K / 8;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < rows * C; i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = FLAT ? 0 : i / C;
    const int64_t k = (i - row * C) * 8, at = row * G + (k >> shift);
    const uint32_t codes = *reinterpret_cast<const uint32_t*>(q + row * (K / 2) + k / 2);
    const float s =
        E8M0 ? e8m0_to_f32(reinterpret_cast<const uint8_t*>(scale)[at]) : reinterpret_cast<const float*>(scale)[at];
    const f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3)};
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a = v[j][0] * s, b = v[j][1] * s;
      // kept apart from the rounding: fused into one multiply-add with +0, fp16 -0 would come out as +0
      if constexpr (F16) asm("" : "+v"(a), "+v"(b));
      r[j] = f32_to_out16(a, F16) | (f32_to_out16(b, F16) << 16);
    }
    *reinterpret_cast<u32x4*>(w + row * ld_w + k) = r;
  }
}

int check_format(int fp16, int group, int e8m0) {
  MOE355_CHECK((fp16 == 0 || fp16 == 1) && (e8m0 == 0 || e8m0 == 1), MOE355_EINVAL);
  MOE355_CHECK(group == 32 || group == 64 || group == 128, MOE355_EUNSUPPORTED);
  return MOE355_OK;
}

bool aligned_scale(const void* s, int e8m0) { return e8m0 || (reinterpret_cast<uintptr_t>(s) & 3u) == 0; }

}  // namespace
}  // namespace moe355

using namespace moe355;

extern "C" int fp4_quant_groups(const uint16_t* w, int fp16, int64_t ld_w, int64_t rows, int K, int group, uint8_t* q,
                                void* scale, int e8m0, hipStream_t stream) {
  if (int st = check_format(fp16, group, e8m0)) return st;
  MOE355_CHECK(rows >= 0 && K >= 0 && ld_w >= K, MOE355_EINVAL);
  MOE355_CHECK(K % 32 == 0, MOE355_EUNSUPPORTED);
  if (rows == 0 || K == 0) return MOE355_OK;
  MOE355_CHECK(w && q && scale, MOE355_EINVAL);
  MOE355_CHECK(aligned16(w) && ld_w % 8 == 0 && aligned16(q) && aligned_scale(scale, e8m0), MOE355_EMISALIGNED);
  const int64_t G = ceil_div64(K, group);
  const int64_t blocks = std::min(kMaxBlocks, ceil_div64(rows * G * (group / 8), kThreads));
  auto go = [&](auto f, auto e, auto flat_c) {
    constexpr bool F = decltype(f)::value, E = decltype(e)::value, FL = decltype(flat_c)::value;
    auto* fn = group == 32   ? &fp4_quant_kernel<F, E, 32, FL>
               : group == 64 ? &fp4_quant_kernel<F, E, 64, FL>
                             : &fp4_quant_kernel<F, E, 128, FL>;
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(kThreads), 0, stream, w, ld_w, FL ? 1 : rows,
                       FL ? rows * K : (int64_t)K, FL ? rows * G : G, q, scale);
    return launch_status();
  };
  const std::true_type yes;
  const std::false_type no;
  const bool flat = K % group == 0 && ld_w == K;
  if (fp16) return e8m0 ? (flat ? go(yes, yes, yes) : go(yes, yes, no)) : (flat ? go(yes, no, yes) : go(yes, no, no));
  return e8m0 ? (flat ? go(no, yes, yes) : go(no, yes, no)) : (flat ? go(no, no, yes) : go(no, no, no));
}

extern "C" int fp4_dequant_groups(const uint8_t* q, const void* scale, int e8m0, int64_t rows, int K, int group,
                                  uint16_t* w, int fp16, int64_t ld_w, hipStream_t stream) {
  if (int st = check_format(fp16, group, e8m0)) return st;
  MOE355_CHECK(rows >= 0 && K >= 0 && ld_w >= K, MOE355_EINVAL);
  MOE355_CHECK(K % 32 == 0, MOE355_EUNSUPPORTED);
  if (rows == 0 || K == 0) return MOE355_OK;
  MOE355_CHECK(w && q && scale, MOE355_EINVAL);
  MOE355_CHECK(aligned16(w) && ld_w % 8 == 0 && aligned16(q) && aligned_scale(scale, e8m0), MOE355_EMISALIGNED);
  const int64_t G = ceil_div64(K, group);
  const int shift = group == 32 ? 5 : group == 64 ? 6 : 7;
  const int64_t blocks = std::min(kMaxBlocks, ceil_div64(rows * (K / 8), kThreads));
  auto go = [&](auto flat_c) {
    constexpr bool FL = decltype(flat_c)::value;
    auto* fn = fp16 ? (e8m0 ? &fp4_dequant_kernel<true, true, FL> : &fp4_dequant_kernel<true, false, FL>)
                    : (e8m0 ? &fp4_dequant_kernel<false, true, FL> : &fp4_dequant_kernel<false, false, FL>);
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(kThreads), 0, stream, q, scale, FL ? 1 : rows,
                       FL ? rows * K : (int64_t)K, shift, FL ? rows * G : G, w, ld_w);
    return launch_status();
  };
  return K % group == 0 && ld_w == K ? go(std::true_type{}) : go(std::false_type{});
}

extern "C" int gemm_fp4_groupscale_workspace(int M, int N, int K, size_t* bytes) {
  MOE355_CHECK(M >= 0 && N >= 0 && K >= 0 && bytes, MOE355_EINVAL);
  MOE355_CHECK(K % 32 == 0, MOE355_EUNSUPPORTED);
  const int splits = M && N && K ? skinny_splits(M, N, K) : 1;
  *bytes = splits > 1 ? (size_t)splits * M * N * sizeof(float) : 0;
  return MOE355_OK;
}

extern "C" int gemm_fp4_groupscale(const uint16_t* x, int fp16, int64_t ld_x, const uint8_t* q, const void* scale,
                                   int e8m0, int group, int M, int N, int K, uint16_t* c, int64_t ldc, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  if (int st = check_format(fp16, group, e8m0)) return st;
  MOE355_CHECK(M >= 0 && N >= 0 && K >= 0 && ld_x >= K && ldc >= N, MOE355_EINVAL);
  MOE355_CHECK(K % 32 == 0 && ld_x <= kMaxLd, MOE355_EUNSUPPORTED);
  if (M == 0 || N == 0) return MOE355_OK;
  MOE355_CHECK(c && (K == 0 || (x && q && scale)), MOE355_EINVAL);
  MOE355_CHECK((K == 0 || (aligned16(x) && ld_x % 8 == 0 && aligned16(q) && aligned_scale(scale, e8m0))) &&
                   (reinterpret_cast<uintptr_t>(c) & 1u) == 0 && aligned16(workspace),
               MOE355_EMISALIGNED);
  const int splits = workspace && K ? skinny_splits(M, N, K) : 1;
  MOE355_CHECK(splits == 1 || workspace_bytes >= (size_t)splits * M * N * sizeof(float), MOE355_EINVAL);
  return launch_skinny(SkinnyArgs{x, q, scale, nullptr, c, ld_x, ldc, M, 1, N, K, splits, static_cast<float*>(workspace)},
                       e8m0 ? kFp4E8M0 : kFp4, group, fp16, stream);
}

extern "C" int grouped_gemm_fp4(const uint16_t* x, int fp16, int64_t ld_x, const uint8_t* q, const void* scale,
                                int e8m0, int group, const int32_t* offsets, int R, int E, int N, int K, uint16_t* c,
                                int64_t ldc, hipStream_t stream) {
  if (int st = check_format(fp16, group, e8m0)) return st;
  MOE355_CHECK(R >= 0 && E >= 0 && N >= 0 && K >= 0 && ld_x >= K && ldc >= N, MOE355_EINVAL);
  MOE355_CHECK(K % 32 == 0 && E < 65536 && ld_x <= kMaxLd, MOE355_EUNSUPPORTED);
  if (R == 0 || E == 0 || N == 0) return MOE355_OK;
  MOE355_CHECK(offsets && c && (K == 0 || (x && q && scale)), MOE355_EINVAL);
  MOE355_CHECK((K == 0 || (aligned16(x) && ld_x % 8 == 0 && aligned16(q) && aligned_scale(scale, e8m0))) &&
                   (reinterpret_cast<uintptr_t>(c) & 1u) == 0 && (reinterpret_cast<uintptr_t>(offsets) & 3u) == 0,
               MOE355_EMISALIGNED);
  return launch_skinny(SkinnyArgs{x, q, scale, offsets, c, ld_x, ldc, R, E, N, K, 1, nullptr}, e8m0 ? kFp4E8M0 : kFp4, group, fp16,
                       stream);
}
