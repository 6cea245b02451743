// 4-bit (OCP e2m1) weights with group scales: packing, unpacking, and the entry points of
// the linear layers on them.
//
//   amax over a group of 32, 64 or 128 along k (the last group of a row may be shorter)
//   fp32 scale: s = fl32(amax / 6), 1 for an all-zero group; E8M0: s = 2^(floor(log2 amax) - 2),
//   the exponent kept in [-127, 127], 1 for an all-zero group
//   code = nearest e2m1 of fl32(w / s), ties to the even code, saturating at +-6, sign kept
#include <type_traits>

#include "device_common.h"
#include "frag16.h"
#include "host_common.h"
#include "skinny.h"

namespace moe355 {
namespace {

constexpr int kThreads = 256;
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

// 8 values a lane; GROUP / 8 lanes own a group.
template <bool F16, bool E8M0, int GROUP>
__global__ __launch_bounds__(kThreads) void fp4_quant_kernel(const uint16_t* __restrict__ w, int64_t ld_w, int64_t rows,
                                                             int K, int G, uint8_t* __restrict__ q, void* scale) {
  constexpr int L = GROUP / 8;
  const int64_t gi = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L;
  const int sub = threadIdx.x % L;
  if (gi >= rows * G) return;  // whole groups leave together
  const int64_t row = gi / G;
  const int gr = (int)(gi - row * G), k = gr * GROUP + sub * 8;
  const bool live = k < K;
  const u32x4 v = live ? *reinterpret_cast<const u32x4*>(w + row * ld_w + k) : u32x4{0, 0, 0, 0};
  float f[8];
  widen8<F16>(v, f);
  float amax = 0.0f;
  bool bad = false;  // a NaN or an infinity in the group: its scale becomes NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    amax = fmaxf(amax, fabsf(f[i]));
    bad |= !(fabsf(f[i]) <= 3.4028234e38f);
  }
  int any = bad;
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) {
    amax = fmaxf(amax, __shfl_xor(amax, o, kWave));
    any |= __shfl_xor(any, o, kWave);
  }
  float y[8];
  if constexpr (E8M0) {
    int ex = amax == 0.0f ? 0 : min(max(__builtin_amdgcn_frexp_expf(amax) - 3, -127), 127);
    if (any) ex = 128;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_ldexpf(f[i], -ex);  // exact where it decides a code
    if (sub == 0) reinterpret_cast<uint8_t*>(scale)[gi] = (uint8_t)(ex + 127);
  } else {
    const float s = any ? __uint_as_float(0x7fc00000u) : amax == 0.0f ? 1.0f : amax / 6.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = f[i] / s;
    if (sub == 0) reinterpret_cast<float*>(scale)[gi] = s;
  }
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], 1.0f, 3);
  if (live) *reinterpret_cast<uint32_t*>(q + row * (K / 2) + k / 2) = c;
}

template <bool F16, bool E8M0>
__global__ __launch_bounds__(kThreads) void fp4_dequant_kernel(const uint8_t* __restrict__ q, const void* scale,
                                                               int64_t rows, int K, int shift, int G,
                                                               uint16_t* __restrict__ w, int64_t ld_w) {
  const int C = K / 8;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= rows * C) return;
  const int64_t row = i / C;
  const int k = (int)(i - row * C) * 8;
  const uint32_t codes = *reinterpret_cast<const uint32_t*>(q + row * (K / 2) + k / 2);
  const int64_t at = row * G + (k >> shift);
  const float s = E8M0 ? e8m0_to_f32(reinterpret_cast<const uint8_t*>(scale)[at]) : reinterpret_cast<const float*>(scale)[at];
  const f32x2 v[4] = {
      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1),
      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3)};
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
  const int G = (int)ceil_div64(K, group);
  const int64_t blocks = ceil_div64(rows * G * (group / 8), kThreads);
  MOE355_CHECK(blocks < (1ll << 31), MOE355_EUNSUPPORTED);
  auto go = [&](auto f, auto e) {
    constexpr bool F = decltype(f)::value, E = decltype(e)::value;
    auto* fn = group == 32 ? &fp4_quant_kernel<F, E, 32> : group == 64 ? &fp4_quant_kernel<F, E, 64> : &fp4_quant_kernel<F, E, 128>;
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(kThreads), 0, stream, w, ld_w, rows, K, G, q, scale);
    return launch_status();
  };
  if (fp16) return e8m0 ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
  return e8m0 ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
}

extern "C" int fp4_dequant_groups(const uint8_t* q, const void* scale, int e8m0, int64_t rows, int K, int group,
                                  uint16_t* w, int fp16, int64_t ld_w, hipStream_t stream) {
  if (int st = check_format(fp16, group, e8m0)) return st;
  MOE355_CHECK(rows >= 0 && K >= 0 && ld_w >= K, MOE355_EINVAL);
  MOE355_CHECK(K % 32 == 0, MOE355_EUNSUPPORTED);
  if (rows == 0 || K == 0) return MOE355_OK;
  MOE355_CHECK(w && q && scale, MOE355_EINVAL);
  MOE355_CHECK(aligned16(w) && ld_w % 8 == 0 && aligned16(q) && aligned_scale(scale, e8m0), MOE355_EMISALIGNED);
  const int G = (int)ceil_div64(K, group), shift = group == 32 ? 5 : group == 64 ? 6 : 7;
  const int64_t blocks = ceil_div64(rows * (K / 8), kThreads);
  MOE355_CHECK(blocks < (1ll << 31), MOE355_EUNSUPPORTED);
  auto* fn = fp16 ? (e8m0 ? &fp4_dequant_kernel<true, true> : &fp4_dequant_kernel<true, false>)
                  : (e8m0 ? &fp4_dequant_kernel<false, true> : &fp4_dequant_kernel<false, false>);
  hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(kThreads), 0, stream, q, scale, rows, K, shift, G, w, ld_w);
  return launch_status();
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
