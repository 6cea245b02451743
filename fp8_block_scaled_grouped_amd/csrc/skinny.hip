// Linear layers with few rows: c[m, n] = sum_k x[m, k] w[n, k] with 4-bit (e2m1) weights and
// group scales, or 16-bit weights; one matrix, or one per expert over ragged row segments.
//
//   4-bit: c[m, n] = round(sum_g s[n, g] sum_{k in group g} x[m, k] q[n, k])
//
// The weights are read once and nothing of them is reused, so they go from memory straight
// into MFMA operands: 16 weight rows are the product's columns, up to 16 MT rows of x its
// rows.  A wave walks a run of 128-wide k blocks; the KW waves that share columns add their
// fp32 tiles in LDS in wave order (one launch, no workspace, deterministic).
//
// A lane loads 16 bytes of a weight row's block: 32 codes, k [32 g, 32 g + 32) for lane group g
// = lane / 16.  The conversion instruction turns 8 codes into an operand in 4 issues.  E8M0
// scales with bf16 x go into the conversion itself (exact).  Else the scale multiplies the
// fp32 tile of its group, so an MFMA's 32 k must lie in one group: groups of 128 take any
// order, for groups of 64 and 32 the lanes of a column exchange codes first (one or two
// lane-swap steps), and x is read in the order that results.
#include "skinny.h"

#include <type_traits>

#include "frag16.h"
#include "host_common.h"

namespace moe355 {
namespace {

constexpr int kWaves = 8;

// vdst's upper 32 lanes <-> vsrc's lower 32 lanes
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
// rows of 16 lanes: a's odd rows <-> b's even rows
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

template <int W, int GROUP, bool F16>
struct Weights {
  static constexpr bool kDirect = W == kFp4E8M0 && !F16;             // scale inside the conversion
  static constexpr int kLoads = W == kW16 ? 4 : 1;                   // 16-byte loads of a row's block per lane
  static constexpr int kScales = W == kW16 ? 0 : kDirect ? 1 : 128 / GROUP;
  static constexpr int kPerScale = W == kW16 || kDirect ? 4 : GROUP / 32;  // MFMAs that share a fold

  u32x4 q[kLoads];
  float s[kScales ? kScales : 1];

  // block kb of weight row `row`; lanes past K get zeros
  __device__ __forceinline__ void load(const uint8_t* row, const void* scale, int64_t srow, int kb, int K, int G, int g) {
    if constexpr (W == kW16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = kb * 128 + 32 * i + 8 * g;
        q[i] = k < K ? *reinterpret_cast<const u32x4*>(row + 2 * (int64_t)k) : u32x4{0, 0, 0, 0};
      }
    } else {
      const int k = kb * 128 + 32 * g;
      q[0] = k < K ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + k / 2)) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kScales; ++i) {
        const int at = kDirect ? (kb * 128 + 32 * g) / GROUP : kb * (128 / GROUP) + i;
        const int in = min(at, G - 1);
        if constexpr (W == kFp4) {
          s[i] = reinterpret_cast<const float*>(scale)[srow + in];
        } else {
          const uint32_t c = reinterpret_cast<const uint8_t*>(scale)[srow + in];
          // the conversion reads the exponent field (0 as 2^-127)
          s[i] = kDirect ? __uint_as_float(c << 23) : e8m0_to_f32(c);
        }
      }
    }
  }
  // 8-wide chunk of x's block that goes with operand i of lane group g
  static __device__ __forceinline__ int chunk(int i, int g) {
    if constexpr (W == kW16 || (!kDirect && GROUP == 32)) return 4 * i + g;
    if constexpr (!kDirect && GROUP == 64) return 8 * (i >> 1) + (i & 1) + 4 * (g & 1) + 2 * (g >> 1);
    return 4 * g + i;
  }
  __device__ __forceinline__ void arrange() {
    if constexpr (W != kW16 && !kDirect && GROUP <= 64) {
      uint32_t d[4] = {q[0][0], q[0][1], q[0][2], q[0][3]};
      swap32(d[0], d[2]);
      swap32(d[1], d[3]);
      if constexpr (GROUP == 32) {
        swap16(d[0], d[1]);
        swap16(d[2], d[3]);
      }
      q[0] = u32x4{d[0], d[1], d[2], d[3]};
    }
  }
  __device__ __forceinline__ s16x8 operand(int i) const {
    if constexpr (W == kW16) return __builtin_bit_cast(s16x8, q[i]);
    return e2m1x8<F16>(q[0][i], kDirect ? s[0] : 1.0f);
  }
};

template <int W, int GROUP, bool F16, int MT, int CW>
__global__ __launch_bounds__(kWaves * 64) void skinny_kernel(SkinnyArgs a) {
  using Wt = Weights<W, GROUP, F16>;
  constexpr int KW = kWaves / CW;
  constexpr int kDepth = W == kW16 || MT >= 4 ? 2 : 4;  // blocks of weights in flight per wave
  __shared__ v4f part[kWaves][MT][64];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cw = w / KW, kw = w % KW;
  const int e = blockIdx.y;
  int lo = 0, hi = a.R;
  if (a.offsets) segment(a.offsets, a.R, e, lo, hi);
  if (lo == hi) return;
  const int n0 = (blockIdx.x * CW + cw) * 16;

  const int KB = (a.K + 127) / 128, G = W == kW16 ? 0 : (a.K + GROUP - 1) / GROUP;
  const int per = (KB + KW - 1) / KW;
  const int kb0 = min(KB, kw * per), kb1 = min(KB, kb0 + per);
  // weight row of this lane (rows past N repeat row N - 1: in bounds, results not stored)
  const int64_t wr = (int64_t)e * a.N + min(n0 + (lane & 15), a.N - 1);
  const uint8_t* row = a.w + wr * (W == kW16 ? 2 * (int64_t)a.K : (int64_t)a.K / 2);
  const int64_t srow = wr * G;

  const int mstep = gridDim.z * 16 * MT;
  for (int m0 = lo + blockIdx.z * 16 * MT; m0 < hi; m0 += mstep) {
    const uint16_t* xrow[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) xrow[t] = a.x + (int64_t)min(m0 + 16 * t + (lane & 15), hi - 1) * a.ldx;
    v4f acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
    Wt wq[kDepth];
    s16x8 xq[MT][4];
    auto load_x = [&](int kb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = kb * 128 + 8 * Wt::chunk(i, g);
#pragma unroll
        for (int t = 0; t < MT; ++t)
          xq[t][i] = k < a.K ? *reinterpret_cast<const s16x8*>(xrow[t] + k) : s16x8{0, 0, 0, 0, 0, 0, 0, 0};
      }
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
      if (kb0 + d < kb1) wq[d].load(row, a.scale, srow, kb0 + d, a.K, G, g);
    if (kb0 < kb1) load_x(kb0);
    for (int kb = kb0; kb < kb1; kb += kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (kb + d < kb1) {
          Wt now = wq[d];
          if (kb + d + kDepth < kb1) wq[d].load(row, a.scale, srow, kb + d + kDepth, a.K, G, g);
          s16x8 xn[MT][4];
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) xn[t][i] = xq[t][i];
          if (kb + d + 1 < kb1) load_x(kb + d + 1);
          now.arrange();
          v4f tile[MT];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const s16x8 b = now.operand(i);
            const bool first = i % Wt::kPerScale == 0, last = i % Wt::kPerScale == Wt::kPerScale - 1;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              if constexpr (Wt::kScales == 0 || Wt::kDirect) {
                acc[t] = mfma16x16x32<F16>(xn[t][i], b, acc[t]);
              } else {
                tile[t] = mfma16x16x32<F16>(xn[t][i], b, first ? v4f{0.f, 0.f, 0.f, 0.f} : tile[t]);
                if (last) acc[t] += tile[t] * now.s[i / Wt::kPerScale];
              }
            }
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[w][t][lane] = acc[t];
    __syncthreads();
    for (int j = tid; j < CW * MT * 64; j += kWaves * 64) {  // whole waves: lane stays
      const int t = j / 64 % MT, c = j / 64 / MT;
      v4f s = part[c * KW][t][lane];
#pragma unroll
      for (int k = 1; k < KW; ++k) s += part[c * KW + k][t][lane];
      const int n = (blockIdx.x * CW + c) * 16 + (lane & 15);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + 16 * t + 4 * g + i;
        if (m < hi && n < a.N) a.c[(int64_t)m * a.ldc + n] = (uint16_t)f32_to_out16(s[i], F16);
      }
    }
    __syncthreads();
  }
}

template <int W, int GROUP, bool F16>
int launch(const SkinnyArgs& g, hipStream_t stream) {
  const int rows = g.offsets ? (int)ceil_div64(g.R, g.E) : g.R;  // of a matrix, on average
  auto go = [&](auto mt, auto cw) {
    constexpr int MT = decltype(mt)::value, CW = decltype(cw)::value;
    const int64_t nx = ceil_div64(g.N, 16 * CW), nz = g.offsets ? 1 : ceil_div64(g.R, 16 * MT);
    MOE355_CHECK(nx < (1ll << 31) && nz < 65536, MOE355_EUNSUPPORTED);
    hipLaunchKernelGGL((skinny_kernel<W, GROUP, F16, MT, CW>), dim3((unsigned)nx, (unsigned)g.E, (unsigned)nz),
                       dim3(kWaves * 64), 0, stream, g);
    return launch_status();
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  const std::integral_constant<int, 4> four;
  if (rows <= 16) return go(one, one);
  if (rows <= 32) return go(two, two);
  return go(four, two);
}

template <int W, bool F16>
int by_group(const SkinnyArgs& g, int group, hipStream_t stream) {
  switch (group) {
    case 32: return launch<W, 32, F16>(g, stream);
    case 64: return launch<W, 64, F16>(g, stream);
    default: return launch<W, 128, F16>(g, stream);
  }
}

}  // namespace

int launch_skinny(const SkinnyArgs& g, int weights, int group, int fp16, hipStream_t stream) {
  if (weights == kW16) return fp16 ? launch<kW16, 128, true>(g, stream) : launch<kW16, 128, false>(g, stream);
  if (weights == kFp4) return fp16 ? by_group<kFp4, true>(g, group, stream) : by_group<kFp4, false>(g, group, stream);
  return fp16 ? by_group<kFp4E8M0, true>(g, group, stream) : by_group<kFp4E8M0, false>(g, group, stream);
}

}  // namespace moe355
