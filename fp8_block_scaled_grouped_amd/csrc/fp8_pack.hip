// FP8 (e4m3) operands of the ragged expert products: activations or gradients with power-of-two
// scales along rows and along columns, and weights with one scale for each 128 x 128.
//
// A workgroup takes a tile of 128 rows x 128 columns: thread t the 8 columns from 8 (t % 16) of the
// 8 rows from 8 (t / 16), which it keeps in registers between the maxima and the codes, so
// the input is read once for both orientations.  The maxima are those of the magnitudes'
// 16 bits (they order as the values do, infinities and NaN above all).  The codes of
// 8 rows of a column are 8 bytes of the transposed tile, which goes through LDS to be stored in whole lines.
// Bound by memory: 2 bytes in, 1 or 2 out for each value.  Both orientations of 32768 x 7168 161 to 196 us (4.8 to 5.8 TB/s), of weights
// 32 x 4096 x 7168 705 to 735 us (5.1 to 5.3 TB/s; as stored alone 515 to 540), with fp32 scales the same.  A few thousand rows wait for their
// own latencies: 5003 x 1168 over 48 experts 11 us run over and over (2.1 TB/s; rows or columns alone 7), 14 behind the launches of a
// training step, 17 with nothing in the caches.
//
// Scales.  E8M0: byte c stands for 2^(c - 127), the smallest power of two that keeps the block in +-448
// (448 = 1.75 * 2^8), so nothing saturates and codes are the nearest e4m3 of x * 2^(127 - c), rounded
// once.  A block that holds an infinity or a NaN gets byte 255 and codes of NaN.
#include "device_common.h"
#include "frag16.h"
#include "host_common.h"

namespace moe355 {
namespace {

constexpr int kThreads = 256;

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 h16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

template <bool F16>
__device__ __forceinline__ float value16(uint32_t bits) {
  return F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)bits) : bf16_to_f32(bits);
}

// E8M0 byte for a block whose largest magnitude has these 16 bits
template <bool F16>
__device__ __forceinline__ uint32_t e8m0_of(uint32_t amax16) {
  if (amax16 >= (F16 ? 0x7c00u : 0x7f80u)) return 255u;
  if (amax16 == 0) return 127u;
  const uint32_t u = __float_as_uint(value16<F16>(amax16));
  return (uint32_t)max(0, (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0));
}

// byte b of the result: byte `at` of w[b]
__device__ __forceinline__ uint32_t gather_bytes(const uint32_t w0, const uint32_t w1, const uint32_t w2, const uint32_t w3,
                                                 int at) {
  const uint32_t sel = (uint32_t)at | ((uint32_t)(at + 4) << 8);
  return __builtin_amdgcn_perm(w1, w0, sel) & 0xffffu | __builtin_amdgcn_perm(w3, w2, sel) << 16;
}

// The thread's 8 x 8 values of a tile: two 16-bit values a word
struct Tile {
  uint32_t v[8][4];
};

// Codes of the four values in two words with the scale of E8M0 byte c.  The conversion divides by the power of two and rounds
// once (held by a test for every value under every byte that its block can have; byte 0, here a scale of +0, counts as 2^-127), NaN for
// byte 255, and takes one instruction in place of nine a pair.
template <bool F16>
__device__ __forceinline__ uint32_t codes4(uint32_t lo, uint32_t hi, uint32_t c) {
  const float s = __uint_as_float(c << 23);
  s16x2 r = {0, 0};
  if constexpr (F16) {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(h16x2, lo), s, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(r, __builtin_bit_cast(h16x2, hi), s, true);
  } else {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(b16x2, lo), s, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(b16x2, hi), s, true);
  }
  return __builtin_bit_cast(uint32_t, r);
}

// Codes of 8 rows of a column -> LDS tile [128 columns][128 rows], i of the thread's columns.  A column's 16-byte
// chunk c stands in slot c ^ (column / 8 % 8).
__device__ __forceinline__ void put_column(uint8_t* lds, uint2 col, int i, int cg, int rg) {
  *reinterpret_cast<uint2*>(lds + (8 * cg + i) * 128 + (((rg >> 1) ^ (cg & 7)) << 4) + 8 * (rg & 1)) = col;
}
// Row-major codes q[8 rows][8 columns of this thread] into that tile
__device__ __forceinline__ void put_transposed(uint8_t* lds, const uint2 (&q)[8], int cg, int rg) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    auto word = [&](int r) { return i < 4 ? q[r].x : q[r].y; };
    const uint2 col = make_uint2(gather_bytes(word(0), word(1), word(2), word(3), i & 3),
                                 gather_bytes(word(4), word(5), word(6), word(7), i & 3));
    put_column(lds, col, i, cg, rg);
  }
}
// chunk c of a column of that tile
__device__ __forceinline__ u32x4 get_transposed(const uint8_t* lds, int col, int c) {
  return *reinterpret_cast<const u32x4*>(lds + col * 128 + ((c ^ ((col >> 3) & 7)) << 4));
}

// the largest halves of 16 lanes side by side, to all of them
__device__ __forceinline__ uint32_t max16x2_row(uint32_t m) {
  m = max16x2(m, __builtin_amdgcn_update_dpp(0, m, 0xb1, 0xf, 0xf, true));   // lanes ^ 1
  m = max16x2(m, __builtin_amdgcn_update_dpp(0, m, 0x4e, 0xf, 0xf, true));   // lanes ^ 2
  m = max16x2(m, __builtin_amdgcn_update_dpp(0, m, 0x141, 0xf, 0xf, true));  // 7 - lane in each 8
  return max16x2(m, __builtin_amdgcn_update_dpp(0, m, 0x140, 0xf, 0xf, true));  // 15 - lane
}

// Block b of 128 rows: expert e's are [off_e / 128 + e, ..), counted from the segment's first row.  Returns
// the rows [r0, r1) of b, none for the indices that no expert has.
__device__ __forceinline__ void block_rows(const int32_t* offsets, int R, int E, int b, int lane, int& r0, int& r1) {
  int before = 0, lo = 0, hi = 0;  // experts whose first block is b or an earlier one; rows of the last such expert
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int l = 0, h = 0;
    if (e < E) segment(offsets, R, e, l, h);
    const int n = __popcll(__ballot(e < E && l / 128 + e <= b));
    if (n == 0) break;
    before += n;
    lo = __builtin_amdgcn_readlane(l, n - 1);
    hi = __builtin_amdgcn_readlane(h, n - 1);
  }
  r0 = r1 = 0;
  if (before == 0) return;
  const int64_t first = lo + (int64_t)max(0, b - (lo / 128 + before - 1)) * 128;
  r0 = (int)min((int64_t)hi, first);
  r1 = (int)min((int64_t)hi, first + 128);
}

struct RaggedPackArgs {
  const uint16_t* x;
  const int32_t* offsets;
  uint8_t *q, *scale, *qt, *tscale;
  int64_t ld_x, ld_q, ssm, sskb;
  int R, E, C;
};

template <bool F16>
__global__ __launch_bounds__(kThreads) void quant_ragged_kernel(RaggedPackArgs g) {
  __shared__ __align__(16) uint8_t lds[128 * 128];
  __shared__ uint32_t cmax[4][64];
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4, w = tid >> 6;
  const int ctiles = (g.C + 127) / 128;
  const int b = (int)(blockIdx.x / ctiles), c0 = (int)(blockIdx.x % ctiles) * 128;
  int r0, r1;
  if (g.offsets) {
    block_rows(g.offsets, g.R, g.E, b, tid & 63, r0, r1);
  } else {
    r0 = b * 128;
    r1 = min(g.R, r0 + 128);
  }
  if (r1 <= r0) return;
  const int c = c0 + 8 * cg;
  const bool in = c < g.C;
  Tile t;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 8 * rg + i;
    const uint4 v = in && r < r1 ? *reinterpret_cast<const uint4*>(g.x + r * g.ld_x + c) : make_uint4(0, 0, 0, 0);
    t.v[i][0] = v.x;
    t.v[i][1] = v.y;
    t.v[i][2] = v.z;
    t.v[i][3] = v.w;
  }
  constexpr uint32_t kAbs = 0x7fff7fffu;
  if (g.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = max16x2(max16x2(t.v[i][0] & kAbs, t.v[i][1] & kAbs), max16x2(t.v[i][2] & kAbs, t.v[i][3] & kAbs));
      m = max16x2_row(m);
      const uint32_t s = e8m0_of<F16>(max(m & 0xffffu, m >> 16));
      const int r = r0 + 8 * rg + i;
      if (r < r1) {
        if (in)
          *reinterpret_cast<uint2*>(g.q + r * g.ld_q + c) =
              make_uint2(codes4<F16>(t.v[i][0], t.v[i][1], s), codes4<F16>(t.v[i][2], t.v[i][3], s));
        if (cg == 0) g.scale[r * g.ssm + (c0 >> 7) * g.sskb] = (uint8_t)s;
      }
    }
  }
  if (g.qt) {
    uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = max16x2(m[j], t.v[i][j] & kAbs);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = max16x2(m[j], __shfl_xor(m[j], 16, 64));
      m[j] = max16x2(m[j], __shfl_xor(m[j], 32, 64));
      if ((tid & 63) < 16) cmax[w][4 * cg + j] = m[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = max16x2(max16x2(cmax[0][4 * cg + j], cmax[1][4 * cg + j]),
                                 max16x2(cmax[2][4 * cg + j], cmax[3][4 * cg + j]));
      const uint32_t s[2] = {e8m0_of<F16>(a & 0xffffu), e8m0_of<F16>(a >> 16)};
      if (rg == 0 && in) *reinterpret_cast<uint16_t*>(g.tscale + (int64_t)b * g.C + c + 2 * j) = (uint16_t)(s[0] | s[1] << 8);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        auto pair = [&](int r) { return __builtin_amdgcn_perm(t.v[r + 1][j], t.v[r][j], h ? 0x07060302u : 0x05040100u); };
        put_column(lds, make_uint2(codes4<F16>(pair(0), pair(2), s[h]), codes4<F16>(pair(4), pair(6), s[h])), 2 * j + h, cg, rg);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = tid + 256 * i, col = id >> 3;
      if (c0 + col < g.C)
        *reinterpret_cast<u32x4*>(g.qt + ((int64_t)b * g.C + c0 + col) * 128 + (id & 7) * 16) = get_transposed(lds, col, id & 7);
    }
  }
}

// One 128 x 128 block of one expert's weights: the codes as stored and transposed.
struct WeightPackArgs {
  const uint16_t* w;
  uint8_t *q, *qt;
  void *scale, *tscale;
  int E, N, K;
};

template <bool F16, bool E8>
__global__ __launch_bounds__(kThreads) void quant_weight_kernel(WeightPackArgs g) {
  __shared__ __align__(16) uint8_t lds[128 * 128];
  __shared__ uint32_t wmax[4];
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
  const int NB = (g.N + 127) / 128, KB = (g.K + 127) / 128;
  const int kb = (int)(blockIdx.x % KB), nb = (int)(blockIdx.x / KB % NB);
  const int64_t e = blockIdx.x / KB / NB;
  const int k = kb * 128 + 8 * cg, n0 = nb * 128;
  const uint16_t* w = g.w + e * g.N * g.K;
  Tile t;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + 8 * rg + i;
    const uint4 v = k < g.K && n < g.N ? *reinterpret_cast<const uint4*>(w + (int64_t)n * g.K + k) : make_uint4(0, 0, 0, 0);
    t.v[i][0] = v.x;
    t.v[i][1] = v.y;
    t.v[i][2] = v.z;
    t.v[i][3] = v.w;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max16x2(m, t.v[i][j] & 0x7fff7fffu);
  }
  m = max(m & 0xffffu, m >> 16);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
  if ((tid & 63) == 0) wmax[tid >> 6] = m;
  __syncthreads();
  m = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  const int64_t at = (e * NB + nb) * KB + kb, tat = (e * KB + kb) * NB + nb;
  uint2 q[8];
  if constexpr (E8) {
    const uint32_t s = e8m0_of<F16>(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = make_uint2(codes4<F16>(t.v[i][0], t.v[i][1], s), codes4<F16>(t.v[i][2], t.v[i][3], s));
    if (tid == 0) {
      static_cast<uint8_t*>(g.scale)[at] = (uint8_t)s;
      if (g.qt) static_cast<uint8_t*>(g.tscale)[tat] = (uint8_t)s;
    }
  } else {
    // scale and quotient are IEEE divisions, as in fp8_quant_1x128
    const bool bad = m >= (F16 ? 0x7c00u : 0x7f80u);
    const float s = bad ? __uint_as_float(0x7fc00000u) : m == 0 ? 1.0f : value16<F16>(m) / kE4M3Max;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = bad ? 0.0f : value16<F16>(t.v[i][j] & 0xffffu) / s;
        f[2 * j + 1] = bad ? 0.0f : value16<F16>(t.v[i][j] >> 16) / s;
      }
      q[i] = make_uint2(f32x4_to_e4m3(f[0], f[1], f[2], f[3]), f32x4_to_e4m3(f[4], f[5], f[6], f[7]));
    }
    if (tid == 0) {
      static_cast<float*>(g.scale)[at] = s;
      if (g.qt) static_cast<float*>(g.tscale)[tat] = s;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = n0 + 8 * rg + i;
    if (k < g.K && n < g.N) *reinterpret_cast<uint2*>(g.q + (e * g.N + n) * g.K + k) = q[i];
  }
  if (g.qt) {
    put_transposed(lds, q, cg, rg);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = tid + 256 * i, col = id >> 3, n = n0 + (id & 7) * 16;
      if (kb * 128 + col < g.K && n < g.N)
        *reinterpret_cast<u32x4*>(g.qt + (e * g.K + kb * 128 + col) * g.N + n) = get_transposed(lds, col, id & 7);
    }
  }
}

constexpr int kMaxDim = 1 << 30;  // columns plus a tile stay below 2^31

inline bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace moe355

using namespace moe355;

extern "C" int fp8_ragged_blocks(int R, int E, int64_t* blocks) {
  MOE355_CHECK(R >= 0 && E >= 0 && blocks, MOE355_EINVAL);
  *blocks = (int64_t)R / 128 + E;
  return MOE355_OK;
}

extern "C" int fp8_quant_ragged(const uint16_t* x, int fp16, int64_t ld_x, const int32_t* offsets, int R, int E, int K, uint8_t* q,
                                int64_t ld_q, uint8_t* scale, int64_t sstride_m, int64_t sstride_kb, uint8_t* qt,
                                uint8_t* tscale, hipStream_t stream) {
  MOE355_CHECK((fp16 == 0 || fp16 == 1) && R >= 0 && K >= 0 && E >= 0 && ld_x >= K && (!q || ld_q >= K), MOE355_EINVAL);
  MOE355_CHECK(K % 8 == 0 && K <= kMaxDim && E < 65536, MOE355_EUNSUPPORTED);
  if (R == 0 || K == 0 || (offsets && E == 0)) return MOE355_OK;
  MOE355_CHECK(x && (q || qt) && (!q || (scale && sstride_m >= 0 && sstride_kb >= 0)) && (!qt || (tscale && offsets)), MOE355_EINVAL);
  MOE355_CHECK(aligned16(x) && ld_x % 8 == 0 && (!q || (aligned16(q) && ld_q % 8 == 0)) && (!qt || aligned16(qt)) &&
                   (reinterpret_cast<uintptr_t>(tscale) & 1u) == 0 && on4(offsets),
               MOE355_EMISALIGNED);
  const int64_t grid = (offsets ? (int64_t)R / 128 + E : ceil_div64(R, 128)) * ceil_div64(K, 128);
  MOE355_CHECK(grid < (1ll << 24), MOE355_EUNSUPPORTED);
  const RaggedPackArgs g{x, offsets, q, scale, qt, tscale, ld_x, ld_q, sstride_m, sstride_kb, R, E, K};
  hipLaunchKernelGGL((fp16 ? &quant_ragged_kernel<true> : &quant_ragged_kernel<false>), dim3((unsigned)grid), dim3(kThreads), 0,
                     stream, g);
  return launch_status();
}

extern "C" int fp8_quant_128x128(const uint16_t* w, int fp16, int E, int N, int K, uint8_t* q, void* scale, uint8_t* qt,
                                 void* tscale, int e8m0, hipStream_t stream) {
  MOE355_CHECK((fp16 == 0 || fp16 == 1) && (e8m0 == 0 || e8m0 == 1) && E >= 0 && N >= 0 && K >= 0, MOE355_EINVAL);
  MOE355_CHECK(K % 8 == 0 && (!qt || N % 16 == 0) && N <= kMaxDim && K <= kMaxDim, MOE355_EUNSUPPORTED);
  if (E == 0 || N == 0 || K == 0) return MOE355_OK;
  MOE355_CHECK(w && q && scale && (!qt || tscale), MOE355_EINVAL);
  MOE355_CHECK(aligned16(w) && aligned16(q) && (!qt || aligned16(qt)) && (e8m0 || (on4(scale) && on4(tscale))), MOE355_EMISALIGNED);
  const int64_t grid = E * ceil_div64(N, 128) * ceil_div64(K, 128);
  MOE355_CHECK(grid < (1ll << 24), MOE355_EUNSUPPORTED);
  const WeightPackArgs g{w, q, qt, scale, tscale, E, N, K};
  auto* fn = fp16 ? (e8m0 ? &quant_weight_kernel<true, true> : &quant_weight_kernel<true, false>)
                  : (e8m0 ? &quant_weight_kernel<false, true> : &quant_weight_kernel<false, false>);
  hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(kThreads), 0, stream, g);
  return launch_status();
}
