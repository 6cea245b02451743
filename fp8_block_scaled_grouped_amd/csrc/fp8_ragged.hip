// FP8 (e4m3) expert products over ragged row segments with a scale for each block of 128, and the
// product over the rows that gives the weights' gradient.
//
//   fwd    y[r, n]     = sum_kb sx[r, kb] sw[e, n / 128, kb] sum_{k in kb} x[r, k] w[e, n, k]
//   wgrad  dw[e, n, k] = sum_b sdy[b, n] sx[b, k] sum_{r in block b of e} dy[r, n] x[r, k]
//
// (the gradient for x is fwd on dy and the transposed weights.)  Both are one tiled product
// C[m, n] = sum_s sa(m, s) sb(n, s) <A_s(m), B_s(n)> whose step s is a block of 128 codes: fwd's lie along the
// rows of x and w, wgrad's in the transposed blocks [b][column][128] that fp8_quant_ragged writes, zeros past the segment's end.
// A step is one 16x16x128 MFMA a 16 x 16 tile.  With power-of-two scales the MFMA applies them and adds to the fp32 sums; with
// fp32 scales its result is folded in, acc += t * (sa * sb).
//
// Ragged edges cost no branch in the loop: every LDS-DMA goes through a buffer descriptor that ends with
// the operand's last valid byte, so rows past it arrive as zeros, and lanes whose chunk lies past the row's
// width are sent past the end.
#include <type_traits>

#include "device_common.h"
#include "frag16.h"
#include "gemm_engine.h"
#include "host_common.h"
#include "ragged_tile.h"

namespace moe355 {
namespace {

enum Fp8Op : int { kFp8Fwd = 0, kFp8Wgrad = 1 };

struct Fp8Args {
  const uint8_t* a;        // fwd: x [R, K]; wgrad: dy [blocks, N, 128]
  const uint8_t* b;        // fwd: w [E, N, K]; wgrad: x [blocks, K, 128]
  const void* sa;          // fwd: (r, kb) at r * ssm + kb * sskb; wgrad: [blocks, N]
  const void* sb;          // fwd: [E, ceil(N / 128), ceil(K / 128)]; wgrad: [blocks, K]
  void* c;                 // fwd: y [R, N]; wgrad: dw [E, N, K]
  const int32_t* offsets;  // [E + 1] on the device
  int64_t lda, ldc, ssm, sskb;
  int R, E, N, K;
  int f16;                 // 16-bit outputs: fp16 or bf16
};

// One operand of a step: ROWS rows of 128 codes, chunk c of row r in slot c ^ (r & 7), filled by NW waves with NI DMAs each.
template <int ROWS, int NW>
struct Operand8 {
  static constexpr int kBytes = ROWS * 128;
  static constexpr int NI = kBytes / 1024 / NW;
  static_assert(NI * NW * 1024 == kBytes, "whole DMAs");
  uint32_t off[NI];
  int kc;  // this lane's k within the step

  __device__ __forceinline__ void init(int w, int lane, int64_t ld) {
    const int c = (lane & 7) ^ (lane >> 3);
    kc = 16 * c;
#pragma unroll
    for (int i = 0; i < NI; ++i) off[i] = (uint32_t)((8 * (w * NI + i) + (lane >> 3)) * ld + kc);
  }
  __device__ __forceinline__ void dma(int i, u32x4 rsrc, uint32_t lds, int w, uint32_t past) const {
    dma16_buf(rsrc, off[i] | past, lds + (w * NI + i) * 1024);
  }
  __device__ __forceinline__ uint32_t past(int krem) const { return kc >= krem ? kPastEnd : 0u; }
};

// Fragment f (16 rows) of a staged operand: lane l row l % 16, chunks l / 16 and l / 16 + 4.  `at` is the lane's place in fragment 0.
__device__ __forceinline__ uint32_t frag_at(int row0, int lane) {
  return (row0 + (lane & 15)) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
}
__device__ __forceinline__ v8i read_frag(uint32_t lds, uint32_t at, int f) {
  typedef __attribute__((address_space(3))) u32x4* p;
  const u32x4 lo = *reinterpret_cast<p>(lds + at + f * 2048);
  const u32x4 hi = *reinterpret_cast<p>(lds + (at ^ 64) + f * 2048);
  return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Lane l's values of 16 T rows (row l % (16 T)) -> for each tile of 16 rows that of row l % 16, in every lane.
template <int T>
__device__ __forceinline__ void spread(uint32_t v, uint32_t (&s)[T]) {
  static_assert(T == 1 || T == 2 || T == 4, "tiles of a wave");
  if constexpr (T == 1) {
    s[0] = v;
  } else if constexpr (T == 2) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    s[0] = r[0];
    s[1] = r[1];
  } else {
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    s[0] = lo[0];
    s[1] = lo[1];
    s[2] = hi[0];
    s[3] = hi[1];
  }
}

// D = A B scaled by 2^(sa - 127) 2^(sb - 127) for each row of A and column of B, + C
__device__ __forceinline__ v4f mfma_scaled(const v8i& a, const v8i& b, const v4f& c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, (int)sa, 0, (int)sb);
}

// E8: power-of-two scales (bytes), else fp32 ones.  Waves stand WM x WN, each with TM x TN tiles of 16 x 16.
// A step reads the wave's TM fragments of A once, ahead of it, and streams the TN fragments of B kAhead ahead.  In the
// middle of step s a wait and a barrier publish the operands of step s + 1; at that point A(s) (in registers since step s - 1)
// and B(s - 1) are done with, so their slots take step s + 2: two slots of A and three of B.
template <int OP, bool E8, bool OUT32, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_ragged_kernel(Fp8Args g) {
  constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr int kAhead = 1, kHold = 2;  // fragments of B ahead, and held
  using OA = Operand8<BM, NW>;
  using OB = Operand8<BN, NW>;
  __shared__ __align__(16) uint8_t smem[2 * OA::kBytes + 3 * OB::kBytes];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (w / WN) * (BM / WM), wn = (w % WN) * (BN / WN);

  const int ndim = OP == kFp8Fwd ? g.N : g.K, ntiles = (ndim + BN - 1) / BN;
  int e, mt, nt, lo, hi;
  if constexpr (OP == kFp8Wgrad) {
    const int mtiles = (g.N + BM - 1) / BM;
    const int64_t total = (int64_t)g.E * mtiles * ntiles, chunk = (total + 7) / 8;
    const int64_t t = (int64_t)(blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= chunk || t >= total) return;
    e = (int)(t / ((int64_t)mtiles * ntiles));
    const int in = (int)(t - (int64_t)e * mtiles * ntiles), band = 8 * ntiles, b0 = in / band * 8;
    const int height = min(8, mtiles - b0);
    mt = b0 + in % band % height;
    nt = in % band / height;
  } else {
    if (!place<BM>(g.offsets, g.R, g.E, ntiles, reinterpret_cast<int*>(smem), e, mt, nt)) return;
    __syncthreads();  // the place has been read: the DMAs may overwrite it
  }
  e = __builtin_amdgcn_readfirstlane(e);
  mt = __builtin_amdgcn_readfirstlane(mt);
  nt = __builtin_amdgcn_readfirstlane(nt);
  segment(g.offsets, g.R, e, lo, hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);

  const int m0 = mt * BM, n0 = nt * BN;
  const int kdim = OP == kFp8Fwd ? g.K : (hi - lo + 127) / 128 * 128;
  const int steps = (kdim + 127) / 128;
  const int mrows = OP == kFp8Wgrad ? g.N - m0 : hi - lo - m0;  // m left from the tile's first on
  const int nrows = ndim - n0;
  const int64_t block0 = lo / 128 + e;  // wgrad: the segment's first block

  // first byte of the tile's operands, what a step adds, and bytes from there to the end
  const int64_t lda = OP == kFp8Fwd ? g.lda : 128, ldb = OP == kFp8Fwd ? g.K : 128;
  const uint8_t* pa = OP == kFp8Fwd ? g.a + (int64_t)(lo + m0) * lda : g.a + (block0 * g.N + m0) * 128;
  const uint8_t* pb = OP == kFp8Fwd ? g.b + ((int64_t)e * g.N + n0) * ldb : g.b + (block0 * g.K + n0) * 128;
  const int64_t stepa = OP == kFp8Fwd ? 128 : (int64_t)g.N * 128, stepb = OP == kFp8Fwd ? 128 : (int64_t)g.K * 128;
  int64_t lena = (min(mrows, BM) - 1) * lda + (OP == kFp8Fwd ? kdim : 128);
  int64_t lenb = (min(nrows, BN) - 1) * ldb + (OP == kFp8Fwd ? kdim : 128);

  OA oa;
  OB ob;
  oa.init(w, lane, lda);
  ob.init(w, lane, ldb);
  const uint32_t ata = frag_at(wm, lane), atb = frag_at(wn, lane);
  const uint32_t lds0 = lds_addr(smem);

  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // scales of a step: this lane's row of A (its last valid one past the end) and, wgrad, its columns of B
  constexpr int kSB = OP == kFp8Wgrad ? (TN + 3) / 4 : 1;
  const int arow = min(wm + lane % (16 * TM), mrows - 1);
  const int64_t sa0 = OP == kFp8Fwd ? (int64_t)(lo + m0 + arow) * g.ssm : block0 * g.N + m0 + arow;
  const int64_t sastep = OP == kFp8Fwd ? g.sskb : g.N;
  int64_t sb0[kSB];
  if constexpr (OP == kFp8Wgrad) {
#pragma unroll
    for (int q = 0; q < kSB; ++q) sb0[q] = block0 * g.K + n0 + min(wn + 64 * q + lane % (16 * min(TN, 4)), nrows - 1);
  } else {
    const int KB = (g.K + 127) / 128;
    sb0[0] = ((int64_t)e * ((g.N + 127) / 128) + (n0 + wn < g.N ? n0 + wn : n0) / 128) * KB;
  }
  auto scale_at = [&](const void* p, int64_t i) {
    if constexpr (E8) return (uint32_t) static_cast<const uint8_t*>(p)[i];
    else return static_cast<const uint32_t*>(p)[i];
  };
  auto scale_a = [&](int s) { return scale_at(g.sa, sa0 + min(s, steps - 1) * sastep); };
  auto scale_b = [&](int s, int q) {
    const int t = min(s, steps - 1);
    return scale_at(g.sb, OP == kFp8Wgrad ? sb0[q] + (int64_t)t * g.K : sb0[q] + t);
  };

  u32x4 da, db;
  uint32_t pasta, pastb;
  int ka = 0, kb = 0;  // first k of the next A and B
  auto next_a = [&] {
    da = dma_buffer(pa, ka < kdim ? lena : 0);
    pasta = OP == kFp8Fwd ? oa.past(kdim - ka) : 0;
    pa += stepa;
    if (OP == kFp8Fwd) lena -= 128;
    ka += 128;
  };
  auto next_b = [&] {
    db = dma_buffer(pb, kb < kdim ? lenb : 0);
    pastb = OP == kFp8Fwd ? ob.past(kdim - kb) : 0;
    pb += stepb;
    if (OP == kFp8Fwd) lenb -= 128;
    kb += 128;
  };

  if (steps > 0) {
    uint32_t rawa[2] = {scale_a(0), scale_a(1)}, rawb[2][kSB];
#pragma unroll
    for (int q = 0; q < kSB; ++q) {
      rawb[0][q] = scale_b(0, q);
      rawb[1][q] = scale_b(1, q);
    }
    uint32_t b0 = lds0 + 2 * OA::kBytes, b1 = b0 + OB::kBytes, b2 = b1 + OB::kBytes;
    vm_wait<0>();
    next_a();
#pragma unroll
    for (int i = 0; i < OA::NI; ++i) oa.dma(i, da, lds0, w, pasta);
    next_b();
#pragma unroll
    for (int i = 0; i < OB::NI; ++i) ob.dma(i, db, b0, w, pastb);
    next_a();
#pragma unroll
    for (int i = 0; i < OA::NI; ++i) oa.dma(i, da, lds0 + OA::kBytes, w, pasta);
    next_b();
#pragma unroll
    for (int i = 0; i < OB::NI; ++i) ob.dma(i, db, b1, w, pastb);
    vm_wait<OA::NI + OB::NI>();
    barrier_only();
    v8i ra[2][TM], rb[kHold];
#pragma unroll
    for (int i = 0; i < TM; ++i) ra[0][i] = read_frag(lds0, ata, i);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) rb[j] = read_frag(b0, atb, j);

    auto step = [&](int s, auto par_c) {
      constexpr int PAR = decltype(par_c)::value;
      const uint32_t acur = lds0 + PAR * OA::kBytes, anext = lds0 + (PAR ^ 1) * OA::kBytes;
      uint32_t sa[TM], sb[kSB][TN < 4 ? TN : 4];
      spread<TM>(rawa[0], sa);
      if constexpr (OP == kFp8Wgrad) {
#pragma unroll
        for (int q = 0; q < kSB; ++q) spread<(TN < 4 ? TN : 4)>(rawb[0][q], sb[q]);
      }
      float f[TM];
      if constexpr (!E8) {
#pragma unroll
        for (int i = 0; i < TM; ++i) f[i] = __uint_as_float(sa[i]) * __uint_as_float(rawb[0][0]);
      }
      const uint32_t sbu = rawb[0][0];
      v4f t[3];
      constexpr int kHalf = TN / 2;
      constexpr int kDmas = (OA::NI + OB::NI + kHalf - 1) / kHalf, kReads = (TM + kHalf - 1) / kHalf;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        if (j == kHalf) {
          vm_wait<0>();    // this wave's share of step s + 1 has landed, and its scales
          barrier_only();  // everyone's has, and nobody reads A(s) and B(s - 1) any more
          rawa[0] = rawa[1];
          rawa[1] = scale_a(s + 2);
#pragma unroll
          for (int q = 0; q < kSB; ++q) {
            rawb[0][q] = rawb[1][q];
            rawb[1][q] = scale_b(s + 2, q);
          }
          next_a();
          next_b();
        }
        if (j + kAhead < TN) rb[(j + kAhead) % kHold] = read_frag(b0, atb, j + kAhead);
        else rb[(j + kAhead) % kHold] = read_frag(b1, atb, j + kAhead - TN);
        if (j >= kHalf) {
#pragma unroll
          for (int d = (j - kHalf) * kReads; d < (j - kHalf + 1) * kReads && d < TM; ++d) ra[PAR ^ 1][d] = read_frag(anext, ata, d);
#pragma unroll
          for (int d = (j - kHalf) * kDmas; d < (j - kHalf + 1) * kDmas; ++d) {
            if (d < OA::NI) oa.dma(d, da, acur, w, pasta);
            else if (d < OA::NI + OB::NI) ob.dma(d - OA::NI, db, b2, w, pastb);
          }
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          if constexpr (E8) {
            acc[i][j] = mfma_scaled(rb[j % kHold], ra[PAR][i], acc[i][j], OP == kFp8Wgrad ? sb[j / 4][j % 4] : sbu, sa[i]);
          } else {
            // the fold of the tile before the last follows each MFMA
            const int q = j * TM + i;
            t[q % 3] = mfma16x16x128_fp8(rb[j % kHold], ra[PAR][i], v4f{0.f, 0.f, 0.f, 0.f});
            if (q >= 2) {
              const int p = q - 2;
              acc[p % TM][p / TM] += t[p % 3] * f[p % TM];
            }
          }
          if constexpr (!E8) __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (!E8) {
#pragma unroll
        for (int p = TM * TN - 2; p < TM * TN; ++p) acc[p % TM][p / TM] += t[p % 3] * f[p % TM];
      }
      const uint32_t was = b0;
      b0 = b1;
      b1 = b2;
      b2 = was;
    };
    int s = 0;
    for (; s + 1 < steps; s += 2) {
      step(s, std::integral_constant<int, 0>{});
      step(s + 1, std::integral_constant<int, 1>{});
    }
    if (s < steps) step(s, std::integral_constant<int, 0>{});
    vm_wait<0>();
  }

  const int64_t row0 = (OP == kFp8Wgrad ? (int64_t)e * g.N : (int64_t)lo) + m0;
  if (OUT32 || !g.f16) {
    store_tile<false, OUT32>(acc, g.c, g.ldc, row0, n0, mrows, nrows, wm, wn, lane);
  } else {
    store_tile<true, false>(acc, g.c, g.ldc, row0, n0, mrows, nrows, wm, wn, lane);
  }
}

template <int OP, bool E8, bool OUT32, int BM, int BN, int WM, int WN>
int launch(const Fp8Args& g, hipStream_t stream) {
  auto* fn = &fp8_ragged_kernel<OP, E8, OUT32, BM, BN, WM, WN>;
  const int64_t nt = ceil_div64(OP == kFp8Fwd ? g.N : g.K, BN);
  // an upper bound of the row tiles: the offsets are on the device
  const int64_t mt = OP == kFp8Wgrad ? (int64_t)g.E * ceil_div64(g.N, BM) : g.R / BM + (g.E < g.R ? g.E : g.R);
  const int64_t grid = ceil_div64(mt * nt, 8) * 8;
  MOE355_CHECK(grid * (64 * WM * WN) < (1ll << 32), MOE355_EUNSUPPORTED);  // threads of a launch
  hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(64 * WM * WN), 0, stream, g);
  return launch_status();
}

// The tile: 256 x 256 where it makes enough work for the CUs, else 128 x 128, else 64 x 64.  The
// offsets are on the device, so the number of row tiles is a guess: half a tile more per expert.
template <int OP, bool E8, bool OUT32>
int run(const Fp8Args& g, hipStream_t stream) {
  const int64_t cols = OP == kFp8Fwd ? g.N : g.K, parts = g.E < g.R ? g.E : g.R;
  auto tiles = [&](int64_t t) {
    return OP == kFp8Wgrad ? g.E * ceil_div64(g.N, t) * ceil_div64(g.K, t) : (g.R / t + (parts + 1) / 2) * ceil_div64(cols, t);
  };
  if (OP == kFp8Wgrad ? tiles(256) >= 512 : tiles(256) >= 200 && g.R >= 112ll * g.E)
    return launch<OP, E8, OUT32, 256, 256, 4, 2>(g, stream);
  if (tiles(128) >= 192) return launch<OP, E8, OUT32, 128, 128, 4, 2>(g, stream);
  return launch<OP, E8, OUT32, 64, 64, 4, 1>(g, stream);
}

bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kMaxLd = 1 << 22;    // 256 rows' byte offsets stay below 2^31
constexpr int kMaxDim = 1 << 22;

}  // namespace
}  // namespace moe355

using namespace moe355;

extern "C" int grouped_gemm_fp8(const uint8_t* x8, const void* x_scale, int64_t ld_x, int64_t sstride_m, int64_t sstride_kb,
                                const uint8_t* w8, const void* w_scale, int e8m0, const int32_t* offsets, int R, int E, int N,
                                int K, uint16_t* y, int64_t ld_y, int fp16, hipStream_t stream) {
  MOE355_CHECK((fp16 == 0 || fp16 == 1) && (e8m0 == 0 || e8m0 == 1) && R >= 0 && E >= 0 && N >= 0 && K >= 0 && ld_x >= K &&
                   ld_y >= N && sstride_m >= 0 && sstride_kb >= 0,
               MOE355_EINVAL);
  MOE355_CHECK(N % 8 == 0 && K % 16 == 0 && N <= kMaxDim && E < 65536 && ld_x <= kMaxLd && ld_y <= (1ll << 40), MOE355_EUNSUPPORTED);
  if (R == 0 || E == 0 || N == 0) return MOE355_OK;
  MOE355_CHECK(offsets && y && (K == 0 || (x8 && w8 && x_scale && w_scale)), MOE355_EINVAL);
  MOE355_CHECK((K == 0 || (aligned16(x8) && ld_x % 16 == 0 && aligned16(w8))) && aligned16(y) && ld_y % 8 == 0 && on4(offsets) &&
                   (e8m0 || (on4(x_scale) && on4(w_scale))),
               MOE355_EMISALIGNED);
  const Fp8Args g{x8, w8, x_scale, w_scale, y, offsets, ld_x, ld_y, sstride_m, sstride_kb, R, E, N, K, fp16};
  return e8m0 ? run<kFp8Fwd, true, false>(g, stream) : run<kFp8Fwd, false, false>(g, stream);
}

extern "C" int grouped_gemm_fp8_wgrad(const uint8_t* dyt, const uint8_t* dyt_scale, const uint8_t* xt, const uint8_t* xt_scale,
                                      const int32_t* offsets, int R, int E, int N, int K, void* dw, int out, hipStream_t stream) {
  MOE355_CHECK(R >= 0 && E >= 0 && N >= 0 && K >= 0 && out >= MOE355_BF16 && out <= MOE355_F32, MOE355_EINVAL);
  MOE355_CHECK(N % 8 == 0 && K % 8 == 0 && N <= kMaxDim && K <= kMaxDim && E < 65536, MOE355_EUNSUPPORTED);
  if (E == 0 || N == 0 || K == 0) return MOE355_OK;  // without rows every gradient is zero: still written
  MOE355_CHECK(offsets && dw && (R == 0 || (dyt && dyt_scale && xt && xt_scale)), MOE355_EINVAL);
  MOE355_CHECK((R == 0 || (aligned16(dyt) && aligned16(xt))) && aligned16(dw) && on4(offsets), MOE355_EMISALIGNED);
  const Fp8Args g{dyt, xt, dyt_scale, xt_scale, dw, offsets, 128, K, 0, 0, R, E, N, K, out == MOE355_F16};
  return out == MOE355_F32 ? run<kFp8Wgrad, true, true>(g, stream) : run<kFp8Wgrad, true, false>(g, stream);
}
