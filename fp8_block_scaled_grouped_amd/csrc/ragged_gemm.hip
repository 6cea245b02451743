// Products grouped by expert over ragged row segments (16-bit operands, fp32 sums)
// and their two gradients.
//
// With C[m, n] = sum_k A(m, k) B(n, k) the three directions are one tiled product:
//   fwd    m = row of the segment, n = output feature, k = input feature
//   dgrad  m = row of the segment, n = input feature,  k = output feature
//   wgrad  m = output feature,     n = input feature,  k = row of the segment
// An operand whose k runs along its rows in memory is staged as BM (or BN) rows of
// 64 k and read as 16-byte fragments; one whose m or n runs along memory rows is
// staged as 64 rows of k and read through the transposing LDS read, so no direction
// needs a transposed copy of anything.
//
// Ragged edges cost no branch in the loop: every LDS-DMA goes through a buffer
// descriptor that ends with the segment's (or matrix's) last valid byte, so rows past it
// arrive as zeros, and lanes whose chunk lies past the row's width are sent past the end.
// Zeros on both operands keep a neighbour expert's infinities and NaN out of the sums.
#include "ragged_gemm.h"

#include <type_traits>

#include "device_common.h"
#include "frag16.h"
#include "gemm_engine.h"
#include "host_common.h"
#include "skinny.h"

namespace moe355 {
namespace {

constexpr int kBK = 64;                      // k per step
// Rotation of the 32-byte column pairs of k-row r in a tile of ROWS columns that is read
// transposed: the 8 k-rows that half a wave touches in one read land in different banks (with 64
// columns, and so 4 pairs a row, in as many as there are).
template <int ROWS>
__device__ __forceinline__ int tr_swz(int r) {
  return ((r & 3) | ((r >> 1) & 4)) & (ROWS / 16 - 1);
}

// One operand of the tile: ROWS rows of m (or n); KMAJOR: k runs along memory rows.
// NW waves fill it with NI DMA instructions each.
template <int ROWS, int NW, bool KMAJOR>
struct Operand {
  static constexpr int kBytes = ROWS * kBK * 2;
  static constexpr int NI = kBytes / 1024 / NW;
  uint32_t off[NI];  // byte offsets of this lane's chunks in a step
  int kc;            // KMAJOR: this lane's k within the step

  __device__ __forceinline__ void init(int w, int lane, int64_t ld, int cols) {
    if constexpr (KMAJOR) {
      const int c = (lane & 7) ^ (lane >> 3);
      kc = 8 * c;
#pragma unroll
      for (int i = 0; i < NI; ++i) off[i] = (uint32_t)((8 * (w * NI + i) + (lane >> 3)) * (ld * 2) + c * 16);
    } else {
      constexpr int CPR = ROWS / 8;  // 16-byte chunks per k-row
      kc = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = (w * NI + i) * (64 / CPR) + lane / CPR;
        const int c = (lane % CPR) ^ (tr_swz<ROWS>(r) << 1);
        off[i] = 8 * c < cols ? (uint32_t)(r * (ld * 2) + c * 16) : kPastEnd;
      }
    }
  }
  // DMA i of a step; past: kPastEnd where this lane's k lies past the end
  __device__ __forceinline__ void dma(int i, u32x4 rsrc, uint32_t lds, int w, uint32_t past) const {
    dma16_buf(rsrc, off[i] | past, lds + (w * NI + i) * 1024);
  }
  // krem: k left from this step's first on
  __device__ __forceinline__ uint32_t past(int krem) const { return KMAJOR && kc >= krem ? kPastEnd : 0u; }
};

// Fragments of 16 rows x 32 k (lane l: row l % 16, k 8 (l / 16) .. + 7) of a staged operand.
template <int ROWS, bool KMAJOR, int T>
struct Fragments {
  uint32_t at[KMAJOR ? 2 : T];  // KMAJOR: per half step; else per fragment

  __device__ __forceinline__ void init(int row0, int lane) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (KMAJOR) {
      at[0] = (row0 + i) * 128 + ((g ^ (i & 7)) << 4);
      at[1] = at[0] ^ 64;
    } else {
      const int r = 8 * g + (i >> 2);
#pragma unroll
      for (int f = 0; f < T; ++f) at[f] = r * (2 * ROWS) + ((((row0 >> 4) + f) ^ tr_swz<ROWS>(r)) << 5) + (i & 3) * 8;
    }
  }
  __device__ __forceinline__ s16x8 read(uint32_t lds, int f, int half) const {
    typedef __attribute__((address_space(3))) s16x8* p8;
    typedef __attribute__((address_space(3))) s16x4* p4;
    if constexpr (KMAJOR) {
      return *reinterpret_cast<p8>(lds + at[half] + f * 2048);
    } else {
      const uint32_t a = lds + at[f] + half * (32 * 2 * ROWS);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<p4>(a));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<p4>(a + 4 * 2 * ROWS));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Row tiles of expert e.
__device__ __forceinline__ int row_tiles(const int32_t* offsets, int R, int e, int BM) {
  int lo, hi;
  segment(offsets, R, e, lo, hi);
  return (hi - lo + BM - 1) / BM;
}

// A workgroup's place: expert, row tile and column tile.  Workgroups go to the 8 XCDs in turn, so
// each XCD takes a contiguous run of the tiles, and inside an expert the tiles advance in
// bands of 8 row tiles: the tiles that an XCD works on at a time share few panels.
template <int BM>
__device__ __forceinline__ bool place(const RaggedArgs& g, int ntiles, int* sh, int& e, int& mt, int& nt) {
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid < 64) {
    const int per = (g.E + 63) / 64;
    const int e0 = min(g.E, lane * per), e1 = min(g.E, e0 + per);
    int mine = 0;
    for (int i = e0; i < e1; ++i) mine += row_tiles(g.offsets, g.R, i, BM);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o, 64);
      if (lane >= o) upto += v;
    }
    const int rows = __shfl(upto, 63, 64);
    const int64_t total = (int64_t)rows * ntiles, chunk = (total + 7) / 8;
    const int64_t t = (int64_t)(blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    if (lane == 0) sh[0] = -1;
    if ((blockIdx.x >> 3) < chunk && t < total) {
      // the lane whose experts hold tile t: tiles before this lane's experts are (upto - mine) * ntiles
      const int64_t first = (int64_t)(upto - mine) * ntiles;
      if (t >= first && t < (int64_t)upto * ntiles) {
        int64_t rest = t - first;
        for (int i = e0; i < e1; ++i) {
          const int m = row_tiles(g.offsets, g.R, i, BM);
          if (rest < (int64_t)m * ntiles) {
            const int band = 8 * ntiles, b0 = (int)(rest / band) * 8, in = (int)(rest % band);
            const int height = min(8, m - b0);
            sh[0] = i;
            sh[1] = b0 + in % height;
            sh[2] = in / height;
            break;
          }
          rest -= (int64_t)m * ntiles;
        }
      }
    }
  }
  __syncthreads();
  e = sh[0];
  mt = sh[1];
  nt = sh[2];
  return e >= 0;
}

template <int OP, bool F16, bool OUT32, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void ragged_gemm_kernel(RaggedArgs g) {
  constexpr bool AK = OP != kRaggedWgrad, BK = OP == kRaggedFwd;  // k along memory rows
  constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
  using OA = Operand<BM, NW, AK>;
  using OB = Operand<BN, NW, BK>;
  constexpr int kSlot = OA::kBytes > OB::kBytes ? OA::kBytes : OB::kBytes;
  __shared__ __align__(16) uint8_t smem[5 * kSlot];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);

  const int mdim = OP == kRaggedWgrad ? g.N : 0, ndim = OP == kRaggedFwd ? g.N : g.K;
  const int ntiles = (ndim + BN - 1) / BN;
  int e, mt, nt, lo, hi;
  if constexpr (OP == kRaggedWgrad) {
    const int mtiles = (mdim + BM - 1) / BM;
    const int64_t total = (int64_t)g.E * mtiles * ntiles, chunk = (total + 7) / 8;
    const int64_t t = (int64_t)(blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= chunk || t >= total) return;
    e = (int)(t / ((int64_t)mtiles * ntiles));
    const int in = (int)(t - (int64_t)e * mtiles * ntiles), band = 8 * ntiles, b0 = in / band * 8;
    const int height = min(8, mtiles - b0);
    mt = b0 + in % band % height;
    nt = in % band / height;
  } else {
    if (!place<BM>(g, ntiles, reinterpret_cast<int*>(smem), e, mt, nt)) return;
    __syncthreads();  // the place has been read: the DMAs may overwrite it
  }
  e = __builtin_amdgcn_readfirstlane(e);
  mt = __builtin_amdgcn_readfirstlane(mt);
  nt = __builtin_amdgcn_readfirstlane(nt);
  segment(g.offsets, g.R, e, lo, hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);

  const int m0 = mt * BM, n0 = nt * BN;
  const int kdim = OP == kRaggedFwd ? g.K : OP == kRaggedDgrad ? g.N : hi - lo;
  const int mrows = OP == kRaggedWgrad ? mdim - m0 : hi - lo - m0;  // m left from the tile's first on
  const int nrows = ndim - n0;

  // first byte of the tile's operands, what a step of 64 k adds, and bytes from there to the end
  const uint16_t* pa = AK ? g.a + (int64_t)(lo + m0) * g.lda : g.a + (int64_t)lo * g.lda + m0;
  const uint16_t* pb = OP == kRaggedFwd     ? g.b + ((int64_t)e * g.N + n0) * g.ldb
                       : OP == kRaggedDgrad ? g.b + (int64_t)e * g.N * g.ldb + n0
                                            : g.b + (int64_t)lo * g.ldb + n0;
  const int64_t stepa = AK ? kBK : kBK * g.lda, stepb = BK ? kBK : kBK * g.ldb;
  int64_t lena = AK ? (min(mrows, BM) - 1) * g.lda + kdim : (kdim - 1) * g.lda + mrows;
  int64_t lenb = BK ? (min(nrows, BN) - 1) * g.ldb + kdim : (kdim - 1) * g.ldb + nrows;

  OA oa;
  OB ob;
  oa.init(w, lane, g.lda, mrows);
  ob.init(w, lane, g.ldb, nrows);
  Fragments<BM, AK, TM> fa;
  Fragments<BN, BK, TN> fb;
  fa.init((w / WN) * (BM / WM), lane);
  fb.init((w % WN) * (BN / WN), lane);
  const uint32_t lds0 = lds_addr(smem);

  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // 16-row tiles of this wave that hold rows of the segment: a last, partial tile multiplies no more
  const int live = min(TM, (mrows - (w / WN) * (BM / WM) + 15) / 16);
  const int steps = (kdim + kBK - 1) / kBK;
  // The operands of the steps, A(0) B(0) A(1) B(1) .., take the slots of a ring of five in turn.  Past the
  // last step the descriptors have no length (zeros, no traffic).
  u32x4 da, db;
  uint32_t pasta, pastb;
  int ka = 0, kb = 0;  // first k of the next A and B
  auto next_a = [&] {
    da = dma_buffer(pa, ka < kdim ? lena * 2 : 0);
    pasta = oa.past(kdim - ka);
    pa += stepa;
    lena -= stepa;
    ka += kBK;
  };
  auto next_b = [&] {
    db = dma_buffer(pb, kb < kdim ? lenb * 2 : 0);
    pastb = ob.past(kdim - kb);
    pb += stepb;
    lenb -= stepb;
    kb += kBK;
  };
  auto fetch = [&](uint32_t slot_a, uint32_t slot_b) {
    next_a();
#pragma unroll
    for (int i = 0; i < OA::NI; ++i) oa.dma(i, da, slot_a, w, pasta);
    next_b();
#pragma unroll
    for (int i = 0; i < OB::NI; ++i) ob.dma(i, db, slot_b, w, pastb);
  };
  s16x8 ra[2][TM], rb[2][TN];
  // The MFMAs of half a step, and spread between them the fragment reads of the next half and the DMAs of
  // one operand (the first half A's, the second B's).  DMAs in a burst cost: with all 8 at the start of
  // one half the product of 65536 rows over 32 experts of 4096 x 7168 took 3.76 ms, spread over that
  // half 3.46, over both 3.32.
  auto half_step = [&](auto half_c, uint32_t read_a, uint32_t read_b, uint32_t fill) {
    constexpr int kHalf = decltype(half_c)::value, kNext = 1 - kHalf;
    constexpr int kCount = kHalf == 0 ? OA::NI : OB::NI, kDmas = (kCount + TM - 1) / TM;
    // reads a row of MFMAs: all are on their way after half of the rows (transposed ones, of two
    // instructions each, after three quarters: dgrad 3.36 ms against 3.43, wgrad 3.35 against 3.44, while fwd
    // went from 3.22 to 3.29)
    constexpr int kReads = OP == kRaggedFwd ? (2 * (TM + TN) + TM - 1) / TM : (4 * (TM + TN) + 3 * TM - 1) / (3 * TM);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int d = 0; d < kDmas; ++d) {
        if (i * kDmas + d >= kCount) break;
        if constexpr (kHalf == 0) {
          oa.dma(i * kDmas + d, da, fill, w, pasta);
        } else {
          ob.dma(i * kDmas + d, db, fill, w, pastb);
        }
      }
#pragma unroll
      for (int d = 0; d < kReads; ++d) {
        const int f = i * kReads + d;
        if (f < TN) {
          rb[kNext][f] = fb.read(read_b, f, kNext);
        } else if (f < TN + TM) {
          ra[kNext][f - TN] = fa.read(read_a, f - TN, kNext);
        }
      }
      if (i < live) {
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mfma16x16x32<F16>(rb[kHalf][j], ra[kHalf][i], acc[i][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  if (steps > 0) {
    uint32_t a0 = lds0, b0 = a0 + kSlot, a1 = b0 + kSlot, b1 = a1 + kSlot, a2 = b1 + kSlot;
    fetch(a0, b0);
    fetch(a1, b1);
    vm_wait<OA::NI + OB::NI>();
    barrier_only();
#pragma unroll
    for (int i = 0; i < TM; ++i) ra[0][i] = fa.read(a0, i, 0);
#pragma unroll
    for (int j = 0; j < TN; ++j) rb[0][j] = fb.read(b0, j, 0);
    lgkm_wait0();
    for (int s = 0; s < steps; ++s) {
      // first half: its fragments are in registers; A(s + 2) follows into its slot
      next_a();
      half_step(std::integral_constant<int, 0>{}, a0, b0, a2);
      lgkm_wait0();
      vm_wait<OA::NI>();  // this wave's share of step s + 1 has landed (that A(s + 2) may be under way)
      barrier_only();     // everyone's has, and nobody reads a0 and b0 any more: B(s + 2), then A(s + 3)
      next_b();
      half_step(std::integral_constant<int, 1>{}, a1, b1, a0);  // reads of the step after the last: not used
      lgkm_wait0();
      const uint32_t was_a = a0, was_b = b0;
      a0 = a1;
      b0 = b1;
      a1 = a2;
      b1 = was_a;
      a2 = was_b;
    }
    vm_wait<0>();
  }

  // lane: row m of the tile, four adjacent n
  const int nw = (w % WN) * (BN / WN) + 4 * (lane >> 4);
  const int64_t row0 = (OP == kRaggedWgrad ? (int64_t)e * g.N : (int64_t)lo) + m0;
  if constexpr (OUT32 && TN % 2 == 0) {
    // pairs of column tiles exchange halves between lanes l and l ^ 8, so that a store covers 8 rows of
    // 128 bytes rather than 16 rows of 64 (16384 rows over 32 experts of 4096 x 2048: 424 us against 437)
    const bool up = lane & 8;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int j = 0; j < TN; j += 2) {
        v4f first, second;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x = up ? acc[i][j][k] : acc[i][j + 1][k];
          const float y = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128, 0xf, 0xf, true));
          first[k] = up ? y : acc[i][j][k];
          second[k] = up ? acc[i][j + 1][k] : y;
        }
        const int n = nw + 16 * (j + (up ? 1 : 0));
        if (n >= nrows) continue;
        const int m = (w / WN) * (BM / WM) + 16 * i + (lane & 7);
        float* out = reinterpret_cast<float*>(g.c) + (row0 + m) * g.ldc + n0 + n;
        if (m < mrows) *reinterpret_cast<v4f*>(out) = first;
        if (m + 8 < mrows) *reinterpret_cast<v4f*>(out + 8 * g.ldc) = second;
      }
    }
  } else {
    const int mw = (w / WN) * (BM / WM) + (lane & 15);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = mw + 16 * i;
      if (m >= mrows) continue;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int n = nw + 16 * j;
        if (n >= nrows) continue;  // nrows % 8 == 0: the four are all in or all out
        const int64_t at = (row0 + m) * g.ldc + n0 + n;
        if constexpr (OUT32) {
          *reinterpret_cast<v4f*>(reinterpret_cast<float*>(g.c) + at) = acc[i][j];
        } else {
          const uint2 r{f32_to_out16(acc[i][j][0], F16) | (f32_to_out16(acc[i][j][1], F16) << 16),
                        f32_to_out16(acc[i][j][2], F16) | (f32_to_out16(acc[i][j][3], F16) << 16)};
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(g.c) + at) = r;
        }
      }
    }
  }
}

template <int OP, bool F16, bool OUT32, int BM, int BN, int WM, int WN>
int launch(const RaggedArgs& g, hipStream_t stream) {
  auto* fn = &ragged_gemm_kernel<OP, F16, OUT32, BM, BN, WM, WN>;
  const int64_t nt = ceil_div64(OP == kRaggedFwd ? g.N : g.K, BN);
  // an upper bound of the row tiles: the offsets are on the device
  const int64_t mt = OP == kRaggedWgrad ? (int64_t)g.E * ceil_div64(g.N, BM)
                                        : g.R / BM + (g.E < g.R ? g.E : g.R);
  const int64_t grid = ceil_div64(mt * nt, 8) * 8;
  MOE355_CHECK(grid * (64 * WM * WN) < (1ll << 32), MOE355_EUNSUPPORTED);  // threads of a launch
  hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(64 * WM * WN), 0, stream, g);
  return launch_status();
}

// The tile: 256 x 256 where it makes enough work for the CUs, else 128 x 128, else 64 x 64.  The
// offsets are on the device, so the number of row tiles is a guess: half a tile more per expert.
// Measured, us with tiles of 256 / 128 / 64:
//   fwd   32 experts of 4096 x 2048, 160 rows each on average 167 / 180 / 216, 64 rows 154 / 140 / 145;
//         2 experts of 2000 x 2000, 500 rows 55 / 29 / 22
//   dgrad the same 123 / 154 / 192, 110 / 103 / 154; 55 / 28 / 22
//   wgrad 8 experts of 1536 x 1536, 750 rows 58 / 47 / 58; 64 of 1024 x 1024, 128 rows 59 / 65 / 79
// The waves stand 4 x 2 in a tile of 256: 8 waves of 128 x 64 (2 x 4) took 3.48 ms where 64 x 128 take
// 3.39 (32 experts of 4096 x 7168, 65536 rows), 4 waves of 128 x 128 3.52.
template <int OP, bool OUT32, bool F16>
int run_type(const RaggedArgs& g, hipStream_t stream) {
  const int64_t cols = OP == kRaggedFwd ? g.N : g.K, parts = g.E < g.R ? g.E : g.R;
  auto tiles = [&](int64_t t) {
    return OP == kRaggedWgrad ? g.E * ceil_div64(g.N, t) * ceil_div64(g.K, t)
                              : (g.R / t + (parts + 1) / 2) * ceil_div64(cols, t);
  };
  if (OP == kRaggedWgrad ? tiles(256) >= 512 : tiles(256) >= 200 && g.R >= 112ll * g.E)
    return launch<OP, F16, OUT32, 256, 256, 4, 2>(g, stream);
  if (tiles(128) >= 192) return launch<OP, F16, OUT32, 128, 128, 4, 2>(g, stream);
  return launch<OP, F16, OUT32, 64, 64, 2, 2>(g, stream);
}

template <int OP, bool OUT32 = false>
int run(const RaggedArgs& g, int f16, hipStream_t stream) {
  return f16 ? run_type<OP, OUT32, true>(g, stream) : run_type<OP, OUT32, false>(g, stream);
}

bool aligned_rows(const void* p, int64_t ld) { return aligned16(p) && ld % 8 == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks the arguments that the three calls share.
int check(int fp16, int R, int E, int N, int K) {
  MOE355_CHECK((fp16 == 0 || fp16 == 1) && R >= 0 && E >= 0 && N >= 0 && K >= 0, MOE355_EINVAL);
  MOE355_CHECK(N % 8 == 0 && K % 8 == 0 && E < 65536, MOE355_EUNSUPPORTED);
  return MOE355_OK;
}

constexpr int64_t kMaxLd = 1 << 21;  // 256 rows' byte offsets stay below 2^31

}  // namespace
}  // namespace moe355

using namespace moe355;

extern "C" int grouped_gemm(const uint16_t* x, int fp16, int64_t ld_x, const uint16_t* w, const int32_t* offsets, int R,
                            int E, int N, int K, uint16_t* y, int64_t ld_y, hipStream_t stream) {
  if (int st = check(fp16, R, E, N, K)) return st;
  MOE355_CHECK(ld_x >= K && ld_y >= N, MOE355_EINVAL);
  MOE355_CHECK(ld_x <= kMaxLd && ld_y <= kMaxLd, MOE355_EUNSUPPORTED);
  if (R == 0 || E == 0 || N == 0) return MOE355_OK;
  MOE355_CHECK(offsets && y && (K == 0 || (x && w)), MOE355_EINVAL);
  MOE355_CHECK((K == 0 || (aligned_rows(x, ld_x) && aligned16(w))) && aligned_rows(y, ld_y) && aligned4(offsets), MOE355_EMISALIGNED);
  // few rows an expert: the weights' bytes bound it (32 experts of 4096 x 2048, 4 rows each: 97 us against
  // 124 with the best tile; 32 rows 133 both, and an expert with more rows than most costs less there)
  if (R <= 8ll * E && K > 0)
    return launch_skinny(SkinnyArgs{x, reinterpret_cast<const uint8_t*>(w), nullptr, offsets, y, ld_x, ld_y, R, E, N, K,
                                    1, nullptr},
                         kW16, 128, fp16, stream);
  return run<kRaggedFwd>(RaggedArgs{x, w, y, offsets, ld_x, K, ld_y, R, E, N, K}, fp16, stream);
}

extern "C" int grouped_gemm_dgrad(const uint16_t* dy, int fp16, int64_t ld_dy, const uint16_t* w,
                                  const int32_t* offsets, int R, int E, int N, int K, uint16_t* dx, int64_t ld_dx,
                                  hipStream_t stream) {
  if (int st = check(fp16, R, E, N, K)) return st;
  MOE355_CHECK(ld_dy >= N && ld_dx >= K, MOE355_EINVAL);
  MOE355_CHECK(ld_dy <= kMaxLd && ld_dx <= kMaxLd, MOE355_EUNSUPPORTED);
  if (R == 0 || E == 0 || K == 0) return MOE355_OK;
  MOE355_CHECK(offsets && dx && (N == 0 || (dy && w)), MOE355_EINVAL);
  MOE355_CHECK((N == 0 || (aligned_rows(dy, ld_dy) && aligned16(w))) && aligned_rows(dx, ld_dx) && aligned4(offsets), MOE355_EMISALIGNED);
  return run<kRaggedDgrad>(RaggedArgs{dy, w, dx, offsets, ld_dy, K, ld_dx, R, E, N, K}, fp16, stream);
}

extern "C" int grouped_gemm_wgrad(const uint16_t* dy, int fp16, int64_t ld_dy, const uint16_t* x, int64_t ld_x,
                                  const int32_t* offsets, int R, int E, int N, int K, void* dw, int out_fp32,
                                  hipStream_t stream) {
  if (int st = check(fp16, R, E, N, K)) return st;
  MOE355_CHECK((out_fp32 == 0 || out_fp32 == 1) && ld_dy >= N && ld_x >= K, MOE355_EINVAL);
  MOE355_CHECK(ld_dy <= kMaxLd && ld_x <= kMaxLd, MOE355_EUNSUPPORTED);
  if (E == 0 || N == 0 || K == 0) return MOE355_OK;  // without rows every gradient is zero: still written
  MOE355_CHECK(offsets && dw && (R == 0 || (dy && x)), MOE355_EINVAL);
  MOE355_CHECK((R == 0 || (aligned_rows(dy, ld_dy) && aligned_rows(x, ld_x))) && aligned16(dw) && aligned4(offsets), MOE355_EMISALIGNED);
  const RaggedArgs g{dy, x, dw, offsets, ld_dy, ld_x, K, R, E, N, K};
  return out_fp32 ? run<kRaggedWgrad, true>(g, fp16, stream) : run<kRaggedWgrad>(g, fp16, stream);
}
