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
// fp32 scales its result is folded in, acc += t * (sa * sb): the scales' product first, so one below 2^-126 is rounded to a multiple of
// 2^-149 and its block off by less than 2^-125.  (Both scales' powers of two applied by the MFMA instead, and the rests folded, would
// hold over all of fp32, and takes 5% longer: 1.70 ms against 1.60 below.)
//
// Ragged edges cost no branch in the loop: every LDS-DMA goes through a buffer descriptor that ends with
// the operand's last valid byte, so rows past it arrive as zeros, and lanes whose chunk lies past the row's
// width are sent past the end; stores past the segment go past the end of one as well.
//
// The unit adds products eight at a time: eight that lie side by side along k are each cut toward zero to 13 bits below the largest
// exponent among them, and their sums are fp32.  So a product below 2^-13 of the largest of its eight may be lost.
//
// What bounds it: the clock that the card's power leaves, 1.6 GHz under this load, at which the matrix unit is busy 71% of the time
// (62% with fp32 scales, whose folds are four VALU instructions an MFMA).  A 256 x 256 step brings 64 KB of operands into LDS for 16.8 MFLOP
// and its waves read 192 KB of fragments back; of an earlier form's 1.48 ms (below) 1.20 remained without the DMAs and 1.49 without
// the MFMAs.  65536 rows over 32 experts of 4096 x 7168: 1.42 to 1.46 ms (2640 to 2710 TFLOP/s) with power-of-two scales, 1.57
// (2460) with fp32 ones, the gradient for w 1.55 to 1.57 (bf16; 1.90 in fp32, 3.8 GB of it); a library product of 8192^3 without block scales runs at
// 2960 to 3000.  Few rows: the weights' bytes, 512 rows over 256 experts of 7168 x 2048 525 us (6.2 TB/s).
#include <math.h>

#include <type_traits>

#include "device_common.h"
#include "frag16.h"
#include "gemm_engine.h"
#include "host_common.h"

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
  int lines;               // wgrad: rows of dw start on lines of 128 bytes
};

// LDS-DMA of a dword a lane, as dma16_buf.
__device__ __forceinline__ void dma4_buf(u32x4 rsrc, uint32_t off, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(off), "s"(rsrc), "s"(m0)
               : "memory");
}

// Fragment f (16 rows) of a staged operand, chunk c of whose row r stands in slot c ^ (r & 7): lane l has row l % 16, chunks
// l / 16 and l / 16 + 4.  `at` is the lane's place in fragment 0.
__device__ __forceinline__ uint32_t frag_at(int row0, int lane) {
  return (row0 + (lane & 15)) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
}
__device__ __forceinline__ v8i read_frag(uint32_t lds, uint32_t at, int f) {
  typedef __attribute__((address_space(3))) u32x4* p;
  const u32x4 lo = *reinterpret_cast<p>(lds + at + f * 2048);
  const u32x4 hi = *reinterpret_cast<p>(lds + (at ^ 64) + f * 2048);
  return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}
__device__ __forceinline__ uint32_t read_u32(uint32_t lds) {
  return *reinterpret_cast<__attribute__((address_space(3))) uint32_t*>(lds);
}

// D = A B scaled by 2^(sa - 127) 2^(sb - 127) for each row of A and column of B, + C; of sa and sb the low bytes count
__device__ __forceinline__ v4f mfma_scaled(const v8i& a, const v8i& b, const v4f& c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, (int)sa, 0, (int)sb);
}

// A workgroup's tiles: what its stream of operands needs of each, by lanes side by side before the first one.
constexpr int kMaxTiles = 64;  // of a workgroup
constexpr int kTab = 512;      // experts, or groups of `per` experts, that are found by their number of row tiles

struct alignas(8) Tile {
  int64_t a, b, sa, sb;              // first bytes of the operands and of their scales
  int64_t row0;                      // first row of c
  int lena, lenb, lensa, lensb;      // bytes from there to the end of the tile's first step (fwd: of its rows)
  int steps, mrows, n0;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Row tiles of expert e.
__device__ __forceinline__ int row_tiles(const int32_t* offsets, int R, int e, int BM) {
  int lo, hi;
  segment(offsets, R, e, lo, hi);
  return (hi - lo + BM - 1) / BM;
}

// Row tiles are numbered one expert after the other: tab[i] becomes the number of the first of expert i * per, INT_MAX past the last
// expert.  By one wave; returns the number of row tiles to all lanes.  No number passes `most`, whatever the offsets hold.
template <int BM>
__device__ __forceinline__ int fill_table(const int32_t* offsets, int R, int E, int per, int most, int* tab, int lane) {
  uint32_t first[kTab / 64], mine = 0;
#pragma unroll
  for (int i = 0; i < kTab / 64; ++i) {
    first[i] = mine;
    const int64_t e0 = (int64_t)(lane * (kTab / 64) + i) * per;
    for (int64_t e = e0; e < e0 + per && e < E; ++e) mine = min(mine + row_tiles(offsets, R, (int)e, BM), (uint32_t)most);
  }
  uint32_t before = __shfl_up(mine, 1, 64);  // tiles of the lanes before this one
  if (lane == 0) before = 0;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(before, o, 64);
    if (lane >= o) before = min(before + v, (uint32_t)most);
  }
#pragma unroll
  for (int i = 0; i < kTab / 64; ++i) {
    const bool in = (int64_t)(lane * (kTab / 64) + i) * per < E;
    tab[lane * (kTab / 64) + i] = in ? (int)min(before + first[i], (uint32_t)most) : 0x7fffffff;
  }
  return (int)__shfl(min(before + mine, (uint32_t)most), 63, 64);
}

// Expert of row tile q, and the number of its first one.
template <int BM>
__device__ __forceinline__ int find_expert(const int32_t* offsets, int R, int E, int per, const int* tab, int q, int& first) {
  int at = 0;
#pragma unroll
  for (int o = kTab / 2; o > 0; o >>= 1)
    if (tab[at + o] <= q) at += o;
  int e = at * per;
  first = tab[at];
  for (; e + 1 < E; ++e) {  // past tab[at]'s first expert where an entry stands for several
    const int m = row_tiles(offsets, R, e, BM);
    if (q < first + m) break;
    first += m;
  }
  return e;
}

// Two sums rounded to 16 bits (hardware conversions, nearest even).
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (F16) return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  else return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// Stores a wave's sums: lane l holds of tile (i, j) the row 16 i + l % 16 and the four columns from 16 j + 4 (l / 16).
// c: the wave's first row and column; rows and cols are left from there on (fewer than none: nothing is stored).  Stores past them
// go past the end of a buffer descriptor, so there is no branch.
// A store covers 8 rows of 128 bytes: lanes l and l ^ 8 change tiles, and before that, with 16 bits, lanes 16 apart, so that one holds
// 8 columns, 16 bytes.  past (if it MAY be): past the caches.
template <bool F16, bool OUT32, bool MAY, int TM, int TN>
__device__ __forceinline__ void store_sums(v4f (&acc)[TM][TN], void* c, int64_t ldc, int rows, int cols, int lane, bool past) {
  constexpr int kSize = OUT32 ? 4 : 2;
  const int r = min(rows, 16 * TM);
  const uint32_t ld = (uint32_t)ldc * kSize;
  const int bytes = rows > 0 && cols > 0 ? (int)((uint32_t)(r - 1) * ld) + min(cols, 16 * TN) * kSize : 0;
  const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(c, 0, bytes, 0x00020000);
  const bool up = lane & 8;
  // p of rows 0 .. 7 and, from lane l ^ 8, q of those; p and q of rows 8 .. 15
  auto halves = [&](const u32x4& p, const u32x4& q, u32x4& first, u32x4& second) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      first[k] = __builtin_amdgcn_update_dpp(p[k], q[k], 0x128, 0xf, 0xc, false);  // lanes 8 .. 15 of each 16 change
      second[k] = __builtin_amdgcn_update_dpp(q[k], p[k], 0x128, 0xf, 0x3, false);
    }
  };
  auto store = [&](const u32x4& p, const u32x4& q, int i, int n) {  // columns n of rows 16 i ..
    u32x4 first, second;
    halves(p, q, first, second);
    const uint32_t at = n < cols ? (16 * i + (lane & 7)) * ld + n * kSize : kPastEnd;
    if (MAY && past) {  // non-temporal
      __builtin_amdgcn_raw_buffer_store_b128(first, rsrc, at, 0, 2);
      __builtin_amdgcn_raw_buffer_store_b128(second, rsrc, at + 8 * ld, 0, 2);
    } else {
      __builtin_amdgcn_raw_buffer_store_b128(first, rsrc, at, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b128(second, rsrc, at + 8 * ld, 0, 0);
    }
  };
  constexpr int kTiles = OUT32 ? 2 : 4;  // 128 bytes
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; j += kTiles) {
      if constexpr (OUT32) {
        store(__builtin_bit_cast(u32x4, acc[i][j]), __builtin_bit_cast(u32x4, acc[i][j + 1]), i, 4 * (lane >> 4) + 16 * (j + (up ? 1 : 0)));
      } else {
        u32x4 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v4f &x = acc[i][j + 2 * h], &y = acc[i][j + 2 * h + 1];
          // lanes of groups 0 and 2 come to hold columns 0 .. 7 and 8 .. 15 of the one tile, those of 1 and 3 of the other
          const auto lo = __builtin_amdgcn_permlane16_swap(pack16<F16>(x[0], x[1]), pack16<F16>(y[0], y[1]), false, false);
          const auto hi = __builtin_amdgcn_permlane16_swap(pack16<F16>(x[2], x[3]), pack16<F16>(y[2], y[3]), false, false);
          v[h] = u32x4{lo[0], hi[0], lo[1], hi[1]};
        }
        store(v[0], v[1], i, 16 * (j + (up ? 2 : 0) + ((lane >> 4) & 1)) + 8 * (lane >> 5));
      }
      if constexpr (OUT32) {  // cleared one by one: else the compiler keeps what was stored as well
#pragma unroll
        for (int k = 0; k < kTiles; ++k) {
          acc[i][j + k] = v4f{0.f, 0.f, 0.f, 0.f};
          asm volatile("" : "+v"(acc[i][j + k]));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// E8: power-of-two scales (bytes), else fp32 ones.  Waves stand WM x WN, each with TM x TN tiles of 16 x 16.
//
// The steps of all tiles of a workgroup are one stream: while one tile's last steps are multiplied and its sums are
// stored, the operands of the next are on their way.  A step's rows j = 0 .. TN - 1 multiply fragment j of B with the TM fragments of A.
// A(s) is read ahead, during step s - 1; B's fragments are read one or two rows ahead.  Two barriers a step:
//   row 1     A(s) is in everyone's registers and B(s - 1) is done with: A(s + D) and its scales follow into A(s)'s slot
//   row TN/2  A(s + 1), B(s + 1) and their scales have landed (the DMAs of later steps may be under way) and the first half of B(s)'s
//             fragments is done with: B(s + D) follows, its halves in the slots of the second half of B(s - 1) and the first of B(s)
// So LDS holds D slots of A and 2 D + 1 halves of B, and DMAs go out in every part of a step.  Measured on 65536 rows over 32 experts of
// 4096 x 7168, E8M0 (fp32 scales; gradient for w): one barrier a step, all DMAs in its second half and scales loaded into registers
// 1.80 ms (1.87; 2.15); so 1.42 (1.57; 1.55), much of the last from one tile's start under another's end: the gradient with 4 steps a tile
// (16384 rows over 32 experts of 4096 x 2048) 0.166 ms against 0.320.  Of its time with 8 steps a tile (32768 rows, 0.96 ms)
// 0.19 is the stores', 0.77 remain where they go nowhere; workgroups that start apart from each
// other gain nothing, and half of a tile's stores between the next one's MFMAs lose (1.03).
template <int OP, bool E8, bool OUT32, int BM, int BN, int WM, int WN, int D>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_ragged_kernel(Fp8Args g) {
  constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr int kAhead = TM * TN >= 32 ? 1 : 2, kHold = 2 * kAhead, kHalf = TN / 2;  // fragments of B ahead, and held
  constexpr int kABytes = BM * 128, kHBytes = BN * 64;  // a slot of A, a half of B
  constexpr int NA = kABytes / 1024 / NW, NH = kHBytes / 1024 / NW;  // DMAs of a wave
  constexpr int kBand = OP == kFp8Wgrad ? 4 : 8;
  constexpr int kStage = NA + 1 + 2 * NH;  // DMAs of a wave for a step
  constexpr int kWinA = (BM + 63) / 64, kWin = kWinA + BN / 64;  // windows of 64 scales: A's rows, then B's columns
  constexpr int kScales = 256 * kWin;                    // scales of a step, a dword each
  static_assert(NA * NW * 1024 == kABytes && NH * NW * 1024 == kHBytes && NW >= kWin && TN >= 4 && TN % 4 == 0, "whole DMAs");
  static_assert(D >= 2 && kHalf >= 2, "A's DMAs go out in rows 1 .. TN/2 - 1");
  __shared__ __align__(16) uint8_t smem[D * kABytes + (2 * D + 1) * kHBytes + (D + 1) * kScales];
  __shared__ Tile tiles[kMaxTiles];
  __shared__ int count_sh;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = uniform(tid >> 6);
  const int wm = (w / WN) * (BM / WM), wi = w % WN;

  const int ndim = OP == kFp8Fwd ? g.N : g.K, ntiles = (ndim + BN - 1) / BN;
  const int KB = (g.K + 127) / 128;
  constexpr int kEsz = E8 ? 1 : 4;
  if (w == 0) {
    const int mtiles = (g.N + BM - 1) / BM, per = (g.E + kTab - 1) / kTab;
    int* tab = reinterpret_cast<int*>(smem);
    const int total = OP == kFp8Fwd ? fill_table<BM>(g.offsets, g.R, g.E, per, g.R / BM + min(g.E, g.R), tab, lane) * ntiles : g.E * mtiles * ntiles;
    // Workgroups go to the eight XCDs in turn.  Small tiles: each XCD takes a run of them, and its workgroups the next one in turn
    // (8192 rows over 32 experts of 2048 x 2048 50 us, else 58).  Large ones, and wgrad's, which cost as much as their
    // expert has rows: the XCDs take as many as they have workgroups in turn (65536 rows over 32 experts of 4096 x 7168 1.41 ms
    // against 1.44; wgrad with 32768 rows that follow Zipf's law 0.98 against 2.7).
    constexpr bool kRuns = OP == kFp8Fwd && BM < 256;
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3, stride = gridDim.x >> 3;
    const int64_t chunk = ((int64_t)total + 7) / 8;
    const int64_t first = xcd * (kRuns ? chunk : (int64_t)stride) + slot, step = kRuns ? stride : 8ll * stride;
    const int64_t end = kRuns ? min((int64_t)total, (xcd + 1) * chunk) : total;
    if (lane == 0) count_sh = first < end ? (int)min((int64_t)kMaxTiles, (end - first + step - 1) / step) : 0;
    const int64_t t = first + lane * step;
    if (t < end) {
      const int q = (int)t / ntiles;
      int e, base, m, lo, hi;
      if constexpr (OP == kFp8Fwd) {
        e = find_expert<BM>(g.offsets, g.R, g.E, per, tab, q, base);
        m = row_tiles(g.offsets, g.R, e, BM);
      } else {
        e = q / mtiles;
        base = e * mtiles;
        m = mtiles;
      }
      segment(g.offsets, g.R, e, lo, hi);
      // inside an expert the tiles advance in bands of row tiles: those that an XCD works on at a time share few panels
      const int rest = (int)t - base * ntiles, band = kBand * ntiles, b0 = max(0, rest) / band * kBand, in = max(0, rest) % band;
      const int height = max(1, min(kBand, m - b0)), mt = b0 + in % height;
      const bool known = rest >= 0 && mt < m;  // always, unless the offsets decrease
      const int m0 = known ? mt * BM : 0, n0 = in / height * BN;
      const int left = !known ? 0 : OP == kFp8Fwd ? hi - lo - m0 : g.N - m0, mrows = min(BM, left), nrows = min(BN, ndim - n0);
      const int64_t block0 = lo / 128 + e;  // wgrad: the segment's first block
      Tile x;
      x.steps = !known || n0 >= ndim ? 0 : OP == kFp8Fwd ? KB : (hi - lo + 127) / 128;
      x.mrows = left;
      x.n0 = n0;
      if constexpr (OP == kFp8Fwd) {
        x.row0 = lo + m0;
        x.a = (int64_t)(lo + m0) * g.lda;
        x.b = ((int64_t)e * g.N + n0) * g.K;
        x.lena = (int)((mrows - 1) * g.lda + g.K);
        x.lenb = (int)((nrows - 1) * (int64_t)g.K + g.K);
        x.sa = (int64_t)(lo + m0) * g.ssm * kEsz;
        x.sb = ((int64_t)e * ((g.N + 127) / 128) + n0 / 128) * KB * kEsz;
        x.lensa = (int)(((mrows - 1) * g.ssm + 1) * kEsz);
        x.lensb = ((nrows - 1) / 128 * KB + 1) * kEsz;
      } else {
        x.row0 = (int64_t)e * g.N + m0;
        x.a = (block0 * g.N + m0) * 128;
        x.b = (block0 * g.K + n0) * 128;
        x.lena = mrows * 128;
        x.lenb = nrows * 128;
        x.sa = block0 * g.N + m0;
        x.sb = block0 * g.K + n0;
        x.lensa = mrows;
        x.lensb = nrows;
      }
      tiles[lane] = x;
    }
  }
  __syncthreads();
  const int count = uniform(count_sh);
  if (count == 0) return;

  // ---- the stream of operands: all uniform but the lanes' offsets, which hold for every tile
  const int64_t lda = OP == kFp8Fwd ? g.lda : 128, ldb = OP == kFp8Fwd ? g.K : 128;
  const int64_t stepa = OP == kFp8Fwd ? 128 : (int64_t)g.N * 128, stepb = OP == kFp8Fwd ? 128 : (int64_t)g.K * 128;
  const int kc = 16 * ((lane & 7) ^ (lane >> 3));  // this lane's k within a step
  const uint32_t offa = (uint32_t)((lane >> 3) * lda + kc), offb = (uint32_t)((lane >> 3) * ldb + kc);
  // DMA i of A moves rows 8 (w NA + i) .., of half h of B 8 rows of the first or second halves of all column waves' fragments
  auto rowa = [&](int i) { return (uint32_t)(8 * (w * NA + i) * lda); };
  auto rowb = [&](int h, int i) {
    constexpr int kPart = BN / WN / 2;
    const int r = 8 * (w * NH + i);
    return (uint32_t)((r / kPart * (2 * kPart) + h * kPart + r % kPart) * ldb);
  };
  // scales: window w % kWin, one lane a row of A or column of B
  const int64_t stepsa = (OP == kFp8Fwd ? g.sskb : g.N) * kEsz, stepsb = OP == kFp8Fwd ? kEsz : g.K;  // from one step to the next
  const int win = w % kWin;
  const bool of_a = win < kWinA;  // uniform
  const int srow = 64 * (of_a ? win : win - kWinA) + lane;
  const uint32_t soff = (uint32_t)((of_a ? srow * (OP == kFp8Fwd ? g.ssm : 1) : OP == kFp8Fwd ? srow / 128 * (int64_t)KB : srow) * kEsz);
  int ft = -1, fs = 0, fsteps = 0;  // tile and step of the next operands
  const uint8_t *pa = nullptr, *pb = nullptr, *ps = nullptr;
  int lena = 0, lenb = 0, lens = 0;
  // E8: where a step's bytes start in their dwords, of A's scales and of B's (this step's, the next one's, .., the one fetched)
  uint32_t lowa = 0, lowb = 0, rema[D + 1], remb[D + 1];
  // to the next tile that has steps; past the last one nothing is fetched
  auto seek = [&]() __attribute__((always_inline)) {
    fs = 0;
    do {
      ++ft;
    } while (ft < count && (fsteps = uniform(tiles[ft].steps)) == 0);
    if (ft < count) {
      const Tile* x = tiles + ft;
      pa = g.a + uniform64(x->a);
      pb = g.b + uniform64(x->b);
      const uint8_t* psa = static_cast<const uint8_t*>(g.sa) + uniform64(x->sa);
      const uint8_t* psb = static_cast<const uint8_t*>(g.sb) + uniform64(x->sb);
      lowa = (uint32_t)(uintptr_t)psa;
      lowb = (uint32_t)(uintptr_t)psb;
      ps = of_a ? psa : psb;
      lena = uniform(x->lena);
      lenb = uniform(x->lenb);
      lens = uniform(of_a ? x->lensa : x->lensb);
    } else {
      lena = lenb = lens = -(1 << 30);
      fsteps = 0x7fffffff;
    }
  };
  u32x4 da, db, ds;
  uint32_t past = 0, srem = 0;
  auto next_a = [&]() __attribute__((always_inline)) {  // and the scales
    da = dma_buffer(pa, lena);
    past = OP == kFp8Fwd && kc >= g.K - fs * 128 ? kPastEnd : 0u;
    pa += stepa;
    if (OP == kFp8Fwd) lena -= 128;
    // scales of a byte are fetched with the dword around them
    srem = E8 ? (uint32_t)(uintptr_t)ps & 3u : 0u;
    ds = dma_buffer(ps - srem, (lens + (int)srem + 3) & ~3);
    ps += of_a ? stepsa : stepsb;
    rema[D] = lowa;
    remb[D] = lowb;
    lowa += (uint32_t)stepsa;
    lowb += (uint32_t)stepsb;
  };
  auto next_b = [&]() __attribute__((always_inline)) {
    db = dma_buffer(pb, lenb);
    pb += stepb;
    if (OP == kFp8Fwd) lenb -= 128;
    ++fs;
  };
  const uint32_t lds0 = lds_addr(smem), ldss = lds0 + D * kABytes + (2 * D + 1) * kHBytes;
  auto dma_a = [&](int i, uint32_t slot) { dma16_buf(da, (offa | past) + rowa(i), slot + (w * NA + i) * 1024); };
  auto dma_b = [&](int h, int i, uint32_t slot) { dma16_buf(db, (offb | past) + rowb(h, i), slot + (w * NH + i) * 1024); };
  auto dma_s = [&](uint32_t slot) { dma4_buf(ds, E8 ? (soff + srem) & ~3u : soff, slot + win * 256); };

  // ---- the products
  const uint32_t ata = frag_at(wm, lane), atb = frag_at(wi * (BN / WN / 2), lane);
  const uint32_t atsa = 4 * (wm + (lane & 15)), atsb = 4 * (64 * kWinA + wi * (BN / WN) + (OP == kFp8Wgrad ? (lane & 15) : 0));
  const uint32_t mod_a = (lane & 15) * (OP == kFp8Fwd ? (uint32_t)g.ssm : 1u);
  const uint32_t mod_b = OP == kFp8Fwd ? (uint32_t)(wi * (BN / WN) / 128 * KB) : lane & 15;
  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  uint32_t sl[D], hb[2 * D + 1], sc[D + 1];  // slots of A, halves of B and scales: this step's, the next one's, ..
#pragma unroll
  for (int i = 0; i < D; ++i) sl[i] = lds0 + i * kABytes;
#pragma unroll
  for (int i = 0; i <= 2 * D; ++i) hb[i] = lds0 + D * kABytes + i * kHBytes;
#pragma unroll
  for (int i = 0; i <= D; ++i) sc[i] = ldss + i * kScales;
  vm_wait<0>();
#pragma unroll
  for (int s = 0; s < D; ++s) {
    if (fs == fsteps) seek();
    next_a();
#pragma unroll
    for (int i = 0; i < NA; ++i) dma_a(i, sl[s]);
    dma_s(sc[s]);
    rema[s] = rema[D];
    remb[s] = remb[D];
    next_b();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NH; ++i) dma_b(h, i, hb[2 * s + h]);
  }
  // two steps: no stores stand behind the second's DMAs yet, as the first wait of a tile takes for granted
  vm_wait<(D - 2) * kStage>();
  barrier_only();
  v8i ra[2][TM], rb[kHold];
  uint32_t rawa[TM], rawb[kHold];  // scales of A's fragments (this step's, then the next one's) and of B's held ones
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    ra[0][i] = read_frag(sl[0], ata, i);
    rawa[i] = read_u32(sc[0] + atsa + 64 * i);
  }
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    rb[j] = read_frag(hb[0], atb, j);
    rawb[j] = read_u32(sc[0] + atsb + (OP == kFp8Wgrad ? 64 * j : 0));
  }

  // first: of a tile, so the sums start from zero, and the stores of the last one's are behind the DMAs that row TN/2 waits for and may
  // be under way
  auto step = [&](auto par_c, auto first_c) __attribute__((always_inline)) {
    constexpr bool kFirst = decltype(first_c)::value, kZero = kFirst && !OUT32;
    constexpr int PAR = decltype(par_c)::value, kLate = kFirst ? TM * TN / (OUT32 ? 2 : 4) * 2 : 0;
    const v4f zero{0.f, 0.f, 0.f, 0.f};
    // a byte's place in its dword is the same for all of a lane's rows (16 apart), and for its columns
    const uint32_t sha = E8 ? 8 * ((mod_a + rema[0]) & 3) : 0, shb = E8 ? 8 * ((mod_b + remb[0]) & 3) : 0;
    uint32_t sa[TM];
    float f[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      if constexpr (E8) sa[i] = rawa[i] >> sha;
      else f[i] = __uint_as_float(rawa[i]) * __uint_as_float(rawb[0]);
    }
    const uint32_t sbu = rawb[0] >> shb;  // fwd: one for all of the wave's columns
    v4f acc2[4];
    auto fold = [&](int p) __attribute__((always_inline)) {
      v4f& sum = acc[p % TM][p / TM];
      sum = kZero ? acc2[p % 4] * f[p % TM] : sum + acc2[p % 4] * f[p % TM];
    };
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if (j == 1) {
        barrier_only();
        next_a();
      }
      if (j == kHalf) {
        vm_wait<NA + 1 + (D - 2) * kStage + kLate>();
        barrier_only();
        next_b();
      }
      const int ahead = j + kAhead;
      rb[ahead % kHold] = read_frag(ahead < TN ? hb[ahead / kHalf] : hb[2], atb, ahead % kHalf);
      if constexpr (OP == kFp8Wgrad) rawb[ahead % kHold] = read_u32(sc[ahead < TN ? 0 : 1] + atsb + 64 * (ahead % TN));
      if (j >= 1 && j < kHalf) {
        constexpr int kRow = (NA + 1 + kHalf - 2) / (kHalf - 1);
#pragma unroll
        for (int d = (j - 1) * kRow; d < j * kRow; ++d) {
          if (d < NA) dma_a(d, sl[0]);
          else if (d == NA) dma_s(sc[D]);
        }
      }
      if (j >= kHalf) {
        constexpr int kRow = 2 * NH / kHalf, kReads = (TM + kHalf - 1) / kHalf;
#pragma unroll
        for (int d = (j - kHalf) * kRow; d < (j - kHalf + 1) * kRow; ++d) dma_b(d / NH, d % NH, hb[d < NH ? 2 * D : 0]);
#pragma unroll
        for (int d = (j - kHalf) * kReads; d < (j - kHalf + 1) * kReads && d < TM; ++d) {
          ra[PAR ^ 1][d] = read_frag(sl[1], ata, d);
          rawa[d] = read_u32(sc[1] + atsa + 64 * d);
        }
      }
      if constexpr (OP == kFp8Fwd) {
        if (j == TN - 1) rawb[0] = read_u32(sc[1] + atsb);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if constexpr (E8) {
          acc[i][j] = mfma_scaled(rb[j % kHold], ra[PAR][i], kZero ? zero : acc[i][j], OP == kFp8Wgrad ? rawb[j % kHold] >> shb : sbu, sa[i]);
        } else {
          // ahead of each MFMA the fold of the tile three before it: the unit is never waited for (65536 rows at random over 32 experts
          // of 4096 x 7168, rounded normal values under scales of one, 1.65 ms; behind the MFMA and two before 1.69, one before 1.76.  On
          // quantised values, which cost more power, 1.74 to 1.81 either way)
          const int q = j * TM + i;
          if (q >= 3) fold(q - 3);
          acc2[q % 4] = mfma16x16x128_fp8(rb[j % kHold], ra[PAR][i], zero);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (!E8) {
#pragma unroll
      for (int p = TM * TN - 3; p < TM * TN; ++p) fold(p);
    }
    // the sums stay in this step's block: products are not moved past the branches between steps
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(acc[i][j]));
    const uint32_t a0 = sl[0], h0 = hb[0], h1 = hb[1], s0 = sc[0];
#pragma unroll
    for (int i = 0; i + 1 < D; ++i) sl[i] = sl[i + 1];
    sl[D - 1] = a0;
#pragma unroll
    for (int i = 0; i + 2 <= 2 * D; ++i) hb[i] = hb[i + 2];
    hb[2 * D - 1] = h0;
    hb[2 * D] = h1;
#pragma unroll
    for (int i = 0; i < D; ++i) {
      sc[i] = sc[i + 1];
      rema[i] = rema[i + 1];
      remb[i] = remb[i + 1];
    }
    sc[D] = s0;
  };
  for (int t = 0; t < count; ++t) {
    int left = uniform(tiles[t].steps);
    using Even = std::integral_constant<int, 0>;
    using Odd = std::integral_constant<int, 1>;
    if (left > 0) {
      if (fs == fsteps) seek();
      step(Even{}, Odd{});
      for (--left; left >= 2; left -= 2) {
        if (fs == fsteps) seek();
        step(Odd{}, Even{});
        if (fs == fsteps) seek();
        step(Even{}, Even{});
      }
      if (left) {
        if (fs == fsteps) seek();
        step(Odd{}, Even{});
      } else {
#pragma unroll
        for (int i = 0; i < TM; ++i) ra[0][i] = ra[1][i];
      }
    } else if (!OUT32) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    }
    const int64_t row0 = uniform64(tiles[t].row0);
    const int mrows = uniform(tiles[t].mrows), n0 = uniform(tiles[t].n0);
    int l = lane;
    asm volatile("" : "+v"(l));  // the stores' addresses are made here, not kept in registers through the steps
    uint8_t* c = static_cast<uint8_t*>(g.c) + ((row0 + wm) * g.ldc + n0 + wi * (BN / WN)) * (OUT32 ? 4 : 2);
    // wgrad's sums are stored past the caches where rows start on lines (nt: 177 us, else 220, for 16384 rows over 32 experts of
    // 4096 x 2048), but 25 us become 56 where they do not (5003 over 48 of 1008 x 1168); fwd's are read by the next product
    const int rows = mrows - wm, cols = ndim - n0 - wi * (BN / WN);
    const bool past = OP == kFp8Wgrad && g.lines;
    constexpr bool kMay = OP == kFp8Wgrad;
    if (OUT32 || !g.f16) store_sums<false, OUT32, kMay>(acc, c, g.ldc, rows, cols, l, past);
    else store_sums<true, false, kMay>(acc, c, g.ldc, rows, cols, l, past);
  }
  vm_wait<0>();
}

template <int OP, bool E8, bool OUT32, int BM, int BN, int WM, int WN, int D = 2>
int launch(const Fp8Args& g, hipStream_t stream) {
  auto* fn = &fp8_ragged_kernel<OP, E8, OUT32, BM, BN, WM, WN, D>;
  const int64_t nt = ceil_div64(OP == kFp8Fwd ? g.N : g.K, BN);
  // an upper bound of the row tiles: the offsets are on the device
  const int64_t mt = OP == kFp8Wgrad ? (int64_t)g.E * ceil_div64(g.N, BM) : g.R / BM + (g.E < g.R ? g.E : g.R);
  MOE355_CHECK(mt * nt < (1ll << 31), MOE355_EUNSUPPORTED);  // tiles are counted in 32 bits
  // as many workgroups as the CUs hold at a time, or tiles; more where one would get more than kMaxTiles
  const int64_t slots = 256 * (BM == 256 ? 1 : 2), need = ceil_div64(ceil_div64(mt * nt, 8), kMaxTiles) * 8;
  const int64_t few = ceil_div64(mt * nt, 8) * 8 < slots ? ceil_div64(mt * nt, 8) * 8 : slots, grid = few > need ? few : need;
  hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(64 * WM * WN), 0, stream, g);
  return launch_status();
}

// Row tiles of t rows that R rows make over E experts: the offsets are on the device, so each row is taken to fall on an
// expert by chance (normal approximation; the number of tiles is sum_k P(rows > k t)).
double expected_tiles(int R, int E, int t) {
  const double a = (double)R / E, sd = sqrt(2 * a * (1 - 1.0 / E)) + 1e-9;
  double n = 0;
  const int64_t sure = (int64_t)((a - 3 * sd) / t);  // (3 * sqrt(2) standard deviations)
  if (sure > 0) n = (double)sure;
  for (int64_t k = sure > 0 ? sure : 0; (double)k * t < a + 3 * sd; ++k) n += 0.5 * erfc((k * (double)t + 0.5 - a) / sd);
  return n * E;
}

// The tile.  One round of tiles, or few rows an expert: 32 x 64 by two waves, two workgroups a CU with four steps on their way each;
// the weights' bytes bound the latter, and what counts is how many of them are under way.  From 13 to 40 rows an expert 64 x 128.
// Beyond, the cheaper one of 256 x 256, in whole rounds of the 256 CUs, and 128 x 128, whose round of 512 costs 0.715 of that.
// Measured, us with tiles of 32 x 64 / 64 x 128 / 128 x 128, weights out of HBM (fp32 scales; the latter two with two steps ahead):
//   one row by 4096 x 7168 24 / 28 / 33; 8 rows over 256 experts of 4096 x 7168 43 / 44 / 45; 512 rows over 256 of 7168 x 2048
//   526 / 540 / 562; 32 experts of 4096 x 7168: 2 rows each on average 139 / 144 / 153, 8 rows 160 / 160 / 164, 32 rows 220 / 168 / 176,
//   64 rows 312 / 234 / 198; 300 rows over 4 experts of 512 x 2048 (E8M0) 11.0 / 12.6 / 14.4; 600 over 8 of 2048 x 1024, more
//   than one round, 12.7 / 10.2 / 11.0.  The 32 x 64 with two steps ahead and four workgroups a CU took 41 for the one row and 53 for
//   the 8; three ahead or six in place of four 44 and more for the 8.
// and of 128 x 128 / 256 x 256 (E8M0; wgrad in brackets):
//   32 experts of 2048 x 2048: 128 rows each on average 35 / 33 (82 / 76), 256 rows 50 / 56 (108 / 101); 160 rows of
//   4096 x 2048 87 / 75 (187 / 162); 2 experts of 2000 x 2000, 500 rows 15 / 26 (12.4 / 14.6); one of 4096 x 7168, 4096 rows
//   124 / 92 (122 / 100)
template <int OP, bool E8, bool OUT32>
int run(const Fp8Args& g, hipStream_t stream) {
  const int64_t cols = OP == kFp8Fwd ? g.N : g.K;
  auto tiles = [&](int tm, int tn) {
    return (OP == kFp8Wgrad ? (double)g.E * ceil_div64(g.N, tm) : expected_tiles(g.R, g.E, tm)) * ceil_div64(cols, tn);
  };
  if constexpr (OP == kFp8Fwd) {
    if (g.R <= 12ll * g.E || tiles(32, 64) <= 512) return launch<OP, E8, OUT32, 32, 64, 2, 1, 4>(g, stream);
    if (g.R <= 40ll * g.E) return launch<OP, E8, OUT32, 64, 128, 4, 2>(g, stream);
  }
  if (ceil(tiles(256, 256) / 256) <= 0.715 * tiles(128, 128) / 512) return launch<OP, E8, OUT32, 256, 256, 4, 2>(g, stream);
  return launch<OP, E8, OUT32, 128, 128, 4, 2>(g, stream);
}

bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kMaxLd = 1 << 22;    // 256 rows' byte offsets stay below 2^31
constexpr int kMaxDim = 1 << 22;
constexpr int64_t kMaxSs = 1 << 21;    // and those of their scales
constexpr int kMaxRows = 0x7fffffff - 255;  // row tiles of a segment are (rows + 255) / 256 in 32 bits

}  // namespace
}  // namespace moe355

using namespace moe355;

extern "C" int grouped_gemm_fp8(const uint8_t* x8, const void* x_scale, int64_t ld_x, int64_t sstride_m, int64_t sstride_kb,
                                const uint8_t* w8, const void* w_scale, int e8m0, const int32_t* offsets, int R, int E, int N,
                                int K, uint16_t* y, int64_t ld_y, int fp16, hipStream_t stream) {
  MOE355_CHECK((fp16 == 0 || fp16 == 1) && (e8m0 == 0 || e8m0 == 1) && R >= 0 && E >= 0 && N >= 0 && K >= 0 && ld_x >= K &&
                   ld_y >= N && sstride_m >= 0 && sstride_kb >= 0,
               MOE355_EINVAL);
  MOE355_CHECK(N % 8 == 0 && K % 16 == 0 && N <= kMaxDim && E < 65536 && ld_x <= kMaxLd && sstride_m <= kMaxSs && ld_y <= kMaxSs && R <= kMaxRows,
               MOE355_EUNSUPPORTED);
  if (R == 0 || E == 0 || N == 0) return MOE355_OK;
  MOE355_CHECK(offsets && y && (K == 0 || (x8 && w8 && x_scale && w_scale)), MOE355_EINVAL);
  MOE355_CHECK((K == 0 || (aligned16(x8) && ld_x % 16 == 0 && aligned16(w8))) && aligned16(y) && ld_y % 8 == 0 && on4(offsets) &&
                   (e8m0 || (on4(x_scale) && on4(w_scale))),
               MOE355_EMISALIGNED);
  const Fp8Args g{x8, w8, x_scale, w_scale, y, offsets, ld_x, ld_y, sstride_m, sstride_kb, R, E, N, K, fp16, 0};
  return e8m0 ? run<kFp8Fwd, true, false>(g, stream) : run<kFp8Fwd, false, false>(g, stream);
}

extern "C" int grouped_gemm_fp8_wgrad(const uint8_t* dyt, const uint8_t* dyt_scale, const uint8_t* xt, const uint8_t* xt_scale,
                                      const int32_t* offsets, int R, int E, int N, int K, void* dw, int out, hipStream_t stream) {
  MOE355_CHECK(R >= 0 && E >= 0 && N >= 0 && K >= 0 && out >= MOE355_BF16 && out <= MOE355_F32, MOE355_EINVAL);
  MOE355_CHECK(N % 8 == 0 && K % 8 == 0 && N <= kMaxDim && K <= kMaxDim && E < 65536 && R <= kMaxRows, MOE355_EUNSUPPORTED);
  if (E == 0 || N == 0 || K == 0) return MOE355_OK;  // without rows every gradient is zero: still written
  MOE355_CHECK(offsets && dw && (R == 0 || (dyt && dyt_scale && xt && xt_scale)), MOE355_EINVAL);
  MOE355_CHECK((R == 0 || (aligned16(dyt) && aligned16(xt))) && aligned16(dw) && on4(offsets), MOE355_EMISALIGNED);
  const int lines = (int64_t)K * (out == MOE355_F32 ? 4 : 2) % 128 == 0 && reinterpret_cast<uintptr_t>(dw) % 128 == 0;
  const Fp8Args g{dyt, xt, dyt_scale, xt_scale, dw, offsets, 128, K, 0, 0, R, E, N, K, out == MOE355_F16, lines};
  return out == MOE355_F32 ? run<kFp8Wgrad, true, true>(g, stream) : run<kFp8Wgrad, true, false>(g, stream);
}
