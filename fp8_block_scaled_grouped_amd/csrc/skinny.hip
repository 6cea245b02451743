// Linear layers with few rows: c[m, n] = sum_k x[m, k] w[n, k] with 4-bit (e2m1) weights and
// group scales, or 16-bit weights; one matrix, or one per expert over ragged row segments.
//
//   4-bit: c[m, n] = round(sum_g s[n, g] sum_{k in group g} x[m, k] q[n, k])
//
// The weights are read once and bound the time, so the kernel is built around their stream:
// two to eight waves of a workgroup do nothing but LDS-DMA, S stages deep, in whole 128-byte lines of
// the weight rows (fragment-shaped loads straight into registers, 16 rows x 64 bytes each,
// ask for twice as many lines and the requests in flight, not the bytes, bounded them).  The
// other waves multiply from LDS: 16 weight rows are an MFMA's columns, 16 rows of x its rows.  A
// stage is 128 H k for each of KW waves that share columns; they add their fp32 tiles in LDS in
// wave order at the end (deterministic, one launch, no workspace).  From 17 rows of one matrix on, where the columns
// leave CUs idle, workgroups split K too: partial sums in a workspace, added by a second launch in order.
//
// A lane takes 16 bytes of a weight row's 128-wide block: 32 codes, k [32 g, 32 g + 32) for
// lane group g = lane / 16.  The conversion instruction turns 8 codes into an operand in 4
// issues.  E8M0 scales with bf16 x go into the conversion itself (exact up to a byte of 252; weights past bf16's
// range are taken again as quarters after the loop), with fp16 x those of 32 relative to the largest of a
// block (Format::kRelative).  Else the scale
// multiplies the fp32 tile of its group, so an MFMA's 32 k must lie in one group: groups of
// 128 take any order, for groups of 64 and 32 the lanes of a column exchange codes first (one
// or two lane-swap steps), and x is read in the order that results.
//
// Columns past N, rows past the segment and k past K lie past the end of the buffer
// descriptors: they arrive as zeros, without traffic.
//
// E8M0 rows of a number of scales that is not a multiple of 4 do not start on dwords, so they cannot be copied as such:
// the multiplying waves read those bytes from memory where they use them (18432 x 7200 against 7168, time a byte:
// bf16 x 1.2 to 1.5 times, fp16 x with scales of 32 twice; experts 1.3 to 3.3 times).
//
// Measured (18432 x 7168, fp32 scales of 128; the same weights in each call, which the last-level cache holds): 1 row
// 15.1 us (4.6 TB/s of weights and scales; fragment-shaped register loads 31 us), 16 rows 17.5 us, 64 rows 32 us.  Weights
// from memory: 17.6, 21.8 and 35.0 us.  64 tokens through 222 of 256 experts of 7168 x 2048 276 to 282 us (6.2 TB/s; 497 us).
// A single copying wave issues too slowly for a CU's share of the stream: with two, 1 row over 2048 x 7168 takes
// 6.8 us instead of 8.4, with 64 rows four take 33 us where one takes 46.
#include "skinny.h"

#include <type_traits>

#include "frag16.h"
#include "gemm_engine.h"
#include "host_common.h"

namespace moe355 {
namespace {

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

// Rotation of the scales of row r in LDS, rows of 2^sh dwords: 16 rows' scales of one group in different banks.
__device__ __forceinline__ int scale_swz(int r, int sh) { return (r & 15) >> (sh < 6 ? 6 - sh : 0); }

// LDS-DMA of a dword per lane.
__device__ __forceinline__ void dma4_buf(u32x4 rsrc, uint32_t off, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(off), "s"(rsrc), "s"(m0)
               : "memory");
}

// Chunk c of row r lies in slot c ^ S(r), so that the 16 lanes that the LDS serves at a time (lanes 0-3 and
// 12-15 of one lane group with 4-11 of the next, or the rest of the two) find their 16-byte chunks in
// different banks.  S is linear: S(a | b) = S(a) ^ S(b) for rows a, b without common bits.
//
// Weights: lane group g reads chunk .. + g of rows 0 to 15; RC chunks a row.
template <int RC>
struct WeightSlots {
  static __device__ __forceinline__ int of(int r) {
    if constexpr (RC >= 16) return r & 15;
    if constexpr (RC == 8) return r & 7;      // two rows a bank round
    const int q = (r >> 2) & 3;               // four rows a bank round
    return ((q << 1) & 2) ^ ((q >> 1) * 3);
  }
};
// x: lane group g reads chunk .. + STEP g of rows 0 to min(ROWS, 16) - 1, which repeat.
template <int ROWS, int STEP>
struct XSlots {
  static __device__ __forceinline__ int of(int r) {
    if constexpr (STEP == 1) return (ROWS < 16 ? r << 1 : r) & 15;
    if constexpr (ROWS <= 4) return r & 3;
    if constexpr (ROWS == 8) return (r & 3) | ((r & 4) << 1);
    return ((r & 3) << 2) | ((r >> 2) & 3);
  }
};

// LDS-DMA of COUNT KB as rows of RC 16-byte chunks, swizzled by SLOTS.
template <int COUNT, int RC, class SLOTS>
struct RowCopy {
  static constexpr int kRows = RC < 64 ? 64 / RC : 1;   // rows of a DMA instruction
  static constexpr int kParts = RC < 64 ? 1 : RC / 64;  // instructions of a row
  uint32_t base;  // byte offset of the lane's first row
  int chunk;      // its chunk in that row

  __device__ __forceinline__ void init(int lane, int64_t stride) {
    const int r = RC < 64 ? lane / RC : 0;
    base = (uint32_t)(r * stride);
    chunk = (RC < 64 ? lane % RC : lane) ^ SLOTS::of(r);
  }
  // TAIL: chunks of `left` and more read zeros;
  // and only instructions `part`, part + PARTS, ... are this wave's.
  template <bool TAIL, int PARTS>
  __device__ __forceinline__ void copy(u32x4 rsrc, uint32_t dst, uint32_t stride, int left, int part) const {
    // The offsets are the same in every stage; kept in registers they would take more of them than
    // the multiplying waves have, so each call computes them (3 VALU a DMA) from values that the
    // compiler must take for new.
    uint32_t base = this->base;
    int chunk = this->chunk;
    asm volatile("" : "+v"(base), "+v"(chunk));
#pragma unroll
    for (int i = 0; i < COUNT / PARTS; ++i) {
      const int j = i * PARTS + part, row = j / kParts * kRows, c = (chunk ^ SLOTS::of(row)) + j % kParts * 64;
      const uint32_t off = base + row * stride + c * 16;
      dma16_buf(rsrc, TAIL && c >= left ? kPastEnd : off, dst + j * 1024);
    }
  }
};

template <int W, int GROUP, bool F16>
struct Format {
  static constexpr bool kDirect = W == kFp4E8M0 && !F16;    // scale inside the conversion
  static constexpr bool kFold = W != kW16 && !kDirect;      // scale on the fp32 tile
  static constexpr int kChunks = W == kW16 ? 16 : 4;        // 16-byte chunks of a row's 128-wide block
  static constexpr int kPerChunk = W == kW16 ? 8 : 32;      // k of a chunk
  static constexpr int kLoads = W == kW16 ? 4 : 1;          // chunks a lane reads per 128-wide block
  // fp16 products with E8M0 scales of 32, four in a block: the conversion takes a scale relative to the
  // block's largest and the fold that one.  Relative scales of at least 2^-13 keep e2m1's values (from 0.5 on)
  // normal in fp16, so exact; a wave that holds a smaller one folds that block's groups one by one.  Four folds
  // a block for all instead: 64 rows, 18432 x 7168, 106 us (38.7 now); 16 rows 25.0 (20.4); 1 row 22.9 (17.3).
  // Groups of 64 could do the same with their two scales; they fold twice a block (35.5, 20.4 and 17.5 us).
  static constexpr bool kRelative = W == kFp4E8M0 && F16 && GROUP == 32;
  static constexpr int kSpread = 13;
  static constexpr int kPerScale = kFold && !kRelative ? GROUP / 32 : 4;  // MFMAs that share a fold
  static constexpr int kFolds = 4 / kPerScale;                            // folds of a block
  static constexpr int kScaleBytes = W == kFp4 ? 4 : 1;

  static constexpr bool kMixed = kFold && !kRelative && GROUP < 128;  // an operand holds one group's codes
  static constexpr bool kNatural = W == kW16 || (kMixed && GROUP == 32);  // lane group g reads x's chunk 4 i + g

  // 8-wide chunk of x's block that goes with operand i of lane group g
  static __device__ __forceinline__ int xchunk(int i, int g) {
    if constexpr (kNatural) return 4 * i + g;
    if constexpr (kMixed && GROUP == 64) return 8 * (i >> 1) + (i & 1) + 4 * (g & 1) + 2 * (g >> 1);
    return 4 * g + i;
  }
  static __device__ __forceinline__ void arrange(u32x4& q) {
    if constexpr (kMixed) {
      uint32_t d[4] = {q[0], q[1], q[2], q[3]};
      swap32(d[0], d[2]);
      swap32(d[1], d[3]);
      if constexpr (GROUP == 32) {
        swap16(d[0], d[1]);
        swap16(d[2], d[3]);
      }
      q = u32x4{d[0], d[1], d[2], d[3]};
    }
  }
};

// MR: rows of x per pass; CT: 16-column tiles per wave; CW x KW multiplying waves; H: 128-wide blocks
// of a wave in a stage; S: stages; NP: copying waves.
template <int W, int GROUP, bool F16, int MR, int CT, int CW, int KW, int H, int S, int NP>
struct Skinny {
  using Fm = Format<W, GROUP, F16>;
  static constexpr int MT = MR > 16 ? MR / 16 : 1;
  static constexpr int NW = CW * KW, NC = 16 * CT * CW;
  static constexpr int kK = 128 * H * KW;                       // k of a stage
  static constexpr int kRowChunks = KW * H * Fm::kChunks;       // of a weight row in a stage
  using WSlots = WeightSlots<kRowChunks>;
  using RowSlots = XSlots<MR, Fm::kNatural ? 1 : 4>;
  static constexpr int kWBytes = NC * kRowChunks * 16;          // weights of a stage
  static constexpr int kXBytes = MR * kK * 2;
  static constexpr int kStage = kWBytes + kXBytes;
  static constexpr int kDmaW = kWBytes / 1024, kDmaX = kXBytes / 1024;
  static constexpr int kInFlight = (S - 2) * (kDmaW + kDmaX) / NP > 63 ? 63 : (S - 2) * (kDmaW + kDmaX) / NP;
  static constexpr int kPart = NW * MT * CT * 1024;
  static constexpr int kWindowStages = 2048 / kK > 4 ? 2048 / kK : 4;  // stages of a window of scales
  static constexpr int kSpan = kWindowStages * kK;                     // and its k
  static constexpr int kWindow = kSpan / GROUP;                        // and its scales of a row
  static_assert(kWindowStages >= S, "a window of scales outlives the stages in flight");
  static_assert(S * kStage + (W == kW16 ? 0 : 2 * NC * kWindow * Fm::kScaleBytes) <= 160 * 1024, "LDS of a workgroup");
  static_assert(kDmaW % NP == 0 && kDmaX % NP == 0, "the copying waves share the DMAs evenly");
  static_assert(kWBytes % 1024 == 0 && kXBytes % 1024 == 0, "whole DMAs");
  static int stages(int K) { return (K + kK - 1) / kK; }
  // slots of a row in a window: a power of two that holds the row's scales or kWindow of them
  static int scale_slots(int K) {
    const int need = (K > kSpan ? kSpan : stages(K) * kK) / GROUP;
    int n = 4;
    while (n < need) n *= 2;
    return n;
  }
  // two windows when a row has more than one
  static int lds_bytes(int K) {
    const int scales = W == kW16 ? 0 : (K > kSpan ? 2 : 1) * NC * scale_slots(K) * Fm::kScaleBytes;
    const int run = S * kStage + scales;
    return run > kPart ? run : kPart;
  }
};

// slots: scales of a row in a window (a power of two); loose: E8M0 rows that do not start on dwords
// (their scales are read from memory where they are used).
template <int W, int GROUP, bool F16, int MR, int CT, int CW, int KW, int H, int S, int NP>
__global__ __launch_bounds__((CW * KW + NP) * 64) void skinny_kernel(SkinnyArgs a, int slots, int loose) {
  using Sk = Skinny<W, GROUP, F16, MR, CT, CW, KW, H, S, NP>;
  using Fm = typename Sk::Fm;
  constexpr int MT = Sk::MT, NW = Sk::NW;
  extern __shared__ __align__(16) uint8_t smem[];  // stages, windows of scales; at the end the waves' tiles
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = blockIdx.y, n0 = blockIdx.x * Sk::NC;
  int lo = 0, hi = a.R;
  if (a.offsets) segment(a.offsets, a.R, e, lo, hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  if (lo == hi) return;
  // this workgroup's stages: all, or one of `splits` runs of them
  const int all = (a.K + Sk::kK - 1) / Sk::kK, per = (all + a.splits - 1) / a.splits;
  const int split = blockIdx.z % a.splits, s0 = min(all, split * per), s1 = min(all, s0 + per);
  const int zrow = blockIdx.z / a.splits, zrows = gridDim.z / a.splits;
  const int G = W == kW16 ? 0 : (a.K + GROUP - 1) / GROUP;
  const int64_t srowbytes = (int64_t)G * Fm::kScaleBytes;
  const uint8_t* scales = reinterpret_cast<const uint8_t*>(a.scale) + ((int64_t)e * a.N + n0) * srowbytes;
  const int cols = min(a.N - n0, Sk::NC);
  const uint32_t lds0 = lds_addr(smem), lds_scale = lds0 + S * Sk::kStage;
  const uint32_t window = Sk::NC * slots * Fm::kScaleBytes;  // bytes

  // unsigned: a row number past the segment may exceed 2^31
  const uint32_t end = hi;
  for (uint32_t m0 = lo + zrow * MR; m0 < end; m0 += zrows * MR) {
    if (w >= NW) {
      const int part = w - NW;
      const int64_t rowbytes = (int64_t)a.K * 16 / Fm::kPerChunk;
      const int rows = min((int)(end - m0), MR);
      const uint8_t* wp = a.w + ((int64_t)e * a.N + n0) * rowbytes + (int64_t)s0 * Sk::kRowChunks * 16;
      const uint8_t* xp = reinterpret_cast<const uint8_t*>(a.x + (int64_t)m0 * a.ldx) + (int64_t)s0 * Sk::kK * 2;
      int64_t wlen = cols * rowbytes - (int64_t)s0 * Sk::kRowChunks * 16;
      int64_t xlen = ((int64_t)(rows - 1) * a.ldx + a.K) * 2 - (int64_t)s0 * Sk::kK * 2;
      RowCopy<Sk::kDmaW, Sk::kRowChunks, typename Sk::WSlots> wc;
      RowCopy<Sk::kDmaX, Sk::kK / 8, typename Sk::RowSlots> xc;
      wc.init(lane, rowbytes);
      xc.init(lane, a.ldx * 2);
      auto fetch = [&](int s) {
        if (s >= s1) return;
        const uint32_t dst = lds0 + (s % S) * Sk::kStage;
        const u32x4 wd = dma_buffer(wp, wlen), xd = dma_buffer(xp, xlen);
        const int left = a.K - s * Sk::kK;
        if (left >= Sk::kK) {
          wc.template copy<false, NP>(wd, dst, (uint32_t)rowbytes, 0, part);
          xc.template copy<false, NP>(xd, dst + Sk::kWBytes, (uint32_t)a.ldx * 2, 0, part);
        } else {
          wc.template copy<true, NP>(wd, dst, (uint32_t)rowbytes, (left + Fm::kPerChunk - 1) / Fm::kPerChunk, part);
          xc.template copy<true, NP>(xd, dst + Sk::kWBytes, (uint32_t)a.ldx * 2, left / 8, part);
        }
        if constexpr (W != kW16) {
          if ((s == s0 || s % Sk::kWindowStages == 0) && !loose) {
            // dword i of the window: row i / (dwords of a row), swizzled; dwords past the row's end are zeros
            const int q = s / Sk::kWindowStages, sh = 31 - __builtin_clz(slots * Fm::kScaleBytes / 4);
            const int first = q * Sk::kWindow * Fm::kScaleBytes;
            const u32x4 sd = dma_buffer(scales, cols * srowbytes);
            const uint32_t win = lds_scale + (q & 1) * window;
            for (int i0 = 64 * part; i0 < (Sk::NC << sh); i0 += 64 * NP) {
              const int i = i0 + lane, r = i >> sh, at = first + ((i - (r << sh)) ^ scale_swz(r, sh)) * 4;
              if (i < Sk::NC << sh)
                dma4_buf(sd, at < srowbytes ? (uint32_t)r * (uint32_t)srowbytes + at : kPastEnd, win + i0 * 4);
            }
          }
        }
        wp += Sk::kRowChunks * 16;
        xp += Sk::kK * 2;
        wlen -= Sk::kRowChunks * 16;
        xlen -= Sk::kK * 2;
      };
#pragma unroll 1
      for (int s = s0; s < s0 + S - 1; ++s) fetch(s);
#pragma unroll 1
      for (int s = s0; s < s1; ++s) {
        // stage s has landed when only the S - 2 stages after it are in flight
        if (s + S - 1 <= s1) {
          vm_wait<Sk::kInFlight>();
        } else {
          vm_wait<0>();
        }
        barrier_only();  // stage s is there; stage s - 1 has been read
        fetch(s + S - 1);
      }
      barrier_only();
    } else {
      const int cw = w / KW, kw = w % KW, r = lane & 15;
      // weights: row r of a tile, chunk (kw, block, g); x: row r, chunk (kw, block, operand)
      uint32_t wat[H][Fm::kLoads], xat[4];
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int i = 0; i < Fm::kLoads; ++i)
          wat[h][i] = (cw * CT * 16 + r) * (Sk::kRowChunks * 16) +
                      ((((kw * H + h) * Fm::kChunks + 4 * i + g) ^ Sk::WSlots::of(r)) << 4);
      const int xr = r & (MR < 16 ? MR - 1 : 15);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xat[i] = Sk::kWBytes + xr * (Sk::kK * 2) + ((kw * H * 16 + (Fm::xchunk(i, g) ^ Sk::RowSlots::of(xr))) << 4);
      const int swz = scale_swz(r, 31 - __builtin_clz(slots * Fm::kScaleBytes / 4)) * (4 / Fm::kScaleBytes);
      // the lane's column, the wave's first group of a stage; E8M0 in the conversion: the lane's own group
      const int col = cw * CT * 16 + r;
      const int sgroup = kw * H * 128 / GROUP + (Fm::kDirect ? 32 * g / GROUP : 0);

      v4f acc[MT][CT];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[t][c] = v4f{0.f, 0.f, 0.f, 0.f};
      typedef __attribute__((address_space(3))) const u32x4* pv;
      typedef __attribute__((address_space(3))) const s16x8* px;
      typedef __attribute__((address_space(3))) const uint32_t* pu;
      typedef __attribute__((address_space(3))) const uint8_t* pb;

#pragma unroll 1
      for (int s = s0; s < s1; ++s) {
        barrier_only();
        const uint32_t st = lds0 + (s % S) * Sk::kStage;
        const uint32_t win = lds_scale + (s / Sk::kWindowStages & 1) * window;
        const int sw = s % Sk::kWindowStages * (Sk::kK / GROUP) + sgroup;  // slot in the window
        // fp16 x with E8M0 scales of 64, 64 x 32 results a wave and 168 registers (more than 8 waves): what takes
        // registers through the loop (without this 7 are spilled, one of them read back in each stage) is computed
        // here, from values that the compiler must take for new.
        constexpr bool kTight = W == kFp4E8M0 && Fm::kFolds > 1 && MT * CT >= 8 && NW + NP > 8;
        int apart = loose;
        uint32_t x0 = xat[0];
        if constexpr (kTight) asm volatile("" : "+s"(apart), "+v"(x0));
        auto scale_of = [&](int c, int at) -> uint32_t {                   // of tile c, group `at` on from sgroup
          const int row = col + 16 * c;
          if constexpr (W == kFp4) {
            return *reinterpret_cast<pu>(win + (row * slots + ((sw + at) ^ swz)) * 4);
          } else {
            if (apart) {
              int from = min(row, cols - 1);
              if constexpr (kTight) asm volatile("" : "+v"(from));
              return scales[from * srowbytes + min(s * (Sk::kK / GROUP) + sgroup + at, G - 1)];
            }
            return *reinterpret_cast<pb>(win + row * slots + ((sw + at) ^ swz));
          }
        };
        auto scales_of = [&](int c, int at) -> uint32_t {  // E8M0 of 32: the four of a block, a byte each
          const int row = col + 16 * c;
          if (!loose) return *reinterpret_cast<pu>(win + row * slots + ((sw + at) ^ swz));
          uint32_t v = 0;
          for (int j = 0; j < 4; ++j) v |= scale_of(c, at + j) << 8 * j;
          return v;
        };
#pragma unroll
        for (int h = 0; h < H; ++h) {
          s16x8 x[MT][4];
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t from = kTight ? x0 ^ (Fm::xchunk(i, 0) << 4) : xat[i];
              x[t][i] = *reinterpret_cast<px>(st + from + h * 256 + t * 16 * (Sk::kK * 2));
            }
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            u32x4 q[Fm::kLoads];
#pragma unroll
            for (int i = 0; i < Fm::kLoads; ++i)
              q[i] = *reinterpret_cast<pv>(st + wat[h][i] + c * 16 * (Sk::kRowChunks * 16));
            uint32_t sv[Fm::kFolds];
            if constexpr (W != kW16) {
#pragma unroll
              for (int i = 0; i < Fm::kFolds && !Fm::kRelative; ++i) sv[i] = scale_of(c, h * (128 / GROUP) + i);
              Fm::arrange(q[0]);
            }
            v4f tile[MT];
            float conv = 1.0f;  // the conversion reads the scale's exponent field (0 as 2^-127)
            if constexpr (Fm::kDirect) conv = __uint_as_float(sv[0] << 23);
            if constexpr (Fm::kRelative) {
              const uint32_t all = scales_of(c, 4 * h);
              sv[0] = max(max(all & 255, all >> 8 & 255), max(all >> 16 & 255, all >> 24));
              const uint32_t below = sv[0] - (all >> 8 * g & 255);
              conv = __uint_as_float((127 - below) << 23);
              if (__any(below > Fm::kSpread)) {  // rare: each group by itself, the other lanes' x and codes zero
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                  const bool mine = g == j;
                  const float scale = e8m0_to_f32(all >> 8 * j & 255);
#pragma unroll
                  for (int t = 0; t < MT; ++t) {
                    tile[t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      uint32_t codes = mine ? q[0][i] : 0u;
                      asm volatile("" : "+v"(codes));  // converted anew for each t: no registers to keep it in
                      tile[t] = mfma16x16x32<F16>(mine ? x[t][i] : s16x8{}, e2m1x8<F16>(codes, 1.0f), tile[t]);
                      __builtin_amdgcn_sched_barrier(0);
                    }
                    acc[t][c] += tile[t] * scale;
                  }
                }
                continue;
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              s16x8 b;
              if constexpr (W == kW16) {
                const u32x4 v = q[i];
                b = __builtin_bit_cast(s16x8, v);
              } else {
                b = e2m1x8<F16>(q[0][i], conv);
              }
              const bool first = i % Fm::kPerScale == 0, last = i % Fm::kPerScale == Fm::kPerScale - 1;
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                if constexpr (!Fm::kFold) {
                  acc[t][c] = mfma16x16x32<F16>(x[t][i], b, acc[t][c]);
                } else {
                  tile[t] = mfma16x16x32<F16>(x[t][i], b, first ? v4f{0.f, 0.f, 0.f, 0.f} : tile[t]);
                  if (last) {
                    const uint32_t u = sv[i / Fm::kPerScale];
                    acc[t][c] += tile[t] * (W == kFp4 ? __uint_as_float(u) : e8m0_to_f32(u));
                  }
                }
              }
            }
            if constexpr (Fm::kFold && MT * CT >= 8) __builtin_amdgcn_sched_barrier(0);  // and of one tile
          }
          __builtin_amdgcn_sched_barrier(0);  // keeps the operands of one block in registers at a time
        }
      }
      if constexpr (Fm::kDirect) {
        // Under a byte of 253 or 254 the larger e2m1 values leave bf16's range: such a weight arrived as an infinity,
        // and none of its products left a finite sum.  If a sum is not finite and a byte is that large, the wave
        // takes its sums again, from memory, with weights of a quarter (18432 x 7168: 1 row 15.8 us without the
        // check and 15.9 with it, 64 rows 32.6 and 33.2; looking at each byte in the loop 19.0 and 36.5, for its
        // branches between the conversions and the MFMAs).
        float z = 0.0f;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) z = __builtin_fmaf(acc[t][c][i], 0.0f, z);
        if (__any(!(z == 0.0f))) {
          int again = lane;
          asm volatile("" : "+v"(again));  // the places below: not kept in registers through the loop above
          const int g = again >> 4, r = again & 15, col = cw * CT * 16 + r;
          const int kend = min(a.K, s1 * Sk::kK);
          bool high = false;
#pragma unroll 1
          for (int k = s0 * Sk::kK + 32 * g; k < kend; k += 128)
#pragma unroll 1
            for (int n = col; n < min(cols, col + 16 * CT); n += 16) {
              const uint32_t byte = scales[n * srowbytes + k / GROUP];
              high |= byte == 253 || byte == 254;
            }
          if (__any(high)) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
              for (int c = 0; c < CT; ++c) acc[t][c] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int j = 0; j < (s1 - s0) * H * 4; ++j) {
              // 8 of the lane's 32 k of a block
              const int b = j >> 2, k = (s0 + b / H) * Sk::kK + (kw * H + b % H) * 128 + 32 * g + 8 * (j & 3);
              s16x8 x[MT];
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                x[t] = s16x8{};
                if (16 * t + r < min((int)(end - m0), MR) && k < a.K)
                  x[t] = *reinterpret_cast<const s16x8*>(a.x + (int64_t)(m0 + 16 * t + r) * a.ldx + k);
              }
#pragma unroll
              for (int c = 0; c < CT; ++c) {
                const int n = col + 16 * c;
                uint32_t codes = 0;
                float quarter = 0.0f;
                if (n < cols && k < a.K) {
                  codes = *reinterpret_cast<const uint32_t*>(a.w + (((int64_t)e * a.N + n0 + n) * a.K + k) / 2);
                  quarter = e8m0_to_f32(scales[n * srowbytes + k / GROUP]) * 0.25f;
                }
                const s16x8 b8 = e2m1x8_times(codes, quarter);
#pragma unroll
                for (int t = 0; t < MT; ++t) acc[t][c] = mfma16x16x32<F16>(x[t], b8, acc[t][c]);
                __builtin_amdgcn_sched_barrier(0);
              }
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
              for (int c = 0; c < CT; ++c) acc[t][c] *= 4.0f;
          }
        }
      }
      barrier_only();  // every stage has been read: the tiles may overwrite them
      v4f* part = reinterpret_cast<v4f*>(smem);
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) part[((w * MT + t) * CT + c) * 64 + lane] = acc[t][c];
    }
    __syncthreads();
    const v4f* part = reinterpret_cast<const v4f*>(smem);
    for (int j = w; j < CW * MT * CT; j += NW + NP) {
      const int c = j % CT, t = j / CT % MT, cc = j / CT / MT;
      v4f s = part[((cc * KW * MT + t) * CT + c) * 64 + lane];
#pragma unroll
      for (int k = 1; k < KW; ++k) s += part[(((cc * KW + k) * MT + t) * CT + c) * 64 + lane];
      const int n = n0 + (cc * CT + c) * 16 + (lane & 15);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t m = m0 + 16 * t + 4 * g + i;
        if (m >= end || m >= m0 + MR || n >= a.N) continue;
        if (a.splits > 1) {
          a.part[((int64_t)split * a.R + m) * a.N + n] = s[i];
        } else {
          a.c[(int64_t)m * a.ldc + n] = (uint16_t)f32_to_out16(s[i], F16);
        }
      }
    }
    __syncthreads();
  }
}

// c = rounded sum of the splits' partial sums, in split order.
template <bool F16>
__global__ __launch_bounds__(256) void skinny_reduce_kernel(SkinnyArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, count = (int64_t)a.R * a.N;
  if (i >= count) return;
  float s = a.part[i];
  for (int k = 1; k < a.splits; ++k) s += a.part[k * count + i];
  const int64_t m = i / a.N;
  a.c[m * a.ldc + (i - m * a.N)] = (uint16_t)f32_to_out16(s, F16);
}

template <int W, int GROUP, bool F16, int MR, int CT, int CW, int KW, int H, int S, int NP>
int launch_tile(SkinnyArgs g, hipStream_t stream) {
  using Sk = Skinny<W, GROUP, F16, MR, CT, CW, KW, H, S, NP>;
  const int64_t nx = ceil_div64(g.N, Sk::NC), passes = ceil_div64(g.R, MR);
  // Passes of one expert run side by side while the grid is small (an expert may hold most of the rows);
  // a large grid of mostly empty workgroups would cost more than it gives.
  const int64_t side = 4096 / (nx * g.E) > 1 ? 4096 / (nx * g.E) : 1;
  const int64_t nz = (g.offsets ? (passes < side ? passes : side) : passes) * g.splits;
  constexpr int kThreads = (CW * KW + NP) * 64;
  MOE355_CHECK(nx * kThreads < (1ll << 32) && nz < 65536, MOE355_EUNSUPPORTED);  // threads of a launch
  auto* fn = &skinny_kernel<W, GROUP, F16, MR, CT, CW, KW, H, S, NP>;
  const int lds = Sk::lds_bytes(g.K), G = (g.K + GROUP - 1) / GROUP;
  const int loose = W == kFp4E8M0 && (G % 4 != 0 || (reinterpret_cast<uintptr_t>(g.scale) & 3u) != 0);
  hipLaunchKernelGGL(fn, dim3((unsigned)nx, (unsigned)g.E, (unsigned)nz), dim3(kThreads), lds, stream, g,
                     Sk::scale_slots(g.K), loose);
  if (g.splits > 1)
    hipLaunchKernelGGL(skinny_reduce_kernel<F16>, dim3((unsigned)ceil_div64((int64_t)g.R * g.N, 256)), dim3(256), 0,
                       stream, g);
  return launch_status();
}

// Columns of a workgroup for one matrix of more than 16 rows: 128 where that gives half of the CUs one.  Else
// K is split over workgroups (skinny_splits): 64 columns above 32 rows where there are many columns and a
// long K, else 32.
int skinny_cols(int64_t M, int64_t N, int64_t K) {
  const int64_t passes = ceil_div64(M, M <= 32 ? 32 : 64);
  if (ceil_div64(N, 128) * passes >= 128) return 128;
  return M > 32 && K > 4096 && ceil_div64(N, 64) * passes >= 64 ? 64 : 32;
}

// The tiling of a launch.  Rows of a pass (MR): the rows of a matrix, of an expert on average; one that
// has more takes another pass over weights that the caches still hold.  Columns of a workgroup: as many
// as still give the CUs enough workgroups.  Measured, us (4-bit weights; the choice first):
//   1 row, 2048 x 7168:      16 columns 6.4, 32 columns 9.2
//   1 row, 18432 x 7168:     32 columns 15.7, 16 16.3, 64 17.2
//   8 rows, 4096 x 7168:     8 rows a pass 7.8, 16 8.4
//   16 rows, 18432 x 7168:   32 columns in two stages of two blocks 22.2, 64 24.0 (E8M0);
//                            128 columns 19.2, 32 22.0 (fp32 scales)
//   32 rows, 18432 x 7168:   128 columns with K in two 24.2, K in one 26.7
//   32 rows, 4096 x 7168:    32 columns and 2 runs of K 11.6, 64 and 4 12.1
//   64 rows, 18432 x 7168:   128 columns with K in two 35.3, 256 columns and 3 runs of K 38.8
//   64 rows, 7168 x 18432:   64 columns and 2 runs of K 36.3, four copying waves 38.5, 32 columns and 1 run 47
//   64 rows, 2048 x 7168:    32 columns and 4 runs of K 11.7, 64 and 7 12.9, 32 and 1 18
//   48 rows, 7168 x 2048:    32 columns 8.5, 64 and 2 runs of K 11.4
//   one token's 8 experts of 4096 x 7168: 64 columns with K in two 34.5, in one 36.6, 128 columns 38.1
//   512 rows over 256 experts: of 7168 x 2048, 16 rows a pass and 128 columns 282, 8 and 64 304;
//                              of 4096 x 7168, 8 rows a pass and 64 columns 572, 16 and 128 632
//   2048 rows over 64 experts of 4096 x 7168: 64 rows a pass and 256 columns 283, 128 292; 32 rows 388
template <int W, int GROUP, bool F16>
int launch(const SkinnyArgs& g, hipStream_t stream) {
  constexpr int H = W == kW16 ? 1 : 2;  // 4-bit rows: whole 128-byte lines
  const int64_t mats = g.offsets && g.R < g.E ? g.R : g.E;       // with rows, at most
  const int64_t rows = g.offsets ? ceil_div64(g.R, g.E) : g.R;  // of a matrix, on average
  auto groups = [&](int cols) { return ceil_div64(g.N, cols) * mats; };
  if constexpr (W != kW16) {
    if (!g.offsets && rows <= 4) {
      if (groups(64) >= 512) return launch_tile<W, GROUP, F16, 4, 2, 2, 2, H, 3, 2>(g, stream);
      if (groups(32) < 192) return launch_tile<W, GROUP, F16, 4, 1, 1, 4, H, 3, 4>(g, stream);
      return launch_tile<W, GROUP, F16, 4, 1, 2, 2, H, 3, 2>(g, stream);
    }
  }
  const bool wide = groups(128) >= 1024;
  // over a short K another pass for the experts of more than 8 rows costs more than wider passes for all
  const bool at_once = W != kW16 && g.offsets && wide && g.K < 4096;
  if (rows <= (g.offsets ? 4 : 8) && !at_once) {
    if constexpr (W == kW16) {
      if (wide) return launch_tile<W, GROUP, F16, 8, 2, 4, 1, 1, 3, 2>(g, stream);
    } else {
      if (wide) return launch_tile<W, GROUP, F16, 8, 1, 4, 1, H, 3, 4>(g, stream);
    }
    if (groups(64) >= 512) return launch_tile<W, GROUP, F16, 8, 2, 2, 2, H, W == kW16 ? 4 : 3, 2>(g, stream);
    if (groups(32) < 192) return launch_tile<W, GROUP, F16, 8, 1, 1, 4, H, 3, 4>(g, stream);
    return launch_tile<W, GROUP, F16, 8, 1, 2, 2, H, 3, 2>(g, stream);
  }
  if (rows <= (g.offsets ? 12 : 16)) {
    if constexpr (W == kW16) {
      if (wide) return launch_tile<W, GROUP, F16, 16, 2, 4, 1, 1, 3, 4>(g, stream);
    } else {
      if (wide) return launch_tile<W, GROUP, F16, 16, 4, 2, 2, 1, 3, 4>(g, stream);
    }
    if (groups(64) >= 512) return launch_tile<W, GROUP, F16, 16, 2, 2, 2, 1, 3, 4>(g, stream);
    if (groups(32) < 192) return launch_tile<W, GROUP, F16, 16, 1, 1, 4, H, 3, 4>(g, stream);
    if constexpr (W == kFp4 && GROUP == 128) {  // the fewest scales: 128 columns' fit beside the stages
      if (groups(128) >= 128) return launch_tile<W, GROUP, F16, 16, 2, 4, 2, H, 3, 4>(g, stream);
    }
    return launch_tile<W, GROUP, F16, 16, 1, 2, 2, H, W == kW16 ? 3 : 2, W == kW16 ? 2 : 4>(g, stream);
  }
  if constexpr (W == kW16) return MOE355_EUNSUPPORTED;  // more rows are the tiled product's
  if constexpr (W != kW16) {
    if (g.offsets) {
      if (rows <= 20) return launch_tile<W, GROUP, F16, 32, 2, 4, 1, 2, 2, 4>(g, stream);
      // 256 columns' fp32 scales of 32 or 64 do not fit, and folding E8M0 of 64 or 128 takes too many registers
      if constexpr (W == kFp4 ? GROUP == 128 : !F16 || GROUP == 32) {
        return launch_tile<W, GROUP, F16, 64, 2, 8, 1, 2, 2, 4>(g, stream);
      } else {
        return launch_tile<W, GROUP, F16, 64, 2, 4, 1, 1, 3, 4>(g, stream);
      }
    }
    const int cols = skinny_cols(g.R, g.N, g.K);
    if (rows <= 32) {
      if (cols == 128) return launch_tile<W, GROUP, F16, 32, 2, 4, 2, 1, 3, 8>(g, stream);
      return launch_tile<W, GROUP, F16, 32, 1, 2, 2, 2, 3, 4>(g, stream);
    }
    constexpr int S = W == kFp4 && GROUP < 128 ? 2 : 3;  // three stages and the fp32 scales do not fit
    if (cols == 128) return launch_tile<W, GROUP, F16, 64, 2, 4, 2, 1, S, 4>(g, stream);
    constexpr int NP = Format<W, GROUP, F16>::kRelative ? 4 : 8;  // 16 waves leave its registers too few
    if (cols == 64) return launch_tile<W, GROUP, F16, 64, 1, 4, 2, 1, 3, NP>(g, stream);
    return launch_tile<W, GROUP, F16, 64, 1, 2, 2, 1, 3, 4>(g, stream);
  }
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

int skinny_splits(int M, int N, int K) {
  const int cols = skinny_cols(M, N, K);
  if (M <= 16 || cols == 128) return 1;
  // as many runs of K, of at least 1024, as give each of the 256 CUs a workgroup
  const int64_t tiles = ceil_div64(N, cols) * ceil_div64(M, M <= 32 ? 32 : 64), runs = ceil_div64(K, 1024);
  const int64_t s = tiles >= 256 ? 1 : 256 / tiles;
  return (int)(s < runs ? s : runs);
}

int launch_skinny(const SkinnyArgs& g, int weights, int group, int fp16, hipStream_t stream) {
  if (weights == kW16) return fp16 ? launch<kW16, 128, true>(g, stream) : launch<kW16, 128, false>(g, stream);
  if (weights == kFp4) return fp16 ? by_group<kFp4, true>(g, group, stream) : by_group<kFp4, false>(g, group, stream);
  return fp16 ? by_group<kFp4E8M0, true>(g, group, stream) : by_group<kFp4E8M0, false>(g, group, stream);
}

}  // namespace moe355
