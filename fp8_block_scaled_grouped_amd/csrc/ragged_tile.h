// What the tiled products over ragged row segments share: a workgroup's expert, row tile and column
// tile, found from the offsets on the device, and the stores of its sums.
#pragma once

#include "frag16.h"

namespace moe355 {
namespace {

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
__device__ __forceinline__ bool place(const int32_t* offsets, int R, int E, int ntiles, int* sh, int& e, int& mt, int& nt) {
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid < 64) {
    const int per = (E + 63) / 64;
    const int e0 = min(E, lane * per), e1 = min(E, e0 + per);
    int mine = 0;
    for (int i = e0; i < e1; ++i) mine += row_tiles(offsets, R, i, BM);
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
          const int m = row_tiles(offsets, R, i, BM);
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

// Stores a wave's sums: lane l holds of tile (i, j) the row 16 i + l % 16 and the four columns from
// 16 j + 4 (l / 16), counted from wm and wn in the workgroup's tile, whose first row and column in c are row0 and
// n0; mrows and nrows (a multiple of 8, or of 4 in fp32) are left from there on.
template <bool F16, bool OUT32, int TM, int TN>
__device__ __forceinline__ void store_tile(const v4f (&acc)[TM][TN], void* c, int64_t ldc, int64_t row0, int n0, int mrows,
                                           int nrows, int wm, int wn, int lane) {
  const int nw = wn + 4 * (lane >> 4);
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
        const int m = wm + 16 * i + (lane & 7);
        float* out = reinterpret_cast<float*>(c) + (row0 + m) * ldc + n0 + n;
        if (m < mrows) *reinterpret_cast<v4f*>(out) = first;
        if (m + 8 < mrows) *reinterpret_cast<v4f*>(out + 8 * ldc) = second;
      }
    }
  } else {
    const int mw = wm + (lane & 15);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = mw + 16 * i;
      if (m >= mrows) continue;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int n = nw + 16 * j;
        if (n >= nrows) continue;  // the four are all in or all out
        const int64_t at = (row0 + m) * ldc + n0 + n;
        if constexpr (OUT32) {
          *reinterpret_cast<v4f*>(reinterpret_cast<float*>(c) + at) = acc[i][j];
        } else {
          const uint2 r{f32_to_out16(acc[i][j][0], F16) | (f32_to_out16(acc[i][j][1], F16) << 16),
                        f32_to_out16(acc[i][j][2], F16) | (f32_to_out16(acc[i][j][3], F16) << 16)};
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(c) + at) = r;
        }
      }
    }
  }
}

}  // namespace
}  // namespace moe355
