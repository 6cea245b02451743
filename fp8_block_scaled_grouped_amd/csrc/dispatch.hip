// Tokens to the rows of their experts and back ("Accelerate DeepSeek-R1 Inference: Integrate AITER
// into SGLang", section "MoE Sorting": token-expert pairs bucketed per expert), without padding:
// the rows of an expert are a segment [offsets[e], offsets[e+1]) as the ragged products take it.
//
// moe_group         the stable order of the pairs by expert
// moe_dispatch      rows[row_of_pair[t, j]] = x[t]
// moe_combine       out[t] = sum_j w[t, j] rows[row_of_pair[t, j]]
// moe_combine_grad  drows[row_of_pair[t, j]] = w[t, j] dout[t],  dw[t, j] = <dout[t], rows[row_of_pair[t, j]]>
//
// A pair without a row (row_of_pair -1) is left out of every sum.  All but moe_group are bound by the
// bytes of the rows, so one wave takes a token's 64 vectors of 16 bytes, the token's places
// come through scalar loads, and every sum has a fixed order.  8192 tokens x 8 of 7168 in bf16, 1.06 GB either way: moe_dispatch 180 us,
// moe_combine 205, and 240 behind a kernel whose writes still leave the caches (5.0 TB/s the two together, a large copy's rate);
// there rows loaded two, four or eight at a time take the same.  Few tokens wait: a pair's place, then its weight and row, then the
// next pair's; 64 tokens x 8 of 7168, less than a wave a SIMD, 3.8 us with the rows in the caches and 7.2 without (bytes: 1.6).
#include "device_common.h"
#include "host_common.h"

namespace moe355 {
namespace {

constexpr int kMaxE = 1024;

// ------------------------------------------------------------------ moe_group
constexpr int kWaves = 16;                   // of a workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kOneChunk = 4096;              // up to here one workgroup takes all pairs
constexpr int kMaxChunks = 256;

// Where pair p's id stands: ids are dense (ld = 0) or in rows of k, ld apart.
__device__ __forceinline__ int expert_of(const int32_t* ids, int64_t ld, uint32_t k, int E, uint32_t p) {
  const int e = ids[ld == 0 ? (int64_t)p : (int64_t)(p / k) * ld + p % k];
  return e >= 0 && e < E ? e : -1;
}

__global__ __launch_bounds__(kThreads) void group_count_kernel(const int32_t* __restrict__ ids, int64_t ld, int k, uint32_t n,
                                                               int E, uint32_t chunk, int32_t* __restrict__ counts) {
  __shared__ int hist[kMaxE];
  for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
  __syncthreads();
  const uint32_t c0 = blockIdx.x * chunk, c1 = min(n, c0 + chunk);
  for (uint32_t p = c0 + threadIdx.x; p < c1; p += kThreads) {
    const int e = expert_of(ids, ld, k, E, p);
    if (e >= 0) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

// Chunk blockIdx.x of the pairs (all of them with one chunk), each wave a contiguous part.  counts: [chunks][E] histograms of the
// chunks, or NULL with one chunk.
// A wave counts its part's experts in LDS; prefixes over waves, chunks and experts give each wave the first row of
// every expert, and a second walk over the part ranks each pair among the 64 at hand: ballots over the bits
// of the expert find the lanes with the same one, and the lowest of them moves the expert's next row on.
// Bound by latency: 64 tokens x 8 of 256 experts, one launch, 5.5 us; 8192 tokens x 8, two launches of 16 workgroups, 3.3 + 8 us (with chunks
// of 1024 pairs and their counts added one by one 25).
__global__ __launch_bounds__(kThreads) void group_kernel(const int32_t* __restrict__ ids, int64_t ld, int k, uint32_t n, int E,
                                                         int bits, uint32_t chunk, const int32_t* __restrict__ counts,
                                                         int32_t* __restrict__ offsets, int32_t* __restrict__ row_of_pair,
                                                         int32_t* __restrict__ pair_of_row) {
  extern __shared__ int next[];  // [kWaves][E], then the sums of the waves
  int* wsum = next + kWaves * E;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const uint32_t c0 = blockIdx.x * chunk, c1 = min(n, c0 + chunk), part = (chunk / kWaves + 63) / 64 * 64;
  const uint32_t p0 = min(c1, c0 + w * part), p1 = min(c1, p0 + part);
  // the ids of a part of up to 256 pairs stay in registers
  constexpr int kHeld = kOneChunk / kThreads;
  int held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = p0 + 64 * i + lane < p1 ? expert_of(ids, ld, k, E, p0 + 64 * i + lane) : -1;
  for (int i = tid; i < kWaves * E; i += kThreads) next[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (held[i] >= 0) atomicAdd(&next[w * E + held[i]], 1);
  for (uint32_t p = p0 + 64 * kHeld + lane; p < p1; p += 64) {
    const int e = expert_of(ids, ld, k, E, p);
    if (e >= 0) atomicAdd(&next[w * E + e], 1);
  }
  __syncthreads();
  // per expert: rows in all chunks, and in the chunks before this one; then the scan over experts (at most one a thread)
  const int e = tid;
  int total = 0, before = 0;
  if (e < E) {
    if (counts) {
      constexpr int kBatch = 16;  // loads on their way at a time
      for (int b = 0; b < (int)gridDim.x; b += kBatch) {
        int v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) v[i] = b + i < (int)gridDim.x ? counts[(int64_t)(b + i) * E + e] : 0;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          total += v[i];
          before += b + i < (int)blockIdx.x ? v[i] : 0;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWaves; ++i) total += next[i * E + e];
    }
  }
  int upto = total;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(upto, o, 64);
    if (lane >= o) upto += v;
  }
  if (lane == 63) wsum[w] = upto;
  __syncthreads();
  int base = upto - total, all = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    base += i < w ? wsum[i] : 0;
    all += wsum[i];
  }
  if (e < E) {
    if (blockIdx.x == 0) {
      offsets[e] = base;
      if (e == E - 1) offsets[E] = all;
    }
    int at = base + before;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const int v = next[i * E + e];
      next[i * E + e] = at;
      at += v;
    }
  }
  __syncthreads();
  auto place = [&](int e, uint32_t p) {
    unsigned long long same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const unsigned long long set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    int row = -1;
    if (e >= 0) {
      // volatile: all lanes read their expert's next row before the lowest of them moves it, and the next 64 read it moved
      volatile int* at = next + w * E + e;
      const unsigned long long lower = same & ((1ull << lane) - 1);
      row = *at + __popcll(lower);
      if (lower == 0) *at = row + __popcll(same);
    }
    if (p < p1) {
      row_of_pair[p] = row;
      if (pair_of_row && row >= 0) pair_of_row[row] = (int)p;
    }
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (p0 + 64 * i < p1) place(held[i], p0 + 64 * i + lane);
  for (uint32_t q = p0 + 64 * kHeld; q < p1; q += 64) place(q + lane < p1 ? expert_of(ids, ld, k, E, q + lane) : -1, q + lane);
  if (pair_of_row)  // rows behind the last segment
    for (uint32_t r = all + blockIdx.x * kThreads + tid; r < n; r += gridDim.x * kThreads) pair_of_row[r] = -1;
}

// Chunks of 4096 pairs, longer ones where there would be more than kMaxChunks.
inline int64_t chunk_of(int64_t n) { return ceil_div64(n > 0 ? ceil_div64(n, kMaxChunks) : 1, kOneChunk) * kOneChunk; }

// ------------------------------------------------------------------ rows
template <int BYTES>
struct Vec;
template <>
struct Vec<16> { typedef u32x4 type; };
template <>
struct Vec<4> { typedef uint32_t type; };
template <>
struct Vec<2> { typedef uint16_t type; };
template <>
struct Vec<1> { typedef uint8_t type; };

// A wave's token and its 64 vectors
struct Place {
  int64_t t, v;
};
__device__ __forceinline__ Place place_of(int64_t chunks) {
  const int64_t i = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = i / chunks;
  return Place{t, (i - t * chunks) * 64 + (threadIdx.x & 63)};
}

template <int BYTES>
__global__ __launch_bounds__(256) void dispatch_kernel(const uint8_t* __restrict__ x, int64_t ld_x, int64_t T, int k, int R,
                                                       int64_t vecs, int64_t chunks,
                                                       const int32_t* __restrict__ row_of_pair,
                                                       uint8_t* __restrict__ rows, int64_t ld_rows) {
  typedef typename Vec<BYTES>::type V;
  const Place at = place_of(chunks);
  if (at.t >= T || at.v >= vecs) return;
  const V v = *reinterpret_cast<const V*>(x + at.t * ld_x + at.v * BYTES);
  const int32_t* to = row_of_pair + at.t * k;
  for (int j = 0; j < k; ++j) {
    const int r = to[j];
    if (r >= 0 && r < R) *reinterpret_cast<V*>(rows + r * ld_rows + at.v * BYTES) = v;
  }
}

// Element types: 0 bf16, 1 fp16, 2 fp32
template <int DT>
struct Elem { typedef uint16_t type; };
template <>
struct Elem<2> { typedef float type; };

template <int DT>
__device__ __forceinline__ float widen(typename Elem<DT>::type v) {
  if constexpr (DT == 2) return v;
  else if constexpr (DT == 1) return (float)__builtin_bit_cast(_Float16, v);
  else return bf16_to_f32(v);
}
template <int DT>
__device__ __forceinline__ typename Elem<DT>::type narrow(float v) {
  if constexpr (DT == 2) return v;
  else {
    // opaque: a product that the compiler joins with its conversion to fp16 (v_fma_mixlo_f16) is rounded once, others by
    // way of fp32, and the result would depend on which loads a call takes
    if constexpr (DT == 1) asm("" : "+v"(v));
    return (uint16_t)f32_to_out16(v, DT == 1);
  }
}

// N elements of a row: 16 bytes at a time where rows start on 16 bytes, else one by one
template <int DT, int N>
struct Pack {
  typename Elem<DT>::type v[N];
};
template <int DT, int N>
__device__ __forceinline__ Pack<DT, N> load_pack(const typename Elem<DT>::type* p) {
  if constexpr (N == 1) return Pack<DT, 1>{{*p}};
  typedef Pack<DT, N> P;
  static_assert(sizeof(P) == 16 || N == 1, "a vector of 16 bytes");
  if constexpr (N != 1) return __builtin_bit_cast(P, *reinterpret_cast<const u32x4*>(p));
}
template <int DT, int N>
__device__ __forceinline__ void store_pack(typename Elem<DT>::type* p, const Pack<DT, N>& v) {
  if constexpr (N == 1) *p = v.v[0];
  else *reinterpret_cast<u32x4*>(p) = __builtin_bit_cast(u32x4, v);
}

template <int DT, int N>
__global__ __launch_bounds__(256) void combine_kernel(const typename Elem<DT>::type* __restrict__ rows, int64_t ld_rows,
                                                      int64_t T, int k, int R, int64_t vecs, int64_t chunks,
                                                      const int32_t* __restrict__ row_of_pair,
                                                      const float* __restrict__ weights, int64_t ld_w,
                                                      typename Elem<DT>::type* __restrict__ out, int64_t ld_out) {
  const Place at = place_of(chunks);
  if (at.t >= T || at.v >= vecs) return;
  const int32_t* from = row_of_pair + at.t * k;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  for (int j = 0; j < k; ++j) {
    const int r = from[j];
    if (r < 0 || r >= R) continue;
    const float wt = weights ? weights[at.t * ld_w + j] : 1.0f;
    const Pack<DT, N> v = load_pack<DT, N>(rows + r * ld_rows + at.v * N);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += wt * widen<DT>(v.v[i]);
  }
  Pack<DT, N> o;
#pragma unroll
  for (int i = 0; i < N; ++i) o.v[i] = narrow<DT>(acc[i]);
  store_pack<DT, N>(out + at.t * ld_out + at.v * N, o);
}

// One wave a pair, four pairs a workgroup: those of a token read its gradient from the caches.  8192 tokens x 8 of 7168 (bf16), 2.0 GB:
// 385 us (5.2 TB/s); with a workgroup a token, pair after pair, 422.
template <int DT, int N>
__global__ __launch_bounds__(256) void combine_grad_kernel(const typename Elem<DT>::type* __restrict__ dout, int64_t ld_dout,
                                                           const typename Elem<DT>::type* __restrict__ rows,
                                                           int64_t ld_rows, int64_t pairs, int k, int R, int vecs,
                                                           const int32_t* __restrict__ row_of_pair,
                                                           const float* __restrict__ weights, int64_t ld_w,
                                                           typename Elem<DT>::type* __restrict__ drows, int64_t ld_drows,
                                                           float* __restrict__ dw) {
  const int64_t p = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (p >= pairs) return;
  const int lane = threadIdx.x & 63;
  const int64_t t = p / k;
  const int r = row_of_pair[p];
  float dot = 0.0f;
  if (r >= 0 && r < R) {
    const float wt = weights[t * ld_w + (p - t * k)];
    const auto* d = dout + t * ld_dout;
    const auto* y = rows + r * ld_rows;
    auto* o = drows + r * ld_drows;
    auto one = [&](int v, const Pack<DT, N>& a, const Pack<DT, N>& b) {
#pragma unroll
      for (int i = 0; i < N; ++i) dot += widen<DT>(a.v[i]) * widen<DT>(b.v[i]);
      if (drows) {
        Pack<DT, N> g;
#pragma unroll
        for (int i = 0; i < N; ++i) g.v[i] = narrow<DT>(wt * widen<DT>(a.v[i]));
        store_pack<DT, N>(o + (int64_t)v * N, g);
      }
    };
    const Pack<DT, N> none{};
    constexpr int kU = 4;  // vectors of a lane on their way
    int v = lane;
    for (; v + 64 * (kU - 1) < vecs; v += 64 * kU) {
      Pack<DT, N> a[kU], b[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        a[u] = load_pack<DT, N>(d + (int64_t)(v + 64 * u) * N);
        b[u] = dw ? load_pack<DT, N>(y + (int64_t)(v + 64 * u) * N) : none;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) one(v + 64 * u, a[u], b[u]);
    }
    for (; v < vecs; v += 64) one(v, load_pack<DT, N>(d + (int64_t)v * N), dw ? load_pack<DT, N>(y + (int64_t)v * N) : none);
  }
  if (dw) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
    if (lane == 0) dw[p] = dot;
  }
}

inline bool multiple(const void* p, int64_t bytes, int64_t stride, int64_t by) {
  return reinterpret_cast<uintptr_t>(p) % by == 0 && bytes % by == 0 && stride % by == 0;
}

// Rows [rows, width] of `size`-byte elements with stride ld: base and rows on whole elements
inline bool on_elements(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % size == 0; }

inline int size_of(int dtype) { return dtype == MOE355_F32 ? 4 : dtype == MOE355_U8 ? 1 : 2; }

}  // namespace
}  // namespace moe355

using namespace moe355;

extern "C" int moe_group_workspace(int T, int topk, int E, size_t* bytes) {
  MOE355_CHECK(T >= 0 && topk >= 1 && E >= 1 && bytes, MOE355_EINVAL);
  MOE355_CHECK(E <= kMaxE && (int64_t)T * topk < (1ll << 31), MOE355_EUNSUPPORTED);
  const int64_t n = (int64_t)T * topk;
  *bytes = n <= kOneChunk ? 0 : (size_t)(ceil_div64(n, chunk_of(n)) * E * 4);
  return MOE355_OK;
}

extern "C" int moe_group(const int32_t* topk_ids, int64_t ld_topk, int T, int topk, int E, int32_t* offsets,
                         int32_t* row_of_pair, int32_t* pair_of_row, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
  size_t need = 0;
  if (int st = moe_group_workspace(T, topk, E, &need)) return st;
  MOE355_CHECK(ld_topk >= topk && offsets, MOE355_EINVAL);
  const int64_t n = (int64_t)T * topk;
  MOE355_CHECK(n == 0 || (topk_ids && row_of_pair), MOE355_EINVAL);
  MOE355_CHECK(need == 0 || (workspace && workspace_bytes >= need), MOE355_EINVAL);
  MOE355_CHECK(on_elements(topk_ids, 4) && on_elements(offsets, 4) && on_elements(row_of_pair, 4) &&
                   on_elements(pair_of_row, 4) && on_elements(workspace, 4),
               MOE355_EMISALIGNED);
  int bits = 0;
  while ((1 << bits) < E) ++bits;
  const uint32_t chunk = (uint32_t)chunk_of(n);
  const unsigned chunks = n <= kOneChunk ? 1 : (unsigned)ceil_div64(n, chunk);
  const int64_t ld = ld_topk == topk ? 0 : ld_topk;
  int32_t* counts = chunks > 1 ? static_cast<int32_t*>(workspace) : nullptr;
  if (counts)
    hipLaunchKernelGGL(group_count_kernel, dim3(chunks), dim3(kThreads), 0, stream, topk_ids, ld, topk, (uint32_t)n, E, chunk, counts);
  hipLaunchKernelGGL(group_kernel, dim3(chunks), dim3(kThreads), (kWaves * E + kWaves) * 4, stream, topk_ids, ld, topk, (uint32_t)n, E,
                     bits, chunk, counts, offsets, row_of_pair, pair_of_row);
  return launch_status();
}

extern "C" int moe_dispatch(const void* x, int dtype, int64_t ld_x, int T, int H, int topk, const int32_t* row_of_pair, int R,
                            void* rows, int64_t ld_rows, hipStream_t stream) {
  MOE355_CHECK(dtype >= MOE355_BF16 && dtype <= MOE355_U8 && T >= 0 && H >= 0 && topk >= 1 && R >= 0 && ld_x >= H && ld_rows >= H,
               MOE355_EINVAL);
  if (T == 0 || H == 0 || R == 0) return MOE355_OK;
  MOE355_CHECK(x && row_of_pair && rows, MOE355_EINVAL);
  const int sz = size_of(dtype);
  MOE355_CHECK(on_elements(x, sz) && on_elements(rows, sz) && on_elements(row_of_pair, 4), MOE355_EMISALIGNED);
  const int64_t bytes = (int64_t)H * sz, sx = ld_x * sz, sr = ld_rows * sz;
  int by = sz;  // the widest vector that every row splits into
  for (int b : {16, 4, 2})
    if (b > by && multiple(x, bytes, sx, b) && multiple(rows, bytes, sr, b)) {
      by = b;
      break;
    }
  const int64_t vecs = bytes / by, chunks = ceil_div64(vecs, 64), grid = ceil_div64(T * chunks, 4);
  MOE355_CHECK(grid < (1ll << 24), MOE355_EUNSUPPORTED);
  auto* fn = by == 16 ? &dispatch_kernel<16> : by == 4 ? &dispatch_kernel<4> : by == 2 ? &dispatch_kernel<2> : &dispatch_kernel<1>;
  hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(256), 0, stream, static_cast<const uint8_t*>(x), sx, (int64_t)T, topk, R, vecs,
                     chunks, row_of_pair, static_cast<uint8_t*>(rows), sr);
  return launch_status();
}

namespace moe355 {
namespace {

template <int DT, int N>
int run_combine(const void* rows, int64_t ld_rows, int T, int H, int k, int R, const int32_t* rop, const float* weights,
                int64_t ld_w, void* out, int64_t ld_out, hipStream_t stream) {
  typedef typename Elem<DT>::type D;
  const int64_t vecs = H / N, chunks = ceil_div64(vecs, 64), grid = ceil_div64(T * chunks, 4);
  MOE355_CHECK(grid < (1ll << 24), MOE355_EUNSUPPORTED);
  hipLaunchKernelGGL((combine_kernel<DT, N>), dim3((unsigned)grid), dim3(256), 0, stream, static_cast<const D*>(rows), ld_rows,
                     (int64_t)T, k, R, vecs, chunks, rop, weights, ld_w, static_cast<D*>(out), ld_out);
  return launch_status();
}

template <int DT, int N>
int run_combine_grad(const void* dout, int64_t ld_dout, const void* rows, int64_t ld_rows, int T, int H, int k, int R,
                     const int32_t* rop, const float* weights, int64_t ld_w, void* drows, int64_t ld_drows, float* dw,
                     hipStream_t stream) {
  typedef typename Elem<DT>::type D;
  const int64_t pairs = (int64_t)T * k, grid = ceil_div64(pairs, 4);
  MOE355_CHECK(grid < (1ll << 24), MOE355_EUNSUPPORTED);
  hipLaunchKernelGGL((combine_grad_kernel<DT, N>), dim3((unsigned)grid), dim3(256), 0, stream, static_cast<const D*>(dout), ld_dout,
                     static_cast<const D*>(rows), ld_rows, pairs, k, R, H / N, rop, weights, ld_w, static_cast<D*>(drows), ld_drows,
                     dw);
  return launch_status();
}

}  // namespace
}  // namespace moe355

extern "C" int moe_combine(const void* rows, int dtype, int64_t ld_rows, int T, int H, int topk, const int32_t* row_of_pair, int R,
                           const float* weights, int64_t ld_weights, void* out, int64_t ld_out, hipStream_t stream) {
  MOE355_CHECK(dtype >= MOE355_BF16 && dtype <= MOE355_F32 && T >= 0 && H >= 0 && topk >= 1 && R >= 0 && ld_rows >= H &&
                   ld_out >= H && (!weights || ld_weights >= topk),
               MOE355_EINVAL);
  if (T == 0 || H == 0) return MOE355_OK;
  MOE355_CHECK((rows || R == 0) && row_of_pair && out, MOE355_EINVAL);
  const int sz = size_of(dtype);
  MOE355_CHECK(on_elements(rows, sz) && on_elements(out, sz) && on_elements(row_of_pair, 4) && on_elements(weights, 4),
               MOE355_EMISALIGNED);
  const int64_t bytes = (int64_t)H * sz;
  const bool wide = multiple(rows, bytes, ld_rows * sz, 16) && multiple(out, bytes, ld_out * sz, 16);
  auto* fn = dtype == MOE355_F32    ? (wide ? &run_combine<2, 4> : &run_combine<2, 1>)
             : dtype == MOE355_F16 ? (wide ? &run_combine<1, 8> : &run_combine<1, 1>)
                                   : (wide ? &run_combine<0, 8> : &run_combine<0, 1>);
  return fn(rows, ld_rows, T, H, topk, R, row_of_pair, weights, ld_weights, out, ld_out, stream);
}

extern "C" int moe_combine_grad(const void* dout, int64_t ld_dout, const void* rows, int64_t ld_rows, int dtype, int T, int H,
                                int topk, const int32_t* row_of_pair, int R, const float* weights, int64_t ld_weights,
                                void* drows, int64_t ld_drows, float* dweights, hipStream_t stream) {
  MOE355_CHECK(dtype >= MOE355_BF16 && dtype <= MOE355_F32 && T >= 0 && H >= 0 && topk >= 1 && R >= 0 && ld_dout >= H &&
                   (!dweights || ld_rows >= H) && (!drows || ld_drows >= H) && ld_weights >= topk,
               MOE355_EINVAL);
  MOE355_CHECK(H <= 0x7fffffff - 255, MOE355_EUNSUPPORTED);  // a lane's next vector is counted in 32 bits
  if (T == 0 || (!drows && !dweights)) return MOE355_OK;
  MOE355_CHECK((H == 0 || dout) && (!dweights || R == 0 || H == 0 || rows) && row_of_pair && weights, MOE355_EINVAL);
  const int sz = size_of(dtype);
  MOE355_CHECK(on_elements(dout, sz) && on_elements(rows, sz) && on_elements(drows, sz) && on_elements(row_of_pair, 4) &&
                   on_elements(weights, 4) && on_elements(dweights, 4),
               MOE355_EMISALIGNED);
  const int64_t bytes = (int64_t)H * sz;
  const bool wide = multiple(dout, bytes, ld_dout * sz, 16) && (!dweights || multiple(rows, bytes, ld_rows * sz, 16)) &&
                    (!drows || multiple(drows, bytes, ld_drows * sz, 16));
  auto* fn = dtype == MOE355_F32    ? (wide ? &run_combine_grad<2, 4> : &run_combine_grad<2, 1>)
             : dtype == MOE355_F16 ? (wide ? &run_combine_grad<1, 8> : &run_combine_grad<1, 1>)
                                   : (wide ? &run_combine_grad<0, 8> : &run_combine_grad<0, 1>);
  return fn(dout, ld_dout, rows, ld_rows, T, H, topk, R, row_of_pair, weights, ld_weights, drows, ld_drows, dweights, stream);
}
