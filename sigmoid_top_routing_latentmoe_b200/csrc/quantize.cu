// Quantisers to e4m3 with one power-of-two scale (E8M0) for each block of 128
// columns of a row, or each 128 x 128 block of a weight matrix.
//
// With amax the largest finite magnitude of a block, the scale is 2^e with the
// smallest e >= -126 such that amax <= 448 * 2^e (448: the largest e4m3
// value); q = round-to-nearest-even e4m3 of x * 2^-e.  The division is exact,
// so each element is rounded once.  The scale is stored as the byte e + 127; a
// block of zeros has scale 1.  A NaN or an infinity becomes NaN: 8 bits hold
// no infinity, and a clamped one would hide an overflow.
//
// Both kernels read each element once (16-byte loads) and keep it in registers
// between the maximum and the rounding.
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "experts_fp8.h"
#include "kernels.h"
#include "launch.h"
#include "quantize.cuh"

namespace lmoe {
namespace {

template <typename T>
constexpr int kVec = 16 / sizeof(T);  // elements of a 16-byte vector

// Element i of a vector.
template <typename T>
__device__ __forceinline__ float elem(const uint4& v, int i) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (kVec<T> == 4) return __uint_as_float(w[i]);
  else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
}
// Magnitudes in order as whole numbers: the bits of |x|, which go from 0 to
// kInfBits for finite and infinite values and beyond for NaN.
constexpr uint32_t kInfBits = 0x7f800000u;
// The largest of a lane's N vectors (bf16: two elements at a time).
template <typename T, int N>
__device__ __forceinline__ uint32_t amax_bits(const uint4 (&v)[N]) {
  constexpr uint32_t kAbs = kVec<T> == 4 ? 0x7fffffffu : 0x7fff7fffu;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (kVec<T> == 4) {
      m = __vimax3_u32(m, v[i].x & kAbs, v[i].y & kAbs);
      m = __vimax3_u32(m, v[i].z & kAbs, v[i].w & kAbs);
    } else {
      m = __vimax3_u16x2(m, v[i].x & kAbs, v[i].y & kAbs);
      m = __vimax3_u16x2(m, v[i].z & kAbs, v[i].w & kAbs);
    }
  }
  return kVec<T> == 4 ? m : max(m & 0xffffu, m >> 16) << 16;
}
// The same over finite elements only, for a block that holds others.
template <typename T, int N>
__device__ __forceinline__ uint32_t finite_amax_bits(const uint4 (&v)[N]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j) m = finite_max(m, elem<T>(v[i], j));
  return __float_as_uint(m);
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t m) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1)
    m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}
// A vector's elements times inv, rounded, four to a word.  FINITE: none is
// infinite.
template <typename T, bool FINITE>
__device__ __forceinline__ void quantize_vec(const uint4& v, float inv, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < kVec<T> / 4; ++i) {
    const float a = elem<T>(v, 4 * i) * inv, b = elem<T>(v, 4 * i + 1) * inv,
                c = elem<T>(v, 4 * i + 2) * inv, d = elem<T>(v, 4 * i + 3) * inv;
    w[i] = FINITE ? pack_e4m3_finite(a, b, c, d) : pack_e4m3(a, b, c, d);
  }
}

// The tile list of a ragged product: expert e's rows [bound[e], bound[e + 1]) in
// tiles of at most tile_m.  bound[e] is the largest of offsets[0 ... e] clamped to
// [0, rows]: the offsets themselves where they ascend, as a dispatch gives them,
// and otherwise still an order in which no row belongs to two experts (two tiles
// would write it, in either order) and the list fits into max_tiles.  One block
// of kTileThreads, each of which takes some neighbouring experts (one pair of
// scans: the quantise step with 896 experts 5.4 us, 7.8 with a scan for every 256).
constexpr int kTileThreads = 256;
// Scan over the block: the result of the threads before this one (MAX: the
// largest, 0 without any; else the sum).  `part` gets the warps' totals.
template <bool MAX>
__device__ __forceinline__ int scan_before(int v, int* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v = MAX ? max(v, o) : v + o;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  v = __shfl_up_sync(0xffffffffu, v, 1);
  if (lane == 0) v = 0;
#pragma unroll
  for (int w = 0; w < kTileThreads / 32; ++w)
    if (w < warp) v = MAX ? max(v, part[w]) : v + part[w];
  return v;
}
__device__ __forceinline__ int clamped_offset(const TileList& t, int i) {
  return min(max(t.offsets[i], 0), (int)t.rows);
}
// bound[first] where the offsets do not ascend.
__device__ __forceinline__ int running_bound(const TileList& t, int first, int last, int* part) {
  int top = clamped_offset(t, first);
  for (int e = first; e < last; ++e) top = max(top, clamped_offset(t, e + 1));
  const int before = scan_before<true>(top, part);
  __syncthreads();
  return max(clamped_offset(t, first), before);
}
__device__ __forceinline__ void build_tile_list(const TileList& t) {
  static_assert(kTileM == 128 && kRoutedPairTileM == 256, "tiles of 2^7 or 2^8 rows");
  __shared__ int part[kTileThreads / 32];
  const int shift = t.tile_m == kRoutedPairTileM ? 8 : 7;
  const int per = (t.R + kTileThreads - 1) / kTileThreads;
  const int first = min((int)threadIdx.x * per, t.R), last = min(first + per, t.R);
  // this thread's experts: first row, end of the first, whether they ascend
  int start = t.offsets[first], end = t.offsets[min(first + 1, t.R)];
  bool ascend = start >= 0 && start <= end && end <= t.rows;
  for (int e = first + 1, lo = end; e < last; ++e) {
    const int hi = t.offsets[e + 1];
    ascend = ascend && lo <= hi && hi <= t.rows;
    lo = hi;
  }
  if (!__syncthreads_and(ascend)) {
    start = running_bound(t, first, last, part);
    end = max(start, clamped_offset(t, min(first + 1, t.R)));
  }
  int n = 0;  // their tiles
  for (int e = first, lo = start, hi = end; e < last;) {
    n += (hi - lo + t.tile_m - 1) >> shift;
    lo = hi;
    if (++e < last) hi = max(lo, clamped_offset(t, e + 1));
  }
  int at = scan_before<false>(n, part);
  if (threadIdx.x == kTileThreads - 1) *t.n_mtiles = min(at + n, t.max_tiles);
  for (int e = first, lo = start, hi = end; e < last;) {
    for (; lo < hi; lo += t.tile_m, ++at)
      if (at < t.max_tiles) t.tiles[at] = make_int4(e, lo, min(t.tile_m, hi - lo), 0);
    lo = hi;
    if (++e < last) hi = max(lo, clamped_offset(t, e + 1));
  }
}
__global__ void __launch_bounds__(kTileThreads) expert_tiles_kernel(TileList t) {
  pdl_trigger();
  pdl_wait();
  build_tile_list(t);
}

// One warp per row, 512 columns a step: a lane holds 16 neighbouring elements,
// eight lanes a block, and the step's four exponents are one word of scales.
// The kernel is bound by issue slots rather than bytes (with 8 elements a lane,
// 140 instructions for every 8, the mid layer's 131072 rows of 1024 took 72 us),
// so 16 elements share the reductions and addresses (51 us; 26 at the copy rate).  One more block writes the
// tile list of the products that follow, when there is one.
constexpr int kLaneElems = 16, kStepCols = 32 * kLaneElems, kRowWarps = 8;
template <typename T, bool FINITE>
__device__ __forceinline__ uint4 lane_q(const uint4 (&v)[kLaneElems / kVec<T>], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < kLaneElems / kVec<T>; ++i)
    quantize_vec<T, FINITE>(v[i], inv, w + i * kVec<T> / 4);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps)
    quantize_rows_kernel(const T* __restrict__ x, int64_t n_src, int64_t ld,
                         const int32_t* __restrict__ index, int64_t rows, int cols,
                         uint8_t* __restrict__ q, uint8_t* __restrict__ scales, TileList tiles) {
  pdl_trigger();
  pdl_wait();
  if (tiles.tiles != nullptr && blockIdx.x == gridDim.x - 1) {  // a block of its own
    if (blockIdx.y == 0) build_tile_list(tiles);
    return;
  }
  constexpr int U = 2;  // steps whose loads are in flight together
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (r >= rows) return;
  int64_t src = r;
  bool have = true;
  if (index != nullptr) {
    src = index[r];
    have = src >= 0 && src < n_src;
  }
  const int steps = (cols + kStepCols - 1) / kStepCols;
  const T* xr = x + (have ? src : 0) * ld + lane * kLaneElems;
  uint8_t* qr = q + r * cols + lane * kLaneElems;
  uint8_t* sr = scales + r * 4 + (lane >> 3);
  // a long row of few rows is shared by gridDim.y warps
  for (int s0 = blockIdx.y * U; s0 < steps; s0 += gridDim.y * U) {
    constexpr int NV = kLaneElems / kVec<T>;
    uint4 v[U][NV];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = have && (s0 + u) * kStepCols + lane * kLaneElems < cols;
      const uint4* at = reinterpret_cast<const uint4*>(xr + (s0 + u) * kStepCols);
#pragma unroll
      for (int j = 0; j < NV; ++j) v[u][j] = in ? at[j] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int step = s0 + u;
      if (step >= steps) break;
      uint32_t m = lanes_max<8>(amax_bits<T>(v[u]));
      const bool finite = !__any_sync(0xffffffffu, m >= kInfBits);
      if (!finite) m = lanes_max<8>(finite_amax_bits<T>(v[u]));
      const int e = scale_exponent(__uint_as_float(m));
      const float inv = pow2_f(-e);
      const uint4 w = finite ? lane_q<T, true>(v[u], inv) : lane_q<T, false>(v[u], inv);
      if (step * kStepCols + lane * kLaneElems < cols)
        *reinterpret_cast<uint4*>(qr + step * kStepCols) = w;
      if ((lane & 7) == 0) sr[(int64_t)step * rows * 4] = (uint8_t)(e + 127);
    }
  }
}

// One thread block per 128 x 128 block (or per block of padding bytes).
template <typename T>
__global__ void __launch_bounds__(256) quantize_weights_kernel(const T* __restrict__ w,
                                                               int64_t rows, int cols, int rb,
                                                               int cb4, uint8_t* __restrict__ q,
                                                               uint8_t* __restrict__ scales) {
  pdl_trigger();
  pdl_wait();
  constexpr int V = kVec<T>, BL = kQBlock / V, RP = 256 / BL, U = kQBlock / RP;
  __shared__ uint32_t part[8];
  const int64_t blk = blockIdx.x;
  const int cbi = (int)(blk % cb4);
  const int rbi = (int)((blk / cb4) % rb);
  const int64_t mat = blk / ((int64_t)cb4 * rb);
  const int c = cbi * kQBlock + (threadIdx.x % BL) * V;
  const int64_t r0 = (int64_t)rbi * kQBlock + threadIdx.x / BL;
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    v[u] = make_uint4(0, 0, 0, 0);
    const int64_t r = r0 + u * RP;
    if (c < cols && r < rows)
      v[u] = *reinterpret_cast<const uint4*>(w + (mat * rows + r) * cols + c);
  }
  uint32_t m = amax_bits<T>(v);
  bool finite = true;  // every element of the block
  for (;;) {
    m = lanes_max<32>(m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, part[i]);
    if (m < kInfBits) break;
    finite = false;
    m = finite_amax_bits<T>(v);
    __syncthreads();
  }
  const int e = scale_exponent(__uint_as_float(m));
  const float inv = pow2_f(-e);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t r = r0 + u * RP;
    if (c < cols && r < rows) {
      uint32_t o[V / 4];
      if (finite) quantize_vec<T, true>(v[u], inv, o);
      else quantize_vec<T, false>(v[u], inv, o);
      uint8_t* dst = q + (mat * rows + r) * cols + c;
      if constexpr (V == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
      else *reinterpret_cast<uint32_t*>(dst) = o[0];
    }
  }
  if (threadIdx.x == 0) scales[blk] = (uint8_t)(e + 127);
}

// Rows of q and their scale words in sorted order, one warp per row.
__global__ void __launch_bounds__(32 * kRowWarps)
    sort_rows_kernel(const uint8_t* __restrict__ q, const uint32_t* __restrict__ words, int64_t n_src,
                     const int32_t* __restrict__ index, int64_t rows, int cols, int n_words,
                     uint8_t* __restrict__ q_out, uint32_t* __restrict__ words_out) {
  pdl_trigger();
  pdl_wait();
  constexpr int U = 4;  // loads in flight
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int64_t src = index[r];
  const bool have = src >= 0 && src < n_src;
  const int nvec = cols / 16;
  const uint4* from = reinterpret_cast<const uint4*>(q + (have ? src : 0) * cols);
  uint4* to = reinterpret_cast<uint4*>(q_out + r * cols);
  for (int w = lane; w < n_words; w += 32)  // 0x7f: scale 1
    words_out[w * rows + r] = have ? words[w * n_src + src] : 0x7f7f7f7fu;
  for (int v0 = lane; v0 < nvec; v0 += 32 * U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = have && v0 + 32 * u < nvec ? from[v0 + 32 * u] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v0 + 32 * u < nvec) to[v0 + 32 * u] = v[u];
  }
}

}  // namespace

template <typename T>
cudaError_t launch_quantize_rows(const T* x, int64_t n_src, int64_t ld, const int32_t* index,
                                 int64_t rows, int cols, uint8_t* q, uint8_t* scales,
                                 cudaStream_t st, const TileList* tiles) {
  static_assert(kTileThreads == 32 * kRowWarps, "one block writes the tile list");
  if (rows == 0) return cudaSuccess;
  const unsigned blocks = (unsigned)((rows + kRowWarps - 1) / kRowWarps);
  // few rows: their steps are spread over up to 8 warps each, towards 1200 blocks
  const int pairs = (cols + 2 * kStepCols - 1) / (2 * kStepCols);
  const unsigned split = std::min<unsigned>(std::min(pairs, 8), std::max(1u, 1200 / blocks));
  count_launch();
  return launch_pdl(quantize_rows_kernel<T>, dim3(blocks + (tiles != nullptr ? 1 : 0), split),
                    dim3(32 * kRowWarps), 0, st, 1, x, n_src, ld, index, rows, cols, q, scales,
                    tiles != nullptr ? *tiles : TileList{});
}
template cudaError_t launch_quantize_rows<float>(const float*, int64_t, int64_t, const int32_t*,
                                                 int64_t, int, uint8_t*, uint8_t*, cudaStream_t,
                                                 const TileList*);
template cudaError_t launch_quantize_rows<__nv_bfloat16>(const __nv_bfloat16*, int64_t, int64_t,
                                                         const int32_t*, int64_t, int, uint8_t*,
                                                         uint8_t*, cudaStream_t, const TileList*);

cudaError_t launch_sort_rows(const uint8_t* q, const uint8_t* scales, int64_t n_src,
                             const int32_t* index, int64_t rows, int cols, uint8_t* q_out,
                             uint8_t* scales_out, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  count_launch();
  return launch_pdl(sort_rows_kernel, dim3((unsigned)((rows + kRowWarps - 1) / kRowWarps)),
                    dim3(32 * kRowWarps), 0, st, 1, q, reinterpret_cast<const uint32_t*>(scales),
                    n_src, index, rows, cols, q_words(cols), q_out,
                    reinterpret_cast<uint32_t*>(scales_out));
}

template <typename T>
cudaError_t launch_quantize_weights(const T* w, int64_t mats, int64_t rows, int cols, uint8_t* q,
                                    uint8_t* scales, cudaStream_t st) {
  if (mats == 0) return cudaSuccess;
  const int rb = q_blocks(rows), cb4 = 4 * q_words(cols);
  count_launch();
  return launch_pdl(quantize_weights_kernel<T>, dim3((unsigned)(mats * rb * cb4)), dim3(256), 0, st,
                    1, w, rows, cols, rb, cb4, q, scales);
}
template cudaError_t launch_quantize_weights<float>(const float*, int64_t, int64_t, int, uint8_t*,
                                                    uint8_t*, cudaStream_t);
template cudaError_t launch_quantize_weights<__nv_bfloat16>(const __nv_bfloat16*, int64_t, int64_t,
                                                            int, uint8_t*, uint8_t*, cudaStream_t);

cudaError_t launch_expert_tiles(const TileList& t, cudaStream_t st) {
  count_launch();
  return launch_pdl(expert_tiles_kernel, dim3(1), dim3(kTileThreads), 0, st, 1, t);
}

}  // namespace lmoe
