// Host interface of the 8-bit routed experts: quantisers and the ragged
// block-scaled product (quantize.cu, experts_fp8.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace lmoe {

// One E8M0 scale per 128 elements; the bytes of four neighbouring blocks make
// a word (512 elements).
constexpr int kQBlock = 128;
inline int q_words(int64_t cols) { return (int)((cols + 511) / 512); }
inline int q_blocks(int64_t n) { return (int)((n + kQBlock - 1) / kQBlock); }

// Tile list of a ragged product, written by launch_expert_tiles or by a block of
// the quantiser of its rows: (expert, first row, rows) of at most
// tile_m rows.
struct TileList {
  const int32_t* offsets;  // [R + 1], clamped to [0, rows]
  int R;
  int64_t rows;
  int tile_m;    // kTileM or kRoutedPairTileM
  int max_tiles;
  int32_t* n_mtiles;
  int4* tiles;
};

// q [rows, cols] e4m3 and scales [words, rows, 4] of x [n_src, cols] (row
// stride ld elements); index != nullptr: row r is x[index[r]], a row of zeros
// where that is outside [0, n_src).  cols a multiple of 16, x 16-byte aligned
// rows.
template <typename T>
cudaError_t launch_quantize_rows(const T* x, int64_t n_src, int64_t ld, const int32_t* index,
                                 int64_t rows, int cols, uint8_t* q, uint8_t* scales,
                                 cudaStream_t st, const TileList* tiles = nullptr);
// Quantised rows in another order: row r is row index[r], zeros outside [0, n_src).
cudaError_t launch_sort_rows(const uint8_t* q, const uint8_t* scales, int64_t n_src,
                             const int32_t* index, int64_t rows, int cols, uint8_t* q_out,
                             uint8_t* scales_out, cudaStream_t st);
// q [mats, rows, cols] e4m3 and scales [mats, ceil(rows / 128), 4 words] of w.
template <typename T>
cudaError_t launch_quantize_weights(const T* w, int64_t mats, int64_t rows, int cols, uint8_t* q,
                                    uint8_t* scales, cudaStream_t st);
cudaError_t launch_expert_tiles(const TileList& t, cudaStream_t st);

// out [rows, n_out] = rows of a against the weights of the tile's expert.
struct Fp8Gemm {
  const uint8_t* a;         // [rows, n_in]
  const uint8_t* a_scales;  // [words, rows, 4]
  int64_t rows;
  int R, n_in, n_out;
  const uint8_t* w;         // [R, n_out, n_in]
  const uint8_t* w_scales;  // [R, ceil(n_out / 128), 4 words]
  // SiTU != 0: w holds the gate and w_up the up projections (n_out hidden
  // units); out gets the quantised hidden units and out_scales their scales.
  int situ;
  const uint8_t* w_up;
  const uint8_t* w_up_scales;
  float beta1, beta2;
  void* out;
  uint8_t* out_scales;
  int out_f32;              // out is fp32, else bf16 (ignored with situ)
  const int4* tiles;        // nullptr: one expert, which has the rows
  const int32_t* offsets;   // [offsets[0], offsets[1]), or every row when that is nullptr
  const int32_t* n_mtiles;
  int max_tiles;
  // CTA pairs over tiles of 256 rows, else single CTAs over tiles of 128; the
  // tile list has to be of that height.
  bool pairs;
};
cudaError_t launch_fp8_gemm(const Fp8Gemm& g, int32_t* status, cudaStream_t st);


}  // namespace lmoe
