// Microscaled 4-bit floating point: element and scale formats, and the layouts
// of the scales.
//
// A row of d values is cut into blocks (32 values for the MX form, 16 for the
// NV form); each value is an e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives) times its block's scale: a power of two (e8m0, bias 127, 255 =
// NaN) for MX, an e4m3 number times one float32 of the whole tensor for NV.
#pragma once

#include <cuda_fp8.h>

#include "qs_internal.cuh"

namespace qs {

__host__ __device__ constexpr int fp4_block(int format) { return format == QS_FP4_MX ? 32 : 16; }

// Tiled scales: tiles of 128 rows x 4 blocks, 512 bytes each, the tiles of one
// row range contiguous.  Within a tile the byte of row r, block b sits at
// (r % 32) * 16 + (r / 32) * 4 + b: 32 lanes of 16 bytes, the form in which the
// tensor core wants the scales in tensor memory.
constexpr int kSfTile = 512;
__host__ __device__ inline size_t fp4_tiles_per_row(int nblocks) { return (size_t)((nblocks + 3) / 4); }
__host__ __device__ inline size_t fp4_tiled_offset(size_t row, int blk, size_t tiles_per_row) {
  return ((row >> 7) * tiles_per_row + (size_t)(blk >> 2)) * kSfTile + (row & 31) * 16 +
         ((row >> 5) & 3) * 4 + (size_t)(blk & 3);
}

// 8 float32 -> 8 e2m1 codes, value i in bits 4i..4i+3 (nearest, ties to even,
// magnitudes above 6 become 6)
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// 8 e2m1 codes -> four pairs of float16 (exact): pair i holds codes 2i, 2i+1.
// (Each byte is brought to the bottom of a 16-bit register first: with the
// word taken apart inside one asm block the upper codes came out as zeros.)
__device__ __forceinline__ uint32_t e2m1x2_to_half2(uint32_t byte) {
  uint32_t h;
  asm("{\n .reg .b8 b0, b1;\n mov.b16 {b0, b1}, %1;\n cvt.rn.f16x2.e2m1x2 %0, b0;\n}\n"
      : "=r"(h)
      : "h"((uint16_t)byte));
  return h;
}
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t c, uint32_t (&h)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = e2m1x2_to_half2((c >> (8 * i)) & 0xffu);
}

// 2^(s - 127) for an e8m0 code (255: NaN)
__device__ __forceinline__ float e8m0_value(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7fc00000u : (s == 0u ? 0x00400000u : s << 23));
}

struct Fp4QuantArgs {
  const void* x = nullptr;          // [R, d] bf16 / f32
  size_t R = 0;
  int d = 0;
  int bf16 = 1;
  int k = 0;                        // launch_fp4_topk_quantize: values kept per row
  int format = QS_FP4_MX;
  int tiled = 1;                    // scale layout
  int pad_rows = 1;                 // tiled: zero the scales of the rows behind the last
  const float* tensor_scale = nullptr;   // NV: 1 float32 (NULL: 1)
  uint8_t* codes = nullptr;         // [R, d/2]
  uint8_t* scales = nullptr;
  void* values = nullptr;           // [R, d] in x's type, or NULL
};
cudaError_t launch_fp4_quantize(const Fp4QuantArgs& a, cudaStream_t s);
// the k largest |x| of each row (ties: lower index), the rest 0; d <= QS_MAX_ROW,
// tiled scales, no rows behind the last
cudaError_t launch_fp4_topk_quantize(const Fp4QuantArgs& a, cudaStream_t s);

struct Fp4GemmPlan {
  int nt = 0;          // tokens per tile: 8, 16, 32, 64 or 128; 256: fp4_gemm_wide.cu
  int mtiles = 0;      // tiles of 128 outputs
  int ntiles = 0;      // tiles of nt tokens
  int nk = 0;          // steps of 256 inputs
  int cluster = 1;     // CTAs that share a tile's steps
  int grid = 0;
};
Fp4GemmPlan plan_fp4_gemm(int T, int d_in, int d_out);

struct Fp4GemmArgs {
  const uint8_t* xc = nullptr;      // [T, d_in/2]
  const uint8_t* xs = nullptr;      // tiled scales
  const uint8_t* wc = nullptr;      // [d_out, d_in/2]
  const uint8_t* ws = nullptr;
  const float* x_scale = nullptr;   // NV tensor scales (NULL: 1)
  const float* w_scale = nullptr;
  void* y = nullptr;                // [T, d_out]
  int y_bf16 = 1;
  int T = 0, d_in = 0, d_out = 0;
  int format = QS_FP4_MX;
  DevStatus* status = nullptr;
  Fp4GemmPlan plan{};
};
bool fp4_gemm_supported();
cudaError_t launch_fp4_gemm(const Fp4GemmArgs& a, cudaStream_t s);
int fp4_wide_pairs();
cudaError_t launch_fp4_gemm_wide(const Fp4GemmArgs& a, cudaStream_t s);

}  // namespace qs
