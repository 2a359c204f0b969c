// Host entry points of the norm, the row-wise 8-bit quantisation and the
// dense int8 layers (norm.hip, int8.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace nvfp4 {

// Rows of h = x (+ res): y = h rstd w and codes with a scale per row.  Row
// strides in elements, multiples of 8.
struct NormArgs {
  int64_t rows;
  int H;
  float eps;
  const void* x;
  int x_f32;
  int64_t ldx;
  const void* res;   // or null
  int res_f32;
  int64_t ldr;
  const void* w;
  int w_f32;
  void* h;           // or null; of the residual's type
  int64_t ldh;
  void* y;           // or null
  int y_f32;
  int64_t ldy;
  int8_t* q;         // [rows][H], or null
  float* s;          // [rows] (with q)
};
constexpr int kNormMaxH = 32768;
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s);
// Codes and scales of the rows of x itself (x, x_f32, ldx, rows, H, q, s).
hipError_t launch_int8_quantize(const NormArgs& a, hipStream_t s);

// Weight W [N][K] int8 in the streaming layout (gated: gate rows [0, N / 2) and
// up rows [N / 2, N) in alternate tiles).
size_t int8_prep_bytes(int64_t N, int64_t K, bool gated);
hipError_t launch_int8_prep(int64_t N, int64_t K, bool gated, const int8_t* q, uint8_t* prep, hipStream_t s);

// y [M][N] = sx[m] sw[n] (a W^T) and the epilogue.
struct Int8Args {
  int M, N, K;
  const int8_t* a;     // [M][lda]
  int64_t lda;
  const float* sx;     // [M]
  const uint8_t* w;    // streaming layout
  const float* sw;     // [N]
  int* part;           // partial sums of a split K
  LinearEpi ep;
};
// Bytes of part that every call of up to M rows is content with.
size_t int8_part_bytes(int64_t M, int64_t N, bool gated);
hipError_t launch_int8_linear(const Int8Args& a, hipStream_t s);

// The launches of a call: its streaming columns [col0, col0 + cols) in tiles of
// rows x columns, K in parts (kind -1: the kernel for a handful of rows).
struct Int8Step {
  int kind, rows, columns, parts;
  int64_t col0, cols;
};
int int8_plan(int64_t M, int64_t N, int64_t K, bool gated, Int8Step (&step)[2]);

}  // namespace nvfp4
