// Epilogue of the dense linear layers: bias, activation (plain or gated),
// residual, one rounding (see nvfp4_epilogue in the header).
//
// All of it runs in FP32 on the accumulator's value: y = act(v + bias) or
// act(gate) * up, then + residual, then one rounding to the output type, so
// a bfloat16 output differs from the real-valued result by half a step plus
// the FP32 error.
#pragma once

#include "common.h"
#include "launch.h"

namespace nvfp4 {

// The activation of N values.  The choice is the same for the whole launch and
// stands outside the values, so that the code of the others is stepped over
// once: instruction fetches of code that is run once are a good part of a
// short kernel's time.
template <int N>
__device__ __forceinline__ void act_apply(int act, float (&z)[N]) {
  switch (act) {
    case kFnRelu:
#pragma unroll
      for (int r = 0; r < N; ++r) z[r] = z[r] > 0.0f ? z[r] : 0.0f;
      break;
    // z / (1 + e^-z): the hardware exponential and reciprocal (1 ulp each).
    case kFnSilu:
#pragma unroll
      for (int r = 0; r < N; ++r) z[r] = silu_fast(z[r]);
      break;
    // z Phi(z): the complementary error function keeps the relative accuracy
    // of the left tail, where 1 + erf cancels.
    case kFnGelu:
#pragma unroll 1
      for (int k = 0; k < N; ++k) {   // (rolled: the values turn through one register)
        const float v = z[0];
#pragma unroll
        for (int r = 0; r + 1 < N; ++r) z[r] = z[r + 1];
        z[N - 1] = 0.5f * v * erfcf(-0.70710678118654752f * v);
      }
      break;
    // 0.5 z (1 + tanh u) = z / (1 + e^-2u)
    case kFnGeluTanh:
#pragma unroll
      for (int r = 0; r < N; ++r) {
        const float u2 = 1.5957691216057308f * (z[r] + 0.044715f * z[r] * z[r] * z[r]);
        z[r] = z[r] * __builtin_amdgcn_rcpf(1.0f + __expf(-u2));
      }
      break;
    default: break;
  }
}

// Residual values and output stores: element (row, col) and four consecutive
// columns (col a multiple of 4; pointers and strides keep 4 elements together).
__device__ __forceinline__ float epi_residual(const LinearEpi& e, int64_t row, int64_t col) {
  if (!e.res) return 0.0f;
  const int64_t i = row * e.ldr + col;
  return e.res_f32 ? static_cast<const float*>(e.res)[i]
                   : bf16_bits_to_f32(static_cast<const uint16_t*>(e.res)[i]);
}
__device__ __forceinline__ void epi_store(const LinearEpi& e, int64_t row, int64_t col, float y) {
  const int64_t o = row * e.ldo + col;
  if (e.out_f32) static_cast<float*>(e.out)[o] = y;
  else static_cast<uint16_t*>(e.out)[o] = (uint16_t)f32_to_bf16_bits(y);
}
__device__ __forceinline__ void epi_finish4(const LinearEpi& e, int64_t row, int64_t col, f32x4 y) {
  if (e.res) {
    const int64_t i = row * e.ldr + col;
    if (e.res_f32) {
      y += *reinterpret_cast<const f32x4*>(static_cast<const float*>(e.res) + i);
    } else {
      const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(e.res) + i);
      y[0] += bf16_bits_to_f32(w[0] & 0xFFFFu);
      y[1] += bf16_bits_to_f32(w[0] >> 16);
      y[2] += bf16_bits_to_f32(w[1] & 0xFFFFu);
      y[3] += bf16_bits_to_f32(w[1] >> 16);
    }
  }
  const int64_t o = row * e.ldo + col;
  if (e.out_f32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(e.out) + o) = y;
  } else {
    const uint32_t lo = f32_to_bf16_bits(y[0]) | (f32_to_bf16_bits(y[1]) << 16);
    const uint32_t hi = f32_to_bf16_bits(y[2]) | (f32_to_bf16_bits(y[3]) << 16);
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(e.out) + o) = u32x2{lo, hi};
  }
}

// Epilogue of a wavefront's MT x NTW accumulator tiles in the matrix
// instruction's layout (lane 16 g + n: rows 4 g .. 4 g + 3 of column n), rows
// row0 + [0, nrows), streaming columns n0 + [0, 16 NTW).  GATED: the column
// tiles alternate gate and up, and column n of pair q is output column
// n0 / 2 + 16 q + n.  One store per value: few rows, or no LDS to turn the
// tile in.
template <bool GATED, int MT, int NTW>
__device__ __forceinline__ void epilogue_linear(const LinearEpi& ep, const f32x4 (&acc)[MT][NTW], float alpha,
                                                int64_t row0, int64_t nrows, int64_t n0, int lane) {
  const int ln = lane & 15, lg = lane >> 4;
  constexpr int Q = GATED ? NTW / 2 : NTW;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int64_t col = (GATED ? n0 / 2 : n0) + 16 * q + ln;
    const float b0 = ep.bias ? ep.bias[col] : 0.0f;
    const float b1 = GATED && ep.bias ? ep.bias[ep.half + col] : 0.0f;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      float y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = alpha * acc[i][GATED ? 2 * q : q][r] + b0;
      act_apply(ep.act, y);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (GATED) y[r] *= alpha * acc[i][2 * q + 1][r] + b1;
        const int64_t row = i * 16 + lg * 4 + r;
        if (row < nrows) epi_store(ep, row0 + row, col, y[r] + epi_residual(ep, row0 + row, col));
      }
    }
  }
}

// The same through a wave-private LDS area sh of 16 x (16 NTW + 4) floats:
// each 16-row tile is turned around and leaves as stores of four consecutive
// columns, and the residual comes in as loads of four.
template <bool GATED, int MT, int NTW>
__device__ __forceinline__ void epilogue_linear_rowmajor(const LinearEpi& ep, const f32x4 (&acc)[MT][NTW],
                                                         float alpha, int64_t row0, int64_t nrows, int64_t n0,
                                                         int lane, float* sh) {
  constexpr int W = 16 * NTW, SW = W + 4;
  constexpr int WO = GATED ? W / 2 : W;   // output columns of the wavefront
  constexpr int LPR = WO / 4, RPP = 64 / LPR;
  const int ln = lane & 15, lg = lane >> 4;
  const int rr = lane / LPR, c4 = (lane % LPR) * 4;
  const int64_t col = (GATED ? n0 / 2 : n0) + c4;
  f32x4 b0 = {0.f, 0.f, 0.f, 0.f}, b1 = {0.f, 0.f, 0.f, 0.f};
  if (ep.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      b0[j] = ep.bias[col + j];
      if constexpr (GATED) b1[j] = ep.bias[ep.half + col + j];
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (i * 16 >= nrows) break;   // (uniform)
#pragma unroll
    for (int j = 0; j < NTW; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) sh[(lg * 4 + r) * SW + 16 * j + ln] = alpha * acc[i][j][r];
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
#pragma unroll
    for (int ps = 0; ps < 16 / RPP; ++ps) {
      const int64_t row = i * 16 + ps * RPP + rr;
      const float* src = sh + (ps * RPP + rr) * SW;
      // (gated: gate columns of the pair; the up columns 16 further)
      const int cg = GATED ? (c4 >> 4) * 32 + (c4 & 15) : c4;
      const f32x4 a = *reinterpret_cast<const f32x4*>(src + cg) + b0;
      float z[4] = {a[0], a[1], a[2], a[3]};
      act_apply(ep.act, z);
      f32x4 y = {z[0], z[1], z[2], z[3]};
      if constexpr (GATED) y *= *reinterpret_cast<const f32x4*>(src + cg + 16) + b1;
      if (row < nrows) epi_finish4(ep, row0 + row, col, y);
    }
    // (the next tile rewrites sh only after every lane has read it)
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

}  // namespace nvfp4
