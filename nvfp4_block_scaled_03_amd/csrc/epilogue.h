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

// z / (1 + e^-z): the hardware exponential and reciprocal (1 ulp each).
__device__ __forceinline__ float act_apply(int act, float z) {
  switch (act) {   // the same for the whole launch
    case kFnRelu: return z > 0.0f ? z : 0.0f;
    case kFnSilu: return silu_fast(z);
    // x P(X <= x): the complementary error function keeps the relative
    // accuracy of the left tail, where 1 + erf cancels.
    case kFnGelu: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    // 0.5 z (1 + tanh u) = z / (1 + e^-2u)
    case kFnGeluTanh: {
      const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
      return z * __builtin_amdgcn_rcpf(1.0f + __expf(-u2));
    }
    default: return z;
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
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t row = i * 16 + lg * 4 + r;
        if (row < nrows) {
          float y;
          if constexpr (GATED)
            y = act_apply(ep.act, alpha * acc[i][2 * q][r] + b0) * (alpha * acc[i][2 * q + 1][r] + b1);
          else
            y = act_apply(ep.act, alpha * acc[i][q][r] + b0);
          epi_store(ep, row0 + row, col, y + epi_residual(ep, row0 + row, col));
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
      f32x4 y;
      if constexpr (GATED) {
        const int cg = (c4 >> 4) * 32 + (c4 & 15);   // gate columns of the pair; the up columns 16 further
        const f32x4 a = *reinterpret_cast<const f32x4*>(src + cg), u = *reinterpret_cast<const f32x4*>(src + cg + 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = act_apply(ep.act, a[j] + b0[j]) * (u[j] + b1[j]);
      } else {
        const f32x4 a = *reinterpret_cast<const f32x4*>(src + c4);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = act_apply(ep.act, a[j] + b0[j]);
      }
      if (row < nrows) epi_finish4(ep, row0 + row, col, y);
    }
    // (the next tile rewrites sh only after every lane has read it)
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

}  // namespace nvfp4
