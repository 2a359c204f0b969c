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

// z Phi(z) = max(z, 0) - |z| erfc(|z| / sqrt 2) / 2: the complementary error
// function keeps the relative accuracy of the left tail, where 1 + erf cancels.
// erfc(w / sqrt 2) = e^(-w^2 / 2) f(w), and f(w) (w + c) / 2 is close to a
// polynomial in u = (w - c) / (w + c), which maps [0, inf) to [-1, 1); degree 8
// with c = 3.75, a least-maximum fit of its own over w <= 14.2, is within
// 1.5e-8 of it.  Beyond, the exponential is 0 in FP32 or nearly so.  Against
// FP64, in FP32 steps of the result (2^20 x 40 arguments a stretch): 8 for
// -1 < z < 1, 10 down to -3, 33 down to -6, growing as z^2 with the exponential,
// 125 at -13; 1.5 above 1 and half a step above 3.  A quarter of the
// instructions of erfcf (a 203 x 4096 layer: 2 us of 16).
__device__ __forceinline__ float gelu_fast(float z) {
  const float w = fminf(fabsf(z), 100.0f);
  const float r = __builtin_amdgcn_rcpf(w + 3.75f), u = __builtin_fmaf(r, -7.5f, 1.0f);
  float q = 0.00044344825f;
  q = __builtin_fmaf(q, u, 0.0005096253f);
  q = __builtin_fmaf(q, u, -0.00416902f);
  q = __builtin_fmaf(q, u, 0.0012000743f);
  q = __builtin_fmaf(q, u, 0.037492506f);
  q = __builtin_fmaf(q, u, -0.15152083f);
  q = __builtin_fmaf(q, u, 0.3529396f);
  q = __builtin_fmaf(q, u, -0.5881883f);
  q = __builtin_fmaf(q, u, 0.7502941f);
  const float e = __builtin_amdgcn_exp2f(w * w * -0.72134752044f);
  const float p = 0.5f * z;
  return (p + fabsf(p)) - (w * r) * (q * e);
}

// The activation of N values.  The choice is the same for the whole launch and
// stands outside the values, so that the code of the others is stepped over
// once: instruction fetches of code that is run once are a good part of a
// short kernel's time.
template <int N>
__device__ __forceinline__ void act_apply(int act, float (&z)[N]) {
  switch (act) {
    case kFnRelu:
#pragma unroll
      for (int r = 0; r < N; ++r) z[r] = z[r] <= 0.0f ? 0.0f : z[r];   // (NaN stays)
      break;
    // z / (1 + e^-z): the hardware exponential and reciprocal (1 ulp each).
    case kFnSilu:
#pragma unroll
      for (int r = 0; r < N; ++r) z[r] = silu_fast(z[r]);
      break;
    case kFnGelu:
#pragma unroll
      for (int r = 0; r < N; ++r) z[r] = gelu_fast(z[r]);
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

// Rounding of an output to bfloat16 bits by the hardware conversion: to the
// nearest, ties to even, and NaN of any payload stays NaN (a caller's bias or
// residual may hold one; integer rounding would carry a payload of ones into the
// sign, 0x7FFFFFFF to -0, and with a test for it cost 5120 x 17408 M = 4096 653
// against 649 us).
__device__ __forceinline__ uint32_t out_bf16_bits(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
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
  else static_cast<uint16_t*>(e.out)[o] = (uint16_t)out_bf16_bits(y);
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
    const uint32_t lo = out_bf16_bits(y[0]) | (out_bf16_bits(y[1]) << 16);
    const uint32_t hi = out_bf16_bits(y[2]) | (out_bf16_bits(y[3]) << 16);
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(e.out) + o) = u32x2{lo, hi};
  }
}

// Epilogue of a wavefront's MT x NTW accumulator tiles in the matrix
// instruction's layout (lane 16 g + n: rows 4 g .. 4 g + 3 of column n), rows
// row0 + [0, nrows), streaming columns n0 + [0, 16 NTW).  GATED: the column
// tiles alternate gate and up, and column n of pair q is output column
// n0 / 2 + 16 q + n.  One store per value: the LDS-staged kernel for operands
// past 2 GiB, whose product takes long.
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

// What the epilogue reads for four consecutive output columns of a row,
// requested ahead of their use (the residual as stored).
template <int N>
struct EpiIn {
  float b0[4], b1[4];
  u32x4 res[N];
};
template <bool GATED, int N>
__device__ __forceinline__ void epi_request_bias(const LinearEpi& ep, int64_t col, EpiIn<N>& d) {
  if (!ep.bias) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    d.b0[j] = ep.bias[col + j];
    if constexpr (GATED) d.b1[j] = ep.bias[ep.half + col + j];
  }
}
__device__ __forceinline__ void epi_request_res(const LinearEpi& ep, int64_t row, int64_t col, u32x4& d) {
  if (!ep.res) return;
  const int64_t i = row * ep.ldr + col;
  if (ep.res_f32) {
    d = *reinterpret_cast<const u32x4*>(static_cast<const float*>(ep.res) + i);
  } else {
    const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(ep.res) + i);
    d[0] = w[0];
    d[1] = w[1];
  }
}
template <bool GATED>
__device__ __forceinline__ void epi_request(const LinearEpi& ep, int64_t row, int64_t col, EpiIn<1>& d) {
  epi_request_bias<GATED>(ep, col, d);
  epi_request_res(ep, row, col, d.res[0]);
}
// Finishes four output columns from col of N rows: z the products (gated: the
// gates; u the up projections), row[n] < 0: none.
template <bool GATED, int N>
__device__ __forceinline__ void epi_finish(const LinearEpi& ep, float (&z)[4 * N], const f32x4 (&u)[N],
                                           const EpiIn<N>& in, const int64_t (&row)[N], int64_t col) {
  if (ep.bias) {
#pragma unroll
    for (int k = 0; k < 4 * N; ++k) z[k] += in.b0[k % 4];
  }
  act_apply(ep.act, z);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    f32x4 y = {z[4 * n], z[4 * n + 1], z[4 * n + 2], z[4 * n + 3]};
    if constexpr (GATED) {
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] *= ep.bias ? u[n][j] + in.b1[j] : u[n][j];
    }
    if (ep.res) {
      if (ep.res_f32) {
        y += __builtin_bit_cast(f32x4, in.res[n]);
      } else {
        y[0] += bf16_bits_to_f32(in.res[n][0] & 0xFFFFu);
        y[1] += bf16_bits_to_f32(in.res[n][0] >> 16);
        y[2] += bf16_bits_to_f32(in.res[n][1] & 0xFFFFu);
        y[3] += bf16_bits_to_f32(in.res[n][1] >> 16);
      }
    }
    if (row[n] < 0) continue;
    const int64_t o = row[n] * ep.ldo + col;
    if (ep.out_f32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(ep.out) + o) = y;
    } else {
      const uint32_t lo = out_bf16_bits(y[0]) | (out_bf16_bits(y[1]) << 16);
      const uint32_t hi = out_bf16_bits(y[2]) | (out_bf16_bits(y[3]) << 16);
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(ep.out) + o) = u32x2{lo, hi};
    }
  }
}

// First streaming column, within a tile, of the thread's four output columns
// (gated: of the gate; its up columns lie 16 further).
template <bool GATED>
__device__ __forceinline__ int tile_col(int c4) {
  return GATED ? (c4 >> 4) * 32 + (c4 & 15) : c4;
}

// Finishes ROWS rows of column block nb (BN streaming columns) of a workgroup's
// tile out of LDS: row_of(r) is row r's row of the output, sum(at) the four
// products at float `at` of LDS, in rows of BN + 4.  A thread keeps its four
// columns and walks down the rows, N at a time; the residuals of the next N are
// requested before the present ones are finished.
template <bool GATED, int ROWS, int BN, int THREADS, class RowOf, class Sum>
__device__ __forceinline__ void emit_tile(const LinearEpi& ep, int64_t M, int64_t n_all, int64_t nb,
                                          const RowOf& row_of, const Sum& sum) {
  constexpr int SW = BN + 4, OUTC = GATED ? BN / 2 : BN, STEP = THREADS / (OUTC / 4),
                N = ROWS >= 4 * STEP ? 4 : ROWS >= 2 * STEP ? 2 : 1;
  static_assert(THREADS % (OUTC / 4) == 0, "a thread's columns stay");
  const int r0 = threadIdx.x / (OUTC / 4), c4 = threadIdx.x % (OUTC / 4) * 4, src = tile_col<GATED>(c4);
  const int64_t col = nb * OUTC + c4;
  if (col >= (GATED ? n_all / 2 : n_all)) return;
  EpiIn<N> in;
  u32x4 ahead[N];
  auto row_at = [&](int r) {
    const int64_t row = r < ROWS ? (int64_t)row_of(r) : M;
    return row < M ? row : -1;
  };
  auto request = [&](int r) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int64_t row = row_at(r + n * STEP);
      if (row >= 0) epi_request_res(ep, row, col, ahead[n]);
    }
  };
  epi_request_bias<GATED>(ep, col, in);
  request(r0);
#pragma unroll 1
  for (int r = r0; r < ROWS; r += N * STEP) {
    int64_t row[N];
    f32x4 u[N];
    float z[4 * N];
#pragma unroll
    for (int n = 0; n < N; ++n) in.res[n] = ahead[n];
    request(r + N * STEP);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      row[n] = row_at(r + n * STEP);
      const int at = row[n] < 0 ? src : (r + n * STEP) * SW + src;
      const f32x4 v = sum(at);
      if constexpr (GATED) u[n] = sum(at + 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) z[4 * n + j] = v[j];
    }
    epi_finish<GATED, N>(ep, z, u, in, row, col);
  }
}

}  // namespace nvfp4
