// The router's product (moe_gate) and the choice of experts (moe_route), for
// gfx950.
#include "common.h"
#include "launch.h"

namespace nvfp4 {
namespace {

// ---------------------------------------------------------------------------
// moe_gate: z[t][e] = sum_h x[t][h] wg[e][h] + b[e], x bf16, FP32 accumulation
// on the 16x16x32 bf16 matrix instruction.
//
// Both operands are row-major along the contraction.  A load of a matrix
// fragment straight from memory has neighbouring lanes in different rows, one
// 16-byte piece from each of 16 lines, and the address unit takes a line a
// cycle: measured at T = 8192, E = 128, H = 2048 that form took 36 us.  So
// chunks of 64 k (one 128-byte line of every row) travel from memory straight
// into a ring of LDS stages, eight neighbouring lanes to a line, and the
// fragments are read from there.  The 16-byte units of a row are XOR-swizzled
// by the row so that the 16 rows of a fragment fall in distinct banks.
//
// A wavefront owns RM x RN tiles of 16 x 16; a group of WR x WC wavefronts
// shares a ring, and KW groups take turns through the chunks of K (their
// partial sums meet in LDS in a fixed order).
//
// float32 weights: w = w0 + w1 + w2 with the top 8 significant bits of what is
// left in each part (truncated, so each difference is exact); three bf16
// products carry all 24 bits, but for parts below the smallest normal number.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t pack_hi16(uint32_t a, uint32_t b) {   // {a >> 16, b >> 16}
  return __builtin_amdgcn_perm(b, a, 0x07060302);
}

// The three bf16 parts of 8 consecutive float32 weights.
struct SplitW {
  u32x4 part[3];
};
__device__ __forceinline__ SplitW split_f32(const f32x4& lo, const f32x4& hi) {
  SplitW s;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = j < 2 ? lo[2 * j] : hi[2 * j - 4], b = j < 2 ? lo[2 * j + 1] : hi[2 * j - 3];
    const uint32_t a0 = (uint32_t)__float_as_int(a), b0 = (uint32_t)__float_as_int(b);
    const float ar = a - __int_as_float((int)(a0 & 0xFFFF0000u)), br = b - __int_as_float((int)(b0 & 0xFFFF0000u));
    const uint32_t a1 = (uint32_t)__float_as_int(ar), b1 = (uint32_t)__float_as_int(br);
    const float as = ar - __int_as_float((int)(a1 & 0xFFFF0000u)), bs = br - __int_as_float((int)(b1 & 0xFFFF0000u));
    s.part[0][j] = pack_hi16(a0, b0);
    s.part[1][j] = pack_hi16(a1, b1);
    s.part[2][j] = pack_hi16((uint32_t)__float_as_int(as), (uint32_t)__float_as_int(bs));
  }
  return s;
}

// s_waitcnt immediate: at most n vector memory operations outstanding, and no
// LDS read (the export counter left at its maximum): the next direct load goes
// into the slot that was read last, and where a group is one wavefront no
// barrier stands between.
constexpr int gate_wait(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

template <bool F32W, int RM, int RN, int WR, int WC, int KW, int D>
__global__ __launch_bounds__(WR * WC * KW * kWave) void gate_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                    const uint8_t* __restrict__ wg,
                                                                    const float* __restrict__ bias, int T, int E,
                                                                    int H, int row_tiles, float* __restrict__ out) {
  constexpr int G = WR * WC;                         // wavefronts of a group
  constexpr int WU = F32W ? 16 : 8;                  // 16-byte units of a weight row's chunk
  constexpr int BM = 16 * RM * WR, BN = 16 * RN * WC;
  constexpr int LA = BM / 8, LB = BN * WU / 64;      // 1 KiB loads of a stage
  constexpr int LPW = (LA + LB) / G;                 // of which each wavefront issues
  static_assert((LA + LB) % G == 0 && D >= 2 && (D - 2) * LPW <= 63, "whole loads per wavefront");
  constexpr int STAGE = (LA + LB) * 1024;
  constexpr int RED = KW > 1 ? (KW - 1) * G * RM * RN * kWave * 16 : 0;
  constexpr int LDS = KW * D * STAGE > RED ? KW * D * STAGE : RED;
  __shared__ __attribute__((aligned(16))) uint8_t lds[LDS];
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int kw = wv / G, wg_i = wv % G, wr = wg_i / WC, wc = wg_i % WC;
  // Row tiles are the faster index: workgroups that run together share the
  // weights' columns.
  const int64_t t0 = (int64_t)(blockIdx.x % row_tiles) * BM;
  const int e0 = (int)(blockIdx.x / row_tiles) * BN;
  const int chunks = H / 64, trips = (chunks + KW - 1) / KW;

  // Sources of this wavefront's loads.  Rows past the end repeat the last one
  // (their results are never stored).
  const uint8_t* src[LPW];
  uint32_t step[LPW];                                // bytes a chunk on
#pragma unroll
  for (int q = 0; q < LPW; ++q) {
    const int ld = wg_i * LPW + q;
    if (ld < LA) {
      const int r = 8 * ld + (lane >> 3), unit = (lane & 7) ^ ((r >> 1) & 7);
      src[q] = reinterpret_cast<const uint8_t*>(x + min(t0 + r, (int64_t)T - 1) * ldx) + unit * 16;
      step[q] = 128;
    } else {
      const int r = (ld - LA) * (64 / WU) + lane / WU;
      const int unit = F32W ? (lane & 15) ^ (r & 15) : (lane & 7) ^ ((r >> 1) & 7);
      src[q] = wg + (int64_t)min(e0 + r, E - 1) * H * (F32W ? 4 : 2) + unit * 16;
      step[q] = WU * 16;
    }
  }
  const uint32_t ring = (uint32_t)(uintptr_t)lds + kw * D * STAGE;
  // Assembly: the compiler would wait for every direct load before any later
  // LDS read.  Completion is awaited explicitly below.
  auto issue = [&](int c, int slot) {
    c = min(c * KW + kw, chunks - 1);                // past the end: the last chunk, not used
#pragma unroll
    for (int q = 0; q < LPW; ++q)
      asm volatile("global_load_lds_dwordx4 %0, off" : : "v"(src[q] + (uint64_t)c * step[q]),
                   "{m0}"(ring + slot * STAGE + (wg_i * LPW + q) * 1024) : "memory");
  };

  f32x4 acc[RM][RN];
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < RN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto multiply = [&](const bf16x8 (&a)[RM], const u32x4& b0, const u32x4& b1, int j) {
    if constexpr (F32W) {
      const SplitW p = split_f32(__builtin_bit_cast(f32x4, b0), __builtin_bit_cast(f32x4, b1));
#pragma unroll
      for (int q = 2; q >= 0; --q)                   // smallest parts first
#pragma unroll
        for (int i = 0; i < RM; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], __builtin_bit_cast(bf16x8, p.part[q]), acc[i][j],
                                                              0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < RM; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], __builtin_bit_cast(bf16x8, b0), acc[i][j], 0, 0, 0);
    }
  };
  auto compute = [&](int slot) {
    const uint8_t* sa = lds + kw * D * STAGE + slot * STAGE;
    const uint8_t* sb = sa + LA * 1024;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int piece = 4 * s + g;                   // lane group g: 8 k from 8 piece on
      bf16x8 a[RM];
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        const int r = (wr * RM + i) * 16 + m;
        a[i] = *reinterpret_cast<const bf16x8*>(sa + r * 128 + ((piece ^ ((r >> 1) & 7)) * 16));
      }
#pragma unroll
      for (int j = 0; j < RN; ++j) {
        const int r = (wc * RN + j) * 16 + m;
        if constexpr (F32W) {
          const u32x4 b0 = *reinterpret_cast<const u32x4*>(sb + r * 256 + (((2 * piece) ^ (r & 15)) * 16));
          const u32x4 b1 = *reinterpret_cast<const u32x4*>(sb + r * 256 + (((2 * piece + 1) ^ (r & 15)) * 16));
          multiply(a, b0, b1, j);
        } else {
          const u32x4 b0 = *reinterpret_cast<const u32x4*>(sb + r * 128 + ((piece ^ ((r >> 1) & 7)) * 16));
          multiply(a, b0, b0, j);
        }
      }
    }
  };

  // Ring: at the top of trip c the chunks c .. c + D - 2 of the group are in
  // flight; once at most (D - 2) LPW loads remain, chunk c has landed.  The
  // barrier publishes it to the group and says that every wavefront is done
  // with the slot refilled next; a group of one wavefront needs none, its own
  // LDS reads being awaited.
  if (chunks > 0) {
#pragma unroll
    for (int c = 0; c < D - 1; ++c) issue(c, c);
    for (int c0 = 0; c0 < trips; c0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (c0 + d < trips) {
          __builtin_amdgcn_s_waitcnt(gate_wait((D - 2) * LPW));
          if constexpr (G > 1) __syncthreads();
          else asm volatile("" ::: "memory");
          issue(c0 + d + D - 1, (d + D - 1) % D);
          if ((c0 + d) * KW + kw < chunks) compute(d);
        }
      }
    }
    // The loads past the end land before the ring is used again or given up.
    __builtin_amdgcn_s_waitcnt(gate_wait(0));
  }
  // The last H % 64 elements (a multiple of 8: a piece is in or out), straight
  // from memory, by the last group.
  if (chunks * 64 < H && kw == KW - 1) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = chunks * 64 + 8 * (4 * s + g);
      const bool in = k < H;
      const u32x4 zero = {0, 0, 0, 0};
      bf16x8 a[RM];
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        const int64_t r = min(t0 + (wr * RM + i) * 16 + m, (int64_t)T - 1);
        const u32x4 v = *reinterpret_cast<const u32x4*>(x + r * ldx + (in ? k : 0));
        a[i] = __builtin_bit_cast(bf16x8, in ? v : zero);
      }
#pragma unroll
      for (int j = 0; j < RN; ++j) {
        const int64_t r = min(e0 + (wc * RN + j) * 16 + m, E - 1);
        const uint8_t* w = wg + (r * H + (in ? k : 0)) * (F32W ? 4 : 2);
        const u32x4 b0 = *reinterpret_cast<const u32x4*>(w);
        const u32x4 b1 = F32W ? *reinterpret_cast<const u32x4*>(w + 16) : zero;
        multiply(a, in ? b0 : zero, in ? b1 : zero, j);
      }
    }
  }

  if constexpr (KW > 1) {
    f32x4* red = reinterpret_cast<f32x4*>(lds);
    __syncthreads();                                 // every group is done with its ring
    if (kw > 0) {
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < RN; ++j) red[((((kw - 1) * G + wg_i) * RM + i) * RN + j) * kWave + lane] = acc[i][j];
    }
    __syncthreads();
    if (kw > 0) return;
#pragma unroll
    for (int w = 0; w < KW - 1; ++w)
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < RN; ++j) acc[i][j] += red[(((w * G + wg_i) * RM + i) * RN + j) * kWave + lane];
  }
#pragma unroll
  for (int j = 0; j < RN; ++j) {
    const int e = e0 + (wc * RN + j) * 16 + m;
    if (e >= E) continue;
    const float b = bias ? bias[e] : 0.0f;
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t t = t0 + (wr * RM + i) * 16 + 4 * g + r;
        if (t < T) out[t * E + e] = bias ? acc[i][j][r] + b : acc[i][j][r];
      }
  }
}

// One or a few tokens (T <= TM): a wavefront per expert, all lanes along the
// contraction, 8 elements each; the time is one trip to memory.
template <bool F32W, int TM>
__global__ __launch_bounds__(256) void gate_rows_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                        const void* __restrict__ wg, const float* __restrict__ bias,
                                                        int T, int E, int H, float* __restrict__ out) {
  const int lane = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (e >= E) return;
  float acc[TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) acc[t] = 0.0f;
#pragma unroll 4
  for (int k = lane * 8; k < H; k += 8 * kWave) {
    float w[8];
    if constexpr (F32W) {
      const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(wg) + (int64_t)e * H + k);
      const f32x4 a = p[0], b = p[1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = a[j];
        w[4 + j] = b[j];
      }
    } else {
      const u32x4 p = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(wg) + (int64_t)e * H + k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[2 * j] = bf16_bits_to_f32(p[j] & 0xFFFFu);
        w[2 * j + 1] = __int_as_float((int)(p[j] & 0xFFFF0000u));
      }
    }
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const u32x4 p = *reinterpret_cast<const u32x4*>(x + (int64_t)min(t, T - 1) * ldx + k);
      float s = acc[t];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s = __builtin_fmaf(bf16_bits_to_f32(p[j] & 0xFFFFu), w[2 * j], s);
        s = __builtin_fmaf(__int_as_float((int)(p[j] & 0xFFFF0000u)), w[2 * j + 1], s);
      }
      acc[t] = s;
    }
  }
  const float b = bias ? bias[e] : 0.0f;
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    float v = acc[t];
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    if (lane == t && t < T) out[(int64_t)t * E + e] = bias ? v + b : v;
  }
}

template <bool F32W, int RM, int RN, int WR, int WC, int KW, int D>
hipError_t launch_gate_t(const uint16_t* x, int64_t ldx, const void* wg, const float* bias, int T, int E, int H,
                         float* out, hipStream_t s) {
  constexpr int BM = 16 * RM * WR, BN = 16 * RN * WC;
  const int row_tiles = (T + BM - 1) / BM, col_tiles = (E + BN - 1) / BN;
  gate_kernel<F32W, RM, RN, WR, WC, KW, D><<<(unsigned)row_tiles * (unsigned)col_tiles, WR * WC * KW * kWave, 0, s>>>(
      x, ldx, static_cast<const uint8_t*>(wg), bias, T, E, H, row_tiles, out);
  return hipGetLastError();
}

template <bool F32W>
hipError_t launch_gate_w(const uint16_t* x, int64_t ldx, const void* wg, const float* bias, int T, int E, int H,
                         float* out, hipStream_t s) {
  if (T <= 4) {
    const unsigned grid = (unsigned)((E + 3) / 4);
    if (T == 1) gate_rows_kernel<F32W, 1><<<grid, 256, 0, s>>>(x, ldx, wg, bias, T, E, H, out);
    else gate_rows_kernel<F32W, 4><<<grid, 256, 0, s>>>(x, ldx, wg, bias, T, E, H, out);
    return hipGetLastError();
  }
  // The smallest tile whose workgroups still run at once, one per CU: a larger
  // tile loads fewer bytes per product, a smaller one uses more CUs.  KW and D
  // fill LDS.  Measured (us, bf16 / float32 weights, H = 2048 with E = 128 and
  // H = 4096 with E = 512), this rule's tile first, then its neighbours:
  //   T =   64, E = 128  16x16  3.6 / 4.7   32x16  4.6 / 5.8
  //   T = 1024, E = 128  32x16  5.5 / 6.6   16x16  6.1 / 9.4   32x32  5.6 / 8.9
  //   T = 2048, E = 128  32x32  6.4 / 9.3   32x16  8.2 / 11.9  32x64  8.2 / 17.0
  //   T = 4096, E = 128  32x64  9.5 / 17.4  32x32 12.6 / 18.6  64x64 10.0 / 20.4
  //   T = 8192, E = 128  64x64 11.7 / 22.2  32x64 19.9 / 33.6  64x128 17.1 / 37.3
  //   T = 4096, E = 512  64x128 28.4 / 68.2  64x64 30.9 / 75.8  128x128 34.6 / 91.3
  //   T = 8192, E = 1024 (H = 4096)  128x128 79.4 / 198  64x128 107 / 267
  // float32 weights leave 16x16 earlier (T = 128, E = 512: 12.5 against 9.1).
  auto fits = [&](int rows, int cols, int most) {
    return (int64_t)((T + rows - 1) / rows) * ((E + cols - 1) / cols) <= most;
  };
  if (fits(16, 16, F32W ? 128 : 256))
    return launch_gate_t<F32W, 1, 1, 1, 1, F32W ? 12 : 4, F32W ? 2 : 4>(x, ldx, wg, bias, T, E, H, out, s);
  if (fits(32, 16, 256)) return launch_gate_t<F32W, 2, 1, 1, 1, F32W ? 8 : 4, F32W ? 2 : 3>(x, ldx, wg, bias, T, E, H, out, s);
  if (fits(32, 32, 256)) return launch_gate_t<F32W, 2, 1, 1, 2, 4, F32W ? 2 : 3>(x, ldx, wg, bias, T, E, H, out, s);
  if (fits(32, 64, 256)) return launch_gate_t<F32W, 2, 2, 1, 2, F32W ? 2 : 4, 3>(x, ldx, wg, bias, T, E, H, out, s);
  if (fits(64, 64, 256)) return launch_gate_t<F32W, 2, 2, 2, 2, 2, F32W ? 3 : 4>(x, ldx, wg, bias, T, E, H, out, s);
  if (fits(64, 128, 256)) return launch_gate_t<F32W, 4, 2, 1, 4, 1, F32W ? 3 : 4>(x, ldx, wg, bias, T, E, H, out, s);
  return launch_gate_t<F32W, 4, 2, 2, 4, 1, F32W ? 3 : 4>(x, ldx, wg, bias, T, E, H, out, s);
}

// ---------------------------------------------------------------------------
// moe_route.  One wavefront per token; lane l holds the EPL consecutive
// experts from l EPL on, so that of equal values the lowest id sits in the
// lowest lane.  Choice values are FP64 (see the header for the definition);
// each of the k rounds finds the largest of their FP32 roundings, which keep
// the order, and looks at the FP64 values only where several round to it.
// The weights of the chosen experts are FP64, rounded once.
//
// The time is instruction issue (a token's bytes are few): lane exchanges run
// on DPP, not through LDS, and the exponentials of all scores on the short
// FP64 series below.
// ---------------------------------------------------------------------------
// e^x for x <= 0: x = n ln 2 + r, |r| <= ln(2) / 2, the Taylor series of e^r
// up to r^13 (the next term is 4e-18), scaled by 2^n.  ln 2 in two parts, the
// first of 32 bits, so that n times it is exact.
__device__ __forceinline__ double exp_neg(double x) {
  x = x > -800.0 ? x : -800.0;   // 2^-1154: zero
  const double n = __builtin_rint(x * 1.4426950408889634);
  double r = __builtin_fma(-n, 0.693147180369123816490, x);
  r = __builtin_fma(-n, 1.90821492927058770002e-10, r);
  constexpr double c[14] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320,
                            1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600, 1.0 / 6227020800.0};
  double p = c[13];
#pragma unroll
  for (int i = 12; i >= 0; --i) p = __builtin_fma(p, r, c[i]);
  return __builtin_amdgcn_ldexp(p, (int)n);
}
// 1 / d for normal d: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double rcp_d(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
  return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

// The value of lane l (the same in all lanes).
__device__ __forceinline__ double lane_value(double v, int l) {
  const int64_t b = __builtin_bit_cast(int64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)b, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
__device__ __forceinline__ float lane_value(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

// Maximum over the wavefront, the same in all lanes: rows of 16 by
// exchanges, then the rows' results handed on to the last lane.
__device__ __forceinline__ float wave_max(float v) {
  v = row16_max(v);
  const int neg = __float_as_int(-INFINITY);
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(neg, __float_as_int(v), 0x142, 0xA, 0xF, false)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(neg, __float_as_int(v), 0x143, 0xC, 0xF, false)));
  return lane_value(v, 63);
}
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const int64_t b = __builtin_bit_cast(int64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}
// Sum over the wavefront (a fixed order), the same in all lanes.
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_d<0xB1>(v);
  v += dpp_d<0x4E>(v);
  v += dpp_d<0x141>(v);
  v += dpp_d<0x140>(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

__device__ __forceinline__ float logit_value(float v) { return v; }
__device__ __forceinline__ float logit_value(uint16_t v) { return bf16_bits_to_f32(v); }

constexpr int kRouteWaves = 4;
constexpr float kFltMax = 3.402823466e38f;

// FULL: a selection bias or expert groups, where the choice needs every
// score; otherwise the experts are in the order of their logits.
template <typename L, int EPL, bool FULL>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_kernel(const L* __restrict__ logits, RouteArgs p) {
  __shared__ double scores[FULL ? kRouteWaves : 1][FULL ? EPL * kWave : 1];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int t = blockIdx.x * kRouteWaves + wv;
  if (t >= p.T) return;   // (no barrier follows: wavefronts work alone)
  const int e0 = lane * EPL;
  const double kNone = -(double)INFINITY;

  // Logits; an expert that is not available (or does not exist) is -infinity.
  const L* zt = logits + (int64_t)t * p.ldl + e0;
  struct __attribute__((packed)) Pack {
    L v[EPL];
  };
  Pack raw;
  if (e0 + EPL <= p.E) {
    raw = *reinterpret_cast<const Pack*>(zt);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) raw.v[i] = e0 + i < p.E ? zt[i] : L(0);
  }
  float z[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const float v = logit_value(raw.v[i]);
    z[i] = e0 + i < p.E && v >= -kFltMax ? fminf(v, kFltMax) : -INFINITY;   // (NaN compares false)
  }
  const bool softmax = p.score == 0;

  // f: the FP32 roundings of the choice values, in their order.
  float f[EPL];
  double c[FULL ? EPL : 1];
  double zmax = 0.0, sum = 1.0;
  if (softmax && (FULL || !p.renormalize)) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, z[i]);
    m = wave_max(m);
    zmax = m > -INFINITY ? (double)m : 0.0;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const double v = exp_neg((double)z[i] - zmax);
      if constexpr (FULL) c[i] = v;
      s += v;
    }
    sum = wave_sum(s);
  }
  if constexpr (FULL) {
    const double inv = softmax && sum > 0.0 ? 1.0 / sum : 1.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      double s;
      if (softmax) {
        s = c[i] * inv;
      } else {
        const double x = (double)z[i], ex = exp_neg(x < 0.0 ? x : -x), r = rcp_d(1.0 + ex);
        s = x < 0.0 ? ex * r : r;
      }
      bool on = z[i] > -INFINITY;
      if (p.bias) {
        const float b = p.bias[min(e0 + i, p.E - 1)];
        on = on && b >= -kFltMax;
        s += (double)fminf(b, kFltMax);
      }
      c[i] = on ? s : kNone;
    }
    uint64_t keep = ~0ull;   // bit (group << shift): the group is chosen from
    int shift = 0;
    if (p.groups > 1) {
      // 2^shift lanes value a group: its largest choice value, and the
      // largest of the others.
#pragma unroll
      for (int i = 0; i < EPL; ++i) scores[wv][e0 + i] = c[i];
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
      const int per = p.E / p.groups;
      while ((p.groups << (shift + 1)) <= kWave) ++shift;
      const int grp = lane >> shift;
      double a = kNone, b = kNone;
      if (grp < p.groups) {
        for (int i = lane & ((1 << shift) - 1); i < per; i += 1 << shift) {
          const double y = scores[wv][grp * per + i];
          b = fmax(b, fmin(a, y));
          a = fmax(a, y);
        }
      }
      for (int off = 1; off < (1 << shift); off <<= 1) {
        const double oa = __shfl_xor(a, off), ob = __shfl_xor(b, off);
        b = fmax(fmax(b, ob), fmin(a, oa));
        a = fmax(a, oa);
      }
      const double v = p.group_top2 && b > kNone ? a + b : a;
      int rank = 0;          // groups before this one: larger, or equal and lower
      for (int h = 0; h < p.groups; ++h) {
        const double o = lane_value(v, h << shift);
        rank += o > v || (o == v && h < grp);
      }
      keep = __ballot(grp < p.groups && rank < p.topk_groups);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = min(e0 + i, p.E - 1);
        if (!((keep >> ((e / per) << shift)) & 1)) {
          c[i] = kNone;
          z[i] = -INFINITY;
        }
      }
    }
    // Without a bias the experts are in the order of their logits.
#pragma unroll
    for (int i = 0; i < EPL; ++i) f[i] = p.bias ? (float)c[i] : z[i];
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) f[i] = z[i];
  }

  int my_id = -1;            // lane j: the expert chosen in round j and its logit
  float my_z = -INFINITY;
  for (int j = 0; j < p.k; ++j) {
    float best = f[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) best = fmaxf(best, f[i]);
    const float top = wave_max(best);
    if (!(top > -INFINITY)) break;
    int at = EPL - 1;        // the first slot that holds it
    float zt_at = z[EPL - 1];
#pragma unroll
    for (int i = EPL - 2; i >= 0; --i) {
      at = f[i] == top ? i : at;
      if constexpr (FULL) zt_at = f[i] == top ? z[i] : zt_at;
    }
    int win = __builtin_ctzll(__ballot(best == top));
    if constexpr (FULL) {
      if (p.bias) {
        int n = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) n += __builtin_popcountll(__ballot(f[i] == top));
        if (n > 1) {         // several round to the same FP32 value
          double bc = kNone;
          at = 0;
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            const bool better = f[i] == top && c[i] > bc;
            bc = better ? c[i] : bc;
            at = better ? i : at;
            zt_at = better ? z[i] : zt_at;
          }
          double m = bc;
          for (int off = 1; off < kWave; off <<= 1) m = fmax(m, __shfl_xor(m, off));
          win = __builtin_ctzll(__ballot(bc == m && bc > kNone));
        }
      }
    }
    const int slot = __builtin_amdgcn_readlane(at, win);
    const float zw = FULL ? lane_value(zt_at, win) : top;
#pragma unroll
    for (int i = 0; i < EPL; ++i) f[i] = lane == win && i == slot ? -INFINITY : f[i];
    if (lane == j) {
      my_id = win * EPL + slot;
      my_z = zw;
    }
  }
  // Weights: lane j's score, renormalised over the chosen ones in their order.
  double s = 0.0;
  if (softmax) {
    const double ref = p.renormalize ? (double)(FULL ? wave_max(my_z) : lane_value(my_z, 0)) : zmax;
    if (my_id >= 0) s = p.renormalize ? exp((double)my_z - ref) : exp((double)my_z - ref) / sum;
  } else if (my_id >= 0) {
    s = 1.0 / (1.0 + exp(-(double)my_z));
  }
  if (p.renormalize) {
    double total = 0.0;
    for (int j = 0; j < p.k; ++j) total += lane_value(s, j);
    s = total > 0.0 ? s / total : 0.0;
  }
  if (lane < p.k) {
    p.ids[(int64_t)t * p.k + lane] = my_id;
    p.weights[(int64_t)t * p.k + lane] = (float)(s * (double)p.scale);
  }
}

template <typename L, int EPL>
void launch_route_e(const L* logits, const RouteArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((a.T + kRouteWaves - 1) / kRouteWaves);
  if (a.bias || a.groups > 1) route_kernel<L, EPL, true><<<grid, kRouteWaves * kWave, 0, s>>>(logits, a);
  else route_kernel<L, EPL, false><<<grid, kRouteWaves * kWave, 0, s>>>(logits, a);
}

template <typename L>
hipError_t launch_route_t(const L* logits, const RouteArgs& a, hipStream_t s) {
  if (a.E <= 64) launch_route_e<L, 1>(logits, a, s);
  else if (a.E <= 128) launch_route_e<L, 2>(logits, a, s);
  else if (a.E <= 256) launch_route_e<L, 4>(logits, a, s);
  else if (a.E <= 512) launch_route_e<L, 8>(logits, a, s);
  else launch_route_e<L, 16>(logits, a, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gate(const uint16_t* x, int64_t ldx, const void* wg, bool w_f32, const float* bias, int T, int E,
                       int H, float* logits, hipStream_t s) {
  return w_f32 ? launch_gate_w<true>(x, ldx, wg, bias, T, E, H, logits, s)
               : launch_gate_w<false>(x, ldx, wg, bias, T, E, H, logits, s);
}

hipError_t launch_route(const void* logits, bool bf16, const RouteArgs& a, hipStream_t s) {
  return bf16 ? launch_route_t(static_cast<const uint16_t*>(logits), a, s)
              : launch_route_t(static_cast<const float*>(logits), a, s);
}

}  // namespace nvfp4
