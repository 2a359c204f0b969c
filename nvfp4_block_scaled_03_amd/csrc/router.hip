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
// Both operands are row-major along the contraction, which is the matrix
// instruction's operand layout (lane 16 g + m: row m, 8 consecutive k of the
// g-th quarter of the step), so fragments load straight from memory, 16 bytes
// a lane.  Which k of a step a quarter takes is free as long as both operands
// agree.  A workgroup owns a 16 x 16 tile and its wavefronts split the steps
// of K; their partial sums meet in LDS in a fixed order.
//
// float32 weights: w = w0 + w1 + w2 with the top 8 significant bits of what is
// left in each part (truncated, so each difference is exact); three bf16
// products carry all 24 bits, but for parts below the smallest normal number.
// ---------------------------------------------------------------------------
constexpr int kGateWaves = 8;

__device__ __forceinline__ uint32_t pack_hi16(uint32_t a, uint32_t b) {   // {a >> 16, b >> 16}
  return __builtin_amdgcn_perm(b, a, 0x07060302);
}

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

template <bool F32W>
__global__ __launch_bounds__(kGateWaves * kWave) void gate_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                  const void* __restrict__ wg,
                                                                  const float* __restrict__ bias, int T, int E,
                                                                  int H, float* __restrict__ out) {
  __shared__ f32x4 red[kGateWaves][kWave];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * 16;
  const int e0 = blockIdx.y * 16;
  const int64_t row = min(t0 + m, (int64_t)T - 1);   // rows and columns past the end repeat the last one
  const int col = min(e0 + m, E - 1);
  const int steps = (H + 31) / 32;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = wv; s < steps; s += kGateWaves) {
    const int k = s * 32 + g * 8;                    // H is a multiple of 8: a piece is in or out
    const bool in = k < H;
    const int kk = in ? k : 0;
    u32x4 a = *reinterpret_cast<const u32x4*>(x + row * ldx + kk);
    a = in ? a : u32x4{0, 0, 0, 0};
    const bf16x8 af = __builtin_bit_cast(bf16x8, a);
    if constexpr (F32W) {
      const float* w = static_cast<const float*>(wg) + (int64_t)col * H + kk;
      f32x4 w0 = *reinterpret_cast<const f32x4*>(w), w1 = *reinterpret_cast<const f32x4*>(w + 4);
      w0 = in ? w0 : f32x4{0.f, 0.f, 0.f, 0.f};
      w1 = in ? w1 : f32x4{0.f, 0.f, 0.f, 0.f};
      const SplitW p = split_f32(w0, w1);
#pragma unroll
      for (int i = 2; i >= 0; --i)                   // smallest parts first
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af, __builtin_bit_cast(bf16x8, p.part[i]), acc, 0, 0, 0);
    } else {
      u32x4 b = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(wg) + (int64_t)col * H + kk);
      b = in ? b : u32x4{0, 0, 0, 0};
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af, __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
    }
  }
  red[wv][lane] = acc;
  __syncthreads();
  if (threadIdx.x >= 256) return;
  // thread (r, lane) of the first four wavefronts: one value of the tile
  const int r = wv;
  float v = 0.0f;
#pragma unroll
  for (int w = 0; w < kGateWaves; ++w) v += reinterpret_cast<const float*>(&red[w][lane])[r];
  const int64_t t = t0 + g * 4 + r;
  const int e = e0 + m;
  if (t < T && e < E) out[t * E + e] = bias ? v + bias[e] : v;
}

// ---------------------------------------------------------------------------
// moe_route.  One wavefront per token; expert e in lane e % 64, slot e / 64.
// The order of the choice values is taken in FP64 (see the header for the
// definition): k rounds of (largest value, lowest id), then the weights of
// the chosen experts in FP64, rounded once.
// ---------------------------------------------------------------------------
__device__ __forceinline__ double shfl_xor_d(double v, int off) { return __shfl_xor(v, off); }

__device__ __forceinline__ float load_logit(const float* z, int64_t i) { return z[i]; }
__device__ __forceinline__ float load_logit(const uint16_t* z, int64_t i) { return bf16_bits_to_f32(z[i]); }

constexpr int kRouteWaves = 4;

template <typename L, int EPL>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_kernel(const L* __restrict__ logits, RouteArgs p) {
  __shared__ double choice[kRouteWaves][EPL * kWave];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int t = blockIdx.x * kRouteWaves + wv;
  if (t >= p.T) return;   // (no barrier follows: wavefronts work alone)
  const L* zt = logits + (int64_t)t * p.ldl;
  float z[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    const float v = e < p.E ? load_logit(zt, e) : -INFINITY;
    z[i] = v > 3.402823466e38f ? 3.402823466e38f : (v >= -3.402823466e38f ? v : -INFINITY);   // NaN: not available
  }
  const bool softmax = p.score == 0;
  // Scores, where the choice or the weights need those of every expert.
  const bool all_scores = p.bias || p.groups > 1 || (softmax && !p.renormalize);
  double c[EPL], zmax = 0.0, sum = 1.0;
  if (all_scores) {
    if (softmax) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < EPL; ++i) m = fmaxf(m, z[i]);
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
      zmax = m > -INFINITY ? (double)m : 0.0;
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        c[i] = exp((double)z[i] - zmax);
        sum += c[i];
      }
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) sum += shfl_xor_d(sum, off);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      double s = softmax ? c[i] / sum : 1.0 / (1.0 + exp(-(double)z[i]));
      if (p.bias && e < p.E) {
        const double b = (double)p.bias[e];
        s = b < INFINITY ? s + b : (b == INFINITY ? s + 3.402823466e38 : -(double)INFINITY);
      }
      c[i] = z[i] > -INFINITY && s == s ? s : -(double)INFINITY;
    }
  }
  uint32_t off_mask = 0;   // slots not to be chosen
  if (p.groups > 1) {
    const int per = p.E / p.groups;
#pragma unroll
    for (int i = 0; i < EPL; ++i) choice[wv][lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    // group g in lane g: its largest value, or the sum of its two largest
    double v = -(double)INFINITY;
    if (lane < p.groups) {
      double a = -(double)INFINITY, b = -(double)INFINITY;
      for (int i = 0; i < per; ++i) {
        const double y = choice[wv][lane * per + i];
        b = y > a ? a : (y > b ? y : b);
        a = y > a ? y : a;
      }
      v = p.group_top2 && b > -(double)INFINITY ? a + b : a;
    }
    int rank = 0;
    for (int h = 0; h < p.groups; ++h) {
      const double o = __shfl(v, h);
      rank += o > v || (o == v && h < lane);
    }
    const uint64_t on = __ballot(lane < p.groups && rank < p.topk_groups);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      if (e >= p.E || !((on >> (e / per)) & 1)) off_mask |= 1u << i;
    }
  }
  // Without a bias the experts are in the order of their logits.
  if (!p.bias) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = (double)z[i];
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) c[i] = (off_mask >> i) & 1 ? -(double)INFINITY : c[i];

  int my_id = -1;          // lane j: the expert chosen in round j and its logit
  float my_z = -INFINITY;
  for (int j = 0; j < p.k; ++j) {
    double bv = -(double)INFINITY;
    float bz = -INFINITY;
    int bi = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const bool better = c[i] > bv;   // ascending ids: the first of equals stays
      bv = better ? c[i] : bv;
      bz = better ? z[i] : bz;
      bi = better ? lane + 64 * i : bi;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const double ov = shfl_xor_d(bv, off);
      const float oz = __shfl_xor(bz, off);
      const int oi = __shfl_xor(bi, off);
      const bool better = ov > bv || (ov == bv && oi < bi);
      bv = better ? ov : bv;
      bz = better ? oz : bz;
      bi = better ? oi : bi;
    }
    if (bi == 0x7FFFFFFF) break;       // none left (the same in every lane)
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = bi == lane + 64 * i ? -(double)INFINITY : c[i];
    if (lane == j) {
      my_id = bi;
      my_z = bz;
    }
  }
  // Weights: lane j's score, renormalised over the chosen ones in their order.
  float zm = my_z;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) zm = fmaxf(zm, __shfl_xor(zm, off));
  double s = 0.0;
  if (my_id >= 0) {
    if (!softmax) s = 1.0 / (1.0 + exp(-(double)my_z));
    else if (p.renormalize) s = exp((double)my_z - (double)zm);
    else s = exp((double)my_z - zmax) / sum;
  }
  if (p.renormalize) {
    double total = 0.0;
    for (int j = 0; j < p.k; ++j) total += __shfl(s, j);
    s = total > 0.0 ? s / total : 0.0;
  }
  if (lane < p.k) {
    p.ids[(int64_t)t * p.k + lane] = my_id;
    p.weights[(int64_t)t * p.k + lane] = (float)(s * (double)p.scale);
  }
}

template <typename L>
hipError_t launch_route_t(const L* logits, const RouteArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((a.T + kRouteWaves - 1) / kRouteWaves);
  const int epl = (a.E + 63) / 64;
  if (epl <= 2) route_kernel<L, 2><<<grid, kRouteWaves * kWave, 0, s>>>(logits, a);
  else if (epl <= 4) route_kernel<L, 4><<<grid, kRouteWaves * kWave, 0, s>>>(logits, a);
  else if (epl <= 8) route_kernel<L, 8><<<grid, kRouteWaves * kWave, 0, s>>>(logits, a);
  else route_kernel<L, 16><<<grid, kRouteWaves * kWave, 0, s>>>(logits, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gate(const uint16_t* x, int64_t ldx, const void* wg, bool w_f32, const float* bias, int T, int E,
                       int H, float* logits, hipStream_t s) {
  const dim3 grid((unsigned)((T + 15) / 16), (unsigned)((E + 15) / 16));
  if (w_f32) gate_kernel<true><<<grid, kGateWaves * kWave, 0, s>>>(x, ldx, wg, bias, T, E, H, logits);
  else gate_kernel<false><<<grid, kGateWaves * kWave, 0, s>>>(x, ldx, wg, bias, T, E, H, logits);
  return hipGetLastError();
}

hipError_t launch_route(const void* logits, bool bf16, const RouteArgs& a, hipStream_t s) {
  return bf16 ? launch_route_t(static_cast<const uint16_t*>(logits), a, s)
              : launch_route_t(static_cast<const float*>(logits), a, s);
}

}  // namespace nvfp4
