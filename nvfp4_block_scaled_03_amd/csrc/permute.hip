// Rows of x in the order of their experts (moe_permute), the weighted sum of a
// token's rows (moe_unpermute) and its gradients, for gfx950.
//
// The permutation is moe_align's: pair f = t topk + j (the shared expert's pairs
// follow, f = T topk + t) has its row at inv_pos[f], or none.  Work goes by
// tokens, so that x, the sums and d_out are read or written once and only the
// rows themselves are scattered or gathered, in whole pieces of 16 bytes.  No
// atomics: a row belongs to one pair.  Sums run in FP32 in the order of j, the
// shared row last.  Bound: bytes.
#include <algorithm>

#include "common.h"
#include "permute.h"

namespace nvfp4 {
namespace {

__device__ __forceinline__ uint32_t bf16_of(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// A piece of 8 (bfloat16) or 4 (float32) elements.
template <bool F32>
struct Piece {
  static constexpr int N = F32 ? 4 : 8;
  __device__ __forceinline__ static void unpack(const u32x4& r, float (&v)[N]) {
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __int_as_float((int)r[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_bits_to_f32(r[j] & 0xFFFFu);
        v[2 * j + 1] = __int_as_float((int)(r[j] & 0xFFFF0000u));
      }
    }
  }
  __device__ __forceinline__ static u32x4 pack(const float (&v)[N]) {
    u32x4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (F32) r[j] = (uint32_t)__float_as_int(v[j]);
      else r[j] = bf16_of(v[2 * j]) | (bf16_of(v[2 * j + 1]) << 16);
    }
    return r;
  }
};

struct KernelArgs {
  int T, topk, shared, P;
  int64_t V;                // pieces of a row
  const int32_t* kept;      // offsets[slots]
  const int32_t* inv_pos;
  const float* w;
};

// Row of pair j of token t, or -1 (also for a value outside the rows).
__device__ __forceinline__ int row_of(const KernelArgs& p, int64_t t, int j) {
  const int r = p.inv_pos[j < p.topk ? t * p.topk + j : (int64_t)p.T * p.topk + t];
  return (unsigned)r < (unsigned)p.P ? r : -1;
}

// Workgroups from `first` on clear the rows behind the last kept one.
__device__ __forceinline__ void clear_tail(const KernelArgs& p, u32x4* rows, int64_t first) {
  const int64_t from = min(max(*p.kept, 0), p.P) * p.V, to = (int64_t)p.P * p.V;
  const int64_t step = ((int64_t)gridDim.x - first) * blockDim.x;
  for (int64_t i = from + ((int64_t)blockIdx.x - first) * blockDim.x + threadIdx.x; i < to; i += step)
    rows[i] = u32x4{0, 0, 0, 0};
}

// A thread moves one piece of a token's row to all its places.
__global__ __launch_bounds__(256) void permute_kernel(KernelArgs p, const uint8_t* __restrict__ x, int64_t ld_bytes,
                                                      u32x4* __restrict__ rows, int64_t blocks) {
  if (blockIdx.x >= blocks) return clear_tail(p, rows, blocks);
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, t = i / p.V, v = i - t * p.V;
  if (t >= p.T) return;
  const u32x4 d = *reinterpret_cast<const u32x4*>(x + t * ld_bytes + v * 16);
  const int n = p.topk + p.shared;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const int r = row_of(p, t, j);
    if (r >= 0) rows[r * p.V + v] = d;
  }
}

// A thread sums one piece over a token's rows.
template <bool F32, bool OUT_F32>
__global__ __launch_bounds__(256) void unpermute_kernel(KernelArgs p, const u32x4* __restrict__ rows,
                                                        void* __restrict__ out) {
  constexpr int N = Piece<F32>::N;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, t = i / p.V, v = i - t * p.V;
  if (t >= p.T) return;
  float acc[N] = {};
  const int n = p.topk + p.shared;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const int r = row_of(p, t, j);
    if (r < 0) continue;
    const float w = p.w && j < p.topk ? p.w[t * p.topk + j] : 1.0f;
    float d[N];
    Piece<F32>::unpack(rows[r * p.V + v], d);
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = __builtin_fmaf(w, d[k], acc[k]);
  }
  if constexpr (F32 == OUT_F32) {
    static_cast<u32x4*>(out)[i] = Piece<F32>::pack(acc);
  } else if constexpr (OUT_F32) {   // bf16 rows, float32 sums
    f32x4* o = static_cast<f32x4*>(out) + 2 * i;
    o[0] = f32x4{acc[0], acc[1], acc[2], acc[3]};
    o[1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
  } else {                          // float32 rows, bf16 sums
    static_cast<u32x2*>(out)[i] =
        u32x2{bf16_of(acc[0]) | (bf16_of(acc[1]) << 16), bf16_of(acc[2]) | (bf16_of(acc[3]) << 16)};
  }
}

// A wavefront per pair: its row's gradient and its weight's.  The workgroups
// of a token are eight apart, on one XCD, whose L2 holds the token's d_out.
template <bool F32, bool OUT_F32>
__global__ __launch_bounds__(256) void unpermute_backward_kernel(KernelArgs p, const void* __restrict__ d_out,
                                                                 const u32x4* __restrict__ rows,
                                                                 u32x4* __restrict__ d_rows, float* __restrict__ d_w,
                                                                 int groups, int64_t blocks) {
  if (blockIdx.x >= blocks) return clear_tail(p, d_rows, blocks);
  constexpr int N = Piece<F32>::N;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)(blockIdx.x / (8 * groups)) * 8 + blockIdx.x % 8;
  const int j = blockIdx.x / 8 % groups * 4 + (threadIdx.x >> 6), n = p.topk + p.shared;
  if (t >= p.T || j >= n) return;
  const int r = row_of(p, t, j);
  const bool weighted = p.w && j < p.topk;
  float dot = 0.0f;
  if (r >= 0) {
    const float w = weighted ? p.w[t * p.topk + j] : 1.0f;
#pragma unroll 4
    for (int64_t v = lane; v < p.V; v += 64) {
      float d[N], x[N];
      if constexpr (F32 == OUT_F32) {
        Piece<F32>::unpack(static_cast<const u32x4*>(d_out)[t * p.V + v], d);
      } else if constexpr (OUT_F32) {
        const f32x4* at = static_cast<const f32x4*>(d_out) + 2 * (t * p.V + v);
        const f32x4 a = at[0], b = at[1];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          d[k] = a[k];
          d[4 + k] = b[k];
        }
      } else {
        const u32x2 a = static_cast<const u32x2*>(d_out)[t * p.V + v];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          d[2 * k] = bf16_bits_to_f32(a[k] & 0xFFFFu);
          d[2 * k + 1] = __int_as_float((int)(a[k] & 0xFFFF0000u));
        }
      }
      if (d_w) {
        Piece<F32>::unpack(rows[r * p.V + v], x);
#pragma unroll
        for (int k = 0; k < N; ++k) dot = __builtin_fmaf(d[k], x[k], dot);
      }
#pragma unroll
      for (int k = 0; k < N; ++k) d[k] *= w;
      if (d_rows) d_rows[r * p.V + v] = Piece<F32>::pack(d);
    }
  }
  if (d_w && j < p.topk) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) dot += __shfl_xor(dot, off);
    if (lane == 0) d_w[t * p.topk + j] = dot;
  }
}

KernelArgs kernel_args(const PermuteArgs& a, bool f32) {
  return KernelArgs{a.T, a.topk, a.shared, a.T * (a.topk + a.shared), a.W / (f32 ? 4 : 8), a.offsets + a.slots,
                    a.inv_pos, a.w};
}
// Workgroups that clear the tail: they leave at once where no pair was dropped.
int64_t tail_blocks(const KernelArgs& k) { return std::min<int64_t>(1024, (k.P * k.V + 255) / 256); }

}  // namespace

hipError_t launch_permute(const PermuteArgs& a, const void* x, bool f32, int64_t ldx, void* rows, bool zero_tail,
                          hipStream_t s) {
  const KernelArgs k = kernel_args(a, f32);
  const int64_t blocks = (k.T * k.V + 255) / 256;
  permute_kernel<<<(unsigned)(blocks + (zero_tail ? tail_blocks(k) : 0)), 256, 0, s>>>(
      k, static_cast<const uint8_t*>(x), ldx * (f32 ? 4 : 2), static_cast<u32x4*>(rows), blocks);
  return hipGetLastError();
}

hipError_t launch_unpermute(const PermuteArgs& a, const void* rows, bool f32, void* out, bool out_f32, hipStream_t s) {
  const KernelArgs k = kernel_args(a, f32);
  const unsigned blocks = (unsigned)((k.T * k.V + 255) / 256);
  const u32x4* r = static_cast<const u32x4*>(rows);
  if (f32 && out_f32) unpermute_kernel<true, true><<<blocks, 256, 0, s>>>(k, r, out);
  else if (f32) unpermute_kernel<true, false><<<blocks, 256, 0, s>>>(k, r, out);
  else if (out_f32) unpermute_kernel<false, true><<<blocks, 256, 0, s>>>(k, r, out);
  else unpermute_kernel<false, false><<<blocks, 256, 0, s>>>(k, r, out);
  return hipGetLastError();
}

hipError_t launch_unpermute_backward(const PermuteArgs& a, const void* d_out, bool out_f32, const void* rows, bool f32,
                                     void* d_rows, float* d_w, bool zero_tail, hipStream_t s) {
  const KernelArgs k = kernel_args(a, f32);
  const int groups = (k.topk + k.shared + 3) / 4;
  const int64_t blocks = (int64_t)((k.T + 7) / 8) * 8 * groups;
  const unsigned grid = (unsigned)(blocks + (zero_tail && d_rows ? tail_blocks(k) : 0));
  const u32x4* r = static_cast<const u32x4*>(rows);
  u32x4* d = static_cast<u32x4*>(d_rows);
  if (f32 && out_f32) unpermute_backward_kernel<true, true><<<grid, 256, 0, s>>>(k, d_out, r, d, d_w, groups, blocks);
  else if (f32) unpermute_backward_kernel<true, false><<<grid, 256, 0, s>>>(k, d_out, r, d, d_w, groups, blocks);
  else if (out_f32) unpermute_backward_kernel<false, true><<<grid, 256, 0, s>>>(k, d_out, r, d, d_w, groups, blocks);
  else unpermute_backward_kernel<false, false><<<grid, 256, 0, s>>>(k, d_out, r, d, d_w, groups, blocks);
  return hipGetLastError();
}

}  // namespace nvfp4
