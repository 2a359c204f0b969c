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
#include <type_traits>

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

// Rows that the last-level cache (256 MB) cannot hold pass it by (NT): nothing of
// them would be left for their reader, and the lines that writes leave dirty
// delay the reads behind them (8192 x 8 rows of 4 KiB there and back 138 -> 105 us;
// rows that fit are read again from the cache: 4095 x 8 rows of 8 KiB, an eighth
// of them kept, 13.7 us, 20.9 past it).
constexpr int64_t kCacheBytes = int64_t(256) << 20;
template <class Body>
__device__ __forceinline__ void by_size(int kept, int V, const Body& body) {
  if ((int64_t)kept * V * 16 >= kCacheBytes) body(std::true_type());
  else body(std::false_type());
}
template <bool NT>
__device__ __forceinline__ u32x4 load_row(const u32x4* at) {
  if constexpr (NT) return __builtin_nontemporal_load(at);
  else return *at;
}
template <bool NT>
__device__ __forceinline__ void store_row(u32x4* at, const u32x4& v) {
  if constexpr (NT) __builtin_nontemporal_store(v, at);
  else *at = v;
}

struct KernelArgs {
  int T, topk, shared, P;
  int V;                    // pieces of a row
  int bpt;                  // workgroups of a token
  const int32_t* kept;      // offsets[slots]
  const int32_t* inv_pos;
  const float* w;
};

// Row of pair j of token t, or -1 (also for a value outside the rows).  The
// same for the whole workgroup or wavefront: read through the scalar cache.
__device__ __forceinline__ int row_of(const KernelArgs& p, int t, int j) {
  const int r = ld_uniform(p.inv_pos + (j < p.topk ? (int64_t)t * p.topk + j : (int64_t)p.T * p.topk + t));
  return (unsigned)r < (unsigned)p.P ? r : -1;
}

// Rows of pairs.
__device__ __forceinline__ int kept_rows(const KernelArgs& p) { return min(max(ld_uniform(p.kept), 0), p.P); }

// Workgroups from `first` on clear the rows behind the last kept one.
__device__ __forceinline__ void clear_tail(const KernelArgs& p, u32x4* rows, unsigned first) {
  const int64_t from = (int64_t)kept_rows(p) * p.V, to = (int64_t)p.P * p.V;
  const int64_t step = (int64_t)(gridDim.x - first) * blockDim.x;
  for (int64_t i = from + (int64_t)(blockIdx.x - first) * blockDim.x + threadIdx.x; i < to; i += step)
    rows[i] = u32x4{0, 0, 0, 0};
}

// Rows and weights of up to 64 pairs of a token, one a lane, read at once (a
// chain of scalar loads, one waiting for the other, had cost more than the rows).
struct Pairs {
  int row;
  float w;
  __device__ __forceinline__ Pairs(const KernelArgs& p, int t, int j, int n) {
    const bool on = j < n, routed = j < p.topk;
    const int64_t f = on ? (routed ? (int64_t)t * p.topk + j : (int64_t)p.T * p.topk + t) : 0;
    const int r = p.inv_pos[f];
    row = on && (unsigned)r < (unsigned)p.P ? r : -1;
    w = 1.0f;
    if (p.w) {
      const float v = p.w[routed ? f : 0];
      w = routed ? v : 1.0f;
    }
  }
  __device__ __forceinline__ int row_at(int j) const { return __builtin_amdgcn_readlane(row, j); }
  __device__ __forceinline__ float w_at(int j) const {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), j));
  }
};

// A thread moves one piece of a token's row to all its places.
__global__ __launch_bounds__(256) void permute_kernel(KernelArgs p, const uint8_t* __restrict__ x, int64_t ld_bytes,
                                                      u32x4* __restrict__ rows, unsigned blocks) {
  if (blockIdx.x >= blocks) return clear_tail(p, rows, blocks);
  const int t = (int)(blockIdx.x / (unsigned)p.bpt);
  const int v = ((int)blockIdx.x - t * p.bpt) * (int)blockDim.x + (int)threadIdx.x;
  const u32x4 d = v < p.V ? *reinterpret_cast<const u32x4*>(x + t * ld_bytes + (int64_t)v * 16) : u32x4{0, 0, 0, 0};
  const int n = p.topk + p.shared;
  by_size(kept_rows(p), p.V, [&](auto nt) {
    for (int j0 = 0; j0 < n; j0 += 64) {
      const Pairs pairs(p, t, j0 + (int)(threadIdx.x & 63), n);
      const int m = min(64, n - j0);
#pragma unroll 4
      for (int j = 0; j < m; ++j) {
        const int r = pairs.row_at(j);
        if (r >= 0 && v < p.V) store_row<decltype(nt)::value>(rows + (int64_t)r * p.V + v, d);
      }
    }
  });
}

// A thread sums one piece over a token's rows.
template <bool F32, bool OUT_F32>
__global__ __launch_bounds__(256) void unpermute_kernel(KernelArgs p, const u32x4* __restrict__ rows,
                                                        void* __restrict__ out) {
  constexpr int N = Piece<F32>::N;
  const int t = (int)(blockIdx.x / (unsigned)p.bpt);
  const int v = ((int)blockIdx.x - t * p.bpt) * (int)blockDim.x + (int)threadIdx.x;
  float acc[N] = {};
  const int n = p.topk + p.shared;
  by_size(kept_rows(p), p.V, [&](auto nt) {
    for (int j0 = 0; j0 < n; j0 += 64) {
      const Pairs pairs(p, t, j0 + (int)(threadIdx.x & 63), n);
      // The pairs that have a row, in their order.  Their pieces are requested
      // together (places past the last one: it once more), without branches
      // between the loads, each of which would wait for the load before (256 x 11
      // rows of 8 KiB: up to 8 at a time 8.6 us, up to 12 7.2).
      uint64_t left = __ballot(pairs.row >= 0);
      auto batch = [&](auto size) {
        constexpr int B = decltype(size)::value;
        const int count = __popcll(left);
        int j = 0, at[B];
        u32x4 d[B];
#pragma unroll
        for (int k = 0; k < B; ++k) {
          if (left) j = __builtin_ctzll(left);
          left &= left - 1;
          at[k] = j;
          d[k] = load_row<decltype(nt)::value>(rows + (int64_t)pairs.row_at(j) * p.V + min(v, p.V - 1));
        }
#pragma unroll
        for (int k = 0; k < B; ++k) {
          if (k < count) {
            const float w = pairs.w_at(at[k]);
            float e[N];
            Piece<F32>::unpack(d[k], e);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = __builtin_fmaf(w, e[i], acc[i]);
          }
        }
      };
      while (left) {
        if (__popcll(left) > 8) batch(std::integral_constant<int, 12>());
        else if (__popcll(left) > 4) batch(std::integral_constant<int, 8>());
        else if (__popcll(left) > 2) batch(std::integral_constant<int, 4>());
        else batch(std::integral_constant<int, 2>());
      }
    }
  });
  if (v >= p.V) return;
  const int64_t i = (int64_t)t * p.V + v;
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

// WPP wavefronts per pair (one: up to four pairs a workgroup): its row's
// gradient and its weight's.  The workgroups of a token are eight apart, on one
// XCD, whose L2 holds the token's d_out.
template <bool F32, bool OUT_F32, int WPP>
__global__ __launch_bounds__(256) void unpermute_backward_kernel(KernelArgs p, const void* __restrict__ d_out,
                                                                 const u32x4* __restrict__ rows,
                                                                 u32x4* __restrict__ d_rows, float* __restrict__ d_w,
                                                                 int groups, unsigned blocks) {
  if (blockIdx.x >= blocks) return clear_tail(p, d_rows, blocks);
  constexpr int N = Piece<F32>::N;
  __shared__ float dots[WPP];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int t = (int)(blockIdx.x / (8u * groups)) * 8 + (int)(blockIdx.x % 8);
  const int j = (int)(blockIdx.x / 8 % groups) * (4 / WPP) + wave / WPP, part = wave % WPP;
  const int n = p.topk + p.shared;
  if (t >= p.T || j >= n) return;
  const int r = row_of(p, t, j);
  const bool weighted = p.w && j < p.topk;
  float dot = 0.0f;
  if (r >= 0) {
    const float w = weighted ? ld_uniform(p.w + (int64_t)t * p.topk + j) : 1.0f;
    const int64_t at_r = (int64_t)r * p.V, at_d = (int64_t)t * p.V;
    by_size(kept_rows(p), p.V, [&](auto nt) {
#pragma unroll 4
      for (int v = part * 64 + lane; v < p.V; v += WPP * 64) {
        float d[N], x[N];
        if constexpr (F32 == OUT_F32) {
          Piece<F32>::unpack(static_cast<const u32x4*>(d_out)[at_d + v], d);
        } else if constexpr (OUT_F32) {
          const f32x4* at = static_cast<const f32x4*>(d_out) + 2 * (at_d + v);
          const f32x4 a = at[0], b = at[1];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            d[k] = a[k];
            d[4 + k] = b[k];
          }
        } else {
          const u32x2 a = static_cast<const u32x2*>(d_out)[at_d + v];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            d[2 * k] = bf16_bits_to_f32(a[k] & 0xFFFFu);
            d[2 * k + 1] = __int_as_float((int)(a[k] & 0xFFFF0000u));
          }
        }
        if (d_w) {
          Piece<F32>::unpack(load_row<decltype(nt)::value>(rows + at_r + v), x);
#pragma unroll
          for (int k = 0; k < N; ++k) dot = __builtin_fmaf(d[k], x[k], dot);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) d[k] *= w;
        if (d_rows) store_row<decltype(nt)::value>(d_rows + at_r + v, Piece<F32>::pack(d));
      }
    });
  }
  if (d_w && j < p.topk) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) dot += __shfl_xor(dot, off);
    if constexpr (WPP > 1) {   // (the same pair for the whole workgroup)
      if (lane == 0) dots[part] = dot;
      __syncthreads();
      dot = dots[0];
#pragma unroll
      for (int w = 1; w < WPP; ++w) dot += dots[w];
    }
    if (lane == 0 && part == 0) d_w[(int64_t)t * p.topk + j] = dot;
  }
}

KernelArgs kernel_args(const PermuteArgs& a, bool f32) {
  return KernelArgs{a.T, a.topk, a.shared, a.T * (a.topk + a.shared), (int)(a.W / (f32 ? 4 : 8)), 1,
                    a.offsets + a.slots, a.inv_pos, a.w};
}
// Threads of a workgroup that takes pieces of one token.
int threads_for(int V) { return std::min(256, (V + 63) / 64 * 64); }
// Workgroups that clear the tail: they leave at once where no pair was dropped.
int64_t tail_blocks(const KernelArgs& k) { return std::min<int64_t>(1024, ((int64_t)k.P * k.V + 255) / 256); }

}  // namespace

hipError_t launch_permute(const PermuteArgs& a, const void* x, bool f32, int64_t ldx, void* rows, bool zero_tail,
                          hipStream_t s) {
  KernelArgs k = kernel_args(a, f32);
  const int threads = threads_for(k.V);
  k.bpt = (k.V + threads - 1) / threads;
  const int64_t blocks = (int64_t)k.T * k.bpt;
  const unsigned grid = (unsigned)(blocks + (zero_tail ? tail_blocks(k) : 0));
  const uint8_t* src = static_cast<const uint8_t*>(x);
  const int64_t ld = ldx * (f32 ? 4 : 2);
  u32x4* r = static_cast<u32x4*>(rows);
  permute_kernel<<<grid, threads, 0, s>>>(k, src, ld, r, (unsigned)blocks);
  return hipGetLastError();
}

hipError_t launch_unpermute(const PermuteArgs& a, const void* rows, bool f32, void* out, bool out_f32, hipStream_t s) {
  KernelArgs k = kernel_args(a, f32);
  const int threads = threads_for(k.V);
  k.bpt = (k.V + threads - 1) / threads;
  const unsigned blocks = (unsigned)((int64_t)k.T * k.bpt);
  const u32x4* r = static_cast<const u32x4*>(rows);
  if (f32 && out_f32) unpermute_kernel<true, true><<<blocks, threads, 0, s>>>(k, r, out);
  else if (f32) unpermute_kernel<true, false><<<blocks, threads, 0, s>>>(k, r, out);
  else if (out_f32) unpermute_kernel<false, true><<<blocks, threads, 0, s>>>(k, r, out);
  else unpermute_kernel<false, false><<<blocks, threads, 0, s>>>(k, r, out);
  return hipGetLastError();
}

template <int WPP>
hipError_t launch_backward_t(const KernelArgs& k, const void* d_out, bool out_f32, const u32x4* r, bool f32, u32x4* d,
                             float* d_w, bool zero_tail, hipStream_t s) {
  const int n = k.topk + k.shared, groups = (n * WPP + 3) / 4, threads = 64 * std::min(4, n * WPP);
  const int64_t blocks = (int64_t)((k.T + 7) / 8) * 8 * groups;
  const unsigned grid = (unsigned)(blocks + (zero_tail && d ? tail_blocks(k) : 0)), b = (unsigned)blocks;
  if (f32 && out_f32) unpermute_backward_kernel<true, true, WPP><<<grid, threads, 0, s>>>(k, d_out, r, d, d_w, groups, b);
  else if (f32) unpermute_backward_kernel<true, false, WPP><<<grid, threads, 0, s>>>(k, d_out, r, d, d_w, groups, b);
  else if (out_f32)
    unpermute_backward_kernel<false, true, WPP><<<grid, threads, 0, s>>>(k, d_out, r, d, d_w, groups, b);
  else unpermute_backward_kernel<false, false, WPP><<<grid, threads, 0, s>>>(k, d_out, r, d, d_w, groups, b);
  return hipGetLastError();
}

hipError_t launch_unpermute_backward(const PermuteArgs& a, const void* d_out, bool out_f32, const void* rows, bool f32,
                                     void* d_rows, float* d_w, bool zero_tail, hipStream_t s) {
  const KernelArgs k = kernel_args(a, f32);
  const u32x4* r = static_cast<const u32x4*>(rows);
  u32x4* d = static_cast<u32x4*>(d_rows);
  // Four wavefronts a pair for long rows, and for shorter ones while there are few
  // pairs (us, bfloat16 of width W, one / four: 8192 x 8 pairs W = 8192 510 / 433, 4096
  // 235 / 202, 2880 150 / 164; 256 x 8 W = 2880 11.6 / 8.8; 512 x 8 W = 1024 6.7 / 8.9;
  // 128 x 2 W = 7168 11.7 / 5.9).  A launch has fewer than 2^32 threads.
  if (k.P < 1 << 23 && (k.V >= 512 || (k.V > 64 && k.P <= 8 * k.V)))
    return launch_backward_t<4>(k, d_out, out_f32, r, f32, d, d_w, zero_tail, s);
  return launch_backward_t<1>(k, d_out, out_f32, r, f32, d, d_w, zero_tail, s);
}

}  // namespace nvfp4
