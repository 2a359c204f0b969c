// Dense int8 layers (int8_linear, int8_linear_fused) for gfx950:
//   y[m][n] = sx[m] sw[n] sum_k xq[m][k] wq[n][k]   (then the epilogue)
// on the 16x16x64 int8 matrix instruction.  The sums are int32 and exact
// (|sum| <= 2^14 K < 2^31), in whatever order they are made.
//
// Weight streaming layout: [N/16 tiles][K/64 chunks][64 lanes][16 B], lane
// 16 g + n: column n of the tile, k in [16 g, 16 g + 16) of the chunk, so that an
// operand of the instruction is one contiguous 1 KiB load.  Tiles past N and k
// past K hold zeros (the tiles come in fours, the chunks in pairs), so whatever
// the activations' side holds there adds nothing.  A gated layer's tiles alternate
// gate and up.
#include <algorithm>

#include "common.h"
#include "epilogue.h"
#include "int8.h"

namespace nvfp4 {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__host__ __device__ constexpr int64_t int8_chunks(int64_t K) { return (K + 127) / 128 * 2; }
__host__ __device__ constexpr int64_t int8_tiles(int64_t N, bool gated) {
  return gated ? ((N / 2 + 15) / 16 * 2 + 3) / 4 * 4 : ((N + 15) / 16 + 3) / 4 * 4;
}

// Row of W in column n of streaming tile t, or -1.
__device__ __forceinline__ int64_t weight_row(int64_t t, int n, int64_t N, bool gated) {
  if (!gated) {
    const int64_t r = t * 16 + n;
    return r < N ? r : -1;
  }
  const int64_t r = (t >> 1) * 16 + n;
  return r < N / 2 ? r + (t & 1) * (N / 2) : -1;
}

// One 16-byte unit a thread.
__global__ __launch_bounds__(256) void int8_prep_kernel(int64_t N, int64_t K, bool gated, const int8_t* __restrict__ q,
                                                        u32x4* __restrict__ prep, int64_t units) {
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const int lane = (int)(u & 63);
  const int64_t KC = int8_chunks(K), c = (u >> 6) % KC, t = (u >> 6) / KC;
  const int64_t row = weight_row(t, lane & 15, N, gated), k = c * 64 + (lane >> 4) * 16;
  u32x4 v = {0, 0, 0, 0};
  if (row >= 0 && k < K) v = *reinterpret_cast<const u32x4*>(q + row * K + k);
  prep[u] = v;
}

// ---------------------------------------------------------------------------
// 16 MT rows x 16 NT columns a workgroup, whose KW wavefronts split K.  Both
// operands come straight from memory into registers, the next chunk's while the
// present one is multiplied; the partial sums meet in LDS and leave in whole rows.
// ---------------------------------------------------------------------------
template <bool GATED, int MT, int NT, int KW>
__global__ __launch_bounds__(KW * 64) void int8_few_kernel(Int8Args p) {
  constexpr int BM = 16 * MT, BN = 16 * NT, SW = BN + 4;
  __shared__ __attribute__((aligned(16))) int sh[KW * BM * SW];
  const int lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  const int kw = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int KC = (int)int8_chunks(p.K);
  const int64_t tiles = int8_tiles(p.N, GATED);
  // Row blocks are the faster index, eight workgroups apart in launch order,
  // so that those of one column block share an XCD's L2.
  const int rb = (p.M + BM - 1) / BM;
  const int grp = blockIdx.x / (8 * rb), rem = blockIdx.x - grp * 8 * rb, nb = grp * 8 + (rem & 7), mb = rem >> 3;
  if ((int64_t)nb * NT >= tiles) return;
  const int c_lo = KC * kw / KW, c_hi = KC * (kw + 1) / KW;
  const uint8_t* wq = p.w + ((int64_t)nb * NT * KC * 64 + lane) * 16;
  const int8_t* aq[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) aq[i] = p.a + (int64_t)min(mb * BM + 16 * i + ln, p.M - 1) * p.lda;
  struct Chunk {
    i32x4 w[NT], a[MT];
  };
  auto load = [&](int c, Chunk& d) {
#pragma unroll
    for (int j = 0; j < NT; ++j) d.w[j] = *reinterpret_cast<const i32x4*>(wq + ((int64_t)j * KC + c) * 1024);
    // (past K the weights are zeros: any 16 bytes of the row will do)
    const int k = min(c * 64 + lg * 16, p.K - 16);
#pragma unroll
    for (int i = 0; i < MT; ++i) d.a[i] = *reinterpret_cast<const i32x4*>(aq[i] + k);
  };
  i32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto compute = [&](const Chunk& d) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(d.a[i], d.w[j], acc[i][j], 0, 0, 0);
  };
  if (c_lo < c_hi) {
    Chunk d0, d1;   // (past the end: the last chunk, not used)
    load(c_lo, d0);
    load(min(c_lo + 1, c_hi - 1), d1);
    for (int c = c_lo; c < c_hi; c += 2) {
      __builtin_amdgcn_sched_barrier(0);
      compute(d0);
      load(min(c + 2, c_hi - 1), d0);
      __builtin_amdgcn_sched_barrier(0);
      if (c + 1 < c_hi) {
        compute(d1);
        load(min(c + 3, c_hi - 1), d1);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) sh[(kw * BM + i * 16 + lg * 4 + r) * SW + 16 * j + ln] = acc[i][j][r];
  __syncthreads();
  constexpr int OUTC = GATED ? BN / 2 : BN, TOTAL = BM * (OUTC / 4);
  const int64_t n_out = GATED ? p.N / 2 : p.N;
#pragma unroll 1
  for (int at = threadIdx.x; at < TOTAL; at += KW * 64) {
    const int r = at / (OUTC / 4), c4 = at % (OUTC / 4) * 4;
    const int64_t row[1] = {(int64_t)mb * BM + r}, col = (int64_t)nb * OUTC + c4;
    if (row[0] >= p.M) break;   // (rows ascend)
    if (col >= n_out) continue;
    EpiIn<1> in;
    epi_request<GATED>(p.ep, row[0], col, in);
    const float sx = p.sx[row[0]];
    auto sum = [&](int cc, const float* sw) {
      i32x4 v = *reinterpret_cast<const i32x4*>(sh + r * SW + cc);
#pragma unroll
      for (int k = 1; k < KW; ++k) v += *reinterpret_cast<const i32x4*>(sh + (k * BM + r) * SW + cc);
      return f32x4{(float)v[0] * (sx * sw[0]), (float)v[1] * (sx * sw[1]), (float)v[2] * (sx * sw[2]),
                   (float)v[3] * (sx * sw[3])};
    };
    const int src = tile_col<GATED>(c4);
    const f32x4 v = sum(src, p.sw + col), up[1] = {GATED ? sum(src + 16, p.sw + p.ep.half + col) : v};
    float z[4] = {v[0], v[1], v[2], v[3]};
    epi_finish<GATED, 1>(p.ep, z, up, in, row, col);
  }
}

template <bool GATED, int MT, int NT, int KW>
hipError_t launch_few_t(const Int8Args& p, hipStream_t s) {
  const int64_t rb = (p.M + 16 * MT - 1) / (16 * MT), groups = (int8_tiles(p.N, GATED) / NT + 7) / 8;
  int8_few_kernel<GATED, MT, NT, KW><<<(unsigned)(groups * 8 * rb), KW * 64, 0, s>>>(p);
  return hipGetLastError();
}
template <bool GATED>
hipError_t launch_few(const Int8Args& p, hipStream_t s) {
  if (p.M <= 16) return launch_few_t<GATED, 1, 4, 4>(p, s);
  if (p.M <= 32) return launch_few_t<GATED, 2, 4, 4>(p, s);
  return launch_few_t<GATED, 4, 4, 4>(p, s);
}

}  // namespace

size_t int8_prep_bytes(int64_t N, int64_t K, bool gated) {
  return (size_t)int8_tiles(N, gated) * (size_t)int8_chunks(K) * 1024;
}

hipError_t launch_int8_prep(int64_t N, int64_t K, bool gated, const int8_t* q, uint8_t* prep, hipStream_t s) {
  const int64_t units = (int64_t)(int8_prep_bytes(N, K, gated) / 16);
  int8_prep_kernel<<<(unsigned)((units + 255) / 256), 256, 0, s>>>(N, K, gated, q, reinterpret_cast<u32x4*>(prep),
                                                                  units);
  return hipGetLastError();
}

hipError_t launch_int8_linear(const Int8Args& p, hipStream_t s) {
  return p.ep.gated ? launch_few<true>(p, s) : launch_few<false>(p, s);
}

}  // namespace nvfp4
