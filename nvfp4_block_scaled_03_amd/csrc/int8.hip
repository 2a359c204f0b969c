// Dense int8 layers (int8_linear) for gfx950:
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
// A handful of rows (kFewRows at most): 16 NT columns a workgroup, whose KW wavefronts
// split K.  Both operands come straight from memory into registers, the next
// chunk's while the present one is multiplied; the partial sums meet in LDS and
// leave in whole rows.  Bound: the weights' bytes.  Read once, they pass the caches
// by (34816 x 5120, M = 1: 32.7 -> 30.1 us, 5.9 TB/s).
// ---------------------------------------------------------------------------
constexpr int kFewRows = 16;
template <bool GATED, int NT, int KW>
__global__ __launch_bounds__(KW * 64) void int8_few_kernel(Int8Args p) {
  constexpr int BN = 16 * NT, SW = BN + 4;
  __shared__ __attribute__((aligned(16))) int sh[KW * 16 * SW];
  const int lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  const int kw = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int KC = (int)int8_chunks(p.K), nb = blockIdx.x;
  const int c_lo = KC * kw / KW, c_hi = KC * (kw + 1) / KW;
  const uint8_t* const wq = p.w + ((int64_t)nb * NT * KC * 64 + lane) * 16;
  const int8_t* const aq = p.a + (int64_t)min(ln, p.M - 1) * p.lda;
  struct Chunk {
    i32x4 w[NT], a;
  };
  auto load = [&](int c, Chunk& d) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      d.w[j] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(wq + ((int64_t)j * KC + c) * 1024));
    // (past K the weights are zeros: any 16 bytes of the row will do)
    d.a = *reinterpret_cast<const i32x4*>(aq + min(c * 64 + lg * 16, p.K - 16));
  };
  i32x4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = i32x4{0, 0, 0, 0};
  auto compute = [&](const Chunk& d) {
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(d.a, d.w[j], acc[j], 0, 0, 0);
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
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) sh[(kw * 16 + lg * 4 + r) * SW + 16 * j + ln] = acc[j][r];
  __syncthreads();
  constexpr int OUTC = GATED ? BN / 2 : BN, TOTAL = 16 * (OUTC / 4);
  const int64_t n_out = GATED ? p.N / 2 : p.N;
#pragma unroll 1
  for (int at = threadIdx.x; at < TOTAL; at += KW * 64) {
    const int r = at / (OUTC / 4), c4 = at % (OUTC / 4) * 4;
    const int64_t row[1] = {r}, col = (int64_t)nb * OUTC + c4;
    if (r >= p.M) break;   // (rows ascend)
    if (col >= n_out) continue;
    EpiIn<1> in;
    epi_request<GATED>(p.ep, row[0], col, in);
    const float sx = p.sx[r];
    auto sum = [&](int cc, const float* sw) {
      i32x4 v = *reinterpret_cast<const i32x4*>(sh + r * SW + cc);
#pragma unroll
      for (int k = 1; k < KW; ++k) v += *reinterpret_cast<const i32x4*>(sh + (k * 16 + r) * SW + cc);
      return f32x4{(float)v[0] * (sx * sw[0]), (float)v[1] * (sx * sw[1]), (float)v[2] * (sx * sw[2]),
                   (float)v[3] * (sx * sw[3])};
    };
    const int src = tile_col<GATED>(c4);
    const f32x4 v = sum(src, p.sw + col), up[1] = {GATED ? sum(src + 16, p.sw + p.ep.half + col) : v};
    float z[4] = {v[0], v[1], v[2], v[3]};
    epi_finish<GATED, 1>(p.ep, z, up, in, row, col);
  }
}

template <bool GATED, int NT, int KW>
hipError_t launch_few_t(const Int8Args& p, hipStream_t s) {
  int8_few_kernel<GATED, NT, KW><<<(unsigned)(int8_tiles(p.N, GATED) / NT), KW * 64, 0, s>>>(p);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Tiles of BM = 16 TM WR rows x BN = 16 TN WC columns for many rows: WR x WC
// wavefronts of 16 TM x 16 TN each.  Both operands travel from memory straight
// into a ring of D LDS stages of 128 k.
//
// Activations are taken row-major: eight neighbouring lanes fetch the 128
// bytes of a row, a whole cache line, and a row's eight 16-byte units are
// swizzled by the row, so that the 16 rows of a fragment (one unit each) fall
// into distinct banks.  A stage's weights are whole operands as they lie.
//
// What bounds it: few row blocks, the weights' bytes (34816 x 5120, M = 64 in 64 x
// 256 tiles: 40 us, 4.5 TB/s from 136 CUs).  Many rows, the matrix units' power: 4096
// x 4096 x 17408 in 256 x 256 tiles takes 225 us (2.6 PFLOP/s), 176 us with operands of
// zeros; the loads alone (25-30 B a cycle and CU from L2 into LDS) take 167-175,
// the products alone 160.  A deeper ring, products of 32 x 32 x 32 (more registers
// than there are), 4 wavefronts of 128 x 128, stages begun at different places and
// rows of x padded apart were no faster.
// ---------------------------------------------------------------------------
constexpr int kMaxParts = 4;                          // of K
constexpr int64_t kPartBytes = int64_t(64) << 20;     // their sums, at most

// s_waitcnt immediate: at most n vector memory operations outstanding, and no LDS
// read (the export counter left at its maximum).  The reads are not left to the
// barrier behind: four kernels (128 x 64 and 64 x 256 tiles with K in parts) came out
// of the compiler without its wait for them, so that a wavefront passed the barrier
// with up to four reads of the slot that is refilled next on their way.
constexpr int wait_loads(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

template <bool GATED, bool SPLIT, int WR, int WC, int TM, int TN, int D, int OCC>
__global__ __launch_bounds__(WR * WC * 64) __attribute__((amdgpu_waves_per_eu(WR * WC * OCC / 4, WR * WC * OCC / 4)))
void int8_tile_kernel(Int8Args p, int nb0, int TNB, int S) {
  constexpr int W = WR * WC, BM = 16 * TM * WR, BN = 16 * TN * WC, SW = BN + 4;
  constexpr int LA = BM / 8, LB = BN / 8;          // 1 KiB loads of a stage
  constexpr int PA = LA / W, PB = LB / W;          // of which each wavefront issues
  static_assert(LA % W == 0 && LB % W == 0, "whole loads per wavefront");
  static_assert(D >= 2 && (D - 1) * (PA + PB) <= 63, "ring depth");
  constexpr int STAGE = (LA + LB) * 1024;
  constexpr int PARTS = TM % 2 == 0 ? 2 : TM, PM = TM / PARTS, EPI = BM / PARTS * SW * 4;   // (the epilogue's)
  constexpr int LDS = D * STAGE > EPI ? D * STAGE : EPI;
  static_assert(LDS * OCC <= 160 * 1024, "LDS of the workgroups on a CU");
  __shared__ __attribute__((aligned(16))) uint8_t lds[LDS];
  const int lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), wr = wv / WC, wc = wv % WC;
  const int KC = (int)int8_chunks(p.K), NS = KC / 2, tiles = (int)int8_tiles(p.N, GATED);
  // Workgroups go to the 8 XCDs in turn: the ones of an XCD take neighbours of a
  // list that walks groups of GM row blocks column block by column block.
  constexpr int GM = 8;
  const int TMB = (p.M + BM - 1) / BM, total = TMB * TNB;   // column blocks nb0 .. nb0 + TNB - 1
  const int per_xcd = (total * S + 7) / 8;
  int L = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
  if ((int)(blockIdx.x / 8) >= per_xcd || L >= total * S) return;
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const int part = SPLIT ? uniform(L / total) : 0;   // of the S parts of K
  L -= part * total;
  const int c_lo = SPLIT ? uniform(NS * part / S) : 0, n_st = SPLIT ? uniform(NS * (part + 1) / S) - c_lo : NS;   // stages
  const int grp = L / (GM * TNB), gh = min(GM, TMB - grp * GM), Lg = L - grp * GM * TNB;
  const int mb = uniform(grp * GM + Lg % gh), nb = uniform(nb0 + Lg / gh);

  // Sources: a lane's offset within the block's rows or tiles; a stage adds to
  // the scalar base.  Rows and tiles past the end repeat the last ones (never
  // stored).
  const int8_t* const a0 = p.a + (int64_t)mb * BM * p.lda;
  const uint8_t* const w0 = p.w + (int64_t)nb * (BN / 16) * KC * 1024;
  uint32_t ra[PA], ua[PA], vb[PB];
#pragma unroll
  for (int q = 0; q < PA; ++q) {
    const int r = 8 * (wv * PA + q) + (lane >> 3);
    ra[q] = (uint32_t)(min(r, p.M - 1 - mb * BM) * (int)p.lda);
    ua[q] = (uint32_t)(((lane & 7) ^ ((r >> 1) & 7)) * 16);
  }
#pragma unroll
  for (int q = 0; q < PB; ++q) {
    const int i = wv * PB + q;                     // tile i / 2, chunk i % 2 of the stage
    vb[q] = (uint32_t)((min(i >> 1, tiles - 1 - nb * (BN / 16)) * KC + (i & 1)) * 1024 + lane * 16);
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)lds;
  // Assembly: the compiler would wait for every direct load before any later
  // LDS read.  Completion is awaited explicitly below.
  auto issue = [&](int c, int slot) {
    c = c_lo + min(c, n_st - 1);                   // past the end: the last stage, not used
    const uint32_t base = lds0 + slot * STAGE;
    // (past K the weights are zeros: any bytes of the row will do; a stage begins
    // before K, so the row's last unit lies at or behind that)
    const uint32_t last = (uint32_t)(p.K - 16 - 128 * c);
    const int8_t* const as = a0 + (int64_t)c * 128;
    const uint8_t* const ws = w0 + (int64_t)c * 2048;
#pragma unroll
    for (int q = 0; q < PA; ++q)
      asm volatile(NVFP4_M0_WAIT "global_load_lds_dwordx4 %0, %1" : : "v"(ra[q] + min(ua[q], last)), "s"(as),
                   "{m0}"(base + (wv * PA + q) * 1024) : "memory");
    if (TMB == 1) {   // weights that are read once pass the caches by
#pragma unroll
      for (int q = 0; q < PB; ++q)
        asm volatile(NVFP4_M0_WAIT "global_load_lds_dwordx4 %0, %1 nt" : : "v"(vb[q]), "s"(ws),
                     "{m0}"(base + LA * 1024 + (wv * PB + q) * 1024) : "memory");
    } else {
#pragma unroll
      for (int q = 0; q < PB; ++q)
        asm volatile(NVFP4_M0_WAIT "global_load_lds_dwordx4 %0, %1" : : "v"(vb[q]), "s"(ws),
                     "{m0}"(base + LA * 1024 + (wv * PB + q) * 1024) : "memory");
    }
  };

  i32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  struct Frags {
    i32x4 a[TM], b[TN];
  };
  // Fragments of chunk s of a stage: row 16 i + ln, unit 4 s + lg at its
  // swizzled place; column tile j as it lies.
  const int at_a = wr * TM * 2048 + ln * 128, at_b = LA * 1024 + wc * TN * 2048 + lane * 16, sw = (ln >> 1) & 7;
  auto read = [&](int slot, int s, Frags& f) {
    const uint8_t* const st = lds + slot * STAGE;
#pragma unroll
    for (int j = 0; j < TN; ++j) f.b[j] = *reinterpret_cast<const i32x4*>(st + at_b + j * 2048 + s * 1024);
#pragma unroll
    for (int i = 0; i < TM; ++i) f.a[i] = *reinterpret_cast<const i32x4*>(st + at_a + i * 2048 + ((4 * s + lg) ^ sw) * 16);
  };
  auto multiply = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
  };
  Frags f0, f1;
#pragma unroll
  for (int c = 0; c < D; ++c) issue(c, c);
  __builtin_amdgcn_s_waitcnt(wait_loads((D - 1) * (PA + PB)));
  __syncthreads();
  read(0, 0, f0);
  read(0, 1, f1);
  multiply(f0);
  // Trip c: stage c + 1 has landed and everybody holds what is left of stage c
  // in registers; refill its slot, and read ahead of the products.
  for (int c0 = 0; c0 < n_st - 1; c0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (c0 + d < n_st - 1) {
        __builtin_amdgcn_s_waitcnt(wait_loads((D - 2) * (PA + PB)));
        __syncthreads();
        issue(c0 + d + D, d);
        read((d + 1) % D, 0, f0);
        multiply(f1);
        read((d + 1) % D, 1, f1);
        multiply(f0);
      }
    }
  }
  multiply(f1);
  // (stages past the end may still be in flight)
  __builtin_amdgcn_s_waitcnt(wait_loads(0));

  const int64_t m0 = (int64_t)mb * BM + wr * 16 * TM;
  if constexpr (SPLIT) {
    // The part's sums, in the launch's streaming columns.
    const int64_t NP = min((int64_t)(tiles - nb0 * (BN / 16)) * 16, (int64_t)TNB * BN);
    int* const at = p.part + (int64_t)part * p.M * NP + (int64_t)((nb - nb0) * (BN / 16) + wc * TN) * 16 + ln;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if (nb * (BN / 16) + wc * TN + j >= tiles) break;
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t row = m0 + i * 16 + lg * 4 + r;
          if (row < p.M) at[row * NP + j * 16] = acc[i][j][r];
        }
    }
    return;
  }
  // Part of the rows at a time through LDS, so that they leave, and residuals
  // come, in whole rows.
  float* const sh = reinterpret_cast<float*>(lds);
  float swv[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int64_t r = weight_row(nb * (BN / 16) + wc * TN + j, ln, p.N, GATED);
    swv[j] = r < 0 ? 0.0f : p.sw[r];
  }
#pragma unroll
  for (int h = 0; h < PARTS; ++h) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float sx = p.sx[min(m0 + (h * PM + i) * 16 + lg * 4 + r, (int64_t)p.M - 1)];
#pragma unroll
        for (int j = 0; j < TN; ++j)
          sh[((wr * PM + i) * 16 + lg * 4 + r) * SW + (wc * TN + j) * 16 + ln] = (float)acc[h * PM + i][j][r] * (sx * swv[j]);
      }
    __syncthreads();
    emit_tile<GATED, WR * 16 * PM, BN, W * 64>(
        p.ep, p.M, p.N, nb,
        [&](int r) { return (int64_t)mb * BM + (r / (16 * PM)) * 16 * TM + h * 16 * PM + r % (16 * PM); },
        [&](int at) { return *reinterpret_cast<const f32x4*>(sh + at); });
  }
}

// Adds the S parts of four output columns and finishes them; the parts hold
// the NP streaming columns from col0 on.
template <bool GATED>
__global__ __launch_bounds__(256) void int8_join_kernel(Int8Args p, int S, int64_t col0, int64_t NP) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, quads = (GATED ? NP / 2 : NP) / 4;
  const int64_t row[1] = {i / quads}, c = (i - row[0] * quads) * 4, col = (GATED ? col0 / 2 : col0) + c;
  if (row[0] >= p.M || col >= (GATED ? p.N / 2 : p.N)) return;
  EpiIn<1> in;
  epi_request<GATED>(p.ep, row[0], col, in);
  const float sx = p.sx[row[0]];
  auto sum = [&](int64_t at, const float* sw) {
    i32x4 v = {0, 0, 0, 0};
    for (int k = 0; k < S; ++k) v += *reinterpret_cast<const i32x4*>(p.part + ((int64_t)k * p.M + row[0]) * NP + at);
    return f32x4{(float)v[0] * (sx * sw[0]), (float)v[1] * (sx * sw[1]), (float)v[2] * (sx * sw[2]),
                 (float)v[3] * (sx * sw[3])};
  };
  const int64_t src = GATED ? (c >> 4) * 32 + (c & 15) : c;
  const f32x4 v = sum(src, p.sw + col), up[1] = {GATED ? sum(src + 16, p.sw + p.ep.half + col) : v};
  float z[4] = {v[0], v[1], v[2], v[3]};
  epi_finish<GATED, 1>(p.ep, z, up, in, row, col);
}

// Column blocks nb0 .. nb0 + nbs - 1 of 16 TN WC columns; K in S parts (SPLIT).
template <bool GATED, bool SPLIT, int WR, int WC, int TM, int TN, int D, int OCC>
hipError_t launch_tile_t(const Int8Args& p, int nb0, int nbs, int S, hipStream_t s) {
  S = std::min(S, (int)int8_chunks(p.K) / 2);   // (a stage or more in every part)
  const int64_t rb = (p.M + 16 * TM * WR - 1) / (16 * TM * WR);
  int8_tile_kernel<GATED, SPLIT, WR, WC, TM, TN, D, OCC>
      <<<(unsigned)((rb * nbs * S + 7) / 8 * 8), WR * WC * 64, 0, s>>>(p, nb0, nbs, S);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !SPLIT) return e;
  const int64_t col0 = (int64_t)nb0 * 16 * TN * WC;
  const int64_t NP = std::min(int8_tiles(p.N, GATED) * 16 - col0, (int64_t)nbs * 16 * TN * WC);
  const int64_t quads = p.M * ((GATED ? NP / 2 : NP) / 4);
  int8_join_kernel<GATED><<<(unsigned)((quads + 255) / 256), 256, 0, s>>>(p, S, col0, NP);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// The choice.  A kernel's time, in us, follows the tiles that a CU gets: with
// u = ceil(tiles / 256) of them, `occ` at a time,
//   a + (u / 2) (f2 + b2 stages) + (u % 2) (f1 + b1 stages)     (occ 1: u (f1 + b1 stages))
// with stages of 128 k; a K in S parts divides the stages, multiplies the tiles
// and costs a launch and the sums' way through memory, 2.4 + 4 S M N / 2.2e6.  The
// weights come from memory meanwhile, N K / 6.0e6, 15 % more for every further row
// block that reads them again: the longer of the two, and a fifth of the shorter.
// Fitted to 3600 timings in graphs of 12 weights from 2048 x 512 to 65536 x 8192
// with M = 16 .. 4096; the choice by it is 1 % slower than the best one on average,
// 21 % at most.  E.g. (us, 16 / 32 / 64 / 128 x 64, 256 x 128, 256 x 256): 4096 x
// 4096 M = 32 9.3 / 10.6 / 11.4 / 15.5 / - / -, M = 512 42 / 26.5 / 18.9 / 17.7 /
// 30.5 / 54, M = 4096 - / - / - / 102 / 76 / 65; 128 x 64 or 64 x 64 against 128 x 256
// or 64 x 256: 34816 x 5120 M = 64 44.6 / 40.9, M = 128 59.9 / 48.2, M = 384 92.8 /
// 87.5; K in 1 / 2 / 3 / 4 parts: 5120 x 17408 M = 16 30.2 / 22.3 / 20.6 / 25.8 (16 x
// 64), M = 128 60.6 / 37.5 / 31.0 / 40.1 (128 x 64), and M = 384 62.6 in 256 x 128
// tiles, 45.6 in 128 x 256 with 4 parts.
// ---------------------------------------------------------------------------
struct TileCost {
  int bm, bn, occ;
  float a, f1, b1, f2, b2;
};
constexpr TileCost kTiles[] = {
    {16, 64, 2, 2.7f, 0.65f, 0.165f, 1.45f, 0.247f},  {32, 64, 2, 3.26f, 0.0f, 0.204f, 0.87f, 0.296f},
    {64, 64, 2, 3.5f, 0.25f, 0.233f, 1.21f, 0.398f},  {128, 64, 2, 3.5f, 0.82f, 0.349f, 1.09f, 0.632f},
    {64, 256, 1, 3.5f, 0.80f, 0.615f, 0.0f, 0.0f},    {128, 256, 1, 1.44f, 3.67f, 0.729f, 0.0f, 0.0f},
    {256, 128, 1, 1.0f, 6.79f, 0.697f, 0.0f, 0.0f},   {256, 256, 1, 1.0f, 10.8f, 1.248f, 0.0f, 0.0f},
};
constexpr int kTileKinds = sizeof(kTiles) / sizeof(kTiles[0]);

float tile_cost(const TileCost& t, int64_t M, int64_t columns, int64_t K, int S) {
  const int64_t n = (M + t.bm - 1) / t.bm * ((columns + t.bn - 1) / t.bn) * S, u = (n + 255) / 256;
  const float st = (float)(((K + 127) / 128 + S - 1) / S), n2 = (float)(u / t.occ), n1 = (float)(u % t.occ);
  float c = t.a + (t.occ == 1 ? n2 * (t.f1 + t.b1 * st) : n2 * (t.f2 + t.b2 * st) + n1 * (t.f1 + t.b1 * st));
  if (S > 1) c += 2.4f + 4.0f * S * M * columns / 2.2e6f;
  const float m = (float)columns * K / 6.0e6f * (0.85f + 0.15f * ((M + t.bm - 1) / t.bm));
  return std::max(c, 3.0f + m) + 0.2f * std::min(c, m);
}

// The same for the few-rows kernel, of whose workgroups three run at once on a CU;
// fitted to 95 timings (1 and 16 rows, us, against the best of the tiles': 34816 x
// 5120 33.2, 41.1 / 34.9, 35.9; 5120 x 5120 7.6, 9.4 / 9.3, 10.6; 16384 x 2048 10.2,
// 11.4 / 8.1, 8.3; 16384 x 16384 56.9, 54.4 / 41.0, 41.9).
float few_cost(int64_t M, int64_t columns, int64_t K) {
  const float rounds = std::max(1.0f, (float)columns / (32.0f * 768.0f));
  const float c = 3.5f + rounds * (float)(((K + 127) / 128 * 2 + 7) / 8) * (0.227f + 0.011f * M);
  const float m = (float)columns * K / 5.5e6f;
  return std::max(c, 3.0f + m) + 0.2f * std::min(c, m);
}

struct Choice {
  int kind, parts;
  float cost;
};
// The fastest kind for `columns` streaming columns.
Choice choose(int64_t M, int64_t columns, int64_t K) {
  Choice best = {0, 1, 3.0e38f};
  for (int kind = 0; kind < kTileKinds; ++kind)
    for (int S = 1; S <= kMaxParts; ++S) {
      if (S > 1 && (S > (K + 127) / 128 || (int64_t)S * M * columns * 4 > kPartBytes)) break;
      const float c = tile_cost(kTiles[kind], M, columns, K, S);
      if (c < best.cost) best = {kind, S, c};
    }
  return best;
}

template <bool GATED>
hipError_t launch_kind(const Int8Args& p, int kind, int parts, int64_t col0, int64_t cols, hipStream_t s) {
  const int bn = kTiles[kind].bn, nb0 = (int)(col0 / bn), nbs = (int)((cols + bn - 1) / bn);
  switch (kind) {
    case 0:
      return parts > 1 ? launch_tile_t<GATED, true, 1, 2, 1, 2, 6, 2>(p, nb0, nbs, parts, s)
                       : launch_tile_t<GATED, false, 1, 2, 1, 2, 6, 2>(p, nb0, nbs, 1, s);
    case 1:
      return parts > 1 ? launch_tile_t<GATED, true, 2, 2, 1, 2, 4, 2>(p, nb0, nbs, parts, s)
                       : launch_tile_t<GATED, false, 2, 2, 1, 2, 4, 2>(p, nb0, nbs, 1, s);
    case 2:
      return parts > 1 ? launch_tile_t<GATED, true, 2, 2, 2, 2, 4, 2>(p, nb0, nbs, parts, s)
                       : launch_tile_t<GATED, false, 2, 2, 2, 2, 4, 2>(p, nb0, nbs, 1, s);
    case 3:
      return parts > 1 ? launch_tile_t<GATED, true, 2, 2, 4, 2, 3, 2>(p, nb0, nbs, parts, s)
                       : launch_tile_t<GATED, false, 2, 2, 4, 2, 3, 2>(p, nb0, nbs, 1, s);
    case 4:
      return parts > 1 ? launch_tile_t<GATED, true, 2, 4, 2, 4, 3, 1>(p, nb0, nbs, parts, s)
                       : launch_tile_t<GATED, false, 2, 4, 2, 4, 3, 1>(p, nb0, nbs, 1, s);
    case 5:
      return parts > 1 ? launch_tile_t<GATED, true, 2, 4, 4, 4, 3, 1>(p, nb0, nbs, parts, s)
                       : launch_tile_t<GATED, false, 2, 4, 4, 4, 3, 1>(p, nb0, nbs, 1, s);
    case 6:
      return parts > 1 ? launch_tile_t<GATED, true, 4, 2, 4, 4, 3, 1>(p, nb0, nbs, parts, s)
                       : launch_tile_t<GATED, false, 4, 2, 4, 4, 3, 1>(p, nb0, nbs, 1, s);
    default:
      return parts > 1 ? launch_tile_t<GATED, true, 2, 4, 8, 4, 2, 1>(p, nb0, nbs, parts, s)
                       : launch_tile_t<GATED, false, 2, 4, 8, 4, 2, 1>(p, nb0, nbs, 1, s);
  }
}

template <bool GATED>
hipError_t launch_chosen(const Int8Args& p, hipStream_t s) {
  Int8Step step[2];
  const int n = int8_plan(p.M, p.N, p.K, GATED, step);
  if (step[0].kind < 0) return launch_few_t<GATED, 2, 8>(p, s);
  for (int i = 0; i < n; ++i)
    if (const hipError_t e = launch_kind<GATED>(p, step[i].kind, step[i].parts, step[i].col0, step[i].cols, s);
        e != hipSuccess)
      return e;
  return hipSuccess;
}

}  // namespace

int int8_plan(int64_t M, int64_t N, int64_t K, bool gated, Int8Step (&step)[2]) {
  auto set = [](Int8Step& s, int kind, int parts, int64_t col0, int64_t cols) {
    s = {kind, kind < 0 ? 0 : kTiles[kind].bm, kind < 0 ? 0 : kTiles[kind].bn, parts, col0, cols};
  };
  const int64_t columns = int8_tiles(N, gated) * 16;
  const Choice one = choose(M, columns, K);
  if (M <= kFewRows && few_cost(M, columns, K) < one.cost) {
    set(step[0], -1, 1, 0, columns);
    return 1;
  }
  // Whole rounds of 256 x 256 tiles, and the columns left over by another kernel
  // (4096 x 5120 x 17408: 393 us in 256 x 256 tiles, 347 in 256 x 128, 312 so: 231 for
  // 4096 columns and 81 for 1024, in 256 x 128 tiles with K in two parts).
  const int64_t rb = (M + 255) / 256, cb = (columns + 255) / 256, whole = rb * cb / 256 * 256 / rb;
  if (whole > 0 && whole < cb) {
    const int64_t rest = columns - whole * 256;
    const Choice two = choose(M, rest, K);
    if (tile_cost(kTiles[kTileKinds - 1], M, whole * 256, K, 1) + two.cost < one.cost) {
      set(step[0], kTileKinds - 1, 1, 0, whole * 256);
      set(step[1], two.kind, two.parts, whole * 256, rest);
      return 2;
    }
  }
  set(step[0], one.kind, one.parts, 0, columns);
  return 1;
}

size_t int8_prep_bytes(int64_t N, int64_t K, bool gated) {
  return (size_t)int8_tiles(N, gated) * (size_t)int8_chunks(K) * 1024;
}

hipError_t launch_int8_prep(int64_t N, int64_t K, bool gated, const int8_t* q, uint8_t* prep, hipStream_t s) {
  const int64_t units = (int64_t)(int8_prep_bytes(N, K, gated) / 16);
  int8_prep_kernel<<<(unsigned)((units + 255) / 256), 256, 0, s>>>(N, K, gated, q, reinterpret_cast<u32x4*>(prep),
                                                                  units);
  return hipGetLastError();
}

size_t int8_part_bytes(int64_t M, int64_t N, bool gated) {
  return (size_t)std::min<int64_t>(kMaxParts * M * int8_tiles(N, gated) * 64, kPartBytes);
}

hipError_t launch_int8_linear(const Int8Args& p, hipStream_t s) {
  return p.ep.gated ? launch_chosen<true>(p, s) : launch_chosen<false>(p, s);
}

}  // namespace nvfp4
