// Dense NVFP4 linear layers with an epilogue (nvfp4_linear_fused,
// nvfp4_linear_w4a16_fused), for gfx950.
//
// Like the grouped kernels, these decode the weight exactly (code * E4M3 block
// scale has at most six significant bits) and multiply on the 16x16x32 f16
// (W4A4) or bf16 (W4A16) matrix instruction with FP32 accumulation; the
// weight streams from memory straight into registers, one coalesced 16-byte
// load per lane per 16 columns x 128 k.
//
// W4A4 activations, and the bf16 ones of 9 rows and more in linear_few_kernel,
// go through one launch into the operand layout
//   [M/16 row tiles][K/128 chunks][4 steps][64 lanes][16 B]
// (lane 16 g + m of step s: row m of the tile, k in [32 g + 8 s, 32 g + 8 s + 8)
// of the chunk), so that a fragment is one contiguous 1 KiB load.  Row-major
// fragments have neighbouring lanes in different rows, and the address unit
// takes one line a cycle for them, a quarter of the rate.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "epilogue.h"
#include "launch.h"
#include "quant.h"

namespace nvfp4 {
namespace {

constexpr int kBK = 128;   // contraction chunk
// Word 3 of a raw buffer descriptor on gfx9 parts (32-bit data format, no
// swizzle, no index stride).
constexpr int kBufferFlags = 0x00020000;

// ---------------------------------------------------------------------------
// Activations into the operand layout.  A workgroup takes 16 rows x 256 k
// (two chunks; the second may lie past K): each thread one 16-element block,
// turned around in LDS so that reads and writes are both whole lines.  Rows
// past M become zeros.
// ---------------------------------------------------------------------------
// Maxima of |x| over stretches of x (kAmaxParts of them), as float bits.
constexpr int kAmaxParts = 512;

__device__ __forceinline__ uint32_t bf16_abs_max(u32x4 w, uint32_t m) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
    lo = lo > 0x7F80u ? 0u : lo;   // a NaN takes no part in the maximum
    hi = hi > 0x7F80u ? 0u : hi;
    m = max(m, max(lo, hi));
  }
  return m;
}

// Maximum over a workgroup of 256 threads, in every thread.
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* red) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  return max(max(red[0], red[1]), max(red[2], red[3]));
}

__global__ __launch_bounds__(256) void linear_amax_kernel(const uint16_t* __restrict__ x, int64_t n8,
                                                          uint32_t* __restrict__ parts) {
  __shared__ uint32_t red[4];
  uint32_t m = 0;
#pragma unroll 4
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256)
    m = bf16_abs_max(*reinterpret_cast<const u32x4*>(x + i * 8), m);
  m = block_max(m, red);
  if (threadIdx.x == 0) parts[blockIdx.x] = m;
}

// QUANT: NVFP4 quantisation (values code * scale as f16); else bf16 as is.
// Where the maxima come from: parts (n_parts > 0), or x itself, read whole by
// every workgroup (small x: one launch less).
template <bool QUANT>
__global__ __launch_bounds__(256) void linear_operand_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                             const uint32_t* __restrict__ parts, int n_parts,
                                                             float* __restrict__ g, uint16_t* __restrict__ a) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[2 * 4 * kWave * 8];   // [chunk][step][lane][8]
  __shared__ uint32_t red[4];
  const int tid = threadIdx.x, r = tid >> 4, b = tid & 15;
  const int64_t KC = K / kBK;
  const unsigned pairs = (unsigned)((KC + 1) / 2);
  const int64_t rt = blockIdx.x / pairs, kc0 = (int64_t)(blockIdx.x % pairs) * 2, row = rt * 16 + r;
  const int64_t k = kc0 * kBK + b * 16;
  const bool in = row < M && k < K;
  u32x4 w0 = {0, 0, 0, 0}, w1 = {0, 0, 0, 0};
  if (in) {
    w0 = *reinterpret_cast<const u32x4*>(x + row * K + k);
    w1 = *reinterpret_cast<const u32x4*>(x + row * K + k + 8);
  }
  if constexpr (QUANT) {
    uint32_t m = 0;
    if (n_parts > 0) {
      for (int i = tid; i < n_parts; i += 256) m = max(m, parts[i]);
    } else {
      const int64_t n8 = M * K / 8;
#pragma unroll 8
      for (int64_t i = tid; i < n8; i += 256) m = bf16_abs_max(*reinterpret_cast<const u32x4*>(x + i * 8), m);
    }
    const float gv = global_scale_of_amax(bf16_bits_to_f32(block_max(m, red)));
    if (blockIdx.x == 0 && tid == 0) *g = gv;
    float v[16], top = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_bits_to_f32(w0[j] & 0xFFFFu);
      v[2 * j + 1] = bf16_bits_to_f32(w0[j] >> 16);
      v[8 + 2 * j] = bf16_bits_to_f32(w1[j] & 0xFFFFu);
      v[8 + 2 * j + 1] = bf16_bits_to_f32(w1[j] >> 16);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) top = fmaxf(top, amax_input(v[j]));
    const uint32_t sc = e4m3_scale_code(top, gv);
    const float s = e4m3_value(sc);
    const E2M1Bounds bd = e2m1_bounds(s, gv);
    uint32_t c0 = 0, c1 = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c0 |= e2m1_code(v[j], bd, sc == 0) << (4 * j);
      c1 |= e2m1_code(v[8 + j], bd, sc == 0) << (4 * j);
    }
    const f16x2 s2 = f16x2_splat(s);
    w0 = __builtin_bit_cast(u32x4, dequant8_f16(c0, s2));
    w1 = __builtin_bit_cast(u32x4, dequant8_f16(c1, s2));
  }
  // block b: chunk b / 8, lane group (b % 8) / 2, steps 2 (b % 2) and 2 (b % 2) + 1
  const int at = ((b >> 3) * 4 + (b & 1) * 2) * kWave + ((b & 7) >> 1) * 16 + r;
  *reinterpret_cast<u32x4*>(tile + at * 8) = w0;
  *reinterpret_cast<u32x4*>(tile + (at + kWave) * 8) = w1;
  __syncthreads();
  uint16_t* dst = a + (rt * KC + kc0) * (4 * kWave * 8);
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (kc0 + c < KC)
      *reinterpret_cast<u32x4*>(dst + (c * 256 + tid) * 8) = *reinterpret_cast<const u32x4*>(tile + (c * 256 + tid) * 8);
}

// ---------------------------------------------------------------------------
// Product and epilogue.  The output is cut into tiles of BM = 16 MT rows x
// BN = 64 CW columns.  A resident workgroup takes whole tiles as long as there
// is one for every workgroup; the remaining tiles' chunks of K are dealt to
// all workgroups in equal runs (stream), so that no CU waits for another at
// the end.  A run that covers part of a tile leaves FP32 partial sums in the
// workspace, and linear_join_kernel adds those of a tile in the order of K and
// finishes it.  The split depends on the sizes alone: results repeat bit for
// bit.
//
// A workgroup's CW x KW wavefronts: each owns 16 MT rows x 64 columns, and the
// KW groups split the chunks of a run.  The activations of a chunk go into LDS
// once for the group's wavefronts, double buffered: M = 64, N = 34816, K = 5120
// moves 190 MB from L2 to the CUs, 435 MB with each wavefront loading its own
// fragments, 64 rows x 64 columns.  The weights of the chunk after next are
// requested as soon as the registers of the present one are read.  Measured,
// whole layers: W4A4 34816 x 5120 M = 64 48 us, of which the activations take 9
// (maximum, quantisation), the product 34 and the join 6; M = 128 67 us (680
// TFLOP/s); W4A16 5120 x 17408 M = 512 113 us (807 TFLOP/s).  What bounds it at M = 64:
// the weight stream (21 us alone) and the matrix work (16 us) run in good part
// one after the other, for the epilogue's LDS leaves room for one workgroup a CU.
// ---------------------------------------------------------------------------
constexpr int kNT = 4;        // column tiles of a wavefront: 64 columns
constexpr int kCUs = 256;
// Dealing out chunks pays where it takes more than kJoinChunks chunks (of 0.3
// to 0.5 us) off the longest path: the join is a launch and a round trip of the
// partial sums, about 5 us.  Measured (us, whole tiles / dealt out, W4A16 and
// W4A4): 9 chunks off (34816 x 2560 M = 64) 30.5 / 33.8, 32.2 / 38.6; 14 (34816 x
// 3840) 40.7 / 39.9, 40.2 / 43.0; 16 (8192 x 8192 M = 330) 73 / 69, 68 / 67; 18
// (34816 x 5120 M = 64) 51 / 46, 48.5 / 48.3; 32 (8192 x 8192 M = 200) 72 / 47,
// 67 / 49.  Where the tiles are fewer than the CUs, a run is kMinRun chunks or
// more, so that its start (the first loads' way from memory) stays the smaller
// part: runs of 4 / 8 / 16, W4A16, 2560 x 4096 M = 200 27.1 / 22.6 / 27.8, 1280 x
// 17408 M = 100 29.3 / 25.2 / 31.5, 640 x 16384 M = 64 22.3 / 21.6 / 26.4.  The few
// tiles left over from whole rounds are dealt to all workgroups all the same,
// down to runs of one chunk: 32896 x 4096 M = 100 (258 tiles) 61 us, 80 in whole
// tiles.
constexpr int kJoinChunks = 16, kMinRun = 8;

// How a layer is cut up, from its sizes.
struct TileSplit {
  int cfg;           // launch_tile's case
  int bm, bn;
  int row_blocks, col_blocks;
  int grid;          // workgroups
  int rounds;        // whole tiles of each workgroup
  int stream;        // tiles whose chunks are dealt out (the last ones)
  int run, extra;    // chunks of a run; the first `extra` runs have one more
};

struct TileParams {
  int M, N, K;
  TileSplit t;
  const uint16_t* a;     // f16 in the operand layout (W4A4), or bf16 [M][K]
  const uint8_t* w_q;    // streaming layout
  const uint8_t* w_sf;
  const float* g_w;
  const float* g_a;      // W4A4, or null
  float* part;           // partial sums: [2 grid][BM][BN], products times alpha
  LinearEpi ep;
};

// First chunk (over the streamed tiles, in order) of workgroup b's run.
__device__ __forceinline__ int stream_start(const TileSplit& t, int b) { return b * t.run + min(b, t.extra); }

// Sends a tile out of LDS: sh holds SUMS copies of [BM][BN + 4], added in
// order.  Whole tiles are finished, parts of one go to the workspace.
template <bool GATED, int BM, int BN, int SUMS, int THREADS>
__device__ __forceinline__ void emit_rows(const TileParams& p, const float* sh, float alpha, float* part, int mb,
                                          int nb) {
  constexpr int SW = BN + 4;
  auto sum = [&](int at) {
    f32x4 v = *reinterpret_cast<const f32x4*>(sh + at);
#pragma unroll
    for (int k = 1; k < SUMS; ++k) v += *reinterpret_cast<const f32x4*>(sh + k * BM * SW + at);
    return alpha * v;
  };
  const int64_t row0 = (int64_t)mb * BM;
  if (part) {
#pragma unroll 4
    for (int at = threadIdx.x; at < BM * (BN / 4); at += THREADS) {
      const int r = at / (BN / 4), c4 = at % (BN / 4) * 4;
      if (row0 + r < p.M) *reinterpret_cast<f32x4*>(part + (int64_t)r * BN + c4) = sum(r * SW + c4);
    }
    return;
  }
  emit_tile<GATED, BM, BN, THREADS>(p.ep, p.M, p.N, nb, [&](int r) { return row0 + r; }, sum);
}

// A workgroup's work: whole tiles, then its run over the streamed tiles.
struct TileWork {
  int b, u, u_end, round = 0, seg = 0;
  int mb, nb, lo = 0, hi = 1 << 30;   // the present piece: tile and chunks
  __device__ __forceinline__ explicit TileWork(const TileSplit& t) {
    // Workgroups go to the 8 XCDs in turn: position b of the work order, in
    // which neighbours share weight columns, runs on one XCD with its
    // neighbours.
    const int q8 = t.grid >> 3, r8 = t.grid & 7, xcd = blockIdx.x & 7;
    b = xcd * q8 + min(xcd, r8) + (int)(blockIdx.x >> 3);
    u = stream_start(t, b);
    u_end = stream_start(t, b + 1);
  }
  __device__ __forceinline__ bool next(const TileSplit& t, int KC) {
    int tile;
    if (round < t.rounds) {
      tile = round * t.grid + b;
      lo = 0;
      hi = KC;
      ++round;
    } else {
      if (u >= u_end) return false;
      seg += hi - lo < KC;     // (the piece before was part of a tile)
      const int st = u / KC;
      tile = t.rounds * t.grid + st;
      lo = u - st * KC;
      hi = min(KC, lo + (u_end - u));
      u += hi - lo;
    }
    nb = tile / t.row_blocks;
    mb = tile - nb * t.row_blocks;
    return true;
  }
  // Where the piece's partial sums go, or null for a whole tile.
  __device__ __forceinline__ float* part(const TileParams& p, int KC) const {
    if (hi - lo == KC) return nullptr;
    return p.part + (int64_t)(2 * b + seg) * p.t.bm * p.t.bn;
  }
};

// The product of one piece after the other.  Weights are requested D chunks
// ahead of their use into registers, activations two chunks ahead into
// registers and from there, a chunk ahead, into LDS (loads complete in order:
// activations requested later than the weights would wait for those).  Trip t
// of a group, between two barriers: request chunk t + 2's activations,
// multiply chunk t from LDS buffer t & 1, request chunk t + D's weights into
// the registers just read, put chunk t + 1's activations into the other
// buffer.  The next piece's first requests precede the end of the present one.
//
// W4A4 activations come in the operand layout, which quantising writes anyway.
// bf16 rows are taken as they are, four rows' 256 bytes of a chunk a load, and
// turned around by the LDS writes: the 16-byte unit u = 4 g + s of row m goes to
// place m ^ u of step s, lane group g, so that neither the writes (16 units of a
// row) nor the fragment reads (16 rows of a unit) meet in a bank.  Against a
// launch that makes the operand layout: 203 x 4096 x 1024 14.2 -> 12.3 us, 512 x 5120 x 17408 118 -> 112 us.
template <bool BF16, bool GATED, int MT, int CW, int KW>
__global__ __launch_bounds__(CW * KW * kWave) __attribute__((amdgpu_waves_per_eu(CW * KW / 4, CW * KW / 4)))
void linear_tile_kernel(TileParams p) {
  constexpr int THREADS = CW * KW * kWave;
  constexpr int D = 2;   // (3: 1 to 2 us slower, for the registers)
  constexpr int BM = 16 * MT, BN = 64 * CW, SW = BN + 4;
  constexpr int STAGE = MT * 4096;                 // activations of a chunk
  constexpr int LPW = MT * 4 / CW;                      // of which each wavefront moves LPW KiB
  static_assert(MT * 4 % CW == 0, "whole loads per wavefront");
  constexpr int RING = KW * 2 * STAGE, EPI = KW * BM * SW * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[RING > EPI ? RING : EPI];
  const int tid = threadIdx.x, lane = tid & 63, ln = lane & 15, lg = lane >> 4, l16 = lane * 16;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kw = wv / CW, wc = wv % CW;
  const int KC = p.K / kBK, row_tiles = (p.M + 15) >> 4, col_tiles = p.N / 16, GS = scale_group(KC);
  const float alpha = p.g_a ? ld_uniform(p.g_a) * ld_uniform(p.g_w) : ld_uniform(p.g_w);
  uint8_t* const ring = lds + kw * 2 * STAGE;

  struct W {
    u32x4 q[kNT];
    uint32_t s[kNT / 2];
  };
  struct A {
    u32x4 v[LPW];
  };
  // The lane's constant offsets within a tile's weights (which span less than
  // 2^31 bytes); a chunk adds a scalar offset.
  int vw[kNT], vs[kNT / 2];
#pragma unroll
  for (int j = 0; j < kNT; ++j) vw[j] = l16 + j * KC * 1024;
#pragma unroll
  for (int j = 0; j < kNT / 2; ++j) vs[j] = lane * GS * 4 + j * KC * 256;

  // A piece's operands and the group's chunks of it; groups run in step, the
  // shorter ones idle.
  struct Piece {
    __amdgpu_buffer_rsrc_t w, s, a;
    int va[LPW];        // one step of one row tile; row tiles past the end repeat the last one
    int c_lo, mine, trips, last;
  };
  auto piece_of = [&](const TileWork& k) {
    Piece P;
    const int len = k.hi - k.lo;
    // Column tiles past N repeat the last ones (loaded, never stored).
    const int nt0 = min(k.nb * (BN / 16) + wc * kNT, col_tiles - kNT);
    P.c_lo = k.lo + len * kw / KW;
    P.mine = k.lo + len * (kw + 1) / KW - P.c_lo;
    P.trips = (len + KW - 1) / KW;
    P.last = max(P.mine, 1) - 1;
    P.w = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w_q + (int64_t)nt0 * KC * 1024), (short)0, 0x7FFFFFFF,
                                            kBufferFlags);
    P.s = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w_sf + (int64_t)(nt0 >> 1) * KC * 256), (short)0, 0x7FFFFFFF,
                                            kBufferFlags);
    // (16 MT rows of either form are MT KC 2048 values)
    P.a = __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + (int64_t)k.mb * MT * KC * 2048), (short)0, 0x7FFFFFFF,
                                            kBufferFlags);
#pragma unroll
    for (int q = 0; q < LPW; ++q) {
      const int at = wc * LPW + q;
      if constexpr (BF16) P.va[q] = min(4 * at + lg, p.M - 1 - k.mb * BM) * KC * 256 + ln * 16;
      else P.va[q] = l16 + min(at / 4, row_tiles - 1 - k.mb * MT) * KC * 4096 + at % 4 * 1024;
    }
    return P;
  };
  // (trips past the end repeat the last chunk: loaded, not used)
  auto load_w = [&](const Piece& P, int t, W& d) {
    const int c = P.c_lo + min(t, P.last);
#pragma unroll
    for (int j = 0; j < kNT; ++j)
      d.q[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(P.w, vw[j], c * 1024, 0));
    const int cg = c / GS, cs = cg * GS * 256 + (c - cg * GS) * 4;
#pragma unroll
    for (int j = 0; j < kNT / 2; ++j) d.s[j] = __builtin_amdgcn_raw_buffer_load_b32(P.s, vs[j], cs, 0);
  };
  auto load_a = [&](const Piece& P, int t, A& d) {
    const int c = P.c_lo + min(t, P.last);
#pragma unroll
    for (int q = 0; q < LPW; ++q)
      d.v[q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(P.a, P.va[q], c * (BF16 ? 256 : 4096), 0));
  };
  auto put_a = [&](int buf, const A& d) {
#pragma unroll
    for (int q = 0; q < LPW; ++q) {
      const int at = wc * LPW + q;   // bf16: rows 4 at + lg, unit ln
      const int to = BF16 ? at / 4 * 4096 + (ln & 3) * 1024 + (ln >> 2) * 256 + ((at % 4 * 4 + lg) ^ ln) * 16
                          : at * 1024 + l16;
      *reinterpret_cast<u32x4*>(ring + buf * STAGE + to) = d.v[q];
    }
  };
  W w[D];
  A a[2];
  auto first_loads = [&](const Piece& P) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (d < 2) load_a(P, d, a[d]);
      load_w(P, d, w[d]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  TileWork work(p.t);
  if (!work.next(p.t, KC)) return;
  Piece P = piece_of(work);
  first_loads(P);
  while (true) {
    f32x4 acc[MT][kNT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < kNT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    // A decoded fragment's matrix instructions are interleaved with the decode
    // of the next: it issues while the matrix unit is busy.
    typedef typename std::conditional<BF16, bf16x8, f16x8>::type frag;
    constexpr int VALU = BF16 ? 16 : 8;                 // instructions of a decode
    auto compute = [&](int buf, const W& w) {
      const uint8_t* st = ring + buf * STAGE;
      f16x2 scale[kNT];
#pragma unroll
      for (int j = 0; j < kNT; ++j) scale[j] = e4m3x2_to_f16x2(w.s[j >> 1] >> ((j & 1) * 16));
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        frag af[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) af[i] = *reinterpret_cast<const frag*>(st + i * 4096 + s * 1024 + (BF16 ? lg * 256 + ((ln ^ (4 * lg)) ^ s) * 16 : l16));
        __builtin_amdgcn_sched_barrier(0);
        frag bf[kNT];
#pragma unroll
        for (int j = 0; j < kNT; ++j) {
          const f16x2 sj = s < 2 ? f16x2_lo(scale[j]) : f16x2_hi(scale[j]);
          if constexpr (BF16) bf[j] = dequant8_bf16(w.q[j][s], (float)sj[0]);
          else bf[j] = dequant8_f16(w.q[j][s], sj);
        }
#pragma unroll
        for (int j = 0; j < kNT; ++j)
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            if constexpr (BF16) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[i], bf[j], acc[i][j], 0, 0, 0);
            else acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(af[i], bf[j], acc[i][j], 0, 0, 0);
          }
        __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
#pragma unroll
        for (int j = 0; j + 1 < kNT; ++j)
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, (VALU + MT - 1) / MT, 0);
          }
        __builtin_amdgcn_sched_group_barrier(0x008, MT, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    put_a(0, a[0]);
    // (unrolled so that register sets and LDS buffers have constant indices)
    static_assert(D == 2, "a period of two trips");
    for (int t0 = 0; t0 < P.trips; t0 += 2) {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const int t = t0 + d;
        if (t < P.trips) {
          // (LDS only: the requests in flight are not waited for)
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
          load_a(P, t + 2, a[d & 1]);
          __builtin_amdgcn_sched_barrier(0);
          if (t < P.mine) compute(d & 1, w[d % D]);
          load_w(P, t + D, w[d % D]);
          __builtin_amdgcn_sched_barrier(0);
          put_a((d + 1) & 1, a[(d + 1) & 1]);
        }
      }
    }
    const TileWork done = work;
    const bool more = work.next(p.t, KC);
    if (more) {
      P = piece_of(work);
      first_loads(P);
    }

    __syncthreads();                                    // the ring is read
    float* const sh = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < kNT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          sh[(kw * BM + i * 16 + lg * 4 + r) * SW + wc * 64 + j * 16 + ln] = acc[i][j][r];
    __syncthreads();
    emit_rows<GATED, BM, BN, KW, THREADS>(p, sh, alpha, done.part(p, KC), done.mb, done.nb);
    if (!more) break;
    __syncthreads();                                    // LDS is free for the next piece
  }
}

// Adds the partial sums of the streamed tiles and finishes them, four output
// columns a thread: a workgroup per 8 rows of a tile.
constexpr int kJoinRows = 8;
template <bool GATED>
__global__ __launch_bounds__(256) void linear_join_kernel(TileParams p) {
  const int BM = p.t.bm, BN = p.t.bn, per_tile = BM / kJoinRows;
  const int st = blockIdx.x / per_tile, r0 = (blockIdx.x % per_tile) * kJoinRows;
  const int KC = p.K / kBK, tile = p.t.rounds * p.t.grid + st;
  const int nb = tile / p.t.row_blocks, mb = tile - nb * p.t.row_blocks;
  if (mb * BM + r0 >= p.M) return;
  // Runs b0 .. b1 hold the tile's chunks [first, last].
  const int first = st * KC, last = first + KC - 1;
  auto run_of = [&](int c) {
    const int head = p.t.extra * (p.t.run + 1);
    return c < head ? c / (p.t.run + 1) : p.t.extra + (c - head) / p.t.run;
  };
  const int b0 = run_of(first), b1 = run_of(last);
  if (b0 == b1) return;                                 // one run: finished there
  const int outc = GATED ? BN / 2 : BN;
  const int64_t cols = GATED ? p.N / 2 : p.N;
  for (int at = threadIdx.x; at < kJoinRows * (outc / 4); at += 256) {
    const int r = r0 + at / (outc / 4), c4 = at % (outc / 4) * 4;
    const int64_t row = (int64_t)mb * BM + r, col = (int64_t)nb * outc + c4;
    if (row >= p.M || col >= cols) continue;
    EpiIn<1> in;
    epi_request<GATED>(p.ep, row, col, in);
    const float* src = p.part + (int64_t)r * BN + tile_col<GATED>(c4);
    f32x4 v = {0.f, 0.f, 0.f, 0.f}, up[1] = {v};
    auto slot = [&](int b) {
      // the run's second part, if it starts in an earlier tile
      return src + (int64_t)(2 * b + (stream_start(p.t, b) < first)) * BM * BN;
    };
#pragma unroll 4
    for (int b = b0; b <= b1; ++b) {
      const float* s = slot(b);
      v += *reinterpret_cast<const f32x4*>(s);
      if constexpr (GATED) up[0] += *reinterpret_cast<const f32x4*>(s + 16);
    }
    float z[4] = {v[0], v[1], v[2], v[3]};
    epi_finish<GATED, 1>(p.ep, z, up, in, {row}, col);
  }
}

// Cases of launch_tile: row tiles, wavefronts over columns and over K.
struct TileCfg {
  int mt, cw, kw;
};
constexpr TileCfg kTileCfgs[] = {{3, 2, 4}, {4, 2, 4}, {3, 4, 2}, {4, 4, 2}};

TileSplit tile_split_as(int cfg, int64_t M, int64_t N, int64_t K) {
  const TileCfg c = kTileCfgs[cfg];
  TileSplit t{};
  t.cfg = cfg;
  t.bm = 16 * c.mt;
  t.bn = 64 * c.cw;
  const int KC = (int)(K / kBK), slots = kCUs;   // one workgroup per CU
  t.row_blocks = (int)((M + t.bm - 1) / t.bm);
  t.col_blocks = (int)((N + t.bn - 1) / t.bn);
  const int64_t tiles = (int64_t)t.row_blocks * t.col_blocks;
  // Chunks on the longest path, with whole tiles only and dealt out evenly.
  const int64_t whole = (tiles + slots - 1) / slots * KC, even = (tiles * KC + slots - 1) / slots;
  if (whole - even > kJoinChunks) {
    t.grid = (int)std::min<int64_t>(slots, std::max<int64_t>(1, tiles * KC / kMinRun));
    t.rounds = (int)(tiles / t.grid);
    t.stream = (int)(tiles % t.grid);
  } else {
    t.grid = (int)tiles;
    t.rounds = 1;
  }
  t.run = t.stream * KC / t.grid;
  t.extra = t.stream * KC % t.grid;
  return t;
}

// Row blocks of even height; 128 columns a workgroup where the tiles are few
// and short, else 256.  Measured (us, the whole layer, W4A16 and W4A4, 128 / 256
// columns): 4096 x 1024 M = 256 13.5 / 17.2, 19.2 / 22.5; 8192 x 512 M = 256 12.0 /
// 13.8, 17.7 / 19.8; longer or more of them: 8192 x 8192 M = 128 36.3 / 34.5, 38.6 /
// 38.3; 34816 x 5120 M = 64 53.8 / 46.5, 53.1 / 49.3.
TileSplit tile_split(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = (M + 15) / 16, blocks = (tiles + 3) / 4;
  const bool low = (tiles + blocks - 1) / blocks <= 3;
  const bool narrow = K <= 2048 && blocks * (N / 128) <= kCUs;
  return tile_split_as((narrow ? 0 : 2) + (low ? 0 : 1), M, N, K);
}

template <bool BF16, bool GATED, int CFG>
hipError_t launch_tile(const TileParams& p, hipStream_t s) {
  constexpr TileCfg c = kTileCfgs[CFG];
  constexpr int waves = c.cw * c.kw;
  linear_tile_kernel<BF16, GATED, c.mt, c.cw, c.kw>
      <<<(unsigned)p.t.grid, waves * kWave, 0, s>>>(p);
  if (p.t.stream > 0)
    linear_join_kernel<GATED><<<(unsigned)(p.t.stream * (p.t.bm / kJoinRows)), 256, 0, s>>>(p);
  return hipGetLastError();
}

template <bool BF16, bool GATED>
hipError_t launch_tiles(const TileParams& p, hipStream_t s) {
  switch (p.t.cfg) {
    case 0: return launch_tile<BF16, GATED, 0>(p, s);
    case 1: return launch_tile<BF16, GATED, 1>(p, s);
    case 2: return launch_tile<BF16, GATED, 2>(p, s);
    default: return launch_tile<BF16, GATED, 3>(p, s);
  }
}

// ---------------------------------------------------------------------------
// Few rows: the weight stream decides, so the grid is wide (16 NT columns a
// workgroup) and the KW wavefronts of a workgroup split K.  The next chunk's
// operands are in flight while the present one is multiplied; the partial sums
// meet in LDS and leave in rows.  Activations (ACT): bf16 rows as they are, for
// a handful of rows (more rows would put neighbouring lanes in different
// lines); codes and scales, likewise; or 16-bit values in the operand layout,
// MT row tiles.  Measured: one row of W4A16 34816 x 5120, 100 MB of weight,
// 25.6 us (3.9 TB/s); 65536 x 8192, 302 MB, 56 us (5.4 TB/s).
//
// W4A4 quantises to codes in one launch, each workgroup taking the maximum over
// all of x, up to kFewQuantMax elements: 5120 x 17408 M = 4 24.4 us against
// 27.2 with the maximum in a launch of its own and the operand layout, M = 8
// 28.7 against 27.5, 8192 x 8192 M = 16 23.5 against 20.5.  W4A16 reads x as it
// is up to kFewRowsMax rows: M = 16 34816 x 5120 38.0 us against 33.5 with the
// operand layout, 5120 x 17408 28.8 against 23.9 (4096 x 1024 6.2 against 6.7).
// ---------------------------------------------------------------------------
constexpr int64_t kFewQuantMax = 98304, kFewRowsMax = 8;
enum FewAct { kFewBf16Rows = 0, kFewCodes = 1, kFewBf16Operand = 2, kFewF16Operand = 3 };
struct FewParams {
  int M, N, K;
  const uint16_t* x;     // bf16 [M][K], or the operand layout, or
  const uint8_t* a_q;    // codes [M][K/2] and
  const uint8_t* a_sf;   // scales [M][K/16]
  const uint8_t* w_q;    // streaming layout
  const uint8_t* w_sf;
  const float* g_w;
  const float* g_a;      // W4A4, or null
  LinearEpi ep;
};

template <int ACT, bool GATED, int MT, int NT, int KW>
__global__ __launch_bounds__(KW * kWave) void linear_few_kernel(FewParams p) {
  constexpr bool BF16 = ACT == kFewBf16Rows || ACT == kFewBf16Operand, CODES = ACT == kFewCodes;
  constexpr bool OPERAND = ACT >= kFewBf16Operand;
  constexpr int BM = 16 * MT, BN = 16 * NT, SW = BN + 4, AW = CODES ? 1 : 4;
  static_assert(OPERAND || MT == 1, "row tiles come in the operand layout");
  // Weights that one workgroup reads pass the caches by where nothing else
  // contends for them: with the operand layout only in the widest layers
  // (W4A4 8192 x 8192 M = 1 15.5 -> 14.4 us; 5120 x 17408 M = 8, operand
  // layout, 27.6 -> 29.1).
  constexpr bool ONCE = !OPERAND || (NT == 4 && KW == 2);
  __shared__ __attribute__((aligned(16))) float sh[KW * BM * SW];
  const int lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
  const int kw = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  // Row blocks are the faster index, eight workgroups apart in launch order,
  // so that those of one column block share an XCD's L2.
  const int rb = OPERAND ? (p.M + BM - 1) / BM : 1;
  const int grp = blockIdx.x / (8 * rb), rem = blockIdx.x - grp * 8 * rb, nb = grp * 8 + (rem & 7), mb = rem >> 3;
  if (nb * BN >= p.N) return;
  const int KC = p.K / kBK, nt0 = nb * NT, GS = scale_group(KC);
  const int c_lo = KC * kw / KW, c_hi = KC * (kw + 1) / KW;
  const float alpha = p.g_a ? ld_uniform(p.g_a) * ld_uniform(p.g_w) : ld_uniform(p.g_w);
  const int64_t row = min(ln, p.M - 1);   // rows past M repeat the last one (never stored)
  const int last_tile = (p.M - 1) >> 4;   // and row tiles past the last one, that
  const uint8_t* wq = p.w_q + ((int64_t)nt0 * KC * kWave + lane) * 16;
  const uint8_t* ws = p.w_sf + (int64_t)(nt0 >> 1) * KC * 256 + lane * GS * 4;
  const uint8_t* ax = CODES     ? p.a_q + row * (p.K / 2) + lg * 16
                      : OPERAND ? reinterpret_cast<const uint8_t*>(p.x) + lane * 16
                                : reinterpret_cast<const uint8_t*>(p.x + row * p.K) + lg * 64;
  const uint8_t* as = CODES ? p.a_sf + row * (p.K / 16) + lg * 2 : nullptr;
  struct Chunk {
    u32x4 w[NT], a[MT][AW];
    uint32_t s[NT / 2], sa;
  };
  auto load = [&](int c, Chunk& d) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const u32x4* at = reinterpret_cast<const u32x4*>(wq + ((int64_t)j * KC + c) * 1024);
      if constexpr (ONCE) d.w[j] = __builtin_nontemporal_load(at);
      else d.w[j] = *at;
    }
    const int cg = c / GS;
#pragma unroll
    for (int j = 0; j < NT / 2; ++j)
      d.s[j] = *reinterpret_cast<const uint32_t*>(ws + (int64_t)j * KC * 256 + cg * GS * 256 + (c - cg * GS) * 4);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int v = 0; v < AW; ++v)
        d.a[i][v] = *reinterpret_cast<const u32x4*>(
            ax + (OPERAND ? ((int64_t)min(mb * MT + i, last_tile) * KC + c) * 4096 + v * 1024 : (int64_t)c * (CODES ? 64 : 256) + v * 16));
    if constexpr (CODES) d.sa = *reinterpret_cast<const uint16_t*>(as + (int64_t)c * 8);
  };
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Chunk& d) {
    f16x2 scale[NT], sa = {};
#pragma unroll
    for (int j = 0; j < NT; ++j) scale[j] = e4m3x2_to_f16x2(d.s[j >> 1] >> ((j & 1) * 16));
    if constexpr (CODES) sa = e4m3x2_to_f16x2(d.sa);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (BF16) {
          const bf16x8 b = dequant8_bf16(d.w[j][s], (float)scale[j][s >> 1]);
#pragma unroll
          for (int i = 0; i < MT; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, d.a[i][s]), b, acc[i][j],
                                                                0, 0, 0);
        } else {
          const f16x8 b = dequant8_f16(d.w[j][s], s < 2 ? f16x2_lo(scale[j]) : f16x2_hi(scale[j]));
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            f16x8 a;
            if constexpr (CODES) a = dequant8_f16(d.a[i][0][s], s < 2 ? f16x2_lo(sa) : f16x2_hi(sa));
            else a = __builtin_bit_cast(f16x8, d.a[i][s]);
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, acc[i][j], 0, 0, 0);
          }
        }
      }
  };
  // The thread's first four output columns: what the epilogue reads for them
  // is requested behind the first chunk.
  constexpr int OUTC = GATED ? BN / 2 : BN, TOTAL = BM * (OUTC / 4);
  EpiIn<1> in;
  int64_t row_out[1] = {(int64_t)mb * BM + threadIdx.x / (OUTC / 4)};
  int64_t col_out = (int64_t)nb * OUTC + threadIdx.x % (OUTC / 4) * 4;
  const bool on = (int)threadIdx.x < TOTAL && row_out[0] < p.M;
  if (c_lo < c_hi) {
    Chunk d0, d1;   // (past the end: the last chunk, not used)
    load(c_lo, d0);
    if (on) epi_request<GATED>(p.ep, row_out[0], col_out, in);
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
  } else if (on) {
    epi_request<GATED>(p.ep, row_out[0], col_out, in);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) sh[(kw * BM + i * 16 + lg * 4 + r) * SW + 16 * j + ln] = acc[i][j][r];
  __syncthreads();
#pragma unroll 1
  for (int at = threadIdx.x; at < TOTAL; at += KW * kWave) {
    const int r = at / (OUTC / 4), c4 = at % (OUTC / 4) * 4;
    row_out[0] = (int64_t)mb * BM + r;
    col_out = (int64_t)nb * OUTC + c4;
    if (row_out[0] >= p.M) break;   // (rows ascend)
    if (at != (int)threadIdx.x) epi_request<GATED>(p.ep, row_out[0], col_out, in);
    auto sum = [&](int col) {
      f32x4 v = *reinterpret_cast<const f32x4*>(sh + r * SW + col);
#pragma unroll
      for (int k = 1; k < KW; ++k) v += *reinterpret_cast<const f32x4*>(sh + (k * BM + r) * SW + col);
      return alpha * v;
    };
    const int src = tile_col<GATED>(c4);
    const f32x4 v = sum(src), up[1] = {GATED ? sum(src + 16) : v};
    float z[4] = {v[0], v[1], v[2], v[3]};
    epi_finish<GATED, 1>(p.ep, z, up, in, row_out, col_out);
  }
}

// Activations of a few rows as codes: the global scale is taken by every
// workgroup from all of x (at most 16 rows and kFewQuantMax elements), so that
// quantising is one launch.
__global__ __launch_bounds__(256) void linear_few_quant_kernel(const uint16_t* __restrict__ x, int64_t M, int64_t K,
                                                               float* __restrict__ g, uint8_t* __restrict__ q,
                                                               uint8_t* __restrict__ sf) {
  __shared__ uint32_t red[4];
  const int64_t n8 = M * K / 8;
  uint32_t m = 0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < n8; i += 256) m = bf16_abs_max(*reinterpret_cast<const u32x4*>(x + i * 8), m);
  const float gv = global_scale_of_amax(bf16_bits_to_f32(block_max(m, red)));
  if (blockIdx.x == 0 && threadIdx.x == 0) *g = gv;
  const int64_t hb = (int64_t)blockIdx.x * 256 + threadIdx.x;   // half blocks: the two of a block are neighbours
  if (hb >= n8) return;
  float v[8];
  load8(x, hb * 8, v);
  const int64_t per = K / 8, row = hb / per;
  quantize_half_block_values(v, row, (hb - row * per) * 8, K, gv, q, sf, nullptr);
}

// x in the operand layout (a), and for W4A4 its global scale (g); parts:
// kAmaxParts words.
hipError_t launch_operand(const uint16_t* x, int64_t M, int64_t K, bool quant, uint32_t* parts, float* g, uint16_t* a,
                          hipStream_t s) {
  const unsigned grid = (unsigned)((K / kBK + 1) / 2 * ((M + 15) / 16));
  if (!quant) {
    linear_operand_kernel<false><<<grid, 256, 0, s>>>(x, M, K, nullptr, 0, nullptr, a);
    return hipGetLastError();
  }
  const int64_t n8 = M * K / 8;
  int n_parts = 0;
  if (n8 > (1 << 13)) {   // (more than a workgroup reads while a launch would start)
    n_parts = (int)std::min<int64_t>(kAmaxParts, (n8 + 255) / 256);
    linear_amax_kernel<<<(unsigned)n_parts, 256, 0, s>>>(x, n8, parts);
    if (hipError_t e = hipGetLastError()) return e;
  }
  linear_operand_kernel<true><<<grid, 256, 0, s>>>(x, M, K, parts, n_parts, g, a);
  return hipGetLastError();
}

}  // namespace

// Which kernel: linear_few_kernel for up to 16 rows, or where its workgroups
// are few and the contraction is not long; the grouped kernels' 128 x 256 tiles
// (launch_linear) once they fill the device; linear_tile_kernel between.
// Measured (us, the whole layer, W4A16 and W4A4), few / tile:
//   12288 x 2048 M = 32 13.2 / 14.6, 17.5 / 19.7; M = 33 16.3 / 14.5, 20.9 / 20.0
//   16384 x 8192 M = 17 33.2 / 29.6, 37.2 / 33.0
//   5120 x 17408 M = 17 30.8 / 30.4, 34.8 / 36.0; M = 64 43.5 / 35.7, 48.1 / 41.7
//   8192 x 8192  M = 64 27.3 / 25.6, 31.6 / 31.7; M = 100 42.6 / 31.0, 46.4 / 35.8
//   4096 x 1024  M = 128 10.3 / 12.4, 14.7 / 17.7; M = 203 15.8 / 12.5, 20.1 / 18.1
// and tile / grouped:
//   34816 x 5120 M = 256 131 / 132, 109 / 121; M = 300 147 / 137, 126 / 128; M = 1024 407 / 336, 342 / 316
//   5120 x 17408 M = 1024 202 / 248, 187 / 239; M = 2048 399 / 404, 367 / 397
//   8192 x 8192  M = 512 81 / 132, 76 / 90; M = 1300 213 / 210, 190 / 199; M = 2048 310 / 247, 274 / 239
static bool uses_few(int64_t M, int64_t N, int64_t K) {
  return M <= 16 || (K <= 8192 && (M + 63) / 64 * (N / 32) <= (M <= 32 ? 384 : kCUs));
}

bool linear_uses_tiles(int64_t M, int64_t N, int64_t K) {
  return uses_few(M, N, K) || M <= 256 || (M + 127) / 128 * ((N + 255) / 256) < kCUs;
}

namespace {
// The activations' form for linear_few_kernel.
FewAct few_act(int64_t M, int64_t K, bool w4a4) {
  if (w4a4) return M <= 16 && M * K <= kFewQuantMax ? kFewCodes : kFewF16Operand;
  return M <= kFewRowsMax ? kFewBf16Rows : kFewBf16Operand;
}

// Workspace of either kernel: W4A4's scale, maxima, the activation operand,
// partial sums; or the scale and the codes and scales of few rows; bf16 rows
// taken as they are need none.
struct TileWs {
  size_t parts, a, part, total;
};
size_t operand_bytes(int64_t M, int64_t K) { return (size_t)((M + 15) / 16 * 16) * K * 2; }
TileWs tile_ws(int64_t M, int64_t N, int64_t K, bool w4a4) {
  const bool few = uses_few(M, N, K);
  const TileSplit t = few ? TileSplit{} : tile_split(M, N, K);
  TileWs w{};
  w.parts = 256;
  w.a = w.parts + kAmaxParts * 4;
  w.part = w.a + (few || w4a4 ? operand_bytes(M, K) : 0);
  w.total = w.part + (t.stream ? (size_t)2 * t.grid * t.bm * t.bn * 4 : 0);
  if (few && few_act(M, K, w4a4) == kFewBf16Rows) w.total = 0;
  if (few && few_act(M, K, w4a4) == kFewCodes) w.total = 256 + (size_t)M * (K / 2) + (size_t)M * (K / 16);
  return w;
}
}  // namespace

size_t linear_tile_ws_bytes(int64_t M, int64_t N, int64_t K, bool w4a4) {
  return M > 0 && linear_uses_tiles(M, N, K) ? tile_ws(M, N, K, w4a4).total : 0;
}

// Of every call with up to M rows, growing with M.  Both rules above hold up to
// some number of rows; the operand grows with the rows, and the partial sums are
// at most two tiles of 64 x 256 for each workgroup of a layer that deals out K.
size_t linear_tile_ws_bound(int64_t M, int64_t N, int64_t K, bool w4a4) {
  auto last = [&](bool (*rule)(int64_t, int64_t, int64_t)) {   // the most rows up to M that it holds for
    int64_t lo = 0, hi = M;
    while (lo < hi) {
      const int64_t m = (lo + hi + 1) / 2;
      if (rule(m, N, K)) lo = m;
      else hi = m - 1;
    }
    return lo;
  };
  const int64_t rows = last(linear_uses_tiles), few = last(uses_few), KC = K / kBK;
  const int64_t operand = w4a4 ? rows : few > kFewRowsMax ? few : 0;
  size_t bytes = 256 + kAmaxParts * 4 + operand_bytes(operand, K);
  if (rows > few && KC > kJoinChunks) {   // (a layer of fewer chunks has nothing to gain from dealing them out)
    const int64_t tiles = (rows + 47) / 48 * ((N + 255) / 256);
    bytes += (size_t)2 * std::min<int64_t>(kCUs, std::max<int64_t>(1, tiles * KC / kMinRun)) * 64 * 256 * 4;
  }
  return rows > 0 ? bytes : 0;
}

namespace {
template <int ACT, bool GATED, int MT, int NT, int KW>
hipError_t launch_few_t(const FewParams& p, hipStream_t s) {
  const unsigned rb = (unsigned)((p.M + 16 * MT - 1) / (16 * MT)), groups = (unsigned)((p.N / (16 * NT) + 7) / 8);
  linear_few_kernel<ACT, GATED, MT, NT, KW><<<groups * 8 * rb, KW * kWave, 0, s>>>(p);
  return hipGetLastError();
}
template <int ACT, bool GATED, int MT>
hipError_t launch_few(const FewParams& p, hipStream_t s) {
  // Columns and wavefronts of a workgroup (us, 32 x 4 / 64 x 4 / 64 x 2).  With
  // two workgroups of 64 columns per CU, a handful of rows take 32 columns and
  // 4 wavefronts, more rows 64 columns and 4: W4A16 34816 x 5120 M = 1 25.6 /
  // 28.3 / 32.3, M = 16 34.9 / 33.7 / 36.0; with four, 64 columns and 2:
  // 65536 x 8192 M = 1 56.3 / 64.6 / 56.6, M = 16 73.2 / 69.4 / 62.7.  Else 32
  // columns and 8 wavefronts: 8192 x 8192 M = 1 11.3, against 14.0 / 18.3 / 31.
  if constexpr (MT == 1) {
    if constexpr (ACT < kFewBf16Operand)
      if (p.N / 64 >= 2 * kCUs && p.M <= 4) return launch_few_t<ACT, GATED, MT, 2, 4>(p, s);
    if (p.N / 64 >= 4 * kCUs) return launch_few_t<ACT, GATED, MT, 4, 2>(p, s);
    if (p.N / 64 >= 2 * kCUs) return launch_few_t<ACT, GATED, MT, 4, 4>(p, s);
  }
  return launch_few_t<ACT, GATED, MT, 2, 8>(p, s);
}
template <int ACT, bool GATED>
hipError_t launch_few_act(const FewParams& p, hipStream_t s) {
  if constexpr (ACT >= kFewBf16Operand) {
    const int tiles = (p.M + 15) / 16, blocks = (tiles + 3) / 4;
    switch ((tiles + blocks - 1) / blocks) {   // row blocks of even height
      case 1: break;
      case 2: return launch_few<ACT, GATED, 2>(p, s);
      case 3: return launch_few<ACT, GATED, 3>(p, s);
      default: return launch_few<ACT, GATED, 4>(p, s);
    }
  }
  return launch_few<ACT, GATED, 1>(p, s);
}
template <int ACT>
hipError_t launch_few_act(const FewParams& p, hipStream_t s) {
  return p.ep.gated ? launch_few_act<ACT, true>(p, s) : launch_few_act<ACT, false>(p, s);
}

hipError_t launch_linear_few(const uint16_t* x, int64_t M, int64_t N, int64_t K, bool w4a4, const uint8_t* w_prep,
                             const float* gw, const LinearEpi& ep, void* ws, hipStream_t s) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  float* g = static_cast<float*>(ws);
  FewParams p{};
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.w_q = w_prep;
  p.w_sf = w_prep + (size_t)N * (K / 2);
  p.g_w = gw;
  p.g_a = w4a4 ? g : nullptr;
  p.ep = ep;
  const FewAct act = few_act(M, K, w4a4);
  if (act == kFewCodes) {
    uint8_t* q = b + 256;
    uint8_t* sf = q + M * (K / 2);
    linear_few_quant_kernel<<<(unsigned)((M * K / 8 + 255) / 256), 256, 0, s>>>(x, M, K, g, q, sf);
    if (hipError_t e = hipGetLastError()) return e;
    p.a_q = q;
    p.a_sf = sf;
    return launch_few_act<kFewCodes>(p, s);
  }
  if (act == kFewBf16Rows) {
    p.x = x;
    return launch_few_act<kFewBf16Rows>(p, s);
  }
  const TileWs L = tile_ws(M, N, K, w4a4);
  uint16_t* a = reinterpret_cast<uint16_t*>(b + L.a);
  if (hipError_t e = launch_operand(x, M, K, w4a4, reinterpret_cast<uint32_t*>(b + L.parts), g, a, s)) return e;
  p.x = a;
  return w4a4 ? launch_few_act<kFewF16Operand>(p, s) : launch_few_act<kFewBf16Operand>(p, s);
}
}  // namespace

hipError_t launch_linear_tiles(const uint16_t* x, int64_t M, int64_t N, int64_t K, bool w4a4, const uint8_t* w_prep,
                               const float* gw, const LinearEpi& ep, void* ws, hipStream_t s) {
  if (uses_few(M, N, K)) return launch_linear_few(x, M, N, K, w4a4, w_prep, gw, ep, ws, s);
  const TileWs L = tile_ws(M, N, K, w4a4);
  uint8_t* b = static_cast<uint8_t*>(ws);
  float* g = reinterpret_cast<float*>(b);
  uint16_t* a = reinterpret_cast<uint16_t*>(b + L.a);
  if (w4a4)
    if (hipError_t e = launch_operand(x, M, K, true, reinterpret_cast<uint32_t*>(b + L.parts), g, a, s)) return e;
  TileParams p{};
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.t = tile_split(M, N, K);
  p.a = w4a4 ? a : x;
  p.w_q = w_prep;
  p.w_sf = w_prep + (size_t)N * (K / 2);
  p.g_w = gw;
  p.g_a = w4a4 ? g : nullptr;
  p.part = reinterpret_cast<float*>(b + L.part);
  p.ep = ep;
  if (w4a4) return ep.gated ? launch_tiles<false, true>(p, s) : launch_tiles<false, false>(p, s);
  return ep.gated ? launch_tiles<true, true>(p, s) : launch_tiles<true, false>(p, s);
}

}  // namespace nvfp4
