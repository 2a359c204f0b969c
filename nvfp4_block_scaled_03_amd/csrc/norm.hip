// Root-mean-square norm with the residual's addition and 8-bit codes
// (rms_norm), and the codes of rows as they are (int8_quantize), for gfx950.
//
//   h = x + residual, rounded to the residual's type (h = x without one)
//   rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd w
//   v = h w,  q = rne(127 v / max |v|),  s = rstd max |v| / 127
//
// The norm's factor leaves the codes alone (it scales a row and its maximum),
// so they are decided on v: a quotient 127 v / max |v| halfway between two
// codes, frequent where h and w are bfloat16, goes to the even one.  A
// candidate k = floor(t) from an approximate quotient is settled by the sign
// of 254 |v| - (2 k + 1) max |v|; near a whole number the candidate may be one
// off, which the comparison sets right.  With bfloat16 h and w all of it is exact
// in FP32 (v has 16 bits, 254 v 23, (2 k + 1) max |v| 24); with float32 ones v is
// exact in FP64 (48 bits) and the comparison takes in what FP64 rounds off 254 |v|
// (55).  FP64 too where a row's magnitudes come near the ends of FP32.
//
// A row stays in registers between its two uses: one read, one write.  Bound:
// bytes.
#include <algorithm>

#include "common.h"
#include "int8.h"

namespace nvfp4 {
namespace {

struct Raw8 {
  u32x4 lo, hi;   // 8 elements as stored (bfloat16: lo alone)
};
template <bool F32>
__device__ __forceinline__ Raw8 load8(const void* p, int64_t i) {
  Raw8 r;
  if constexpr (F32) {
    const u32x4* at = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i);
    r.lo = at[0];
    r.hi = at[1];
  } else {
    r.lo = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void unpack8(const Raw8& r, float (&v)[8]) {
  if constexpr (F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __int_as_float((int)r.lo[j]);
      v[4 + j] = __int_as_float((int)r.hi[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_bits_to_f32(r.lo[j] & 0xFFFFu);
      v[2 * j + 1] = __int_as_float((int)(r.lo[j] & 0xFFFF0000u));
    }
  }
}
// (the hardware conversion: nearest, ties to even, NaN stays NaN)
__device__ __forceinline__ uint32_t bf16_of(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (F32) {
    f32x4* at = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
    at[0] = f32x4{v[0], v[1], v[2], v[3]};
    at[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = bf16_of(v[2 * j]) | (bf16_of(v[2 * j + 1]) << 16);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = o;
  }
}

// Reductions over a row's lanes: DPP steps within 16 lanes, the four groups by
// lane reads (every lane gets the result).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
  return (uint64_t)dpp32<CTRL>((uint32_t)(v >> 32)) << 32 | dpp32<CTRL>((uint32_t)v);
}
__device__ __forceinline__ uint64_t lane64(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
// What a row's lanes gather: the sum of squares and the largest magnitude (as
// bits: NaN above infinity above the rest).
struct Gathered {
  double ss;
  uint64_t top;
  __device__ __forceinline__ void add(double s, uint64_t t) {
    ss += s;
    top = max(top, t);
  }
};
__device__ __forceinline__ uint64_t bits_of(double v) { return (uint64_t)__double_as_longlong(v); }
__device__ __forceinline__ double of_bits(uint64_t v) { return __longlong_as_double((long long)v); }
__device__ __forceinline__ void reduce16(Gathered& g) {
  g.add(of_bits(dpp64<0xB1>(bits_of(g.ss))), dpp64<0xB1>(g.top));     // lane ^ 1
  g.add(of_bits(dpp64<0x4E>(bits_of(g.ss))), dpp64<0x4E>(g.top));     // lane ^ 2
  g.add(of_bits(dpp64<0x141>(bits_of(g.ss))), dpp64<0x141>(g.top));   // mirror of 8
  g.add(of_bits(dpp64<0x140>(bits_of(g.ss))), dpp64<0x140>(g.top));   // mirror of 16
}
template <int WAVES>
__device__ __forceinline__ void row_reduce(Gathered& g, Gathered* red) {
  reduce16(g);
  Gathered r = {of_bits(lane64(bits_of(g.ss), 0)), lane64(g.top, 0)};
#pragma unroll
  for (int l = 16; l < 64; l += 16) r.add(of_bits(lane64(bits_of(g.ss), l)), lane64(g.top, l));
  g = r;
  if constexpr (WAVES > 1) {
    static_assert(WAVES <= 16, "a result per lane of a group");
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = g;
    __syncthreads();
    const int l = threadIdx.x & 15;
    g = red[l % WAVES];
    if (l >= WAVES) g.ss = 0.0;
    reduce16(g);
  }
}

// 1 / sqrt(x) by Newton steps on the hardware's estimate (2^-14 or better): two reach
// 2^-54 but for their own roundings, which a third takes back.
__device__ __forceinline__ double rsqrt64(double x) {
  const double y0 = __builtin_amdgcn_rsq(x), hx = 0.5 * x;
  double y = y0 * __builtin_fma(-hx * y0, y0, 1.5);
  y = y * __builtin_fma(-hx * y, y, 1.5);
  y = y * __builtin_fma(-hx * y, y, 1.5);
  return x > 0.0 && x < (double)INFINITY ? y : y0;
}

// |code| of one value: k = floor(t), one more beyond k + 1/2 (at it: if k is odd).
__device__ __forceinline__ int code_f32(float a, float top, float inv) {
  const float k = floorf(a * inv);
  const float d = __builtin_fmaf(-(2.0f * k + 1.0f), top, 254.0f * a);
  const int c = (int)k;
  return c + (d > 0.0f || (d == 0.0f && (c & 1)));
}
// (254 a is p + e.  Where p - (2 k + 1) top comes near e it is exact: a whole
// multiple of the last places of p and top, and far below either.)
__device__ __forceinline__ int code_f64(double a, double top, double inv) {
  const double k = floor(a * inv), p = 254.0 * a, e = __builtin_fma(254.0, a, -p);
  const double d = __builtin_fma(-(2.0 * k + 1.0), top, p) + e;
  const int c = (int)k;
  return min(c + (d > 0.0 || (d == 0.0 && (c & 1))), 127);
}

__device__ __forceinline__ uint64_t magnitude_bits(double v) {
  return (uint64_t)__double_as_longlong(v) & 0x7FFFFFFFFFFFFFFFull;
}

constexpr float kTiny = 8.673617379884035e-19f, kHuge = 1.2676506002282294e30f;   // 2^-60, 2^100

// TPR threads a row (64: a wavefront, four rows a workgroup), VPT pieces of 8
// elements a thread.  RES: 0 none, 1 bfloat16, 2 float32.  NORM false: the codes
// of x itself.
template <bool NORM, bool XF32, int RES, int TPR, int VPT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void row_kernel(NormArgs p) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1, WAVES = TPR / 64;
  constexpr bool HF32 = RES == 2 || (RES == 0 && XF32);   // type of h
  __shared__ Gathered red[WAVES > 1 ? WAVES : 1], red2[WAVES > 1 ? WAVES : 1];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
  if (ROWS > 1 && row >= p.rows) return;   // (whole wavefronts)
  const int V = p.H / 8;
  constexpr bool KEEP_W = VPT <= 2;   // the weights stay in registers (else they are read twice, from the caches)
  Raw8 xr[VPT], rr[VPT], wr[KEEP_W ? VPT : 1];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * TPR + t;
    if (v < V) {
      xr[i] = load8<XF32>(p.x, row * p.ldx + v * 8);
      if constexpr (RES != 0) rr[i] = load8<RES == 2>(p.res, row * p.ldr + v * 8);
      if constexpr (NORM && KEEP_W) wr[i] = p.w_f32 ? load8<true>(p.w, v * 8) : load8<false>(p.w, v * 8);
    }
  }
  const bool wide = HF32 || (NORM && p.w_f32);   // v needs FP64
  float h[VPT][8];
  Gathered g = {0.0, 0};
  uint32_t top_bits = 0;
  auto weights = [&](int i, float (&w)[8]) {
    if constexpr (NORM) {
      Raw8 r;
      if constexpr (KEEP_W) r = wr[i];
      else r = p.w_f32 ? load8<true>(p.w, (i * TPR + t) * 8) : load8<false>(p.w, (i * TPR + t) * 8);
      if (p.w_f32) unpack8<true>(r, w);
      else unpack8<false>(r, w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 1.0f;
    }
  };
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * TPR + t;
    if (v < V) {
      unpack8<XF32>(xr[i], h[i]);
      if constexpr (RES != 0) {
        float r[8];
        unpack8<RES == 2>(rr[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[i][j] += r[j];
          if constexpr (!HF32) h[i][j] = __int_as_float((int)(bf16_of(h[i][j]) << 16));
        }
        if (p.h) store8<HF32>(p.h, row * p.ldh + v * 8, h[i]);
      }
      if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g.ss = __builtin_fma((double)h[i][j], (double)h[i][j], g.ss);
      }
      if (p.q) {
        float w[8];
        weights(i, w);
        if (wide) {
#pragma unroll
          for (int j = 0; j < 8; ++j) g.top = max(g.top, magnitude_bits((double)h[i][j] * (double)w[j]));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            top_bits = max(top_bits, (uint32_t)__float_as_int(h[i][j] * w[j]) & 0x7FFFFFFFu);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
    }
  }
  if (!wide) g.top = top_bits;
  row_reduce<WAVES>(g, red);
  const double rstd = NORM ? rsqrt64(g.ss / p.H + (double)p.eps) : 1.0;
  const float rs = (float)rstd;
  bool far = NORM && !(rs >= kTiny && rs <= kHuge);   // (NaN too)
  double top = 0.0;
  if (p.q) {
    top = wide ? of_bits(g.top) : (double)__int_as_float((int)(uint32_t)g.top);
    far = far || !(top >= kTiny && top <= kHuge);
    if (far && !wide) {   // (the same for the whole row)
      g = {0.0, 0};
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (i * TPR + t < V) {
          float w[8];
          weights(i, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) g.top = max(g.top, magnitude_bits((double)h[i][j] * (double)w[j]));
        }
      }
      row_reduce<WAVES>(g, red2);
      top = of_bits(g.top);
    }
  }
  const float top32 = (float)top, inv32 = 127.0f * __builtin_amdgcn_rcpf(top32);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * TPR + t;
    if (v >= V) continue;
    float w[8];
    weights(i, w);
    if (NORM && p.y) {
      float y[8];
      if (!far) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = h[i][j] * rs * w[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = (float)((double)h[i][j] * rstd * (double)w[j]);
      }
      if (p.y_f32) store8<true>(p.y, row * p.ldy + v * 8, y);
      else store8<false>(p.y, row * p.ldy + v * 8, y);
    }
    if (p.q) {
      int c[8];
      if (!(far || wide)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float vj = h[i][j] * w[j];
          const int k = code_f32(fabsf(vj), top32, inv32);
          c[j] = vj < 0.0f ? -k : k;
        }
      } else {
        const double inv64 = 127.0 / top;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double vj = (double)h[i][j] * (double)w[j];
          const int k = top > 0.0 ? code_f64(fabs(vj), top, inv64) : 0;
          c[j] = vj < 0.0 ? -k : k;
        }
      }
      u32x2 o;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        o[j] = (c[4 * j] & 0xFF) | (c[4 * j + 1] & 0xFF) << 8 | (c[4 * j + 2] & 0xFF) << 16 | (c[4 * j + 3] & 0xFF) << 24;
      *reinterpret_cast<u32x2*>(p.q + row * p.H + v * 8) = o;
    }
  }
  // (a row with NaN or infinity: scale NaN)
  if (p.q && t == 0) p.s[row] = top < (double)INFINITY ? (float)(rstd * top / 127.0) : __builtin_nanf("");
}

template <bool NORM, bool XF32, int RES, int TPR, int VPT>
hipError_t launch_rows_t(const NormArgs& a, hipStream_t s) {
  constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
  // (a launch has fewer than 2^32 threads)
  constexpr int64_t STEP = (int64_t(1) << 31) / TPR;
  NormArgs p = a;
  auto past = [](const void* at, int64_t bytes) {
    return at ? const_cast<char*>(static_cast<const char*>(at)) + bytes : nullptr;
  };
  for (int64_t r = 0; r < a.rows; r += STEP) {
    p.rows = std::min(a.rows - r, STEP);
    row_kernel<NORM, XF32, RES, TPR, VPT>
        <<<(unsigned)((p.rows + ROWS - 1) / ROWS), TPR < 256 ? 256 : TPR, 0, s>>>(p);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    p.x = past(p.x, STEP * p.ldx * (XF32 ? 4 : 2));
    p.res = past(p.res, STEP * p.ldr * (RES == 2 ? 4 : 2));
    p.h = past(p.h, STEP * p.ldh * (RES == 2 ? 4 : 2));
    p.y = past(p.y, STEP * p.ldy * (p.y_f32 ? 4 : 2));
    p.q = reinterpret_cast<int8_t*>(past(p.q, STEP * p.H));
    p.s = reinterpret_cast<float*>(past(p.s, STEP * 4));
  }
  return hipSuccess;
}
// Threads and pieces a thread ("codes alone" are int8_quantize's).  A piece a thread
// for the latency (H = 5120, both outputs, us: 1 row 256 x 3 6.4, 512 x 2 4.7, 1024 x 1 4.2) as long as the workgroups
// take turns in loading and reducing (both outputs / codes alone: 1024 rows of 8192
// 256 x 4 23.7 / 9.5, 1024 x 1 20.1 / 9.5; 4096 rows of 4096 256 x 2 35.6 / 13.9, 512 x
// 1 32.2 / 14.8; 16384 rows of 2048 64 x 4 68.7 / 21.6, 256 x 1 59.4 / 27.0).  Fewer
// reductions and barriers a byte for many rows that are short or leave threads idle,
// and for the codes alone, whose rows have a third of the bytes (16384 rows of 1024 64
// x 2 35.5 / 13.2, 256 x 1 39.1 / 20.8; of 5120 256 x 3 151.6 / 47.7, 1024 x 1 155.6 /
// 77.7), and for long ones, which do not fit a piece a thread (4096 rows of 16384 512 x
// 4 125.8 / 36.2, 1024 x 2 137.4 / 43.1).  151.6 us are 755 MB at 5.0 TB/s.  8192 rows of
// 4096, both outputs: 512 x 1 57, 256 x 2 60, with one set of inputs or with twelve
// (3.6 GB, past any cache).  rms_norm takes the layout for both outputs whatever is
// asked for; y or codes alone without a residual would gain from the other one (16384
// rows of 4096, y / codes: 512 x 1 56.8 / 70.0, 256 x 2 47.8 / 60.7).
template <bool NORM, bool XF32, int RES>
hipError_t launch_rows(const NormArgs& a, hipStream_t s) {
  const int V = a.H / 8;
  const bool many = a.rows > (NORM ? 4096 : 1024);
  if (V <= 64) return launch_rows_t<NORM, XF32, RES, 64, 1>(a, s);
  if (many) {
    if (V <= 128) return launch_rows_t<NORM, XF32, RES, 64, 2>(a, s);
    if constexpr (!NORM) {
      if (V <= 256) return launch_rows_t<NORM, XF32, RES, 64, 4>(a, s);
      if (V <= 512) return launch_rows_t<NORM, XF32, RES, 256, 2>(a, s);
      if (V > 768 && V <= 1024) return launch_rows_t<NORM, XF32, RES, 256, 4>(a, s);
    }
    if (V > 512 && V <= 768) return launch_rows_t<NORM, XF32, RES, 256, 3>(a, s);
  }
  if (V <= 256) return launch_rows_t<NORM, XF32, RES, 256, 1>(a, s);
  if (V <= 512) return launch_rows_t<NORM, XF32, RES, 512, 1>(a, s);
  if (V <= 1024) return launch_rows_t<NORM, XF32, RES, 1024, 1>(a, s);
  if (a.rows <= 256) {   // (17408, 1 row: 1024 x 3 7.7, 256 x 9 14.9)
    if (V <= 2048) return launch_rows_t<NORM, XF32, RES, 1024, 2>(a, s);
    if (V <= 3 * 1024) return launch_rows_t<NORM, XF32, RES, 1024, 3>(a, s);
  }
  if (V <= 2048) return launch_rows_t<NORM, XF32, RES, 512, 4>(a, s);
  if (V <= 2560) return launch_rows_t<NORM, XF32, RES, 512, 5>(a, s);
  return launch_rows_t<NORM, XF32, RES, 512, 8>(a, s);
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  const int res = !a.res ? 0 : a.res_f32 ? 2 : 1;
  if (a.x_f32) {
    if (res == 0) return launch_rows<true, true, 0>(a, s);
    if (res == 1) return launch_rows<true, true, 1>(a, s);
    return launch_rows<true, true, 2>(a, s);
  }
  if (res == 0) return launch_rows<true, false, 0>(a, s);
  if (res == 1) return launch_rows<true, false, 1>(a, s);
  return launch_rows<true, false, 2>(a, s);
}

hipError_t launch_int8_quantize(const NormArgs& a, hipStream_t s) {
  return a.x_f32 ? launch_rows<false, true, 0>(a, s) : launch_rows<false, false, 0>(a, s);
}

}  // namespace nvfp4
