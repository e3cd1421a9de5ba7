// Rows of 8-bit codes: a row y of f32 values is held as one scale, max|y| / 127,
// and a code for each element, rint(127 y / max|y|).  Three kinds of row:
// y = x; the RMSNorm of x + other; silu(gate) * up.  And the way back.
//
// The codes are those of the exact values (SwiGLU's: of values known to 2^-38).  In f32
// the quotient t = 127 y / max|y| is known to within kBand; where t lies that near to a
// border between two codes, and only there, it is taken again in f64, with the row's
// largest value in f64 too.  A row whose largest value or sum of squares leaves the middle
// of the f32 range is done in f64 as a whole, so neither squares nor products overflow or
// vanish.  The norm's 1 / rms multiplies every element alike: it is in the scale and not
// in the codes.  A scale is found in f32.  Rows: one rounding.  The norm, in units of 2^-24:
// the sum of squares 52 (chains of 16, a warp's 5 steps, up to 31 warps more), / n and + eps
// 2, all halved by the root; the root, its reciprocal, the largest h g, its product with
// that, / 127: 5; 32 in all.  SwiGLU: its largest value 8 (see kBand), / 127: 9.
#include <cuda_runtime.h>
#include <float.h>

#include "tqd_device.cuh"
#include "tqd_i8.cuh"
#include "tqd_internal.h"

namespace tqd {
namespace {

constexpr int kSms = 152;

// The relative errors that reach t, in units of 2^-24, times 127: of y (exact for rows; the
// product h g, 1; silu: e^-g 5, 1 + e, the quotient and the product with up 1 each), of the
// largest y the same, of 127 / max and of the product with it 1 each.
// 2 * 127 * 2^-24 < 2^-16, 4 * 127 * 2^-24 < 2^-15, 18 * 127 * 2^-24 < 1.125 * 2^-13.
template <int kKind>
constexpr float kBand = kKind == kI8Rows ? 0x1p-16f : kKind == kI8Norm ? 0x1p-15f : 0x1.2p-13f;

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: added, it leaves the nearest whole number in the low bits

// e^x for x <= 87 within 5 units: 2^t, t = x log2 e rounded, times 1 + ln 2 (x log2 e - t).
// (Far below zero 2^t is 0.)
__device__ __forceinline__ float exp_near(float x) {
  constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596303e-8f, kLn2 = 0.693147182f;
  const float t = x * kLog2e, left = fmaf(x, kLog2eRest, fmaf(x, kLog2e, -t));
  float e;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
  return fmaf(e * kLn2, left, e);
}
// g / (1 + e^-g): the quotient from the approximate reciprocal and one step of Newton's
// iteration, within a unit.  (e^87 is the largest that leaves the reciprocal in range.  Below
// it the value is too large, by |g| e^-87 at most, 2^-89 of gates down to -2^36: nothing beside
// the largest of a row that is done here.)
__device__ __forceinline__ float silu(float g) {
  const float d = 1.f + exp_near(fminf(-g, 87.f));
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
  const float q = g * r;
  return fmaf(fmaf(-d, q, g), r, q);
}

// silu(g) u to 2^-38 (the worst found: 2^-41), for gates whose e^-g is within f32: of a row whose
// largest |y| is at least 2^-40 and whose |g| and |u| are at most 2^36, elements of at least a
// 2^8th of the largest have g > -62.  The f64 pipe does a warp's instruction in 15 clocks, so
// this takes the reduction to |r| <= ln 2 / 2 with ln 2 in two parts (Cody and Waite), the Taylor
// series with the terms from r^6 on in f32 (less than 2^-18 of the whole), and one step of
// Newton's iteration from the f32 reciprocal in place of exp and a division.
constexpr double kLn2High = 0.6931471804855391, kLn2Low = 7.440617110012397e-11;  // 33 bits after the point, and the rest
__device__ __forceinline__ double near_silu(float g, float u) {
  const float xf = fmaxf(-g, -64.f);  // (e^-64 is nothing beside 1)
  const float kf = rintf(xf * 1.44269504f);
  const double k = kf, r = fma(k, -kLn2Low, fma(k, -kLn2High, static_cast<double>(xf)));
  const float rf = static_cast<float>(r);
  float h = 1.f / 3628800;
  h = fmaf(h, rf, 1.f / 362880);
  h = fmaf(h, rf, 1.f / 40320);
  h = fmaf(h, rf, 1.f / 5040);
  h = fmaf(h, rf, 1.f / 720);
  double e = h;
  e = fma(e, r, 1.0 / 120);
  e = fma(e, r, 1.0 / 24);
  e = fma(e, r, 1.0 / 6);
  e = fma(e, r, 0.5);
  e = fma(e, r, 1.0);
  e = fma(e, r, 1.0);
  const double d = fma(e, __hiloint2double((1023 + static_cast<int>(kf)) << 20, 0), 1.0);
  const double q = 1.f / static_cast<float>(d);
  return fma(fma(-d, q, 1.0), q, q) * (static_cast<double>(g) * u);
}

// Element i of a row in f64, from memory again (the norm: without 1 / rms; h is its sum in f32).
template <int kKind>
__device__ __noinline__ double exact_element(const I8RowsArgs& a, int64_t row, int i, double& h) {
  const float x = a.x[row * a.x_stride + i];
  h = 0.0;
  if (kKind == kI8Rows) return x;
  if (kKind == kI8Norm) {
    // the sum may stand where x or other stood
    h = a.sum ? a.sum[row * a.sum_stride + i] : a.other ? x + a.other[row * a.other_stride + i] : x;
    return h * a.g[i];
  }
  const float u = a.other[row * a.other_stride + i];
  if ((x == 0.f && isfinite(u)) || (u == 0.f && isfinite(x))) return 0.0;
  return x / (1.0 + exp(-static_cast<double>(x))) * u;
}

// The code next to the border between `low` and low + 1: by the side of it that 127 y / most lies on, and on it the even
// one.  Where y and most are exact (rows: 24 bits; the norm's products: 48) so is the side: the border times most has 56 bits,
// in two parts.
__device__ __forceinline__ float code_beside(float low, double y, double most) {
  const double at = low + 0.5f, p = at * most, side = fma(127.0, y, -p) - fma(at, most, -p);
  return side > 0.0 || (side == 0.0 && (static_cast<int>(low) & 1)) ? low + 1.f : low;
}

// The code of y in a row whose largest value is `most`.  (For the norm's products a quotient in f64 tells a border from what
// lies beside it no more; up to a unit it finds what is below, for which a product with the reciprocal is enough.)
__device__ __noinline__ float exact_code(double y, double most) { return static_cast<float>(rint(127.0 * y / most)); }
__device__ __noinline__ float exact_code(double y, double inv, double most) {
  return code_beside(static_cast<float>(floor(y * inv)), y, most);
}

// The largest of a and |b|, |c|; NaN where one of them is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <bool kVec>
__device__ __forceinline__ void load4(const float* p, int i, int n, float (&v)[4]) {
  if (kVec) {
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) t = __ldg(reinterpret_cast<const float4*>(p + i));
    v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + j < n ? p[i + j] : 0.f;
  }
}

// `some` (of four) elements from p on into 16 bytes of shared memory.
template <bool kVec>
__device__ __forceinline__ void fetch4(uint32_t to, const float* p, int some) {
  if (kVec) {
    if (some > 0) asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < some) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4 * j), "l"(p + j) : "memory");
  }
}

// Reductions over the kT threads of a row: one warp, or the whole block.
template <int kT>
struct RowGroup {
  static __device__ __forceinline__ void sync() {
    if (kT == 32) __syncwarp();
    else __syncthreads();
  }
  static __device__ __forceinline__ bool any(bool p) {
    return kT == 32 ? __any_sync(0xFFFFFFFFu, p) : __syncthreads_or(p) != 0;
  }
  template <class F>
  static __device__ double all(double v, double* sh, F join) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (kT == 32) return v;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh[0];
    for (int w = 1; w < kT / 32; ++w) v = join(v, sh[w]);
    return v;
  }
};

// A row in f64 as a whole, or its codes only.
template <int kKind, int kT>
__device__ __noinline__ void whole_row(const I8RowsArgs& a, int64_t row, int t, double* sh, bool codes_only) {
  const int n = a.n;
  RowGroup<kT>::sync();  // (a sum that was written is read by other threads)
  double most = 0.0, squares = 0.0, h;
  bool lost = false;
  for (int i = t; i < n; i += kT) {
    const double y = exact_element<kKind>(a, row, i, h);
    lost = lost || !(fabs(y) <= DBL_MAX);
    most = fmax(most, fabs(y));
    squares += h * h;
  }
  most = RowGroup<kT>::all(most, sh, [](double p, double q) { return fmax(p, q); });
  lost = RowGroup<kT>::any(lost);
  double top = most;
  if (kKind == kI8Norm) {
    squares = RowGroup<kT>::all(squares, sh, [](double p, double q) { return p + q; });
    const double at = squares / n + a.eps;
    top = at > 0.0 ? most / sqrt(at) : 0.0;
  }
  if (!isfinite(static_cast<float>(top))) lost = true;
  int8_t* q = a.q + row * a.q_stride;
  if (kKind == kI8Norm) {
    const bool none = lost || most == 0.0;
    const double inv = none ? 0.0 : 127.0 / most;
    for (int i = t; i < n; i += kT) {
      q[i] = none ? 0 : static_cast<int8_t>(exact_code(exact_element<kKind>(a, row, i, h), inv, most));
    }
  } else {
    for (int i = t; i < n; i += kT)
      q[i] = lost || most == 0.0 ? 0 : static_cast<int8_t>(exact_code(exact_element<kKind>(a, row, i, h), most));
  }
  if (t == 0 && !codes_only) a.scale[row] = lost ? __uint_as_float(0x7FC00000u) : static_cast<float>(top / 127.0);
}

// The code of y where 127 y / most is known to lie at a border.
__device__ __forceinline__ int8_t code_at_border(double y, double most) {
  return static_cast<int8_t>(code_beside(floorf(static_cast<float>(y) * (127.f / static_cast<float>(most))), y, most));
}

// Elements next to borders, and those that may be a row's largest, of up to kWindow rows of a group of threads: they
// are worked out together, a lane each.  (At once, one lane of a row's threads each, they took 12 of 40 us of
// 2053 x 8192 silu rows: f64's latency, and two barriers.)
constexpr int kWindow = 16;
template <int kT>
struct Pending {
  static constexpr int room = kT == 32 ? 64 : 256;
  uint32_t count, borders, over;   // entries; whether some are at borders; bit r: row r of the window had more than there was room for
  unsigned long long most[kWindow];  // the largest |y| of each row, as bits
  uint32_t entry[room];            // row of the window << 16 | largest << 15 | element
  double y[room];

  __device__ __forceinline__ void clear(int t) {
    if (t < kWindow) most[t] = 0ull;
    if (t == 0) count = borders = over = 0u;
  }
  __device__ __forceinline__ void add(int r, bool largest, int i) {
    const uint32_t at = atomicAdd(&count, 1u);
    if (at < room) entry[at] = static_cast<uint32_t>(r) << 16 | static_cast<uint32_t>(largest) << 15 | static_cast<uint32_t>(i);
    else atomicOr(&over, 1u << r);
    if (!largest) borders = 1u;
  }
};

// The codes next to borders of a SwiGLU row that had no room in the list: the same elements by the same values as the list's,
// so that what a row becomes does not depend on what else was in the list.  (The norm's values are exact either way.)
template <int kT>
__device__ __noinline__ void settle_silu(const I8RowsArgs& a, int64_t row, int t, double* sh) {
  const int n = a.n;
  const float *gate = a.x + row * a.x_stride, *up = a.other + row * a.other_stride;
  float m = 0.f;
#pragma unroll 1
  for (int i = t; i < n; i += kT) m = fmaxf(m, fabsf(silu(gate[i]) * up[i]));
  auto larger = [](double p, double q) { return fmax(p, q); };
  const float inv = 127.f / static_cast<float>(RowGroup<kT>::all(m, sh, larger));
  double most = 0.0;
#pragma unroll 1
  for (int i = t; i < n; i += kT)
    if (fabsf(fmaf(silu(gate[i]) * up[i], inv, kMagic) - kMagic) > 126.f) most = fmax(most, fabs(near_silu(gate[i], up[i])));
  most = RowGroup<kT>::all(most, sh, larger);
#pragma unroll 1
  for (int i = t; i < n; i += kT) {
    const float v = silu(gate[i]) * up[i], c = fmaf(v, inv, kMagic);
    if (fabsf(fmaf(v, inv, kMagic - c)) > 0.5f - kBand<kI8Silu>) a.q[row * a.q_stride + i] = code_at_border(near_silu(gate[i], up[i]), most);
  }
}

template <int kKind, int kT>
__device__ __noinline__ void settle(const I8RowsArgs& a, Pending<kT>& p, int64_t first, int64_t step, int t, double* sh) {
  RowGroup<kT>::sync();
  const int n = static_cast<int>(min(p.count, static_cast<uint32_t>(p.room)));
  const uint32_t over = p.over, some = p.borders;
  for (int e = some ? t : n; e < n; e += kT) {
    const uint32_t x = p.entry[e];
    const int r = x >> 16, i = x & 0x7FFF;
    const int64_t row = first + r * step;
    double h, y;
    if (kKind == kI8Silu) y = near_silu(a.x[row * a.x_stride + i], a.other[row * a.other_stride + i]);
    else y = exact_element<kKind>(a, row, i, h);
    p.y[e] = y;
    if (x & 0x8000u) atomicMax(&p.most[r], static_cast<unsigned long long>(__double_as_longlong(fabs(y))));
  }
  RowGroup<kT>::sync();
  if (!some) {  // (nothing to settle, however many may be the largest)
    p.clear(t);
    if (kT == 32) __syncwarp();
    return;
  }
  for (int e = t; e < n; e += kT) {
    const uint32_t x = p.entry[e];
    const int r = x >> 16, i = x & 0x7FFF;
    if (!(x & 0x8000u) && !((over >> r) & 1u))
      a.q[(first + r * step) * a.q_stride + i] = code_at_border(p.y[e], __longlong_as_double(static_cast<long long>(p.most[r])));
  }
  for (int r = 0; over && r < kWindow; ++r)
    if ((over >> r) & 1u) {
      if (kKind == kI8Silu) settle_silu<kT>(a, first + r * step, t, sh);
      else whole_row<kKind, kT>(a, first + r * step, t, sh, true);  // (its scale depends on no other row)
    }
  RowGroup<kT>::sync();
  p.clear(t);  // (a block's next entries come after the next row's barrier)
  if (kT == 32) __syncwarp();
}

// How many rows' inputs a thread has under way, and CTAs an SM.
template <int kKind, int kT, int kE>
struct RowsCfg {
  static constexpr int block = kT < 128 ? 128 : kT;
  static constexpr int inputs = kKind == kI8Rows ? 1 : 2, ahead = kKind == kI8Rows ? 2 : 1;
  // The norm's g is kept beside the rows up to 2048 columns (8192 x 1024 23.4 -> 21.2 us, 8191 x 2048 39.7 -> 38.3), and read
  // again for each wider row, which leaves L1 more room (4099 x 4096 39.7 us and kept 42.2, 2053 x 8192 47.2 and 55.8).
  static constexpr bool keeps_g = kKind == kI8Norm && kT * kE <= 512;
  static constexpr int parts = inputs * ahead + keeps_g;  // of kE groups a thread
  static constexpr int smem = block * kE * 16 * parts;
  static constexpr int ctas = kT >= 1024 ? 1 : kT == 512 ? 2 : kT == 256 ? (kE == 4 ? 3 : 5)
                              : kE == 4 ? 5 : kKind == kI8Rows ? 8 : kKind == kI8Norm ? 6 : 7;
  };

// kT threads a row, kE groups of four elements a thread.  Measured, in TB/s of the bytes that it must move (a copy of
// as many: 6.8): rows 4099 x 4096 5.1 (16.4 us), norm with a sum that is kept 5.5 (39.6), SwiGLU 5.2
// (28.8); a single row of 1024 1.2, 2.0 and 2.1 us.  HBM bounds the norm up to 4096 columns; wider rows have two
// CTAs or one an SM, which wait at a row's barrier together (1500 x 12288 norm 3.8 TB/s); SwiGLU's instructions
// (2.6 a clock and SM) and its barrier bound it.  kVec: every row of every tensor
// begins on a 16-byte boundary (codes: 4) and is whole groups of four.  CTAs go from row to
// row; a thread copies its elements of the next row into its own part of shared memory
// while it works on this one, so that loads are always under way.
template <int kKind, int kT, int kE, bool kVec>
__global__ void __launch_bounds__(RowsCfg<kKind, kT, kE>::block, RowsCfg<kKind, kT, kE>::ctas)
    k_rows_i8(const __grid_constant__ I8RowsArgs a) {
  using Cfg = RowsCfg<kKind, kT, kE>;
  extern __shared__ float4 next_rows[];  // [ahead][inputs][kE][block], then g, [kE][block]
  __shared__ uint32_t sh_max[2][32];     // the largest |y| of each warp, as bits
  __shared__ float sh_sum[2][32];
  __shared__ double sh_d[32];
  __shared__ Pending<kT> pending[kKind == kI8Rows ? 1 : Cfg::block / kT];
  Pending<kT>& later = pending[kKind == kI8Rows ? 0 : threadIdx.x / kT];
  const int t = threadIdx.x % kT, lane = threadIdx.x & 31, n = a.n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (Cfg::block / kT);
  int64_t row = static_cast<int64_t>(blockIdx.x) * (Cfg::block / kT) + threadIdx.x / kT;
  const bool two = kKind == kI8Silu || (kKind == kI8Norm && a.other);
  pdl_launch_dependents();
  pdl_wait();
  // (past a row's end its places hold zeros from here on: copies leave them)
#pragma unroll
  for (int i = 0; i < Cfg::parts * kE; ++i)
    if ((i % kE * kT + t) * 4 + 3 >= n) next_rows[i * Cfg::block + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  const uint32_t place = smem_addr(next_rows + threadIdx.x);
  auto fetch = [&](int at, int64_t r) {  // (a row past the last: nothing, but a group of its own)
    if (r < a.rows) {
      const uint32_t to = place + at * (Cfg::inputs * kE * Cfg::block * 16);
      const float* p = a.x + r * a.x_stride + 4 * t;
#pragma unroll(kVec ? kE : 1)
      for (int e = 0; e < kE; ++e) fetch4<kVec>(to + e * (Cfg::block * 16), p + e * (4 * kT), n - (e * kT + t) * 4);
      if (two) {
        p = a.other + r * a.other_stride + 4 * t;
#pragma unroll(kVec ? kE : 1)
        for (int e = 0; e < kE; ++e) fetch4<kVec>(to + (kE + e) * (Cfg::block * 16), p + e * (4 * kT), n - (e * kT + t) * 4);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (Cfg::keeps_g) {  // g, once for all of its rows (comes with the first)
#pragma unroll(kVec ? kE : 1)
    for (int e = 0; e < kE; ++e)
      fetch4<kVec>(place + (Cfg::inputs * Cfg::ahead * kE + e) * (Cfg::block * 16), a.g + (e * kT + t) * 4, n - (e * kT + t) * 4);
  }
#pragma unroll
  for (int i = 0; i < Cfg::ahead; ++i) fetch(i, row + i * step);
  if (kKind != kI8Rows) {
    later.clear(t);
    if (kT == 32) __syncwarp();  // (a block's first entries come after the first row's barrier)
  }
  int turn = 0;
#pragma unroll 1
  for (; row < a.rows; row += step, ++turn) {
  if (kKind != kI8Rows && turn && turn % kWindow == 0) settle<kKind, kT>(a, later, row - kWindow * step, step, t, sh_d);
  const int odd = turn & 1;
  float v[kE][4], w[kE][4];  // y; what else came in (the norm: then h)
  asm volatile("cp.async.wait_group %0;" ::"n"(Cfg::ahead - 1) : "memory");
  {
    const float4* from = next_rows + turn % Cfg::ahead * (Cfg::inputs * kE * Cfg::block) + threadIdx.x;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const float4 f = from[e * Cfg::block];
      v[e][0] = f.x, v[e][1] = f.y, v[e][2] = f.z, v[e][3] = f.w;
      if (two) {
        const float4 o = from[(kE + e) * Cfg::block];
        w[e][0] = o.x, w[e][1] = o.y, w[e][2] = o.z, w[e][3] = o.w;
      }
    }
  }
  fetch(turn % Cfg::ahead, row + Cfg::ahead * step);
  float top = 0.f, ss = 0.f, ins = 0.f;  // the largest |y| (a NaN or an infinity is above all), the sum of h^2, the largest |gate| and |up|
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int i = (e * kT + t) * 4;
    if (kKind == kI8Silu) {
      ins = max_abs(max_abs(ins, v[e][0], v[e][1]), v[e][2], v[e][3]);
      ins = max_abs(max_abs(ins, w[e][0], w[e][1]), w[e][2], w[e][3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[e][j] = silu(v[e][j]) * w[e][j];
    }
    if (kKind == kI8Norm) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[e][j] = two ? v[e][j] + w[e][j] : v[e][j];
      if (a.sum) {
        float* s = a.sum + row * a.sum_stride + i;
        if (kVec) {
          if (i < n) *reinterpret_cast<float4*>(s) = make_float4(w[e][0], w[e][1], w[e][2], w[e][3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (i + j < n) s[j] = w[e][j];
        }
      }
      float g[4];
      if (Cfg::keeps_g) {
        const float4 kept = next_rows[(Cfg::inputs * Cfg::ahead * kE + e) * Cfg::block + threadIdx.x];
        g[0] = kept.x, g[1] = kept.y, g[2] = kept.z, g[3] = kept.w;
      } else {
        load4<kVec>(a.g, i, n, g);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ss = fmaf(w[e][j], w[e][j], ss);
        v[e][j] = w[e][j] * g[j];
      }
    }
    top = max_abs(max_abs(top, v[e][0], v[e][1]), v[e][2], v[e][3]);
  }
  if (kKind == kI8Silu && ins > 0x1p36f) top = INFINITY;  // silu may be below f32's range, and count: the row in f64
  uint32_t high = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top) & 0x7FFFFFFFu);
  if (kKind == kI8Norm) ss = warp_sum(ss);
  if (kT > 32) {
    if (lane == 0) {
      sh_max[odd][threadIdx.x >> 5] = high;
      if (kKind == kI8Norm) sh_sum[odd][threadIdx.x >> 5] = ss;
    }
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < kT / 32; ++i) {
      high = max(high, sh_max[odd][i]);
      if (kKind == kI8Norm) ss += sh_sum[odd][i];
    }
  }
  const float m = __uint_as_float(high);

  // (false for NaN)
  bool whole = !(m >= (kKind == kI8Silu ? 0x1p-40f : 0x1p-60f) && m <= 0x1p60f);
  if (kKind == kI8Norm) whole = whole || !(ss >= 0x1p-60f && ss <= 0x1p100f);
  if (m == 0.f) {
    // a row of zeros (a batch's padding; zeros in up are enough) needs no more; products that vanished do
    whole = false;
    if (kKind != kI8Rows) {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        if (kKind == kI8Silu) {  // (w: up; the gates' place has the next row's)
          float g[4];
          load4<kVec>(a.x + row * a.x_stride, (e * kT + t) * 4, n, g);
#pragma unroll
          for (int j = 0; j < 4; ++j) whole = whole || (g[j] != 0.f && w[e][j] != 0.f);
        } else {
          whole = whole || max_abs(max_abs(0.f, w[e][0], w[e][1]), w[e][2], w[e][3]) != 0.f;
        }
      }
      whole = RowGroup<kT>::any(whole);
    }
  }
  if (whole) {
    whole_row<kKind, kT>(a, row, t, sh_d, false);
    continue;
  }
  const float inv = m > 0.f ? 127.f / m : 0.f;
  float c[kE][4], far = 0.f;  // kMagic + code; the largest distance of a quotient from its code
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    float d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[e][j] = fmaf(v[e][j], inv, kMagic);
      d[j] = fmaf(v[e][j], inv, kMagic - c[e][j]);
    }
    far = max_abs(max_abs(far, d[0], d[1]), d[2], d[3]);
  }
  // Quotients next to a border: one bit each for rows as they are, which know their largest value; else noted for later,
  // with the elements that may be the largest (those that f32 cannot tell from it: silu 8 units each).
  uint32_t near = 0u;
  if (far > 0.5f - kBand<kKind>) {
#pragma unroll
    for (int e = 0; e < kE; ++e)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (fabsf(fmaf(v[e][j], inv, kMagic - c[e][j])) > 0.5f - kBand<kKind>) near |= 1u << (e * 4 + j);
  }
  auto place = [&](uint32_t bits) {
    const int b = __ffs(bits) - 1;
    return (b / 4 * kT + t) * 4 + b % 4;
  };
  if (kKind != kI8Rows) {
    for (; near; near &= near - 1) later.add(turn % kWindow, false, place(near));
    if (__float_as_uint(top) >= high - (kKind == kI8Silu ? 32u : 0u)) {
      uint32_t tops = 0u;
#pragma unroll
      for (int e = 0; e < kE; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (fabsf(c[e][j] - kMagic) > 126.f) tops |= 1u << (e * 4 + j);
      for (; tops; tops &= tops - 1) later.add(turn % kWindow, true, place(tops));
    }
  }
  float scale = m / 127.f;
  if (kKind == kI8Norm && m > 0.f) scale = m * (1.f / sqrtf(ss / n + a.eps)) / 127.f;
  int8_t* q = a.q + row * a.q_stride;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int i = (e * kT + t) * 4;
    if (i >= n) continue;
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(c[e][j]);
    if (kVec) {
      *reinterpret_cast<uint32_t*>(q + i) = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) q[i + j] = static_cast<int8_t>(b[j] & 0xFFu);
    }
  }
  if (t == 0) a.scale[row] = scale;
  if (kKind == kI8Rows) {
    for (; near; near &= near - 1) {
      const int i = place(near);
      q[i] = code_at_border(a.x[row * a.x_stride + i], m);
    }
  }
  }
  if (kKind != kI8Rows && turn) {
    const int64_t rows_left = (turn - 1) % kWindow + 1;
    settle<kKind, kT>(a, later, row - rows_left * step, step, t, sh_d);
  }
}

template <int kKind, int kT, int kE>
cudaError_t launch_rows(const I8RowsArgs& a, bool vec, cudaStream_t st) {
  using Cfg = RowsCfg<kKind, kT, kE>;
  const auto kernel = vec ? k_rows_i8<kKind, kT, kE, true> : k_rows_i8<kKind, kT, kE, false>;
  if (Cfg::smem > 40 * 1024) {  // (of 48 KB that need no leave, the rest is for what has a fixed place)
    static unsigned long long done[2] = {0, 0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Cfg::smem, &done[vec]);
    if (e != cudaSuccess) return e;
  }
  const int per = Cfg::block / kT, blocks = (a.rows + per - 1) / per, most = kSms * Cfg::ctas;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), Cfg::block, Cfg::smem, st, a);
}

template <int kKind>
cudaError_t launch_kind(const I8RowsArgs& a, cudaStream_t st) {
  auto on16 = [&](const float* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.rows == 1 || stride % 4 == 0);
  };
  const bool vec = a.n % 4 == 0 && on16(a.x, a.x_stride) && on16(a.other, a.other_stride) && on16(a.g, 0) &&
                   on16(a.sum, a.sum_stride) && reinterpret_cast<uintptr_t>(a.q) % 4 == 0 &&
                   (a.rows == 1 || a.q_stride % 4 == 0);
  // Few threads a row where that leaves an SM more rows under way, as a barrier of each row stands between its loads and
  // its codes; many where a row's elements would not fit the registers.  Measured (us, 8191 x 2048): 128 x 4 and 256 x 2
  // norm 39.1 and 45.4, SwiGLU 31.7 and 35.6, but rows as they are 17.3 and 15.0, which need few registers.  4099 x 4096,
  // 256 x 4 and 512 x 2: 39.4 and 54.6, 28.5 and 38.8, 16.3 and 15.8.  8192 x 1024, 128 x 2, 256 x 1 and 64 x 4: norm 23.4, 31.3 and
  // 22.1, SwiGLU 18.5, 23.9 and 20.2.  8192 x 512, 32 x 4 and 128 x 1: norm 12.2 and 16.5, SwiGLU 11.6 and 13.8, rows 6.0 and 6.7.
  if (a.n <= 128) return launch_rows<kKind, 32, 1>(a, vec, st);
  if (a.n <= 512) return launch_rows<kKind, 32, 4>(a, vec, st);
  if (a.n <= 1024) return launch_rows<kKind, 128, 2>(a, vec, st);
  if (a.n <= 2048) return launch_rows<kKind, kKind == kI8Rows ? 256 : 128, kKind == kI8Rows ? 2 : 4>(a, vec, st);
  if (a.n <= 4096) return launch_rows<kKind, 256, 4>(a, vec, st);
  if (a.n <= 8192) return launch_rows<kKind, 512, 4>(a, vec, st);
  return launch_rows<kKind, 1024, 4>(a, vec, st);
}

// The values that rows of codes stand for: four codes a thread and step, a block's 4096 codes from one row or several
// short ones (groups: of four codes a row; mul = floor(2^32 / groups) + 1, or 0 for one).
template <bool kVec>
__global__ void __launch_bounds__(256) k_rows_i8_read(const int8_t* q, int64_t q_stride, const float* scale, int64_t all,
                                                      int n, float* out, int64_t out_stride, int groups, uint32_t mul) {
  constexpr int kRead = 1024;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRead, row0 = first / groups;
  const int skip = static_cast<int>(first - row0 * groups);  // below 4096
  uint32_t w[kRead / 256];
  float s[kRead / 256];
#pragma unroll
  for (int k = 0; k < kRead / 256; ++k) {
    const int f = skip + k * 256 + static_cast<int>(threadIdx.x);
    const int r = mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(f), mul)) : f;
    const int64_t row = row0 + r;
    const int i = (f - r * groups) * 4;
    if (first + k * 256 + threadIdx.x >= all) continue;
    s[k] = __ldg(scale + row);
    const int8_t* src = q + row * q_stride + i;
    if (kVec) {
      w[k] = __ldg(reinterpret_cast<const uint32_t*>(src));
    } else {
      w[k] = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) w[k] |= static_cast<uint32_t>(static_cast<uint8_t>(src[j])) << (8 * j);
    }
  }
#pragma unroll
  for (int k = 0; k < kRead / 256; ++k) {
    const int f = skip + k * 256 + static_cast<int>(threadIdx.x);
    const int r = mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(f), mul)) : f;
    const int i = (f - r * groups) * 4;
    if (first + k * 256 + threadIdx.x >= all) continue;
    float* dst = out + (row0 + r) * out_stride + i;
    float v[4];
    i8x4_to_f32(w[k], v[0], v[1], v[2], v[3]);
    if (kVec) {
      *reinterpret_cast<float4*>(dst) = make_float4(v[0] * s[k], v[1] * s[k], v[2] * s[k], v[3] * s[k]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) dst[j] = v[j] * s[k];
    }
  }
}

}  // namespace

cudaError_t launch_rows_i8(int kind, const I8RowsArgs& a, cudaStream_t st) {
  if (kind == kI8Norm) return launch_kind<kI8Norm>(a, st);
  if (kind == kI8Silu) return launch_kind<kI8Silu>(a, st);
  return launch_kind<kI8Rows>(a, st);
}

cudaError_t launch_rows_i8_read(const int8_t* q, int64_t q_stride, const float* scale, int rows, int n, float* out,
                                int64_t out_stride, cudaStream_t st) {
  const bool vec = n % 4 == 0 && reinterpret_cast<uintptr_t>(q) % 4 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0 &&
                   (rows == 1 || (q_stride % 4 == 0 && out_stride % 4 == 0));
  const int groups = (n + 3) / 4;
  const int64_t all = static_cast<int64_t>(rows) * groups;
  const uint32_t mul = groups > 1 ? static_cast<uint32_t>((1ull << 32) / groups + 1) : 0u;
  return launch_pdl(vec ? k_rows_i8_read<true> : k_rows_i8_read<false>, dim3(static_cast<unsigned>((all + 1023) / 1024)), 256, 0, st,
                    q, q_stride, scale, all, n, out, out_stride, groups, mul);
}

}  // namespace tqd
