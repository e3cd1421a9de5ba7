// Rows of 8-bit codes: a row y of f32 values is held as one scale, max|y| / 127,
// and a code for each element, rint(127 y / max|y|).  Three kinds of row:
// y = x; the RMSNorm of x + other; silu(gate) * up.  And the way back.
//
// The codes are those of the exact values.  In f32 the quotient t = 127 y / max|y| is
// known to within kBand; where t lies that near to a border between two codes,
// and only there, it is taken again in f64, with the row's largest value in f64
// too (found among the elements whose code is 127 in magnitude).  A row whose
// largest value or sum of squares leaves the middle of the f32 range is done in
// f64 as a whole, so neither squares nor products overflow or vanish.  The norm's
// 1 / rms multiplies every element alike: it is in the scale and not in the codes.
#include <cuda_runtime.h>
#include <float.h>

#include "tqd_device.cuh"
#include "tqd_i8.cuh"
#include "tqd_internal.h"

namespace tqd {
namespace {

// The relative errors that reach t, in units of 2^-24, times 127: of y (exact for
// rows; the product h g, 1; expf 4, 1 + e, the quotient and the product with up 3), of the
// largest y the same, of 127 / max and of the product with it 1 each.  2 * 127 * 2^-24 =
// 2^-16, 4 * 127 * 2^-24 = 2^-15, 16 * 127 * 2^-24 = 2^-13.
template <int kKind>
constexpr float kBand = kKind == kI8Silu ? 0x1p-12f : 0x1p-14f;

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: added, it leaves the nearest whole number in the low bits

__device__ __forceinline__ float silu(float g) { return g / (1.f + expf(-g)); }

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

// Reductions over the kT threads of a row: one warp, or the whole block.
template <int kT>
struct RowGroup {
  static __device__ __forceinline__ uint32_t max_u32(uint32_t v, uint32_t* sh) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if (kT == 32) return v;
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh[0];
#pragma unroll
    for (int w = 1; w < kT / 32; ++w) v = max(v, sh[w]);
    return v;
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

// kT threads a row, kE groups of four elements a thread.  kVec: every row of every tensor
// begins on a 16-byte boundary (codes: 4) and is whole groups of four.
template <int kKind, int kT, int kE, bool kVec>
__global__ void __launch_bounds__(kT < 128 ? 128 : kT) k_rows_i8(const I8RowsArgs a) {
  __shared__ uint32_t sh_max[32];
  __shared__ float sh_sum[32];
  __shared__ double sh_d[32];
  const int t = threadIdx.x % kT;
  const int64_t row = kT < 128 ? static_cast<int64_t>(blockIdx.x) * (128 / kT) + threadIdx.x / kT : blockIdx.x;
  if (row >= a.rows) return;  // whole warps, of blocks without barriers
  const int n = a.n;
  const float* x = a.x + row * a.x_stride;
  const float* other = a.other ? a.other + row * a.other_stride : nullptr;

  float v[kE][4], w[kE][4];
#pragma unroll
  for (int e = 0; e < kE; ++e) load4<kVec>(x, (e * kT + t) * 4, n, v[e]);
  if (kKind == kI8Silu || (kKind == kI8Norm && other)) {
#pragma unroll
    for (int e = 0; e < kE; ++e) load4<kVec>(other, (e * kT + t) * 4, n, w[e]);
  }
  uint32_t top = 0u;  // the largest |y|, as bits: a NaN or an infinity is above all
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int i = (e * kT + t) * 4;
    if (kKind == kI8Silu) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[e][j] = silu(v[e][j]) * w[e][j];
    }
    if (kKind == kI8Norm) {
      if (other) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[e][j] += w[e][j];
      }
      if (a.sum) {
        float* s = a.sum + row * a.sum_stride + i;
        if (kVec) {
          if (i < n) *reinterpret_cast<float4*>(s) = make_float4(v[e][0], v[e][1], v[e][2], v[e][3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (i + j < n) s[j] = v[e][j];
        }
      }
      float g[4];
      load4<kVec>(a.g, i, n, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ss = fmaf(v[e][j], v[e][j], ss);
        v[e][j] *= g[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(v[e][j]) & 0x7FFFFFFFu);
  }
  if (kKind == kI8Norm) {
    ss = warp_sum(ss);
    if (kT > 32 && (threadIdx.x & 31) == 0) sh_sum[threadIdx.x >> 5] = ss;
  }
  const float m = __uint_as_float(RowGroup<kT>::max_u32(top, sh_max));
  if (kKind == kI8Norm && kT > 32) {
    ss = sh_sum[0];
#pragma unroll
    for (int i = 1; i < kT / 32; ++i) ss += sh_sum[i];
  }

  // (false for NaN; zeros of rows as they are need nothing)
  bool whole = !(m >= 0x1p-60f && m <= 0x1p60f);
  if (kKind == kI8Rows && m == 0.f) whole = false;
  if (kKind == kI8Norm) whole = whole || !(ss >= 0x1p-60f && ss <= 0x1p100f);
  float scale = m / 127.f;
  if (kKind == kI8Norm) scale = m * (1.f / sqrtf(ss / n + a.eps)) / 127.f;
  const float inv = m > 0.f ? 127.f / m : 0.f;
  uint32_t near = 0u;  // elements whose quotient is next to a border
#pragma unroll
  for (int e = 0; e < kE; ++e) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float q = v[e][j] * inv;
      v[e][j] = q + kMagic;
      if (fabsf(q - (v[e][j] - kMagic)) > 0.5f - kBand<kKind>) near |= 1u << (e * 4 + j);
    }
  }
  if (RowGroup<kT>::any(near != 0u || whole)) {
    double most = 0.0, squares = 0.0, h;
    bool lost = false;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = (e * kT + t) * 4 + j;
        if (i < n && (whole || fabsf(v[e][j] - kMagic) > 126.f)) {
          const double y = exact_element<kKind>(a, row, i, h);
          lost = lost || !(fabs(y) <= DBL_MAX);
          most = fmax(most, fabs(y));
          squares += h * h;
        }
      }
    }
    most = RowGroup<kT>::all(most, sh_d, [](double p, double q) { return fmax(p, q); });
    if (whole) {
      lost = RowGroup<kT>::any(lost);
      if (kKind == kI8Norm) {
        squares = RowGroup<kT>::all(squares, sh_d, [](double p, double q) { return p + q; });
        const double at = squares / n + a.eps;
        scale = at > 0.0 ? static_cast<float>(most / sqrt(at) / 127.0) : 0.f;
        if (at > 0.0 && !isfinite(static_cast<float>(most / sqrt(at)))) lost = true;
      } else {
        scale = static_cast<float>(most / 127.0);
        if (!isfinite(static_cast<float>(most))) lost = true;
      }
      if (lost) scale = __uint_as_float(0x7FC00000u);
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = (e * kT + t) * 4 + j;
        if (i < n && (whole || ((near >> (e * 4 + j)) & 1u))) {
          double c = 0.0;
          if (!lost && most > 0.0) c = rint(127.0 * exact_element<kKind>(a, row, i, h) / most);
          v[e][j] = static_cast<float>(c) + kMagic;
        }
      }
    }
  }
  int8_t* q = a.q + row * a.q_stride;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int i = (e * kT + t) * 4;
    if (i >= n) break;
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(v[e][j]);
    if (kVec) {
      *reinterpret_cast<uint32_t*>(q + i) = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) q[i + j] = static_cast<int8_t>(b[j] & 0xFFu);
    }
  }
  if (t == 0) a.scale[row] = scale;
}

template <int kKind, int kT, int kE>
cudaError_t launch_rows(const I8RowsArgs& a, bool vec, cudaStream_t st) {
  const unsigned per = kT < 128 ? 128 / kT : 1, grid = static_cast<unsigned>((a.rows + per - 1) / per);
  const unsigned block = kT < 128 ? 128 : kT;
  if (vec) k_rows_i8<kKind, kT, kE, true><<<grid, block, 0, st>>>(a);
  else k_rows_i8<kKind, kT, kE, false><<<grid, block, 0, st>>>(a);
  return cudaGetLastError();
}

template <int kKind>
cudaError_t launch_kind(const I8RowsArgs& a, cudaStream_t st) {
  auto on16 = [&](const float* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.rows == 1 || stride % 4 == 0);
  };
  const bool vec = a.n % 4 == 0 && on16(a.x, a.x_stride) && on16(a.other, a.other_stride) && on16(a.g, 0) &&
                   on16(a.sum, a.sum_stride) && reinterpret_cast<uintptr_t>(a.q) % 4 == 0 &&
                   (a.rows == 1 || a.q_stride % 4 == 0);
  if (a.n <= 1024 && a.rows > 1024) return launch_rows<kKind, 32, 8>(a, vec, st);
  if (a.n <= 2048) return launch_rows<kKind, 256, 2>(a, vec, st);
  if (a.n <= 4096) return launch_rows<kKind, 256, 4>(a, vec, st);
  if (a.n <= 8192) return launch_rows<kKind, 256, 8>(a, vec, st);
  return launch_rows<kKind, 512, 8>(a, vec, st);
}

// The values that rows of codes stand for: four a thread and step.
template <bool kVec>
__global__ void __launch_bounds__(256) k_rows_i8_read(const int8_t* q, int64_t q_stride, const float* scale, int rows,
                                                      int n, float* out, int64_t out_stride, int groups) {
  // blockIdx.x: kRead groups of four of one row
  constexpr int kRead = 1024;
  const int64_t row = blockIdx.x / groups;
  const int first = static_cast<int>(blockIdx.x - row * groups) * kRead;
  const float s = scale[row];
  const int8_t* src = q + row * q_stride;
  float* dst = out + row * out_stride;
#pragma unroll
  for (int k = 0; k < kRead / 256; ++k) {
    const int i = (first + k * 256 + static_cast<int>(threadIdx.x)) * 4;
    if (i >= n) continue;
    if (kVec) {
      float4 f;
      i8x4_to_f32(*reinterpret_cast<const uint32_t*>(src + i), f.x, f.y, f.z, f.w);
      *reinterpret_cast<float4*>(dst + i) = make_float4(f.x * s, f.y * s, f.z * s, f.w * s);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) dst[i + j] = src[i + j] * s;
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
  const int groups = (n + 4095) / 4096;
  const unsigned grid = static_cast<unsigned>(rows) * groups;
  if (vec) k_rows_i8_read<true><<<grid, 256, 0, st>>>(q, q_stride, scale, rows, n, out, out_stride, groups);
  else k_rows_i8_read<false><<<grid, 256, 0, st>>>(q, q_stride, scale, rows, n, out, out_stride, groups);
  return cudaGetLastError();
}

}  // namespace tqd
