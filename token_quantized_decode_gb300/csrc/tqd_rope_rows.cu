// Rotary positions for many tokens' heads at once: halves or neighbouring pairs,
// the whole head or its first part, angles from a table; and tables whose angles
// are scaled for long contexts.
#include <cuda_runtime.h>

#include "tqd_device.cuh"
#include "tqd_i8.cuh"
#include "tqd_internal.h"

namespace tqd {
namespace {

// f / d for f, d < 2^16: mul = floor(2^32 / d) + 1, or 0 for d = 1.
__device__ __forceinline__ int div_by(int f, uint32_t mul) {
  return mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(f), mul)) : f;
}

// kW neighbouring floats (of one 4 kW-byte load).
template <int kW>
struct Run;
template <>
struct Run<4> {
  using Type = float4;
};
template <>
struct Run<2> {
  using Type = float2;
};
template <>
struct Run<1> {
  using Type = float;
};
template <int kW>
__device__ __forceinline__ void get(float (&v)[kW], const float* p) {
  *reinterpret_cast<typename Run<kW>::Type*>(v) = *reinterpret_cast<const typename Run<kW>::Type*>(p);
}
template <int kW>
__device__ __forceinline__ void put(float* p, const float (&v)[kW]) {
  *reinterpret_cast<typename Run<kW>::Type*>(p) = *reinterpret_cast<const typename Run<kW>::Type*>(v);
}

// A unit is 2 kW elements of a head: two runs of kW that turn together (halves), neighbours, or what follows the rotated part
// (with kW = 1 one element of that).  A thread does one at a time, in few registers, so that an SM holds 2048 threads: that
// many 16-byte loads are under way (8191 tokens of 20 heads of 128: 28.3 us, 89 % of the copy rate; with four units a
// thread at once, half as many threads, 34.7).
template <int kW, bool kInter>
__global__ void __launch_bounds__(256, 8) k_rope_rows(const RopeRowsArgs a, int tokens, int units, int per_head,
                                                      uint32_t mul_units, uint32_t mul_head) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * tokens;
  const int all = static_cast<int>(min(static_cast<int64_t>(tokens), a.n - first)) * units, half = a.rotary / 2;
  for (int f = threadIdx.x; f < all; f += 256) {
    const int tok = div_by(f, mul_units), u = f - tok * units, head = div_by(u, mul_head), g = u - head * per_head;
    const bool turn = g * kW < half;
    if (!turn && a.out == a.x) continue;
    const int pos = __ldg(a.positions + first + tok);
    if (pos < 0 || pos >= a.max_pos) continue;
    // where the unit's two runs begin
    const int i0 = turn ? (kInter ? 2 : 1) * kW * g : kW == 1 ? half + g : 2 * kW * g;
    const int i1 = turn ? kInter ? i0 + kW : half + kW * g : kW == 1 ? i0 : i0 + kW;
    const float* src = a.x + (first + tok) * a.x_stride + head * a.head_dim;
    float* dst = a.out + (first + tok) * a.out_stride + head * a.head_dim;
    float p[kW], q[kW], r[kW], w[kW];
    get<kW>(p, src + i0);
    get<kW>(q, src + i1);
    if (turn) {
      const float* row = reinterpret_cast<const float*>(a.table + static_cast<int64_t>(pos) * half) + 2 * kW * g;
      float t[2 * kW];  // (cos, sin) of the unit's pairs
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float c[kW];
        get<kW>(c, row + h * kW);
#pragma unroll
        for (int i = 0; i < kW; ++i) t[h * kW + i] = c[i];
      }
      if (!kInter || kW == 1) {
#pragma unroll
        for (int i = 0; i < kW; ++i) {
          r[i] = p[i] * t[2 * i] - q[i] * t[2 * i + 1];
          w[i] = q[i] * t[2 * i] + p[i] * t[2 * i + 1];
        }
      } else {
#pragma unroll
        for (int i = 0; i + 1 < kW; i += 2) {
          r[i] = p[i] * t[i] - p[i + 1] * t[i + 1];
          r[i + 1] = p[i + 1] * t[i] + p[i] * t[i + 1];
          w[i] = q[i] * t[kW + i] - q[i + 1] * t[kW + i + 1];
          w[i + 1] = q[i + 1] * t[kW + i] + q[i] * t[kW + i + 1];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kW; ++i) r[i] = p[i], w[i] = q[i];
    }
    put<kW>(dst + i0, r);
    if (kW > 1 || turn) put<kW>(dst + i1, w);
  }
}

// A table is made once, when a program begins, and not tuned: every entry finds its frequency again, by pow in f64, and its
// sincos (40960 positions of 128: 0.66 ms unscaled, 0.84 by rotations, 1.47 by index; its bytes take 3 us).
__global__ void k_rope_table_scaled(double theta, int rotary, int64_t pairs, RopeScaling sc, float2* table) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (at >= pairs) return;
  const int half = rotary / 2, i = static_cast<int>(at % half);
  const int64_t p = at / half;
  double f = pow(theta, -static_cast<double>(i) / half);
  if (sc.kind == kRopeLinear) {
    f /= sc.factor;
  } else if (sc.kind == kRopeByRotations || sc.kind == kRopeByIndex) {
    constexpr double kTurn = 6.283185307179586;
    double keep;
    if (sc.kind == kRopeByRotations) {
      keep = (sc.original * f / kTurn - sc.low) / (sc.high - sc.low);
    } else {
      // the index whose pair turns r times over the original length
      auto index = [&](double r) { return rotary * log(sc.original / (r * kTurn)) / (2.0 * log(theta)); };
      const double from = fmax(floor(index(sc.high)), 0.0), to = fmin(ceil(index(sc.low)), rotary - 1.0);
      keep = 1.0 - (i - from) / (to > from ? to - from : 0.001);
    }
    keep = fmin(1.0, fmax(0.0, keep));
    f *= keep + (1.0 - keep) / sc.factor;
  }
  double s, c;
  sincos(p * f, &s, &c);
  table[at] = make_float2(static_cast<float>(c * sc.attention), static_cast<float>(s * sc.attention));
}

}  // namespace

cudaError_t launch_rope_table_scaled(double theta, int rotary, int max_pos, const RopeScaling& sc, float2* table,
                                     cudaStream_t st) {
  const int64_t pairs = static_cast<int64_t>(max_pos) * (rotary / 2);
  k_rope_table_scaled<<<static_cast<unsigned>((pairs + 255) / 256), 256, 0, st>>>(theta, rotary, pairs, sc, table);
  return cudaGetLastError();
}

cudaError_t launch_rope_rows(const RopeRowsArgs& a, bool interleaved, cudaStream_t st) {
  // the widest run that head sizes, strides and addresses allow
  auto fits = [&](int w) {
    auto on = [&](const float* p, int64_t stride) {
      return reinterpret_cast<uintptr_t>(p) % (4 * w) == 0 && (a.n == 1 || stride % w == 0);
    };
    return a.head_dim % (2 * w) == 0 && a.rotary % (2 * w) == 0 && on(a.x, a.x_stride) && on(a.out, a.out_stride) &&
           reinterpret_cast<uintptr_t>(a.table) % (4 * w) == 0;
  };
  const int w = fits(4) ? 4 : fits(2) ? 2 : 1;
  const int per_head = w > 1 ? a.head_dim / (2 * w) : a.rotary / 2 + (a.head_dim - a.rotary);
  const int units = a.heads * per_head;
  const int tokens = units >= 256 ? 1 : 256 / units;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.n) + tokens - 1) / tokens);  // (n: up to 2^31 - 1)
  auto mul = [](int d) { return d > 1 ? static_cast<uint32_t>((1ull << 32) / d + 1) : 0u; };
  const auto kernel = w == 4   ? interleaved ? k_rope_rows<4, true> : k_rope_rows<4, false>
                      : w == 2 ? interleaved ? k_rope_rows<2, true> : k_rope_rows<2, false>
                               : interleaved ? k_rope_rows<1, true> : k_rope_rows<1, false>;
  return launch_pdl(kernel, dim3(grid), 256, 0, st, a, tokens, units, per_head, mul(units), mul(per_head));
}

}  // namespace tqd
