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

// A unit is eight elements of a head (kVec) or two: two runs of four that turn
// together (halves), eight neighbours, or what follows the rotated part.  Without
// kVec: one pair, or one element of the rest.  A block does `tokens` tokens' units,
// four a thread at a time, so that their loads are under way together.
template <bool kVec, bool kInter>
__global__ void __launch_bounds__(256) k_rope_rows(const RopeRowsArgs a, int tokens, int units, int per_head,
                                                   uint32_t mul_units, uint32_t mul_head) {
  constexpr int kAt = 4;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * tokens;
  const int here = static_cast<int>(min(static_cast<int64_t>(tokens), a.n - first));
  const int all = here * units, half = a.rotary / 2;
  const bool copies = a.out != a.x;
  for (int f0 = threadIdx.x; f0 < all; f0 += 256 * kAt) {
    const float *src[kAt], *row[kAt];
    float* dst[kAt];
    int i0[kAt], i1[kAt];
    bool turn[kAt];
#pragma unroll
    for (int k = 0; k < kAt; ++k) {
      const int f = f0 + k * 256;
      src[k] = nullptr, row[k] = nullptr, dst[k] = nullptr, turn[k] = false, i0[k] = i1[k] = 0;
      if (f >= all) continue;
      const int tok = div_by(f, mul_units), u = f - tok * units, head = div_by(u, mul_head), g = u - head * per_head;
      const int pos = a.positions[first + tok];
      if (pos < 0 || pos >= a.max_pos) continue;
      turn[k] = g < (kVec ? a.rotary / 8 : half);
      if (!turn[k] && !copies) continue;
      src[k] = a.x + (first + tok) * a.x_stride + static_cast<int64_t>(head) * a.head_dim;
      dst[k] = a.out + (first + tok) * a.out_stride + static_cast<int64_t>(head) * a.head_dim;
      if (kVec) {
        i0[k] = turn[k] && !kInter ? 4 * g : 8 * g;
        i1[k] = turn[k] && !kInter ? half + 4 * g : 8 * g + 4;
      } else {
        i0[k] = turn[k] ? (kInter ? 2 * g : g) : half + g;
        i1[k] = turn[k] ? (kInter ? 2 * g + 1 : half + g) : i0[k];
      }
      // (cos, sin) of the unit's pairs
      row[k] = reinterpret_cast<const float*>(a.table + static_cast<int64_t>(pos) * half) + (kVec ? 8 : 2) * g;
    }
    if (kVec) {
      float4 p[kAt], q[kAt], c[kAt], s[kAt];
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
        if (!dst[k]) continue;
        p[k] = *reinterpret_cast<const float4*>(src[k] + i0[k]);
        q[k] = *reinterpret_cast<const float4*>(src[k] + i1[k]);
        if (turn[k]) {
          c[k] = __ldg(reinterpret_cast<const float4*>(row[k]));
          s[k] = __ldg(reinterpret_cast<const float4*>(row[k]) + 1);
        }
      }
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
        if (!dst[k]) continue;
        float4 u = p[k], w = q[k];
        if (turn[k] && !kInter) {
          u = make_float4(p[k].x * c[k].x - q[k].x * c[k].y, p[k].y * c[k].z - q[k].y * c[k].w,
                          p[k].z * s[k].x - q[k].z * s[k].y, p[k].w * s[k].z - q[k].w * s[k].w);
          w = make_float4(q[k].x * c[k].x + p[k].x * c[k].y, q[k].y * c[k].z + p[k].y * c[k].w,
                          q[k].z * s[k].x + p[k].z * s[k].y, q[k].w * s[k].z + p[k].w * s[k].w);
        } else if (turn[k]) {
          u = make_float4(p[k].x * c[k].x - p[k].y * c[k].y, p[k].y * c[k].x + p[k].x * c[k].y,
                          p[k].z * c[k].z - p[k].w * c[k].w, p[k].w * c[k].z + p[k].z * c[k].w);
          w = make_float4(q[k].x * s[k].x - q[k].y * s[k].y, q[k].y * s[k].x + q[k].x * s[k].y,
                          q[k].z * s[k].z - q[k].w * s[k].w, q[k].w * s[k].z + q[k].z * s[k].w);
        }
        *reinterpret_cast<float4*>(dst[k] + i0[k]) = u;
        *reinterpret_cast<float4*>(dst[k] + i1[k]) = w;
      }
    } else {
      float p[kAt], q[kAt], c[kAt], s[kAt];
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
        if (!dst[k]) continue;
        p[k] = src[k][i0[k]];
        q[k] = src[k][i1[k]];
        if (turn[k]) c[k] = __ldg(row[k]), s[k] = __ldg(row[k] + 1);
      }
#pragma unroll
      for (int k = 0; k < kAt; ++k) {
        if (!dst[k]) continue;
        dst[k][i0[k]] = turn[k] ? p[k] * c[k] - q[k] * s[k] : p[k];
        if (turn[k]) dst[k][i1[k]] = q[k] * c[k] + p[k] * s[k];
      }
    }
  }
}

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
  auto on16 = [&](const float* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.n == 1 || stride % 4 == 0);
  };
  const bool vec = a.head_dim % 8 == 0 && a.rotary % 8 == 0 && on16(a.x, a.x_stride) && on16(a.out, a.out_stride) &&
                   reinterpret_cast<uintptr_t>(a.table) % 16 == 0;
  const int per_head = vec ? a.head_dim / 8 : a.rotary / 2 + (a.head_dim - a.rotary);
  const int units = a.heads * per_head;
  const int tokens = units >= 1024 ? 1 : 1024 / units;
  const unsigned grid = static_cast<unsigned>((a.n + tokens - 1) / tokens);
  auto mul = [](int d) { return d > 1 ? static_cast<uint32_t>((1ull << 32) / d + 1) : 0u; };
  const auto kernel = vec ? interleaved ? k_rope_rows<true, true> : k_rope_rows<true, false>
                          : interleaved ? k_rope_rows<false, true> : k_rope_rows<false, false>;
  return launch_pdl(kernel, dim3(grid), 256, 0, st, a, tokens, units, per_head, mul(units), mul(per_head));
}

}  // namespace tqd
