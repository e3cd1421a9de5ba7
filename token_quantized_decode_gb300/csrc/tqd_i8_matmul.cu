// Products of int8 matrices with a scale for each token and each channel:
// y[j][r] = x_scale[j] w_scale[r] sum_c x[j][c] w[r][c].
//
// The sums are exact.  The int8 tensor instructions of this part run at a sixteenth of the
// f16 ones' rate, so codes become f16 operands (exact), products are exact in the f32
// accumulator, and so are sums of up to 1024 of them (128 * 128 * 1024 = 2^24); a run of
// at most 1024 columns is added to a 32-bit whole number.  So the order of the sums, and how
// they are split, changes nothing.
#include <cuda_runtime.h>

#include "tqd_device.cuh"
#include "tqd_i8.cuh"
#include "tqd_internal.h"

namespace tqd {
namespace {

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- few tokens
//
// The weights pass once through registers: a warp takes 16 rows, lane (g, c) = (lane / 4,
// lane % 4) sixteen bytes of rows g and g + 8, which are its share of four 16 x 16
// operands (the columns' order within a unit of 64 does not matter, as long as both operands have
// the same).  The tokens' codes stand in shared memory as f16 operands, per unit and eight
// tokens 1 KB.  kw warps share 16 rows, each with every kw-th pair of units.
constexpr int kFewWarps = 8;
constexpr int kFewCtas = 304;         // two an SM
constexpr int kFewStage = 64 * 1024;  // bytes of operands in shared memory

template <int kNT>
__global__ void __launch_bounds__(32 * kFewWarps, 2) k_i8_few(const I8MatmulArgs a, int kw, int groups) {
  extern __shared__ uint4 xs[];                 // [unit][tile of 8][2][lane]
  __shared__ int sums[kFewWarps][kNT * 4][32];  // of the warps that share rows
  constexpr int kUnits = kFewStage / (kNT * 1024);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int units = (a.cols + 63) / 64, share = kFewWarps / kw, part = warp % kw;
  const int j0 = blockIdx.y * (kNT * 8);

  for (int group = blockIdx.x; group < groups; group += gridDim.x) {
    const int r0 = (group * share + warp / kw) * 16 + g;
    const int8_t* w0 = a.w + static_cast<int64_t>(min(r0, a.rows - 1)) * a.cols + c * 16;
    const int8_t* w1 = a.w + static_cast<int64_t>(min(r0 + 8, a.rows - 1)) * a.cols + c * 16;
    int total[kNT][4];
    float acc[kNT][4];
#pragma unroll
    for (int t = 0; t < kNT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[t][i] = 0, acc[t][i] = 0.f;
    int run = 0;  // units in acc

    uint4 now[2][2], next[2][2];  // [unit][row]
    auto load = [&](uint4(&v)[2][2], int u) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool in = (u + k) * 64 + c * 16 < a.cols;
        v[k][0] = in ? ld_weights16(w0 + (u + k) * 64) : make_uint4(0u, 0u, 0u, 0u);
        v[k][1] = in ? ld_weights16(w1 + (u + k) * 64) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    load(now, 2 * part);
    for (int u0 = 0; u0 < units; u0 += kUnits) {
      const int here = min(kUnits, units - u0);
      if (units > kUnits || group == static_cast<int>(blockIdx.x)) {
        __syncthreads();
        for (int i = threadIdx.x; i < here * kNT * 32; i += 32 * kFewWarps) {
          const int l = i & 31, t = (i >> 5) % kNT, u = (i >> 5) / kNT;
          const int j = j0 + t * 8 + (l >> 2), col = (u0 + u) * 64 + (l & 3) * 16;
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (j < a.n && col < a.cols) v = *reinterpret_cast<const uint4*>(a.x + j * a.x_stride + col);
          uint4 p, q;
          i8x4_to_f16(v.x, p.x, p.y);
          i8x4_to_f16(v.y, p.z, p.w);
          i8x4_to_f16(v.z, q.x, q.y);
          i8x4_to_f16(v.w, q.z, q.w);
          xs[(u * kNT + t) * 64 + l] = p;
          xs[(u * kNT + t) * 64 + 32 + l] = q;
        }
        __syncthreads();
      }
      for (int u = 2 * part; u < here; u += 2 * kw) {
        // the next pair of units, which may be of the next stage
        load(next, u + 2 * kw < kUnits ? u0 + u + 2 * kw : u0 + kUnits + 2 * part);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (u + k < here) {
            const uint32_t r0w[4] = {now[k][0].x, now[k][0].y, now[k][0].z, now[k][0].w};
            const uint32_t r1w[4] = {now[k][1].x, now[k][1].y, now[k][1].z, now[k][1].w};
            uint32_t op[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              i8x4_to_f16(r0w[i], op[i][0], op[i][2]);
              i8x4_to_f16(r1w[i], op[i][1], op[i][3]);
            }
#pragma unroll
            for (int t = 0; t < kNT; ++t) {
              const uint4 p = xs[((u + k) * kNT + t) * 64 + lane], q = xs[((u + k) * kNT + t) * 64 + 32 + lane];
              mma16816(acc[t], op[0], p.x, p.y);
              mma16816(acc[t], op[1], p.z, p.w);
              mma16816(acc[t], op[2], q.x, q.y);
              mma16816(acc[t], op[3], q.z, q.w);
            }
          }
        }
        run += 2;
        if (run == 16) {
          run = 0;
#pragma unroll
          for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) total[t][i] += __float2int_rn(acc[t][i]), acc[t][i] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) now[k][0] = next[k][0], now[k][1] = next[k][1];
      }
    }
#pragma unroll
    for (int t = 0; t < kNT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[t][i] += __float2int_rn(acc[t][i]);
    if (kw > 1) {
      __syncthreads();
#pragma unroll
      for (int t = 0; t < kNT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[warp][t * 4 + i][lane] = total[t][i];
      __syncthreads();
    }
    // warp `part` of those that share rows writes every kw-th of their sums
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (kw > 1 && (t * 4 + i) % kw != part) continue;
        int s = total[t][i];
        if (kw > 1) {
          s = 0;
          for (int w = warp - part; w < warp - part + kw; ++w) s += sums[w][t * 4 + i][lane];
        }
        const int r = r0 + (i >> 1) * 8, j = j0 + t * 8 + 2 * c + (i & 1);
        if (r < a.rows && j < a.n)
          a.y[j * a.y_stride + r] = static_cast<float>(s) * a.x_scale[j] * a.w_scale[r];
      }
    }
  }
}

template <int kNT>
cudaError_t launch_few(const I8MatmulArgs& a, cudaStream_t st) {
  static unsigned long long done = 0;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_i8_few<kNT>), kFewStage, &done);
  if (e != cudaSuccess) return e;
  // how many warps share 16 rows: what makes the busiest CTA's share least
  const int tiles = (a.rows + 15) / 16, pairs = (a.cols + 127) / 128, blocks = (a.n + kNT * 8 - 1) / (kNT * 8);
  int kw = 1, groups = 0;
  int64_t best = -1;
  for (int k = 1; k <= kFewWarps; k *= 2) {
    const int gr = (tiles + kFewWarps / k - 1) / (kFewWarps / k);
    const int64_t waves = (static_cast<int64_t>(gr) * blocks + kFewCtas - 1) / kFewCtas;
    const int64_t cost = waves * ((pairs + k - 1) / k + 1);
    if (best < 0 || cost < best) best = cost, kw = k, groups = gr;
  }
  const int units = (a.cols + 63) / 64;
  const size_t smem = units * kNT * 1024 < kFewStage ? units * kNT * 1024 : kFewStage;
  const dim3 grid(static_cast<unsigned>(groups < kFewCtas ? groups : kFewCtas), static_cast<unsigned>(blocks));
  k_i8_few<kNT><<<grid, 32 * kFewWarps, smem, st>>>(a, kw, groups);
  return cudaGetLastError();
}

}  // namespace

size_t i8_matmul_scratch_bytes(int rows, int cols, int n) { return 0; }

cudaError_t launch_i8_matmul(const I8MatmulArgs& a, cudaStream_t st) {
  if (a.n <= 8) return launch_few<1>(a, st);
  if (a.n <= 16) return launch_few<2>(a, st);
  return launch_few<4>(a, st);
}

}  // namespace tqd
