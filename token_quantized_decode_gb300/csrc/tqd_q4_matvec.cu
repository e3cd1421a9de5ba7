// Matrix-vector products with Q4_0 weights (4-bit codes, one f16 scale per
// 32 columns).
#include <cuda_runtime.h>

#include "tqd_internal.h"
#include "tqd_q4.cuh"

namespace tqd {
namespace {

// One thread per 32-bit word of a tile's codes or scales.
__global__ void __launch_bounds__(288) k_q4_repack(const uint8_t* src, int64_t rows, int64_t groups, int64_t strips,
                                                   uint8_t* dst) {
  const int64_t tile = blockIdx.x, rt = tile / strips, st = tile - rt * strips;
  const int w = threadIdx.x;  // 256 words of codes, 32 of scales
  uint32_t word;
  if (w < 256) {
    const int g = w & 3, c = (w >> 2) & 3, row = (w >> 4);  // row: half * 8 + r
    const int64_t r = rt * 16 + row, grp = st * 4 + g;
    word = 0x88888888u;
    if (r < rows && grp < groups) {
      const uint8_t* b = src + (r * groups + grp) * 18 + 2;
      word = 0u;
      for (int i = 0; i < 8; ++i) {
        const int e = 8 * c + i;
        word |= ((static_cast<uint32_t>(b[e & 15]) >> (e < 16 ? 0 : 4)) & 15u) << (4 * i);
      }
    }
  } else {
    word = 0u;
    for (int i = 0; i < 2; ++i) {
      const int e = (w - 256) * 2 + i;
      const int64_t r = rt * 16 + e / 4, grp = st * 4 + e % 4;
      if (r < rows && grp < groups) {
        const uint8_t* b = src + (r * groups + grp) * 18;
        word |= (static_cast<uint32_t>(b[0]) | (static_cast<uint32_t>(b[1]) << 8)) << (16 * i);
      }
    }
  }
  reinterpret_cast<uint32_t*>(dst + tile * kQ4TileBytes)[w] = word;
}

// One warp per (row, vector).
__global__ void __launch_bounds__(256) k_q4_matvec(const uint8_t* w, int rows, int cols, int strips, const float* x,
                                                   int64_t x_stride, int n, float* y, int64_t y_stride) {
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t row = task / n;
  if (row >= rows) return;
  const int vec = static_cast<int>(task - row * n);
  const int r = static_cast<int>(row & 15);
  float s = 0.f;
  for (int g = 0; g < cols / 32; ++g) {
    const uint8_t* tile = w + (row / 16 * strips + g / 4) * kQ4TileBytes;
    const uint32_t word = reinterpret_cast<const uint32_t*>(tile)[r * 16 + (lane >> 3) * 4 + (g & 3)];
    const float d = __half2float(reinterpret_cast<const __half*>(tile + kQ4TileScales)[r * 4 + (g & 3)]);
    const float q = static_cast<float>(static_cast<int>((word >> (4 * (lane & 7))) & 15u) - 8);
    s += q * d * x[vec * x_stride + g * 32 + lane];
  }
  s = warp_sum(s);
  if (lane == 0) y[vec * y_stride + row] = s;
}

}  // namespace

cudaError_t launch_q4_repack(const uint8_t* src, int64_t rows, int64_t cols, uint8_t* dst, cudaStream_t st) {
  const int64_t strips = (cols + kQ4TileCols - 1) / kQ4TileCols;
  const int64_t tiles = (rows + kQ4TileRows - 1) / kQ4TileRows * strips;
  k_q4_repack<<<static_cast<unsigned>(tiles), 288, 0, st>>>(src, rows, cols / 32, strips, dst);
  return cudaGetLastError();
}

cudaError_t launch_q4_matvec(const uint8_t* w, int rows, int cols, const float* x, int n, int64_t x_stride, float* y,
                             int64_t y_stride, cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(rows) * n;
  k_q4_matvec<<<static_cast<unsigned>((warps + 7) / 8), 256, 0, st>>>(w, rows, cols, (cols + 127) / 128, x, x_stride, n,
                                                                      y, y_stride);
  return cudaGetLastError();
}

}  // namespace tqd
