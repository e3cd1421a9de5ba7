// Rows of 8-bit codes: arguments of the kernels that make and read them, and the
// codes as f16 operands.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace tqd {

enum { kI8Rows = 0, kI8Norm = 1, kI8Silu = 2 };

struct I8RowsArgs {
  const float* x;      // the rows; kI8Silu: the gate rows
  const float* other;  // kI8Norm: rows to add, or null; kI8Silu: the up rows
  const float* g;      // kI8Norm: gains
  float* sum;          // kI8Norm: x + other, or null
  int8_t* q;
  float* scale;
  int64_t x_stride, other_stride, sum_stride, q_stride;
  int rows, n;
  float eps;
};

enum { kRopeUnscaled = 0, kRopeLinear = 1, kRopeByRotations = 2, kRopeByIndex = 3 };
struct RopeScaling {
  int kind;
  double factor, original, low, high, attention;
};

struct RopeRowsArgs {
  const float* x;
  float* out;
  const int32_t* positions;
  const float2* table;
  int64_t x_stride, out_stride;
  int n, heads, head_dim, rotary, max_pos;
};

struct I8MatmulArgs {
  const int8_t* w;
  const float* w_scale;
  const int8_t* x;
  const float* x_scale;
  float* y;
  void* scratch;
  int64_t x_stride, y_stride;
  int rows, cols, n;
};

// How a product is made (tqd_i8_matmul_way in tqd.h).
struct I8Way {
  int kind, tokens, warps, cluster;
  int64_t tiles, rounds;
};
I8Way i8_matmul_way(int rows, int cols, int n);

// Four codes of a word as f16, exactly: a code's byte with its top bit turned is
// code + 128, and as the low byte of 0x64xx it makes 1024 + code + 128.  lo holds
// bytes 0 and 2, hi bytes 1 and 3; both operands of a product are taken apart in
// this way, so their columns meet.
__device__ __forceinline__ void i8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  const uint32_t a = (w & 0x00FF00FFu) ^ 0x64806480u, b = ((w >> 8) & 0x00FF00FFu) ^ 0x64806480u;
  const __half2 l = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&l);
  hi = *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace tqd
