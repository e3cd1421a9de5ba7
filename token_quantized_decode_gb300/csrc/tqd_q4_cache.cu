// Appending to and reading from the paged Q4 cache.
#include <cuda_runtime.h>

#include "tqd_internal.h"
#include "tqd_q4.cuh"

namespace tqd {
namespace {

// Address of the block holding position pos of sequence seq, head h; nullptr
// when the sequence, the position or the page lies outside the cache.
__device__ __forceinline__ uint8_t* q4_block_of(const Q4Cache& c, int seq, int pos, int h, int hd) {
  if (seq < 0 || seq >= c.n_seq || pos < 0) return nullptr;
  const int slot = pos / c.page_size;
  if (slot >= c.table_stride) return nullptr;
  const int page = c.table[static_cast<size_t>(seq) * c.table_stride + slot];
  if (page < 0 || page >= c.n_pages) return nullptr;
  const int in_page = pos - slot * c.page_size;
  return c.pages + static_cast<size_t>(page) * c.page_bytes +
         (static_cast<size_t>(h) * (c.page_size / kQ4Block) + in_page / kQ4Block) * q4_block_bytes(hd);
}

// One group of 32 (a lane's element each): the codes are rint(7 y / max|y|)
// and the scale f16(max|y| / 7) of the exact rotated values.
struct Q4Code {
  uint32_t code;   // 1..15 (8: zero)
  uint32_t scale;  // f16 bits, the same in every lane
};

__device__ __noinline__ Q4Code q4_code_exact(double y) {
  double a = fabs(y);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmax(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  Q4Code r;
  r.code = a > 0.0 ? static_cast<uint32_t>(__double2int_rn(7.0 * y / a) + 8) : 8u;
  const float d = __double2float_rn(a / 7.0);
  r.scale = d < 65520.f ? __half_as_ushort(__float2half_rn(d)) : 0x7E00u;
  return r;
}

// y: the lane's element in f32; e: |x0| + |x1| of the rotation that made it
// (0: y is exact).  exact(): the element in f64, called by whole warps only.
//
// The f32 rotation is off by at most 2^-23 e, so 7 y / max|y| by at most
// 2^-19 (M / max|y| + 1) with M the largest e of the group; where a code lies
// closer than that to the border between two, or the scale to the border
// between two f16, the group is coded again from f64.  That happens to about
// one group in 3,000; coding every group in f64 would bound the kernel by the
// f64 units (about two operations a clock per SM).
template <class F>
__device__ __forceinline__ Q4Code q4_code(float y, float e, F exact) {
  const float a = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(y))));
  const float M = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(e)));
  const float d = __fdiv_rn(a, 7.f);
  Q4Code r;
  // a NaN or an infinity in the group, or a scale past the f16 range: the
  // scale is NaN, so the group stands for NaN
  if (!(d < 65520.f)) {
    r.code = 8u;
    r.scale = 0x7E00u;
    return r;
  }
  const float rel = a > 0.f ? M / a : 0.f;
  const float t = y * __fdiv_rn(7.f, a);
  const float q = rintf(t);
  const float band = 1.9073486e-6f * (rel + 1.f);  // 2^-19
  const float slack = d * (2.3841858e-7f * (rel + 1.f));  // 2^-22
  bool unsure = fabsf(t - q) > 0.5f - band;
  if (M > 0.f) {
    const uint16_t lo = __half_as_ushort(__float2half_rn(d - slack)), hi = __half_as_ushort(__float2half_rn(d + slack));
    unsure |= lo != hi || rel > 256.f;
  }
  unsure |= a < 1e-30f && (a > 0.f || M > 0.f);
  if (__any_sync(0xFFFFFFFFu, unsure)) return q4_code_exact(exact());
  r.code = a > 0.f ? static_cast<uint32_t>(static_cast<int>(q) + 8) : 8u;
  r.scale = __half_as_ushort(__float2half_rn(d));
  return r;
}

struct AppendArgs {
  Q4Cache c;
  const float* k;
  const float* v;
  const float* q;
  float* q_out;
  int64_t k_stride, v_stride, q_stride, qo_stride;
  const int32_t* positions;
  const int32_t* seqs;
  const float2* rope;
  int n_tokens, n_heads, max_pos;
};

// One warp per (token, head): the first n_kv heads are the cache's (the key
// rotated, both rows coded and stored), the others rotate a query head.  A
// lane holds elements lane + 32 j, so a group of 32 is one element per lane
// and its maximum one redux instruction; loads are whole 128-byte lines
// whatever the rows' alignment.
template <int HD>
__global__ void __launch_bounds__(256) k_kv_append_q4(AppendArgs a) {
  constexpr int NG = HD / 32;
  const int lane = threadIdx.x & 31;
  const int per = a.c.n_kv + a.n_heads;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t token = task / per;
  if (token >= a.n_tokens) return;
  const int item = static_cast<int>(task - token * per);
  const int pos = a.positions[token];
  const int seq = a.seqs ? a.seqs[token] : static_cast<int>(token);
  if (pos < 0 || seq < 0 || seq >= a.c.n_seq || (a.rope && pos >= a.max_pos)) return;  // padding

  const bool is_kv = item < a.c.n_kv;
  const float* src = is_kv ? a.k + token * a.k_stride + static_cast<int64_t>(item) * HD
                           : a.q + token * a.q_stride + static_cast<int64_t>(item - a.c.n_kv) * HD;
  float x[NG], y[NG], cs[NG / 2], sn[NG / 2];
#pragma unroll
  for (int j = 0; j < NG; ++j) x[j] = src[lane + 32 * j];
#pragma unroll
  for (int j = 0; j < NG / 2; ++j) {
    const float2 w = a.rope ? a.rope[static_cast<size_t>(pos) * (HD / 2) + lane + 32 * j] : make_float2(1.f, 0.f);
    cs[j] = w.x;
    sn[j] = w.y;
    y[j] = a.rope ? fmaf(x[j], w.x, -__fmul_rn(x[j + NG / 2], w.y)) : x[j];
    y[j + NG / 2] = a.rope ? fmaf(x[j + NG / 2], w.x, __fmul_rn(x[j], w.y)) : x[j + NG / 2];
  }
  if (!is_kv) {
    float* dst = a.q_out + token * a.qo_stride + static_cast<int64_t>(item - a.c.n_kv) * HD;
#pragma unroll
    for (int j = 0; j < NG; ++j) dst[lane + 32 * j] = y[j];
    return;
  }
  const float* vsrc = a.v + token * a.v_stride + static_cast<int64_t>(item) * HD;
  float vx[NG];
#pragma unroll
  for (int j = 0; j < NG; ++j) vx[j] = vsrc[lane + 32 * j];
  uint8_t* blk = q4_block_of(a.c, seq, pos, item, HD);
  if (!blk) return;

  const int b = (pos % a.c.page_size) % kQ4Block;
  uint32_t kword = 0, ksc[2] = {0u, 0u}, vsc[2] = {0u, 0u}, vpiece[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    const int p = j % (NG / 2);
    const bool second = j >= NG / 2;
    const Q4Code kc = q4_code(y[j], a.rope ? fabsf(x[p]) + fabsf(x[p + NG / 2]) : 0.f, [&] {
      if (!a.rope) return static_cast<double>(x[j]);
      const double x0 = x[p], x1 = x[p + NG / 2], c = cs[p], s = sn[p];
      return second ? x1 * c + x0 * s : x0 * c - x1 * s;
    });
    // the eight codes of an octet of lanes into one word; lane i of the octet keeps group i's
    uint32_t w = kc.code << (4 * (lane & 7));
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 1);
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 2);
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 4);
    if ((lane & 7) == j) kword = w;
    ksc[j >> 1] |= kc.scale << (16 * (j & 1));

    const Q4Code vc = q4_code(vx[j], 0.f, [&] { return static_cast<double>(vx[j]); });
    // elements n, n + 8, n + 16, n + 24 of the group into 16 bits at lane n
    uint32_t u = vc.code << (4 * (lane >> 3));
    u |= __shfl_xor_sync(0xFFFFFFFFu, u, 8);
    u |= __shfl_xor_sync(0xFFFFFFFFu, u, 16);
    vpiece[j >> 1] |= u << (16 * (j & 1));
    vsc[j >> 1] |= vc.scale << (16 * (j & 1));
  }
  if ((lane & 7) < NG)
    *reinterpret_cast<uint32_t*>(blk + q4_k_row(b, HD) + (lane >> 3) * (4 * NG) + (lane & 7) * 4) = kword;
  if (HD == 128) {
    if (lane < 8) *reinterpret_cast<uint2*>(blk + q4_v_piece(b, lane, HD)) = make_uint2(vpiece[0], vpiece[1]);
    if (lane == 8) *reinterpret_cast<uint2*>(blk + q4_ks_off(HD) + b * 8) = make_uint2(ksc[0], ksc[1]);
    if (lane == 9) *reinterpret_cast<uint2*>(blk + q4_vs_off(HD) + b * 8) = make_uint2(vsc[0], vsc[1]);
  } else {
    if (lane < 8) *reinterpret_cast<uint32_t*>(blk + q4_v_piece(b, lane, HD)) = vpiece[0];
    if (lane == 8) *reinterpret_cast<uint32_t*>(blk + q4_ks_off(HD) + b * 4) = ksc[0];
    if (lane == 9) *reinterpret_cast<uint32_t*>(blk + q4_vs_off(HD) + b * 4) = vsc[0];
  }
}

struct ReadArgs {
  Q4Cache c;
  const int32_t* positions;
  const int32_t* seqs;
  float* k_out;
  float* v_out;
  int64_t k_stride, v_stride;
  int n_tokens;
};

// One warp per (token, kv head); a lane writes elements lane + 32 j.
template <int HD>
__global__ void __launch_bounds__(256) k_kv_read_q4(ReadArgs a) {
  constexpr int NG = HD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t token = task / a.c.n_kv;
  if (token >= a.n_tokens) return;
  const int h = static_cast<int>(task - token * a.c.n_kv);
  const int pos = a.positions[token];
  const int seq = a.seqs ? a.seqs[token] : static_cast<int>(token);
  const uint8_t* blk = q4_block_of(a.c, seq, pos, h, HD);
  const float nan = __int_as_float(0x7FC00000);
  const int b = pos >= 0 ? (pos % a.c.page_size) % kQ4Block : 0;
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    float kv = nan, vv = nan;
    if (blk) {
      const uint32_t kb = blk[q4_k_row(b, HD) + (lane >> 3) * (4 * NG) + j * 4 + ((lane & 7) >> 1)];
      const uint32_t vb = blk[q4_v_piece(b, lane & 7, HD) + 2 * j + (lane >> 4)];
      const __half ks = *reinterpret_cast<const __half*>(blk + q4_ks_off(HD) + (b * NG + j) * 2);
      const __half vs = *reinterpret_cast<const __half*>(blk + q4_vs_off(HD) + (b * NG + j) * 2);
      kv = static_cast<float>(static_cast<int>((kb >> (4 * (lane & 1))) & 15u) - 8) * __half2float(ks);
      vv = static_cast<float>(static_cast<int>((vb >> (4 * ((lane >> 3) & 1))) & 15u) - 8) * __half2float(vs);
    }
    if (a.k_out) a.k_out[token * a.k_stride + static_cast<int64_t>(h) * HD + lane + 32 * j] = kv;
    if (a.v_out) a.v_out[token * a.v_stride + static_cast<int64_t>(h) * HD + lane + 32 * j] = vv;
  }
}

}  // namespace

cudaError_t allow_smem(const void* kernel, size_t bytes, unsigned long long* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (__atomic_load_n(done, __ATOMIC_RELAXED) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && dev < 64) __atomic_fetch_or(done, bit, __ATOMIC_RELAXED);
  return e;
}

cudaError_t launch_kv_append_q4(const Q4Cache& c, int hd, const float* k, int64_t k_stride, const float* v,
                                int64_t v_stride, const int32_t* positions, const int32_t* seqs, int n_tokens,
                                const float2* rope, int max_pos, const float* q, int64_t q_stride, int n_heads,
                                float* q_out, int64_t qo_stride, cudaStream_t st) {
  AppendArgs a{c, k, v, q, q_out, k_stride, v_stride, q_stride, qo_stride, positions, seqs, rope, n_tokens, n_heads,
               max_pos};
  const int64_t warps = static_cast<int64_t>(n_tokens) * (c.n_kv + n_heads);
  const unsigned blocks = static_cast<unsigned>((warps + 7) / 8);
  if (hd == 128)
    k_kv_append_q4<128><<<blocks, 256, 0, st>>>(a);
  else
    k_kv_append_q4<64><<<blocks, 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_read_q4(const Q4Cache& c, int hd, const int32_t* positions, const int32_t* seqs, int n_tokens,
                              float* k_out, int64_t k_stride, float* v_out, int64_t v_stride, cudaStream_t st) {
  ReadArgs a{c, positions, seqs, k_out, v_out, k_stride, v_stride, n_tokens};
  const int64_t warps = static_cast<int64_t>(n_tokens) * c.n_kv;
  const unsigned blocks = static_cast<unsigned>((warps + 7) / 8);
  if (hd == 128)
    k_kv_read_q4<128><<<blocks, 256, 0, st>>>(a);
  else
    k_kv_read_q4<64><<<blocks, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace tqd
