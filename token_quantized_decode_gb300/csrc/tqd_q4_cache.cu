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
  // (a page is a multiple of 16 positions: the position in its block is pos % 16)
  return c.pages + static_cast<size_t>(page) * c.page_bytes +
         (static_cast<size_t>(h) * (c.page_size / kQ4Block) + in_page / kQ4Block) * q4_block_bytes(hd);
}

// Codes and scale of one group of 32, a lane's element each: rint(7 y / max|y|)
// + 8 and f16(max|y| / 7) of the exact values.
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

// The same in f32, and whether the result is sure.  M: the group's largest
// |x0| + |x1| of the rotation that made y (0: y is exact).
//
// The f32 rotation is off by at most 2^-23 M, so 7 y / max|y| by at most
// 2^-19 (M / max|y| + 1), the approximate reciprocal's 2^-23 included; where a
// code lies closer than that to the border between two, or the scale to the
// border between two f16, the group is coded again from f64.  That happens to
// about one group in 2,000; coding every group in f64 would bound the kernel by
// the f64 units (about two operations a clock per SM).
__device__ __forceinline__ Q4Code q4_code(float y, float M, bool& unsure) {
  const float a = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(y))));
  // a / 7 rounded: one step from a times the nearest f32 to 1 / 7
  float d = a * 0.14285715f;
  d = fmaf(fmaf(-7.f, d, a), 0.14285715f, d);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(a));
  const float rel = M * inv;
  const float t = y * (7.f * inv);
  const float q = rintf(t);
  Q4Code r;
  const __half h = __float2half_rn(d);
  r.scale = __half_as_ushort(h);
  r.code = static_cast<uint32_t>(static_cast<int>(q) + 8);
  unsure = fabsf(t - q) > fmaf(rel, -1.9073486e-6f, 0.49999809f);  // 1/2 - 2^-19 (rel + 1)
  if (M > 0.f) {
    const float slack = d * fmaf(rel, 2.3841858e-7f, 2.3841858e-7f);  // 2^-22
    unsure |= __half_as_ushort(__float2half_rn(d - slack)) != __half_as_ushort(__float2half_rn(d + slack)) || rel > 256.f;
  }
  if (!(a > 1e-30f && d < 65520.f)) {
    // All 0; so small that the steps above lose bits; or a NaN or an infinity
    // in the group, or a scale past the f16 range: the scale is NaN, so the
    // group stands for NaN.
    unsure = d < 65520.f && (a > 0.f || M > 0.f);
    r.code = 8u;
    r.scale = d < 65520.f ? 0u : 0x7E00u;
  }
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

// One warp per (token, kv head): it rotates that head's key and its share of the
// query heads, and codes and stores the key and the value.  A lane holds
// elements lane + 32 j, so a group of 32 is one element per lane and its maximum
// one redux instruction; loads are whole 128-byte lines whatever the rows'
// alignment.  All rows are loaded before the first is used: the kernel is bound
// by that latency for a few tokens and by instructions for many (a row of K and V costs
// about 450).
template <int HD>
__global__ void __launch_bounds__(256) k_kv_append_q4(AppendArgs a) {
  constexpr int NG = HD / 32;
  const int lane = threadIdx.x & 31;
  const unsigned task = blockIdx.x * 8 + (threadIdx.x >> 5);  // (at most 2^30)
  const unsigned token = task / static_cast<unsigned>(a.c.n_kv);
  pdl_wait();
  pdl_launch_dependents();
  if (token >= static_cast<unsigned>(a.n_tokens)) return;
  const int item = static_cast<int>(task - token * a.c.n_kv);
  const int pos = a.positions[token];
  const int seq = a.seqs ? a.seqs[token] : static_cast<int>(token);
  const float* ksrc = a.k + token * a.k_stride + item * HD + lane;
  const float* vsrc = a.v + token * a.v_stride + item * HD + lane;
  float x[NG], y[NG], vx[NG], cs[NG / 2], sn[NG / 2];
#pragma unroll
  for (int j = 0; j < NG; ++j) x[j] = ksrc[32 * j];
#pragma unroll
  for (int j = 0; j < NG; ++j) vx[j] = vsrc[32 * j];
  if (pos < 0 || seq < 0 || seq >= a.c.n_seq || (a.rope && pos >= a.max_pos)) return;  // padding
#pragma unroll
  for (int j = 0; j < NG / 2; ++j) {
    const float2 w = a.rope ? a.rope[static_cast<size_t>(pos) * (HD / 2) + lane + 32 * j] : make_float2(1.f, 0.f);
    cs[j] = w.x;
    sn[j] = w.y;
  }
  auto rotate = [&](const float (&in)[NG], float (&out)[NG]) {
#pragma unroll
    for (int j = 0; j < NG / 2; ++j) {
      out[j] = a.rope ? fmaf(in[j], cs[j], -__fmul_rn(in[j + NG / 2], sn[j])) : in[j];
      out[j + NG / 2] = a.rope ? fmaf(in[j + NG / 2], cs[j], __fmul_rn(in[j], sn[j])) : in[j + NG / 2];
    }
  };
  uint8_t* blk = q4_block_of(a.c, seq, pos, item, HD);
  for (int h = item; h < a.n_heads; h += 2 * a.c.n_kv) {  // two query heads at a time
    const bool two = h + a.c.n_kv < a.n_heads;
    const float* q = a.q + token * a.q_stride + static_cast<int64_t>(h) * HD + lane;
    float* o = a.q_out + token * a.qo_stride + static_cast<int64_t>(h) * HD + lane;
    const int64_t next = static_cast<int64_t>(a.c.n_kv) * HD;
    float q0[NG], q1[NG], r[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) q0[j] = q[32 * j];
    if (two)
#pragma unroll
      for (int j = 0; j < NG; ++j) q1[j] = q[next + 32 * j];
    rotate(q0, r);
#pragma unroll
    for (int j = 0; j < NG; ++j) o[32 * j] = r[j];
    if (two) {
      rotate(q1, r);
#pragma unroll
      for (int j = 0; j < NG; ++j) o[next + 32 * j] = r[j];
    }
  }
  rotate(x, y);
  if (!blk) return;

  const int b = pos % kQ4Block;
  uint32_t kcode[NG], vcode[NG], ksc[NG], vsc[NG], again = 0;
  float M[NG / 2];
#pragma unroll
  for (int p = 0; p < NG / 2; ++p)
    M[p] = a.rope ? __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(x[p]) + fabsf(x[p + NG / 2]))))
                  : 0.f;
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    bool unsure;
    const Q4Code kc = q4_code(y[j], M[j % (NG / 2)], unsure);
    kcode[j] = kc.code;
    ksc[j] = kc.scale;
    again |= unsure ? 1u << j : 0u;
    const Q4Code vc = q4_code(vx[j], 0.f, unsure);
    vcode[j] = vc.code;
    vsc[j] = vc.scale;
    again |= unsure ? 256u << j : 0u;
  }
  again = __reduce_or_sync(0xFFFFFFFFu, again);
  if (again) {
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      if (again >> j & 1u) {
        const int p = j % (NG / 2);
        const double x0 = x[p], x1 = x[p + NG / 2], c = cs[p], s = sn[p];
        const Q4Code r = q4_code_exact(!a.rope ? static_cast<double>(x[j]) : j < NG / 2 ? x0 * c - x1 * s : x1 * c + x0 * s);
        kcode[j] = r.code;
        ksc[j] = r.scale;
      }
      if (again >> j & 256u) {
        const Q4Code r = q4_code_exact(static_cast<double>(vx[j]));
        vcode[j] = r.code;
        vsc[j] = r.scale;
      }
    }
  }

  // K: an octet's eight codes of a group are a word.  In three exchanges each
  // lane gives away the groups that its partner keeps and ends with one group's word.
  const bool l2 = lane & 2, l4 = lane & 4;
  uint32_t kword;
  {
    uint32_t u = 0;  // byte g: codes of lanes 2 i, 2 i + 1 of group g
#pragma unroll
    for (int j = 0; j < NG; ++j) u |= kcode[j] << (8 * j + 4 * (lane & 1));
    u |= __shfl_xor_sync(0xFFFFFFFFu, u, 1);
    if constexpr (NG == 4) {
      // lane bit 1 keeps groups 2, 3 or 0, 1; then bit 2 keeps the odd or the even one
      uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, l2 ? u : u >> 16, 2) & 0xFFFFu;
      const uint32_t mine = l2 ? u >> 16 : u & 0xFFFFu;
      // halves: codes of the quad for the lower and the higher group kept
      const uint32_t lo4 = l2 ? got : mine, hi4 = l2 ? mine : got;  // lanes 0, 1 of the quad first
      const uint32_t even = (lo4 & 0xFFu) | (hi4 & 0xFFu) << 8, odd = lo4 >> 8 | (hi4 & 0xFF00u);
      got = __shfl_xor_sync(0xFFFFFFFFu, l4 ? even : odd, 4);
      kword = l4 ? got | odd << 16 : even | got << 16;
    } else {
      uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, l2 ? u : u >> 8, 2) & 0xFFu;
      const uint32_t mine = l2 ? u >> 8 & 0xFFu : u & 0xFFu;
      const uint32_t quad = l2 ? got | mine << 8 : mine | got << 8;
      got = __shfl_xor_sync(0xFFFFFFFFu, quad, 4);
      kword = l4 ? got | quad << 16 : quad | got << 16;
    }
  }
  // V: the codes of elements n + 8 i in nibble i of the piece of lane n
  uint32_t vpiece[2] = {0u, 0u}, ks2[2] = {0u, 0u}, vs2[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    vpiece[j >> 1] |= vcode[j] << (16 * (j & 1) + 4 * (lane >> 3));
    ks2[j >> 1] |= ksc[j] << (16 * (j & 1));
    vs2[j >> 1] |= vsc[j] << (16 * (j & 1));
  }
#pragma unroll
  for (int h = 0; h < NG / 2; ++h) {
    vpiece[h] |= __shfl_xor_sync(0xFFFFFFFFu, vpiece[h], 8);
    vpiece[h] |= __shfl_xor_sync(0xFFFFFFFFu, vpiece[h], 16);
  }
  const int g = NG == 4 ? (l2 ? 2 : 0) + (l4 ? 1 : 0) : (l2 ? 1 : 0);
  if (NG == 4 ? !(lane & 1) : !(lane & 5))
    *reinterpret_cast<uint32_t*>(blk + q4_k_row(b, HD) + (lane >> 3) * (4 * NG) + g * 4) = kword;
  if (HD == 128) {
    if (lane < 8) *reinterpret_cast<uint2*>(blk + q4_v_piece(b, lane, HD)) = make_uint2(vpiece[0], vpiece[1]);
    if (lane == 8) *reinterpret_cast<uint2*>(blk + q4_ks_off(HD) + b * 8) = make_uint2(ks2[0], ks2[1]);
    if (lane == 9) *reinterpret_cast<uint2*>(blk + q4_vs_off(HD) + b * 8) = make_uint2(vs2[0], vs2[1]);
  } else {
    if (lane < 8) *reinterpret_cast<uint32_t*>(blk + q4_v_piece(b, lane, HD)) = vpiece[0];
    if (lane == 8) *reinterpret_cast<uint32_t*>(blk + q4_ks_off(HD) + b * 4) = ks2[0];
    if (lane == 9) *reinterpret_cast<uint32_t*>(blk + q4_vs_off(HD) + b * 4) = vs2[0];
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
  const unsigned task = blockIdx.x * 8 + (threadIdx.x >> 5);
  const unsigned token = task / static_cast<unsigned>(a.c.n_kv);
  pdl_wait();
  pdl_launch_dependents();
  if (token >= static_cast<unsigned>(a.n_tokens)) return;
  const int h = static_cast<int>(task - token * a.c.n_kv);
  const int pos = a.positions[token];
  const int seq = a.seqs ? a.seqs[token] : static_cast<int>(token);
  const uint8_t* blk = q4_block_of(a.c, seq, pos, h, HD);
  const float nan = __int_as_float(0x7FC00000);
  const int b = pos & (kQ4Block - 1);
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
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(n_tokens) * c.n_kv + 7) / 8);
  return hd == 128 ? launch_pdl(k_kv_append_q4<128>, dim3(blocks), 256, 0, st, a)
                   : launch_pdl(k_kv_append_q4<64>, dim3(blocks), 256, 0, st, a);
}

cudaError_t launch_kv_read_q4(const Q4Cache& c, int hd, const int32_t* positions, const int32_t* seqs, int n_tokens,
                              float* k_out, int64_t k_stride, float* v_out, int64_t v_stride, cudaStream_t st) {
  ReadArgs a{c, positions, seqs, k_out, v_out, k_stride, v_stride, n_tokens};
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(n_tokens) * c.n_kv + 7) / 8);
  return hd == 128 ? launch_pdl(k_kv_read_q4<128>, dim3(blocks), 256, 0, st, a)
                   : launch_pdl(k_kv_read_q4<64>, dim3(blocks), 256, 0, st, a);
}

}  // namespace tqd
