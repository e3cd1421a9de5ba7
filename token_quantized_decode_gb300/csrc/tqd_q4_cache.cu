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

// Codes and scale of one group of 32, four elements in each of eight
// neighbouring lanes: rint(7 y / max|y|) + 8 and f16(max|y| / 7) of the exact values.
struct Q4Code {
  uint32_t codes;  // the lane's four, a nibble each (1..15, 8: zero)
  uint32_t scale;  // f16 bits, the same in the eight lanes
};

__device__ __noinline__ Q4Code q4_code_exact(double y0, double y1, double y2, double y3) {
  double a = fmax(fmax(fabs(y0), fabs(y1)), fmax(fabs(y2), fabs(y3)));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) a = fmax(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  const float d = __double2float_rn(a / 7.0);
  Q4Code r;
  r.codes = 0x8888u;
  if (a > 0.0 && d < 65520.f) {
    r.codes = static_cast<uint32_t>(__double2int_rn(7.0 * y0 / a) + 8);
    r.codes |= static_cast<uint32_t>(__double2int_rn(7.0 * y1 / a) + 8) << 4;
    r.codes |= static_cast<uint32_t>(__double2int_rn(7.0 * y2 / a) + 8) << 8;
    r.codes |= static_cast<uint32_t>(__double2int_rn(7.0 * y3 / a) + 8) << 12;
  }
  r.scale = d < 65520.f ? __half_as_ushort(__float2half_rn(d)) : 0x7E00u;
  return r;
}

// The largest of a group's f32 of no sign, as bits, so that a NaN or an infinity is the largest.
__device__ __forceinline__ float group_max(uint32_t m) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return __uint_as_float(m);
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
__device__ __forceinline__ Q4Code q4_code(const float (&y)[4], float M, bool& unsure) {
  const float a = group_max(max(max(__float_as_uint(fabsf(y[0])), __float_as_uint(fabsf(y[1]))),
                                max(__float_as_uint(fabsf(y[2])), __float_as_uint(fabsf(y[3])))));
  // a / 7 rounded: one step from a times the nearest f32 to 1 / 7
  float d = a * 0.14285715f;
  d = fmaf(fmaf(-7.f, d, a), 0.14285715f, d);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(a));
  const float rel = M * inv, inv7 = 7.f * inv;
  const float edge = fmaf(rel, -1.9073486e-6f, 0.49999809f);  // 1/2 - 2^-19 (rel + 1)
  Q4Code r;
  r.scale = __half_as_ushort(__float2half_rn(d));
  r.codes = 0u;
  float far = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float t = y[e] * inv7, q = rintf(t);
    far = fmaxf(far, fabsf(t - q));
    r.codes |= static_cast<uint32_t>(static_cast<int>(q) + 8) << (4 * e);
  }
  unsure = far > edge;
  const float slack = d * fmaf(rel, 2.3841858e-7f, 2.3841858e-7f);  // 2^-22 d (rel + 1)
  if (M > 0.f) {
    unsure |= __half_as_ushort(__float2half_rn(d - slack)) != __half_as_ushort(__float2half_rn(d + slack)) || rel > 256.f;
  }
  if (!(a > 1e-30f && d < 65520.f)) {
    // All 0; so small that the steps above lose bits; or a NaN or an infinity
    // in the group, or a scale past the f16 range: the scale is NaN, so the
    // group stands for NaN.  (A scale that the rotation's error may have taken
    // past it is looked at again; that of a NaN or an infinity compares false.)
    unsure = d < 65520.f ? a > 0.f || M > 0.f : M > 0.f && d - slack < 65520.f;
    r.codes = 0x8888u;
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
  bool wide_kv, wide_q, wide_rope;  // rows and table on 16-byte boundaries
};

__device__ __forceinline__ void load4(const float* p, bool wide, float (&v)[4]) {
  if (wide) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else {
    v[0] = p[0]; v[1] = p[1]; v[2] = p[2]; v[3] = p[3];
  }
}

// One warp per (token, kv head): it rotates that head's key and its share of the
// query heads, and codes and stores the key and the value.  A lane holds four
// consecutive elements, so a row is a warp (head_dim 128) or half of one (64: the key's
// and the value's row side by side, and two query heads), a group eight lanes, and
// what a group shares is computed once for four elements.  All rows are loaded
// before the position is looked at: with 40 warps an SM the chain of loads
// (position, page, table of angles) is what a warp waits for.
//
// 5003 tokens of 16/8 heads of 128 take 33 us (130 MB: 3.9 TB/s), 8192 of 32/8
// heads 65 us (5.4 TB/s, 80 % of a copy's rate); with an element a lane they took
// 37.5 and 74 us, with the queries loaded after the position 37.5 and 74 as well.
// About 570 instructions a warp, so issue (70 % of its slots) is next to the
// loads in what bounds it.  Up to 1024 tokens a call is its launch (9 to 11 us
// back to back).
template <int HD>
__global__ void __launch_bounds__(256) k_kv_append_q4(AppendArgs a) {
  constexpr int NG = HD / 32, LR = HD / 4, ROWS = 32 / LR;  // lanes of a row, rows side by side
  const int lane = threadIdx.x & 31, l = lane % LR, side = lane / LR;
  const unsigned task = blockIdx.x * 8 + (threadIdx.x >> 5);  // (at most 2^30)
  const unsigned token = task / static_cast<unsigned>(a.c.n_kv);
  pdl_wait();
  pdl_launch_dependents();
  if (token >= static_cast<unsigned>(a.n_tokens)) return;
  const int item = static_cast<int>(task - token * a.c.n_kv);
  const int pos = a.positions[token];
  const int seq = a.seqs ? a.seqs[token] : static_cast<int>(token);
  const float* ksrc = a.k + token * a.k_stride + item * HD + 4 * l;
  const float* vsrc = a.v + token * a.v_stride + item * HD + 4 * l;
  float x[4], vx[4];  // head_dim 64: x is the key's row in the lower lanes, the value's in the upper ones
  load4(ROWS == 2 && side ? vsrc : ksrc, a.wide_kv, x);
  if constexpr (ROWS == 1) load4(vsrc, a.wide_kv, vx);
  // query heads item, item + n_kv, ...: as many side by side as rows, two rounds at a time
  float q[2][4];
  auto load_q = [&](int h0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int h = h0 + (u * ROWS + side) * a.c.n_kv;
      q[u][0] = q[u][1] = q[u][2] = q[u][3] = 0.f;
      if (h < a.n_heads) load4(a.q + token * a.q_stride + static_cast<int64_t>(h) * HD + 4 * l, a.wide_q, q[u]);
    }
  };
  load_q(item);
  if (pos < 0 || seq < 0 || seq >= a.c.n_seq || (a.rope && pos >= a.max_pos)) return;  // padding
  // cos and sin of the lane's four elements (the second half of a row has those of the first)
  float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.rope) {
    const float* w = reinterpret_cast<const float*>(a.rope + static_cast<size_t>(pos) * (HD / 2) + 4 * l % (HD / 2));
    float lo[4], hi[4];
    load4(w, a.wide_rope, lo);
    load4(w + 4, a.wide_rope, hi);
    cs[0] = lo[0]; sn[0] = lo[1]; cs[1] = lo[2]; sn[1] = lo[3];
    cs[2] = hi[0]; sn[2] = hi[1]; cs[3] = hi[2]; sn[3] = hi[3];
  }
  const bool second = 4 * l >= HD / 2;
  // y = x c - x1 s in the first half of a row, x c + x1 s in the second, x1 the element half a row away
  auto rotate = [&](const float (&in)[4], float (&other)[4], float (&out)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      other[e] = __shfl_xor_sync(0xFFFFFFFFu, in[e], LR / 2);
      const float p = __fmul_rn(other[e], sn[e]);
      out[e] = a.rope ? fmaf(in[e], cs[e], second ? p : -p) : in[e];
    }
  };
  uint8_t* blk = q4_block_of(a.c, seq, pos, item, HD);
  for (int h0 = item; h0 < a.n_heads; h0 += 2 * ROWS * a.c.n_kv) {
    if (h0 != item) load_q(h0);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int h = h0 + (u * ROWS + side) * a.c.n_kv;
      if (h - side * a.c.n_kv >= a.n_heads) break;
      float other[4], out[4];
      rotate(q[u], other, out);
      if (h < a.n_heads) {
        float* o = a.q_out + token * a.qo_stride + static_cast<int64_t>(h) * HD + 4 * l;
        if (a.wide_q)
          *reinterpret_cast<float4*>(o) = make_float4(out[0], out[1], out[2], out[3]);
        else
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = out[e];
      }
    }
  }

  float y[4], x1[4];
  rotate(x, x1, y);
  if (!blk) return;
  const int b = pos % kQ4Block, g = l / 8;
  bool unsure;
  // ---- the key's row (head_dim 64: and the value's, which is not rotated)
  const bool is_v = ROWS == 2 && side;
  uint32_t em = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (is_v) y[e] = x[e];
    em = max(em, __float_as_uint(fabsf(x[e]) + fabsf(x1[e])));
  }
  const float M = group_max(a.rope && !is_v ? em : 0u);
  Q4Code kc = q4_code(y, M, unsure);
  uint32_t again = __ballot_sync(0xFFFFFFFFu, unsure);
  if (again) {
    double w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double xe = x[e], oe = x1[e], c = cs[e], s = sn[e];
      w[e] = !a.rope || is_v ? xe : second ? xe * c + oe * s : xe * c - oe * s;
    }
    const Q4Code r = q4_code_exact(w[0], w[1], w[2], w[3]);
    if (again >> (lane & 24) & 0xFFu) kc = r;
  }
  Q4Code vc = kc;
  if constexpr (ROWS == 1) {
    vc = q4_code(vx, 0.f, unsure);
    again = __ballot_sync(0xFFFFFFFFu, unsure);
    if (again) {
      const Q4Code r = q4_code_exact(vx[0], vx[1], vx[2], vx[3]);
      if (again >> (lane & 24) & 0xFFu) vc = r;
    }
  }

  // K: two neighbouring lanes hold the eight codes of a word
  const uint32_t kword = kc.codes | __shfl_xor_sync(0xFFFFFFFFu, kc.codes, 1) << 16;
  // V: nibble i of piece n is element n + 8 i, this lane's are n = 4 (l % 2) + e,
  // i = l / 2.  In three exchanges over the lanes of a word (8 values of i)
  // each lane gives away the pieces that its partner keeps.
  const int shift = 4 * (l / 2 % 8);
  uint32_t p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = (vc.codes >> (4 * e) & 15u) << shift;
  const bool l2 = lane & 2, l4 = lane & 4;
  const uint32_t s0 = __shfl_xor_sync(0xFFFFFFFFu, l2 ? p[0] : p[2], 2) | (l2 ? p[2] : p[0]);
  const uint32_t s1 = __shfl_xor_sync(0xFFFFFFFFu, l2 ? p[1] : p[3], 2) | (l2 ? p[3] : p[1]);
  uint32_t vword = __shfl_xor_sync(0xFFFFFFFFu, l4 ? s0 : s1, 4) | (l4 ? s1 : s0);
  vword |= __shfl_xor_sync(0xFFFFFFFFu, vword, 8);
  const int n = 4 * (l & 1) + (l2 ? 2 : 0) + (l4 ? 1 : 0);

  if (!is_v) {
    if (!(l & 1)) *reinterpret_cast<uint32_t*>(blk + q4_k_row(b, HD) + l % 8 / 2 * (4 * NG) + g * 4) = kword;
    if (l % 8 == 0) *reinterpret_cast<uint16_t*>(blk + q4_ks_off(HD) + (b * NG + g) * 2) = static_cast<uint16_t>(kc.scale);
  }
  if (ROWS == 1 || is_v) {
    if (!(l & 8)) *reinterpret_cast<uint32_t*>(blk + q4_v_piece(b, n, HD) + l / 16 * 4) = vword;
    if (l % 8 == 0) *reinterpret_cast<uint16_t*>(blk + q4_vs_off(HD) + (b * NG + g) * 2) = static_cast<uint16_t>(vc.scale);
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

// One warp per (token, kv head); a lane writes elements lane + 32 j.  A reading for
// hand-overs, off the decode path: 5003 rows of 8 heads of 128 take 12 us (47 MB, 3.9 TB/s).
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

cudaError_t launch_kv_append_q4(const Q4Cache& c, int hd, const float* k, int64_t k_stride, const float* v,
                                int64_t v_stride, const int32_t* positions, const int32_t* seqs, int n_tokens,
                                const float2* rope, int max_pos, const float* q, int64_t q_stride, int n_heads,
                                float* q_out, int64_t qo_stride, cudaStream_t st) {
  auto wide = [](const void* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 4 == 0; };
  AppendArgs a{c, k, v, q, q_out, k_stride, v_stride, q_stride, qo_stride, positions, seqs, rope, n_tokens, n_heads,
               max_pos, wide(k, k_stride) && wide(v, v_stride), wide(q, q_stride) && wide(q_out, qo_stride),
               wide(rope, 0)};
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
