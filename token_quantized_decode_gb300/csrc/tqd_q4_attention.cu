// Attention over the paged Q4 cache.
#include <cuda_runtime.h>

#include "tqd_internal.h"
#include "tqd_q4.cuh"

namespace tqd {
namespace {

// One warp per (query token, head), positions one after the other.
template <int HD>
__global__ void __launch_bounds__(128) k_attention_q4(Q4AttnArgs a) {
  constexpr int NG = HD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int token = static_cast<int>(task / a.n_heads);
  if (token >= a.n_tokens) return;
  const int head = static_cast<int>(task - static_cast<int64_t>(token) * a.n_heads);
  int seq = -1, nq = 1, i = 0;
  if (!a.q_start) {
    seq = token;
  } else {
    for (int s = 0; s < a.c.n_seq; ++s)
      if (token >= a.q_start[s] && token < a.q_start[s + 1]) {
        seq = s;
        nq = a.q_start[s + 1] - a.q_start[s];
        i = token - a.q_start[s];
        break;
      }
  }
  if (seq < 0) return;
  const int last = a.lens[seq] - nq + i;
  float q[NG], o[NG], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    q[j] = a.q[token * a.q_stride + head * HD + lane + 32 * j] * a.scale;
    o[j] = 0.f;
  }
  const int h = head / (a.n_heads / a.c.n_kv);
  for (int t = 0; t <= last; ++t) {
    const int slot = t / a.c.page_size;
    const int page = slot < a.c.table_stride ? a.c.table[static_cast<size_t>(seq) * a.c.table_stride + slot] : -1;
    float s = 0.f, v[NG];
    if (page < 0 || page >= a.c.n_pages) {
      l = __int_as_float(0x7FC00000);
      break;
    }
    const int in_page = t % a.c.page_size, b = in_page % kQ4Block;
    const uint8_t* blk = a.c.pages + static_cast<size_t>(page) * a.c.page_bytes +
                         (static_cast<size_t>(h) * (a.c.page_size / kQ4Block) + in_page / kQ4Block) * q4_block_bytes(HD);
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const uint32_t kb = blk[q4_k_row(b, HD) + (lane >> 3) * (4 * NG) + j * 4 + ((lane & 7) >> 1)];
      const uint32_t vb = blk[q4_v_piece(b, lane & 7, HD) + 2 * j + (lane >> 4)];
      const __half ks = *reinterpret_cast<const __half*>(blk + q4_ks_off(HD) + (b * NG + j) * 2);
      const __half vs = *reinterpret_cast<const __half*>(blk + q4_vs_off(HD) + (b * NG + j) * 2);
      s += q[j] * (static_cast<float>(static_cast<int>((kb >> (4 * (lane & 1))) & 15u) - 8) * __half2float(ks));
      v[j] = static_cast<float>(static_cast<int>((vb >> (4 * ((lane >> 3) & 1))) & 15u) - 8) * __half2float(vs);
    }
    s = warp_sum(s);
    const float mn = fmaxf(m, s);
    const float c = m == -INFINITY ? 0.f : expf(m - mn);
    const float p = s == -INFINITY ? 0.f : expf(s - mn);
    l = l * c + p;
#pragma unroll
    for (int j = 0; j < NG; ++j) o[j] = o[j] * c + p * v[j];
    m = mn;
  }
#pragma unroll
  for (int j = 0; j < NG; ++j)
    a.out[token * a.out_stride + head * HD + lane + 32 * j] = l == 0.f ? 0.f : o[j] / l;
}

}  // namespace

size_t attention_q4_scratch_bytes(int hd) { return static_cast<size_t>(hd) * 4; }

cudaError_t launch_attention_q4(const Q4AttnArgs& a, int hd, cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(a.n_tokens) * a.n_heads;
  const unsigned blocks = static_cast<unsigned>((warps + 3) / 4);
  if (hd == 128)
    k_attention_q4<128><<<blocks, 128, 0, st>>>(a);
  else
    k_attention_q4<64><<<blocks, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace tqd
