// Attention over the paged Q4 cache: out = softmax(q . K / sqrt(hd)) V, one or
// several queries per sequence.
//
// Mathematics.  Scores are kept in units of log2 (q is multiplied by
// log2(e) / sqrt(hd)), the running reference of a row is ref = M + ex - 11 with M
// its largest score so far and 2^ex above the largest V scale so far, and with
// p = 2^(score - ref) the row is (sum p v) / (sum p), rescaled when M or the V
// scale grows past a slack of 2 octaves.  K and V elements are (code - 8) * scale,
// so  q . k = sum over groups scale_g (sum_d q_d code_d - 8 sum_d q_d)  and
// sum_t p_t v_t = sum_t (p_t scale_t) (code_t - 8).  (The second is not split like
// the first: over many positions sum p code is 8 sum p but for a small rest,
// and the rest is the result.)
//
// Both contractions run on the tensor cores by mma.sync m16n8k16 with f16
// operands: codes are exact (a masked word is an operand, tqd_q4.cuh), q and
// p * scale are split into two f16 parts (22 bits; 2^-11 would show in f32
// outputs), one in rows 0-7 of the 16-row operand and one in rows 8-15, so the
// split costs no instruction more; sums are f32.  tcgen05 does not fit here:
// its weight-side operand would have to pass through shared memory as f16, four
// times the bytes that the cache holds, and that is more than shared memory
// moves at the rate HBM delivers the codes.
//
// Few query rows share a kv head (G = 2 to 8), and the operand has 8.  The free
// rows carry other groups: with GV groups side by side, row (h, gv) holds
// query row h for group gv only, one chain of MMAs sums each group in its own
// row, and a p * scale operand is made once instead of GV times.  GV is 4 for up
// to 2 rows, 2 for up to 4, 1 otherwise.
//
// Split.  The unit is a block of 16 positions of one (sequence, kv head, tile
// of query rows); units are laid end to end and each CTA takes an equal run of
// them (kCtas at three per SM), its 4 warps every fourth unit with a running
// softmax each, whatever the lengths.  Rows that one CTA finishes are written
// out; where a run begins or ends inside a row's units the CTA leaves a partial
// (ref, sum p, sum p v) and a second kernel, already launched (programmatic
// dependent launch), joins them.  The order of every sum is fixed by the sizes.
#include <cuda_runtime.h>

#include "tqd_internal.h"
#include "tqd_q4.cuh"

namespace tqd {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kCtas = 456;      // three per SM
constexpr int kSegment = 16;    // units that beginning and ending a segment is counted as
constexpr int kCombine = 512;   // threads of the joining kernel
constexpr float kNaN = __builtin_nanf("");

// Stages of a warp's ring of blocks.
template <int HD>
struct Ring {
  static constexpr int stages = HD == 128 ? 5 : 8;
  static constexpr int bytes = q4_block_bytes(HD);
};

// A partial result: R rows of HD sums, then the 8 operand rows' ref and sum p.
__host__ __device__ constexpr int partial_floats(int hd) { return 8 * hd + 16; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x0, x1 as two f16 parts each: hi = f16(x), lo = f16(x - hi).
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_f16(x0 - f.x, x1 - f.y);
}

// The codes in bits 0-3 (lo) or 4-7 (hi) of each half of x as f16 pairs of
// code - 8: 1024 + code and 1024 + 16 code are exact f16, so is the result.
__device__ __forceinline__ uint32_t signed_lo(uint32_t x) {
  const uint32_t v = (x & 0x000F000Fu) | 0x64006400u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), __halves2half2(__ushort_as_half(0x6408), __ushort_as_half(0x6408)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t signed_hi(uint32_t x) {
  const uint32_t v = (x & 0x00F000F0u) | 0x64006400u;
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(0.0625f), __float2half2_rn(-72.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ unsigned long long udiv(unsigned long long a, unsigned b) {
  return a >> 32 ? a / b : static_cast<unsigned>(a) / b;
}

// The units of a call, the same in every CTA of both kernels.
struct Plan {
  const unsigned long long* pre;  // [n_seq + 1] units before each sequence (shared memory)
  const int* len;                 // [n_seq] cached positions, >= 0
  const int* nq;                  // [n_seq] queries
  unsigned long long total, per;  // units, and units of one CTA
  int n_seq, n_kv, G, R;

  // Units of a segment: its blocks, and kSegment more that stand for the cost
  // of beginning and ending it.
  __device__ int blocks(int s) const {
    return len[s] > 0 ? (len[s] + kQ4Block - 1) / kQ4Block + kSegment : 0;
  }
  __device__ int tiles(int s) const { return static_cast<int>((static_cast<long long>(nq[s]) * G + R - 1) / R); }
  // Sequence of unit u < total.
  __device__ int seq_of(unsigned long long u) const {
    int lo = 0, hi = n_seq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= u) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
  // Row tile of a segment: light and heavy tiles of a prompt in turn, so that
  // equal runs of units hold equal work.
  __device__ int tile_of(int s, unsigned long long seg, int* kvh) const {
    const int rt = tiles(s);
    const unsigned long long k = udiv(seg, rt);
    const int i = static_cast<int>(seg - k * rt);
    *kvh = static_cast<int>(k);
    return i & 1 ? rt - 1 - (i >> 1) : i >> 1;
  }
  // Positions that query row `row` of sequence s sees (0 for a row past the last).
  __device__ int seen(int s, int row) const {
    const int q = row / G;
    if (q >= nq[s]) return 0;
    const int v = len[s] - nq[s] + q + 1;
    return v > 0 ? v : 0;
  }
};

// First query token of a sequence.
__device__ __forceinline__ int q_first(const Q4AttnArgs& a, int s) { return a.q_start ? a.q_start[s] : s; }

// Build the plan: every thread of the block calls it; blocks of up to 32 warps.
// Shared memory: pre [n_seq + 1] u64, len [n_seq], nq [n_seq], warp sums.
__device__ Plan make_plan(const Q4AttnArgs& a, int R, int ctas, unsigned char* smem) {
  __shared__ unsigned long long wsum[33];
  Plan p;
  const int n = a.c.n_seq, t = threadIdx.x, nt = blockDim.x;
  auto* pre = reinterpret_cast<unsigned long long*>(smem);
  auto* len = reinterpret_cast<int*>(pre + n + 1);
  auto* nq = len + n;
  p.pre = pre;
  p.len = len;
  p.nq = nq;
  p.n_seq = n;
  p.n_kv = a.c.n_kv;
  p.G = a.n_heads / a.c.n_kv;
  p.R = R;
  const int each = (n + nt - 1) / nt, s0 = t * each;
  unsigned long long mine = 0;
  for (int s = s0; s < s0 + each && s < n; ++s) {
    len[s] = max(a.lens[s], 0);
    int q = 1;
    if (a.q_start) {  // clipped to the query rows there are
      const int b = a.q_start[s], e = a.q_start[s + 1];
      q = b >= 0 && b <= a.n_tokens && e > b ? min(e, a.n_tokens) - b : 0;
    }
    nq[s] = q;
    pre[s] = mine;
    mine += static_cast<unsigned long long>(p.n_kv) * p.tiles(s) * p.blocks(s);
  }
  unsigned long long run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long v = __shfl_up_sync(0xFFFFFFFFu, run, o);
    if ((t & 31) >= o) run += v;
  }
  if ((t & 31) == 31) wsum[t >> 5] = run;
  __syncthreads();
  unsigned long long before = run - mine, total = 0;
  for (int w = 0; w < nt / 32; ++w) {
    if (w < (t >> 5)) before += wsum[w];
    total += wsum[w];
  }
  for (int s = s0; s < s0 + each && s < n; ++s) pre[s] += before;
  if (t == 0) pre[n] = total;
  __syncthreads();
  p.total = total;
  const unsigned long long per = (total + ctas - 1) / ctas;
  p.per = (per + kWarps - 1) / kWarps * kWarps;
  if (p.per == 0) p.per = kWarps;
  return p;
}

size_t plan_bytes(int n_seq) { return (static_cast<size_t>(n_seq) * 16 + 8 + 15) / 16 * 16; }

template <int HD, int GV>
__global__ void __launch_bounds__(kThreads, 3) k_attention_q4(Q4AttnArgs a) {
  constexpr int NG = HD / 32, NS = NG / GV, R = 8 / GV;
  constexpr int ST = Ring<HD>::stages, BB = Ring<HD>::bytes;
  extern __shared__ __align__(128) unsigned char sm[];
  unsigned char* ring = sm;
  float* merge = reinterpret_cast<float*>(ring + kWarps * ST * BB);  // [warps][R * HD], then [warps][8] ref, l
  float* mref = merge + kWarps * R * HD;
  float* ml = mref + kWarps * 8;
  auto* bars = reinterpret_cast<uint64_t*>(ml + kWarps * 8);  // [warps][ST]
  int* flags = reinterpret_cast<int*>(bars + kWarps * ST);    // [warps][ST] 0 block, 1 no such page, 2 not seen
  unsigned char* plan_mem = reinterpret_cast<unsigned char*>(flags + kWarps * ST);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r8 = lane >> 2, c = lane & 3, h = r8 / GV, gv = r8 % GV;
  pdl_launch_dependents();
  uint64_t* bar = bars + warp * ST;
  int* flag = flags + warp * ST;
  if (lane < ST) mbar_init(&bar[lane], 1);
  fence_mbar_init();
  const Plan plan = make_plan(a, R, gridDim.x, plan_mem);

  // sequences without positions: their queries see nothing
  for (int s = blockIdx.x; s < plan.n_seq; s += gridDim.x) {
    if (plan.len[s] > 0) continue;
    const int64_t width = static_cast<int64_t>(a.n_heads) * HD, first = q_first(a, s);
    for (int64_t i = threadIdx.x; i < plan.nq[s] * width; i += kThreads)
      a.out[(first + i / width) * a.out_stride + i % width] = 0.f;
  }

  const unsigned long long u0 = blockIdx.x * plan.per;
  if (u0 >= plan.total) return;
  const unsigned long long u1 = min(u0 + plan.per, plan.total);
  const int n_it = static_cast<int>((u1 - u0 - warp + kWarps - 1) / kWarps) * (u0 + warp < u1);
  unsigned char* my_ring = ring + warp * ST * BB;
  const int ppb = a.c.page_size / kQ4Block;  // blocks per page

  // Issue unit number i of this warp: lane i % 32 knows its address (found for
  // 32 units at a time, a lane each).
  const uint8_t* src = nullptr;
  int src_flag = 0;
  auto locate = [&](int i) {
    const unsigned long long u = u0 + warp + static_cast<unsigned long long>(i) * kWarps;
    if (u >= u1) return;
    const int s = plan.seq_of(u);
    const unsigned long long uq = u - plan.pre[s];
    const int nb = plan.blocks(s);
    const unsigned long long seg = udiv(uq, nb);
    const int blk = static_cast<int>(uq - seg * nb);
    int kvh;
    const int rt = plan.tile_of(s, seg, &kvh);
    const int last = min(rt * R + R, plan.nq[s] * plan.G) - 1;
    if (blk * kQ4Block >= plan.seen(s, last)) {
      src_flag = 2;
      return;
    }
    const int slot = blk / ppb;
    const int page = slot < a.c.table_stride ? a.c.table[static_cast<size_t>(s) * a.c.table_stride + slot] : -1;
    src_flag = page < 0 || page >= a.c.n_pages;
    src = a.c.pages + static_cast<size_t>(page) * a.c.page_bytes +
          (static_cast<size_t>(kvh) * ppb + (blk - slot * ppb)) * BB;
  };
  auto issue = [&](int i) {
    if (i >= n_it) return;
    if ((i & 31) == 0) locate(i + lane);
    if (lane == (i & 31)) {
      const int st = i % ST;
      flag[st] = src_flag;
      if (src_flag == 0) {
        mbar_arrive_expect_tx(&bar[st], BB);
        bulk_g2s(my_ring + st * BB, src, BB, &bar[st]);
      } else {
        mbar_arrive_expect_tx(&bar[st], 0);
      }
    }
  };
  for (int i = 0; i < ST - 1; ++i) issue(i);

  int it = 0;
  bool dead = false;  // a copy that did not arrive within the wait's limit: the rows become NaN
  int s = plan.seq_of(u0);
  unsigned long long u = u0;
  while (u < u1) {
    // ---- the segment of unit u: one (sequence, kv head, tile of rows)
    while (plan.pre[s + 1] <= u) ++s;
    const int nb = plan.blocks(s);
    const unsigned long long seg = udiv(u - plan.pre[s], nb);
    const unsigned long long seg0 = plan.pre[s] + seg * nb, seg1 = seg0 + nb;
    const unsigned long long uend = min(seg1, u1);
    int kvh;
    const int rt = plan.tile_of(s, seg, &kvh);
    const int n_rows = min(R, plan.nq[s] * plan.G - rt * R);
    const int min_seen = plan.seen(s, rt * R);
    const int row = rt * R + min(h, n_rows - 1);  // rows past the last repeat it
    const int seen = plan.seen(s, row);
    const int head = kvh * plan.G + row % plan.G;
    const int64_t token = q_first(a, s) + row / plan.G;

    // ---- the query rows as operands
    uint32_t qa[NG][2][4];
    float zq[NS][2], fac[NS];
    {
      const float* q = a.q + token * a.q_stride + static_cast<int64_t>(head) * HD;
      // A power of two for each group of 32 brings its largest element to 2^10
      // .. 2^11; the high part is then the nearest whole number, so that a group's sum
      // of high parts times codes is exact in the tensor cores' f32, which truncate
      // (f16 parts with their own exponents cost four times the error).
      // (The clip of fac is met past 2^113, where distinct scores differ by
      // more than 2^80 however they are scaled.)
#pragma unroll
      for (int t = 0; t < NS; ++t) {
        float x[8], m = 0.f, zh = 0.f, zl = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = q[(gv * NS + t) * 32 + 8 * c + i] * a.scale;
          m = fmaxf(m, fabsf(x[i]));
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const int e = max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -100);
        const float f = pow2(10 - e);
        fac[t] = pow2(min(24 - 10 + e, 127));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= f;
          zh += rintf(x[i]);
          zl += round_f16(x[i] - rintf(x[i]));  // what the operand holds
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          zh += __shfl_xor_sync(0xFFFFFFFFu, zh, o);
          zl += __shfl_xor_sync(0xFFFFFFFFu, zl, o);
        }
        zq[t][0] = -8.f * 0x1p-24f * zh;
        zq[t][1] = -8.f * 0x1p-24f * zl;
#pragma unroll
        for (int k = 0; k < GV; ++k) {
          const int g = k * NS + t;
          const float on = k == gv ? 1.f : 0.f;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float y0 = on * x[2 * w], y1 = on * x[2 * w + 4];
            const float y2 = on * x[2 * w + 1], y3 = on * x[2 * w + 5];
            const float i0 = rintf(y0), i1 = rintf(y1), i2 = rintf(y2), i3 = rintf(y3);
            qa[g][w][0] = pack_f16(i0, i1);
            qa[g][w][1] = pack_f16(y0 - i0, y1 - i1);
            qa[g][w][2] = pack_f16(0.0625f * i2, 0.0625f * i3);
            qa[g][w][3] = pack_f16(0.0625f * (y2 - i2), 0.0625f * (y3 - i3));
          }
        }
      }
    }

    float o[NG * 4][4], l = 0.f, M = -INFINITY, S = 0.f, ref = 0.f;
#pragma unroll
    for (int i = 0; i < NG * 4; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    // ---- this warp's units of it
    for (;; ++it) {
      const unsigned long long ui = u0 + warp + static_cast<unsigned long long>(it) * kWarps;
      if (ui >= uend) break;
      issue(it + ST - 1);
      __syncwarp();
      const int st = it % ST;
      if (!dead) dead = !mbar_wait_bounded(&bar[st], (it / ST) & 1, nullptr);
      const int t0 = static_cast<int>(ui - seg0) * kQ4Block;
      const int fl = flag[st];
      if (fl || dead) {
        if (fl != 2 && t0 < seen) l = kNaN;
        __syncwarp();
        continue;
      }
      const unsigned char* blk = my_ring + st * BB;

      // scales of positions 4c .. 4c + 3, this row's groups
      float ks[4][NS], vs[4][NS];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < NS; ++t) {
          const int at = ((4 * c + i) * NG + gv * NS + t) * 2;
          ks[i][t] = __half2float(*reinterpret_cast<const __half*>(blk + q4_ks_off(HD) + at));
          vs[i][t] = __half2float(*reinterpret_cast<const __half*>(blk + q4_vs_off(HD) + at));
        }

      // scores of positions 4c .. 4c + 3
      float sc[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t kw[NG];
        const unsigned char* kr = blk + (j * 8 + r8) * (HD / 2) + c * (4 * NG);
        if constexpr (HD == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(kr);
          kw[0] = v.x; kw[1] = v.y; kw[2] = v.z; kw[3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(kr);
          kw[0] = v.x; kw[1] = v.y;
        }
        float p0 = 0.f, p1 = 0.f;
#pragma unroll
        for (int t = 0; t < NS; ++t) {
          float d[4] = {zq[t][0], zq[t][0], zq[t][1], zq[t][1]};
#pragma unroll
          for (int k = 0; k < GV; ++k) {
            const int g = k * NS + t;
            mma_f16(d, qa[g][0], kw[g] & 0x000F000Fu, kw[g] & 0x00F000F0u);
            const uint32_t w = kw[g] >> 8;
            mma_f16(d, qa[g][1], w & 0x000F000Fu, w & 0x00F000F0u);
          }
          p0 += ks[2 * j][t] * (fac[t] * (d[0] + d[2]));
          p1 += ks[2 * j + 1][t] * (fac[t] * (d[1] + d[3]));
        }
#pragma unroll
        for (int x = 4; x < 4 * GV; x <<= 1) {
          p0 += __shfl_xor_sync(0xFFFFFFFFu, p0, x);
          p1 += __shfl_xor_sync(0xFFFFFFFFu, p1, x);
        }
        sc[2 * j] = p0;
        sc[2 * j + 1] = p1;
      }
      if (t0 + kQ4Block > min_seen) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t0 + 4 * c + i >= seen) {
            sc[i] = -INFINITY;
#pragma unroll
            for (int t = 0; t < NS; ++t) vs[i][t] = 0.f;  // a NaN scale behind the end weighs nothing
          }
      }

      // the reference: kept while neither the scores nor the V scales grow past the slack
      const float bm = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
      float bs = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < NS; ++t) bs = fmaxf(bs, vs[i][t]);
      if (__any_sync(0xFFFFFFFFu, bm > M + 2.f || bs > 4.f * S)) {
        float m2 = bm, s2 = bs;
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
          m2 = fmaxf(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, x));
          s2 = fmaxf(s2, __shfl_xor_sync(0xFFFFFFFFu, s2, x));
        }
        m2 = fmaxf(m2, M);
        S = fmaxf(s2, S);
        const int ex = max(static_cast<int>(__float_as_uint(S) >> 23) - 126, -24);
        const float nref = m2 == -INFINITY ? 0.f : m2 + static_cast<float>(ex - 11);
        const float k = M == -INFINITY ? 1.f : ex2(ref - nref);
        M = m2;
        ref = nref;
        l *= k;
#pragma unroll
        for (int i = 0; i < NG * 4; ++i) {
          o[i][0] *= k; o[i][1] *= k; o[i][2] *= k; o[i][3] *= k;
        }
      }

      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = ex2(sc[i] - ref);
      l += (p[0] + p[1]) + (p[2] + p[3]);

      uint4 v0, v1;
      if constexpr (HD == 128) {
        v0 = *reinterpret_cast<const uint4*>(blk + q4_v_off(HD) + c * 128 + r8 * 16);
        v1 = *reinterpret_cast<const uint4*>(blk + q4_v_off(HD) + 512 + c * 128 + r8 * 16);
      } else {
        v0 = *reinterpret_cast<const uint4*>(blk + q4_v_off(HD) + c * 128 + r8 * 16);
      }
#pragma unroll
      for (int t = 0; t < NS; ++t) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = p[i] * vs[i][t];
        uint32_t pa[4];
        split_f16(w[0], w[1], pa[0], pa[1]);
        split_f16(w[2], w[3], pa[2], pa[3]);
#pragma unroll
        for (int k = 0; k < GV; ++k) {
          const int g = k * NS + t;
          const uint32_t sel = g & 1 ? 0x7632u : 0x5410u;
          uint32_t x0, x1;
          if constexpr (HD == 128) {
            x0 = __byte_perm(g < 2 ? v0.x : v0.y, g < 2 ? v0.z : v0.w, sel);
            x1 = __byte_perm(g < 2 ? v1.x : v1.y, g < 2 ? v1.z : v1.w, sel);
          } else {
            x0 = __byte_perm(v0.x, v0.y, sel);
            x1 = __byte_perm(v0.z, v0.w, sel);
          }
          mma_f16(o[4 * g], pa, signed_lo(x0), signed_lo(x1));
          mma_f16(o[4 * g + 1], pa, signed_hi(x0), signed_hi(x1));
          x0 >>= 8;
          x1 >>= 8;
          mma_f16(o[4 * g + 2], pa, signed_lo(x0), signed_lo(x1));
          mma_f16(o[4 * g + 3], pa, signed_hi(x0), signed_hi(x1));
        }
      }
      __syncwarp();  // every lane has read the stage before it is filled again
    }

    // ---- the warps' sums into one
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
    float* mo = merge + warp * R * HD + h * HD;
#pragma unroll
    for (int g = 0; g < NG; ++g)
      if (g / NS == gv) {
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const float (&d)[4] = o[4 * g + tt];
          *reinterpret_cast<float2*>(mo + 32 * g + 8 * tt + 2 * c) = make_float2(d[0] + d[2], d[1] + d[3]);
        }
      }
    if (c == 0) {
      mref[warp * 8 + r8] = M == -INFINITY && l == 0.f ? -INFINITY : ref;
      ml[warp * 8 + r8] = l;
    }
    __syncthreads();
    const bool whole = u0 <= seg0 && seg1 <= u1;
    // slot 0: the units from the CTA's first on; slot 1: those up to its last
    float* part = static_cast<float*>(a.scratch) +
                  (static_cast<size_t>(blockIdx.x) * 2 + (u == u0 ? 0 : 1)) * partial_floats(HD);
    for (int i = threadIdx.x; i < R * HD; i += kThreads) {
      const int hr = i / HD, d = i % HD, r = hr * GV + d / 32 / NS;
      float ref2 = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ref2 = fmaxf(ref2, mref[w * 8 + r]);
      float acc = 0.f, ls = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (mref[w * 8 + r] > -INFINITY) {
          const float k = ex2(mref[w * 8 + r] - ref2);
          acc += k * merge[w * R * HD + i];
          ls += k * ml[w * 8 + r];
        }
      if (whole) {
        if (hr < n_rows) {
          const int rr = rt * R + hr;
          a.out[(q_first(a, s) + rr / plan.G) * a.out_stride + static_cast<int64_t>(kvh * plan.G + rr % plan.G) * HD + d] =
              ls == 0.f ? 0.f : acc / ls;
        }
      } else {
        part[i] = acc;
        if (d % (32 * NS) == 0) {
          part[8 * HD + r] = ref2;
          part[8 * HD + 8 + r] = ls;
        }
      }
    }
    __syncthreads();
    u = uend;
  }
}

// Joins the partials of the rows that a CTA's run of units begins and does not
// end: block i looks at the last segment of run i.
template <int HD, int GV>
__global__ void __launch_bounds__(kCombine) k_attention_q4_join(Q4AttnArgs a) {
  constexpr int NG = HD / 32, NS = NG / GV, R = 8 / GV;
  extern __shared__ __align__(128) unsigned char sm[];
  const Plan plan = make_plan(a, R, gridDim.x, sm);
  pdl_wait();
  const unsigned long long u0 = blockIdx.x * plan.per, u1 = u0 + plan.per;
  if (u1 >= plan.total) return;  // nothing behind this run
  const int s = plan.seq_of(u1 - 1);
  const int nb = plan.blocks(s);
  const unsigned long long seg = udiv(u1 - 1 - plan.pre[s], nb);
  const unsigned long long seg0 = plan.pre[s] + seg * nb, seg1 = seg0 + nb;
  if (seg0 < u0 || seg1 <= u1) return;  // begun by an earlier run, or ended by this one
  const int runs = static_cast<int>((seg1 - 1) / plan.per) - static_cast<int>(blockIdx.x) + 1;
  int kvh;
  const int rt = plan.tile_of(s, seg, &kvh);
  const int n_rows = min(R, plan.nq[s] * plan.G - rt * R);
  const float* first = static_cast<const float*>(a.scratch) +
                       (static_cast<size_t>(blockIdx.x) * 2 + (seg0 == u0 ? 0 : 1)) * partial_floats(HD);
  const float* rest = static_cast<const float*>(a.scratch) + static_cast<size_t>(blockIdx.x) * 2 * partial_floats(HD);
  auto part = [&](int k) { return k ? rest + static_cast<size_t>(k) * 2 * partial_floats(HD) : first; };
  __shared__ float wt[kCtas * 8], lsum[8];  // each partial's weight; a row's sum p
  __shared__ float4 red[kCombine];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < 8) {  // a warp per operand row
    float ref = -INFINITY, ls = 0.f;
    for (int k = lane; k < runs; k += 32) ref = fmaxf(ref, part(k)[8 * HD + warp]);
    ref = warp_max(ref);
    for (int k = lane; k < runs; k += 32) {
      const float pr = part(k)[8 * HD + warp];
      const float w = pr > -INFINITY ? ex2(pr - ref) : 0.f;
      wt[k * 8 + warp] = w;
      if (pr > -INFINITY) ls += w * part(k)[8 * HD + 8 + warp];
    }
    ls = warp_sum(ls);
    if (lane == 0) lsum[warp] = ls;
  }
  __syncthreads();
  // four elements a thread, the partials dealt over the threads left
  constexpr int kQuads = R * HD / 4, kDeal = kCombine / kQuads;
  const int i = threadIdx.x % kQuads * 4, deal = threadIdx.x / kQuads;
  const int hr = i / HD, d = i % HD, r = hr * GV + d / 32 / NS;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = deal; k < runs; k += kDeal) {
    const float w = wt[k * 8 + r];
    const float4 v = *reinterpret_cast<const float4*>(part(k) + i);
    acc.x += w * v.x;
    acc.y += w * v.y;
    acc.z += w * v.z;
    acc.w += w * v.w;
  }
  red[threadIdx.x] = acc;
  __syncthreads();
  if (deal == 0 && hr < n_rows) {
#pragma unroll
    for (int k = 1; k < kDeal; ++k) {
      const float4 v = red[k * kQuads + threadIdx.x];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    const int rr = rt * R + hr;
    const float ls = lsum[r];
    float* out = a.out + (q_first(a, s) + rr / plan.G) * a.out_stride + static_cast<int64_t>(kvh * plan.G + rr % plan.G) * HD + d;
    out[0] = ls == 0.f ? 0.f : acc.x / ls;
    out[1] = ls == 0.f ? 0.f : acc.y / ls;
    out[2] = ls == 0.f ? 0.f : acc.z / ls;
    out[3] = ls == 0.f ? 0.f : acc.w / ls;
  }
}

template <int HD, int GV>
cudaError_t launch(const Q4AttnArgs& a, cudaStream_t st) {
  constexpr int R = 8 / GV;
  const size_t plan_b = plan_bytes(a.c.n_seq);
  const size_t smem = static_cast<size_t>(kWarps) * Ring<HD>::stages * (Ring<HD>::bytes + 12) +
                      static_cast<size_t>(kWarps) * (R * HD + 16) * 4 + plan_b;
  cudaError_t e = cudaFuncSetAttribute(k_attention_q4<HD, GV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  k_attention_q4<HD, GV><<<kCtas, kThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kCombine);
  cfg.dynamicSmemBytes = plan_b;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attention_q4_join<HD, GV>, a);
}

}  // namespace

size_t attention_q4_scratch_bytes(int hd) { return static_cast<size_t>(kCtas) * 2 * partial_floats(hd) * 4; }

cudaError_t launch_attention_q4(const Q4AttnArgs& args, int hd, cudaStream_t st) {
  Q4AttnArgs a = args;
  a.scale *= 1.4426950408889634f;  // scores in log2
  // rows that share a kv head; with q_start their number is on the device
  const int rows = a.q_start ? 8 : a.n_heads / a.c.n_kv;
  if (hd == 128) {
    if (rows <= 2) return launch<128, 4>(a, st);
    if (rows <= 4) return launch<128, 2>(a, st);
    return launch<128, 1>(a, st);
  }
  return rows <= 4 ? launch<64, 2>(a, st) : launch<64, 1>(a, st);
}

}  // namespace tqd
