// Attention over the paged Q4 cache: out = softmax(q . K / sqrt(hd)) V, one or
// several queries per sequence.
//
// Mathematics.  Scores are kept in units of log2 (q is multiplied by
// log2(e) / sqrt(hd)), and with p = 2^(score - ref) a row is (sum p v) / (sum p).  The
// running reference of a row goes by its largest product p * V scale so far,
// which it keeps between 2^12 and 2^15; all sums are rescaled when it moves.  (By
// the largest score and the largest scale, which may be of two positions, a
// position of no weight with values 2^24 times the others' left these 11 bits; it
// costs 1 % at 131072 positions.)  K and V elements are (code - 8) * scale, so
// q . k = sum over groups scale_g (sum_d q_d code_d - 8 sum_d q_d)  and
// sum_t p_t v_t = sum_t (p_t scale_t) (code_t - 8).  (The second is not split like
// the first: over many positions sum p code is 8 sum p but for a small rest,
// and the rest is the result.)
//
// Both contractions run on the tensor cores by mma.sync m16n8k16 with f16
// operands, the cache as the 16-row operand: codes are exact (a masked word is
// an operand, tqd_q4.cuh; V's are made signed by one packed operation), q and
// p * scale are split into two f16 parts (22 bits; 2^-11 would show in f32
// outputs) in two of the 8 columns, so the split costs no instruction more;
// sums are f32.  p * scale passes from the scores' layout to the operand's by
// movmatrix.  tcgen05 does not fit here: the cache would have to pass through
// shared memory as f16, four times the bytes that HBM delivers, and that is
// more than shared memory moves at HBM's rate.
//
// 8 columns hold 4 query rows.  Where fewer share a kv head, GV groups lie side
// by side: column pair (h, gv) holds row h for group gv only, one chain of MMAs
// sums each group in its own column, and a p * scale operand is made once
// instead of GV times.  GV is 4 for one row, 2 for two; for more than four rows
// (NT = 2) two column tiles share the unpacked cache.
//
// Split.  The unit is 32 positions of one segment: (sequence, kv head, tile of
// query rows).  Units, and a few empty ones at each segment's beginning for what
// that costs, are laid end to end and each warp takes an equal run of them,
// whatever the lengths, with a running softmax for each segment it meets.  A
// segment inside a warp's run is written out by the warp alone; the partial
// results (ref, sum p, sum p v) of one that several warps of a CTA share are
// joined in shared memory at the CTA's end, and those of one that several CTAs
// share by a second kernel, already launched (programmatic dependent launch).  The
// order of every sum is fixed by the sizes.
//
// Where every sequence has one query and the page table holds few positions
// (use_clusters), a cluster of 1 to 8 CTAs takes a segment instead, and joins its
// parts through distributed shared memory: no plan and no second kernel, half the time of a
// short call.
//
// What it measures (GB300, 1.9 GHz).  131071 positions of 32/8 heads of 128: 42.0 us for
// 151 MB (3.6 TB/s; 22 us at a copy's rate), of which a warp's instructions take most:
// 752 for each unit of 32 positions and 4 rows, 40,500 a scheduler, 21 us at one a
// cycle; the three warps that the registers leave a scheduler reach 0.7 of that between
// the copies' arrival and the last unit, and 12 us are the beginning (lengths, pages,
// queries: 6 us) and the two joins (3 and 3).  The same 12 us bound short calls by
// runs (33 ragged to 4160 positions of 16/8 heads: 18.5 us); 1 x 575 positions by
// clusters take 6.7 us, a launch and one chain of loads.  Prompts' tiles are
// bound by the same instructions (2048 queries of 16/8 heads of 128: 295 us, 58 TFLOP/s).
#include <cuda_runtime.h>

#include <type_traits>

#include "tqd_internal.h"
#include "tqd_q4.cuh"

namespace tqd {
namespace {

constexpr int kCtas = 304;      // two per SM
constexpr int kUnit = 32;       // positions of a unit: two blocks
constexpr int kCombine = 256;   // threads of the joining kernel
constexpr float kNaN = __builtin_nanf("");
constexpr float kNoRef = -3.402823466e38f;  // the reference of a row that has seen no position

// One instantiation: head size, column tiles, groups side by side.
template <int HD, int NT, int GV>
struct Cfg {
  static constexpr int NG = HD / 32;      // groups of a row
  static constexpr int NS = NG / GV;      // chains: column pair gv holds groups gv * NS + 0 .. NS - 1
  static constexpr int P = 4 * NT;        // column pairs
  static constexpr int R = P / GV;        // query rows of a tile
  static constexpr int B = R == 1 ? 1 : 2;  // blocks that join a run
  // Warps: what the registers leave room for twice an SM.  Spills cost more than
  // warps: 131072 positions of 32/8 heads of 128 took 51 us with eight warps of 128
  // registers, 45 with six of 168 (three CTAs of four: 47); of 64/8 heads 101 us with
  // six, 66 with four of 255.
  static constexpr int W = HD == 64 ? (NT == 1 ? 8 : 6) : NT == 2 ? 4 : GV == 1 ? 6 : 8;
  static constexpr int T = 32 * W;
  static constexpr int BB = q4_block_bytes(HD);
  static constexpr int JB = NT == 1 ? 2 : 1;  // blocks of a unit taken at once: two where the registers hold them
  static constexpr int ST = HD == 64 ? 4 : W == 8 ? 2 : 3;  // stages (units) of a warp's ring
  // Empty units that a segment begins with in the plan: about what a warp loses at a
  // segment's beginning and end.  Without them the warps that meet two or more
  // segments ended 5 us after the others: 40 ragged batches (20 of one query, 20 of 8
  // to 400 a sequence) took 20.9 and 38.5 us in the geometric mean with none, 18.7
  // and 34.8 with two, 19.3 and 34.0 with four (33 ragged to 4160: 22.4, 18.6, 20.0; 2048
  // queries of 16/8 heads of 128, where all runs are long: 280, 285, 288).
  static constexpr int LEAD = NT == 1 ? 2 : 4;
  static constexpr int LD = HD + 8;       // floats of a row in the merge buffer
  static constexpr int PART = R * LD + 2 * P;  // floats of a warp's partial result
  static constexpr size_t smem = static_cast<size_t>(W) * ST * (2 * BB + 12) + static_cast<size_t>(W) * PART * 4;
  static_assert(PART * 4 <= ST * 2 * BB, "a partial result fits a warp's ring");
  static_assert(W * ST % 2 == 0, "the plan behind the flags starts on 8 bytes");
  static_assert(NT == 1 || GV == 1, "groups side by side only where columns are free");
};

// A partial result: R rows of HD sums, then the column pairs' ref and sum p.
__host__ __device__ constexpr int partial_floats(int hd) { return 8 * hd + 16; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two sums by one instruction.
__device__ __forceinline__ void add_f32x2(float& x0, float& x1, float y0, float y1) {
  asm("{\n.reg .b64 x, y;\nmov.b64 x, {%0, %1};\nmov.b64 y, {%2, %3};\nadd.rn.f32x2 x, x, y;\nmov.b64 {%0, %1}, x;\n}"
      : "+f"(x0), "+f"(x1)
      : "f"(y0), "f"(y1));
}

// Two products, and two sums of squares, by one instruction.
__device__ __forceinline__ void mul_f32x2(float& x0, float& x1, float a0, float a1, float b0, float b1) {
  asm("{\n.reg .b64 x, y;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmul.rn.f32x2 x, x, y;\nmov.b64 {%0, %1}, x;\n}"
      : "=f"(x0), "=f"(x1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void square_f32x2(float& s0, float& s1, float x0, float x1) {
  asm("{\n.reg .b64 x, y;\nmov.b64 x, {%0, %1};\nmov.b64 y, {%2, %3};\nfma.rn.f32x2 x, y, y, x;\nmov.b64 {%0, %1}, x;\n}"
      : "+f"(s0), "+f"(s1)
      : "f"(x0), "f"(x1));
}

// x as two f16 parts in one word: the leading 11 bits low, the rest high.
__device__ __forceinline__ uint32_t split_f16(float x) {
  const float hi = __uint_as_float(__float_as_uint(x) & 0xFFFFE000u);
  return pack_f16(hi, x - hi);
}

// Element (i, j) of an 8 x 8 matrix of f16 (lane 4 i + j / 2, half j % 2) to (j, i).
__device__ __forceinline__ uint32_t transpose_f16(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ unsigned long long udiv(unsigned long long a, unsigned b) {
  return a >> 32 ? a / b : static_cast<unsigned>(a) / b;
}

// The units of a call, the same in every CTA of both kernels.
struct Plan {
  const unsigned long long* pre;  // [n_seq + 1] units before each sequence (shared memory)
  const int* len;                 // [n_seq] cached positions, >= 0
  const int* nq;                  // [n_seq] queries
  unsigned long long total, per;  // units, and units of one warp
  int n_seq, n_kv, G, rbits;      // 2^rbits rows of a tile
  int most;                       // positions of the page table, and a unit
  int lead;                       // empty units that a segment begins with

  // Units of a segment: the empty ones, its positions', and where they pass the page
  // table one behind the table's end (which makes the rows that see it NaN).
  __device__ int units(int s) const { return len[s] > 0 ? lead + (min(len[s], most) + kUnit - 1) / kUnit : 0; }
  // (rows are at most tokens * heads, 2^30)
  __device__ int tiles(int s) const { return (nq[s] * G + (1 << rbits) - 1) >> rbits; }
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
  // Query of row `row` (a division only where there are several).
  __device__ int query(int row) const { return row < G ? 0 : row / G; }
  // Positions that query row `row` of sequence s sees (0 for a row past the last).
  __device__ int seen(int s, int row) const {
    const int q = query(row);
    if (q >= nq[s]) return 0;
    const int v = len[s] - nq[s] + q + 1;
    return v > 0 ? v : 0;
  }
};

// First query token of a sequence.
__device__ __forceinline__ int q_first(const Q4AttnArgs& a, int s) { return a.q_start ? a.q_start[s] : s; }

// Build the plan: every thread of the block calls it; blocks of up to 32 warps.
// Shared memory: pre [n_seq + 1] u64, len [n_seq], nq [n_seq], warp sums.
__device__ Plan make_plan(const Q4AttnArgs& a, int R, int W, int lead, int ctas, unsigned char* smem) {
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
  p.lead = lead;
  p.n_kv = a.c.n_kv;
  p.G = a.n_heads / a.c.n_kv;
  p.most = static_cast<int>(min(static_cast<long long>(a.c.table_stride) * a.c.page_size, 1ll << 30)) + kUnit;
  p.rbits = R == 8 ? 3 : R == 4 ? 2 : R == 2 ? 1 : 0;
  auto sizes = [&](int s) {  // fills in a sequence's entries, returns its units
    len[s] = min(max(__ldcg(a.lens + s), 0), 1 << 30);
    int q = 1;
    if (a.q_start) {  // clipped to the query rows there are
      const int b = __ldcg(a.q_start + s), e = __ldcg(a.q_start + s + 1);
      q = b >= 0 && b <= a.n_tokens && e > b ? min(e, a.n_tokens) - b : 0;
    }
    nq[s] = q;
    return static_cast<unsigned long long>(p.n_kv) * p.tiles(s) * p.units(s);
  };
  auto scan = [&](unsigned long long v) {  // inclusive, over a warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if ((t & 31) >= o) v += u;
    }
    return v;
  };
  if (n <= 32) {  // one warp does it
    if (t < 32) {
      const unsigned long long mine = t < n ? sizes(t) : 0, run = scan(mine);
      if (t < n) pre[t] = run - mine;
      if (t == 31) pre[n] = run;
    }
    __syncthreads();
  } else {
    const int each = (n + nt - 1) / nt, s0 = t * each;
    unsigned long long mine = 0;
    for (int s = s0; s < s0 + each && s < n; ++s) {
      pre[s] = mine;
      mine += sizes(s);
    }
    const unsigned long long run = scan(mine);
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
  }
  p.total = pre[n];
  const unsigned warps = static_cast<unsigned>(ctas * W);
  p.per = max(udiv(p.total + warps - 1, warps), 1ull);
  return p;
}

size_t plan_bytes(int n_seq) { return (static_cast<size_t>(n_seq) * 16 + 8 + 15) / 16 * 16; }

// A segment whose parts the warps of a CTA join at its end.
struct Shared {
  unsigned long long seg0, seg1;
  int64_t token;            // first query token of its sequence
  int n_rows, row0, head0;  // rows of the tile, its first row, first query head of the kv head
};

// CL: clusters of `cluster` CTAs, one a segment; else equal runs of units.
template <int HD, int NT, int GV, bool CL>
__global__ void __launch_bounds__(Cfg<HD, NT, GV>::T, 2) k_attention_q4(Q4AttnArgs a, int cluster) {
  using C = Cfg<HD, NT, GV>;
  constexpr int NG = C::NG, NS = C::NS, P = C::P, R = C::R, W = C::W, ST = C::ST, BB = C::BB, LD = C::LD, JB = C::JB, PART = C::PART;
  extern __shared__ __align__(128) unsigned char sm[];
  unsigned char* ring = sm;
  // A warp's partial result of the segment that it shares with the warp before
  // it; that of one shared with the warp behind it goes to its ring, done with by then.
  float* parts = reinterpret_cast<float*>(ring + W * ST * 2 * BB);  // [W][PART]: [R][LD], [P] ref, [P] sum p
  auto* bars = reinterpret_cast<uint64_t*>(parts + W * PART);      // [W][ST]
  int* flags = reinterpret_cast<int*>(bars + W * ST);    // [W][ST] 1, 2: no page for the first, second block; 4: not seen
  unsigned char* plan_mem = reinterpret_cast<unsigned char*>(flags + W * ST);

  __shared__ int ends[W];
  __shared__ Shared shared[W + 1];  // the last segment of each warp's run, and the CTA's first one

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;  // operand row (and r + 8), and column pair of the sums
  const int h = c / GV, gv = c % GV;      // the pair's query row in its tile and first group's chain
  uint64_t* bar = bars + warp * ST;
  int* flag = flags + warp * ST;
  if (lane < ST) mbar_init(&bar[lane], 1);
  fence_mbar_init();
  pdl_wait();
  pdl_launch_dependents();
  Plan plan;
  unsigned long long c0 = 0, c1, u0, u1;  // the CTA's run of units, and the warp's
  int cl_s = 0, cl_kvh = 0, cl_rt = 0, cl_len = 0;
  if constexpr (CL) {
    plan.G = a.n_heads / a.c.n_kv;
    const int tiles = (plan.G + R - 1) / R;
    const int seg = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    cl_s = seg / (a.c.n_kv * tiles);
    cl_kvh = seg / tiles - cl_s * a.c.n_kv;
    cl_rt = seg % tiles;
    cl_len = min(max(a.lens[cl_s], 0), 1 << 30);
    const int most = static_cast<int>(min(static_cast<long long>(a.c.table_stride) * a.c.page_size, 1ll << 30)) + kUnit;
    const unsigned units = (min(cl_len, most) + kUnit - 1) / kUnit, warps = cluster * W;
    plan.per = (units + warps - 1) / warps;
    c1 = units;
    u0 = min((rank * W + warp) * plan.per, c1);
    u1 = min(u0 + plan.per, c1);
  } else {
    plan = make_plan(a, R, W, C::LEAD, gridDim.x, plan_mem);
    // sequences without positions: their queries see nothing
    for (int s = blockIdx.x; s < plan.n_seq; s += gridDim.x) {
      if (plan.len[s] > 0) continue;
      const int64_t first = q_first(a, s);
      for (int q = 0; q < plan.nq[s]; ++q)
        for (int i = threadIdx.x; i < a.n_heads * HD; i += C::T) a.out[(first + q) * a.out_stride + i] = 0.f;
    }
    c0 = blockIdx.x * plan.per * W;
    if (c0 >= plan.total) return;
    c1 = min(c0 + plan.per * W, plan.total);
    u0 = min(c0 + warp * plan.per, c1);
    u1 = min(u0 + plan.per, c1);
  }
  const int n_it = static_cast<int>(u1 - u0);
  unsigned char* my_ring = ring + warp * ST * 2 * BB;
  const int ppb = a.c.page_size / kQ4Block;  // blocks per page

  // Issue unit number i of this warp: lane i % 32 knows its address (found for
  // 32 units at a time, a lane each).
  const uint8_t *src0 = nullptr, *src1 = nullptr;
  int src_flag = 0;
  auto locate = [&](int i) {
    if (i >= n_it) return;
    const unsigned long long u = u0 + i;
    int s = cl_s, kvh = cl_kvh, t0, seen;
    if constexpr (CL) {
      t0 = static_cast<int>(u) * kUnit;
      seen = cl_len;
    } else {
      s = plan.seq_of(u);
      const unsigned long long uq = u - plan.pre[s];
      const int nb = plan.units(s);
      const unsigned long long seg = udiv(uq, nb);
      t0 = (static_cast<int>(uq - seg * nb) - C::LEAD) * kUnit;
      const int rt = plan.tile_of(s, seg, &kvh);
      seen = plan.seen(s, min(rt * R + R, plan.nq[s] * plan.G) - 1);
    }
    src0 = src1 = nullptr;
    src_flag = t0 >= 0 && t0 < seen ? 0 : 4;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = t0 + j * kQ4Block;
      if (t < 0 || t >= seen) break;
      const int slot = t / a.c.page_size;
      const int page = slot < a.c.table_stride ? a.c.table[static_cast<size_t>(s) * a.c.table_stride + slot] : -1;
      if (page < 0 || page >= a.c.n_pages) {
        src_flag |= 1 << j;
        continue;
      }
      (j ? src1 : src0) = a.c.pages + static_cast<size_t>(page) * a.c.page_bytes +
                          (static_cast<size_t>(kvh) * ppb + (t - slot * a.c.page_size) / kQ4Block) * BB;
    }
  };
  bool dead = false;  // a copy that did not arrive within the wait's limit: the rows become NaN
  int issued = 0, issue_st = 0;
  auto issue = [&] {
    if (issued >= n_it || dead) return;
    if ((issued & 31) == 0) locate(issued + lane);
    if (lane == (issued & 31)) {
      flag[issue_st] = src_flag;
      unsigned char* to = my_ring + issue_st * 2 * BB;
      mbar_arrive_expect_tx(&bar[issue_st], (src0 ? BB : 0) + (src1 ? BB : 0));
      if (src1 == src0 + BB && src0) {
        bulk_g2s(to, src0, 2 * BB, &bar[issue_st]);
      } else {
        if (src0) bulk_g2s(to, src0, BB, &bar[issue_st]);
        if (src1) bulk_g2s(to + BB, src1, BB, &bar[issue_st]);
      }
    }
    ++issued;
    issue_st = issue_st + 1 == ST ? 0 : issue_st + 1;
  };
  // ---- the segment of unit u: one (sequence, kv head, tile of rows)
  unsigned long long u = u0, seg0 = 0, seg1 = c1;
  int s = cl_s, kvh = cl_kvh, rt = cl_rt, rows = plan.G, min_seen = cl_len, n_rows = 0;
  auto segment = [&] {
    if constexpr (!CL) {
      while (plan.pre[s + 1] <= u) ++s;
      const int nb = plan.units(s);
      const unsigned long long seg = udiv(u - plan.pre[s], nb);
      seg0 = plan.pre[s] + seg * nb;
      seg1 = seg0 + nb;
      rt = plan.tile_of(s, seg, &kvh);
      rows = plan.nq[s] * plan.G;
      min_seen = plan.seen(s, rt * R);
    }
    n_rows = min(R, rows - rt * R);
  };
  // A lane's operand column is a pair's high or low part; its elements of query row
  // (rows past the last repeat it) t:
  const int pair = lane >> 3, part = (lane >> 2) & 1;
  auto row_of = [&](int t) {
    const int row = rt * R + min(t * 4 + pair / GV, n_rows - 1);
    return a.q + (q_first(a, s) + plan.query(row)) * a.q_stride +
           static_cast<int64_t>(kvh * plan.G + (row - plan.query(row) * plan.G)) * HD + pair % GV * NS * 32 + 8 * c;
  };
  if (u < u1) {  // on their way while the first units' pages are looked up and their copies issued
    if constexpr (!CL) s = plan.seq_of(u);
    segment();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float* q = row_of(t);
#pragma unroll
      for (int k = 0; k < NS; ++k) asm volatile("prefetch.global.L1 [%0];" ::"l"(q + k * 32));
    }
  }
  for (int i = 0; i < ST - 1; ++i) issue();

  const Unpack unpack;
  int rel = 0, st = 0, phase = 0;  // the warp's next unit, counted from u0, and its stage
  int goes_on = 0;
  bool begun = false;
  while (u < u1) {
    const unsigned long long uend = min(seg1, u1);
    const int rel_end = static_cast<int>(uend - u0);
    const int unit0 = static_cast<int>(static_cast<long long>(u0 - seg0)) - (CL ? 0 : C::LEAD);  // unit rel is the segment's rel + unit0

    // ---- the query rows as column operands
    int seen[NT];
    uint32_t qb[NT][NG][2][2];
    float zh[NT][NS], zl[NT][NS], fac[NT][NS];
    if (CL || uend > seg0 + C::LEAD) {  // (else the run ends before the segment's first positions)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float* q = row_of(t);
        seen[t] = CL ? cl_len : plan.seen(s, rt * R + min(t * 4 + h, n_rows - 1));
        // A power of two for each group of 32 brings its largest element to 2^10
        // .. 2^11; the high part is then the nearest whole number, so that a
        // group's sum of high parts times codes is exact in the tensor cores' f32,
        // which truncate (f16 parts with their own exponents cost four times
        // the error).  (The clip of fac is met past 2^113, where distinct
        // scores differ by more than 2^80 however they are scaled.)
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          float x[8], m = 0.f, z = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = q[k * 32 + i] * a.scale;
            m = fmaxf(m, fabsf(x[i]));
          }
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
          const int e = max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -100);
          const float f = pow2(10 - e);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float y = x[i] * f;
            x[i] = part ? round_f16(y - rintf(y)) : rintf(y);
            z += x[i];  // (counts what the operand holds)
          }
          z += __shfl_xor_sync(0xFFFFFFFFu, z, 1);
          z += __shfl_xor_sync(0xFFFFFFFFu, z, 2);
          z *= -8.f * 0x1p-24f;
          zh[t][k] = __shfl_sync(0xFFFFFFFFu, z, c * 8);
          zl[t][k] = __shfl_sync(0xFFFFFFFFu, z, c * 8 + 4);
          fac[t][k] = __shfl_sync(0xFFFFFFFFu, pow2(min(24 - 10 + e, 127)), c * 8);
          zl[t][k] *= fac[t][k];
#pragma unroll
          for (int v = 0; v < GV; ++v) {
            const float on = v == pair % GV ? 1.f : 0.f;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              qb[t][v * NS + k][w][0] = pack_f16(on * x[2 * w], on * x[2 * w + 4]);
              qb[t][v * NS + k][w][1] = pack_f16(on * 0.0625f * x[2 * w + 1], on * 0.0625f * x[2 * w + 5]);
            }
          }
        }
      }
    }

    float o[NT][NG * 2][4], l[NT], ref[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      l[t] = 0.f;
      ref[t] = kNoRef;
#pragma unroll
      for (int i = 0; i < NG * 2; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
    }

    // ---- this warp's units of it
    // positions of operand rows r and r + 8 in a block
    const int b0 = 4 * (r >> 1) + (r & 1), b1 = b0 + 2;
    auto blocks = [&](auto masked_c, const unsigned char* from, int t0, int bad) {
      constexpr bool masked = decltype(masked_c)::value;
      float sc[NT][2 * JB];  // positions b0, b1 of each block
      const int at0 = (b0 * NG + gv * NS) * 2, at1 = (b1 * NG + gv * NS) * 2;  // their scales
      constexpr int SW = NS == 4 ? 2 : 1;  // words of a position's scales
      auto scale_words = [&](const unsigned char* p, uint32_t (&w)[SW]) {
        if constexpr (NS == 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          w[0] = v.x;
          w[1] = v.y;
        } else if constexpr (NS == 2) {
          w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
          w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
      };
      auto scales = [&](const uint32_t (&w)[SW], float (&d)[NS]) {
#pragma unroll
        for (int i = 0; i < SW; ++i) {
          const float2 x = unpack_f16(w[i]);
          d[2 * i] = x.x;
          if constexpr (NS > 1) d[2 * i + 1] = x.y;
        }
      };
      uint32_t vw[2 * JB][SW];  // the V scales as they lie
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        const unsigned char* blk = from + j * BB;
        // scores of the block's two positions
        float ks0[NS], ks1[NS];
        uint32_t kw0[SW], kw1[SW];
        scale_words(blk + q4_ks_off(HD) + at0, kw0);
        scale_words(blk + q4_ks_off(HD) + at1, kw1);
        scales(kw0, ks0);
        scales(kw1, ks1);
        scale_words(blk + q4_vs_off(HD) + at0, vw[2 * j]);
        scale_words(blk + q4_vs_off(HD) + at1, vw[2 * j + 1]);
        uint32_t k0[NG], k1[NG];
        const unsigned char* kr = blk + r * (HD / 2) + c * (4 * NG);
        if constexpr (HD == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(kr), w = *reinterpret_cast<const uint4*>(kr + 512);
          k0[0] = v.x; k0[1] = v.y; k0[2] = v.z; k0[3] = v.w;
          k1[0] = w.x; k1[1] = w.y; k1[2] = w.z; k1[3] = w.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(kr), w = *reinterpret_cast<const uint2*>(kr + 256);
          k0[0] = v.x; k0[1] = v.y;
          k1[0] = w.x; k1[1] = w.y;
        }
        float d[NT][NS][4];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int k = g % NS;
          const uint32_t p = k0[g], q = k1[g], p8 = p >> 8, q8 = q >> 8;
          const uint32_t a0[4] = {p & unpack.lo, q & unpack.lo, p & unpack.hi, q & unpack.hi};
          const uint32_t a1[4] = {p8 & unpack.lo, q8 & unpack.lo, p8 & unpack.hi, q8 & unpack.hi};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (g < NS)
              mma_f16(d[t][k], a0, qb[t][g][0][0], qb[t][g][0][1], 0.f, 0.f, 0.f, 0.f);
            else
              mma_f16(d[t][k], a0, qb[t][g][0][0], qb[t][g][0][1]);
            mma_f16(d[t][k], a1, qb[t][g][1][0], qb[t][g][1][1]);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int k = 0; k < NS; ++k) {
            // (the high parts' sum and its -8 sum q are whole: their difference is exact)
            s0 = fmaf(ks0[k], fmaf(fac[t][k], d[t][k][0] + zh[t][k] + d[t][k][1], zl[t][k]), s0);
            s1 = fmaf(ks1[k], fmaf(fac[t][k], d[t][k][2] + zh[t][k] + d[t][k][3], zl[t][k]), s1);
          }
#pragma unroll
          for (int x = 1; x < GV; x <<= 1) {
            s0 += __shfl_xor_sync(0xFFFFFFFFu, s0, x);
            s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, x);
          }
          if (masked) {
            if (t0 + j * kQ4Block + b0 >= seen[t] || (bad >> j & 1)) s0 = -INFINITY;
            if (t0 + j * kQ4Block + b1 >= seen[t] || (bad >> j & 1)) s1 = -INFINITY;
          }
          sc[t][2 * j] = s0;
          sc[t][2 * j + 1] = s1;
        }
      }

      // p * scale as column operands.  The reference stays while a lane's products have
      // a sum of squares up to 2^30, so each is at most 2^15 (f16 ends at 2^16), and no
      // sum of p passes 2^100; else it moves to where the largest product is 2^12, or to
      // 60 below the largest score where that is more (a position whose scale is 0
      // has a p too).  Squares, two to an operation, cost less than maxima.
      uint32_t pb[JB][NT][NS][2];
      float sum[NT];
#pragma unroll 1
      for (bool again = false;; again = true) {
        // (converted within the loop: as f32 they would take more registers on the other path)
#pragma unroll
        for (int i = 0; i < 2 * JB * SW; ++i) asm volatile("" : "+r"(vw[i / SW][i % SW]));
        float top0 = 0.f, top1 = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) sum[t] = l[t];
#pragma unroll
        for (int j = 0; j < JB; ++j) {
          float vs0[NS], vs1[NS];
          scales(vw[2 * j], vs0);
          scales(vw[2 * j + 1], vs1);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float p0 = ex2(sc[t][2 * j] - ref[t]), p1 = ex2(sc[t][2 * j + 1] - ref[t]);
            sum[t] += p0 + p1;
#pragma unroll
            for (int k = 0; k < NS; ++k) {
              float w0, w1;
              mul_f32x2(w0, w1, p0, p1, vs0[k], vs1[k]);
              if (masked) {  // a NaN scale of a position that this row does not see
                if (t0 + j * kQ4Block + b0 >= seen[t] || (bad >> j & 1)) w0 = 0.f;
                if (t0 + j * kQ4Block + b1 >= seen[t] || (bad >> j & 1)) w1 = 0.f;
              }
              square_f32x2(top0, top1, w0, w1);
              pb[j][t][k][0] = transpose_f16(split_f16(w0));
              pb[j][t][k][1] = transpose_f16(split_f16(w1));
            }
          }
        }
        bool grow = !(top0 + top1 <= 0x1p30f);  // (a NaN may hide another one)
#pragma unroll
        for (int t = 0; t < NT; ++t) grow |= sum[t] > 0x1p100f;
        if (!__any_sync(0xFFFFFFFFu, grow) || again) break;
        float best[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) best[t] = ref[t];
#pragma unroll
        for (int i = 0; i < 2 * JB; ++i) {
          float v[NS], size = 0.f;
          scales(vw[i], v);
#pragma unroll
          for (int k = 0; k < NS; ++k) size = fmaxf(size, fabsf(v[k]) <= 65504.f ? fabsf(v[k]) : 0.f);  // (not NaN or infinite)
          const float high = fmaxf(__log2f(size) - 12.f, -60.f);
#pragma unroll
          for (int t = 0; t < NT; ++t) best[t] = fmaxf(best[t], sc[t][i] + high);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) best[t] = fmaxf(best[t], __shfl_xor_sync(0xFFFFFFFFu, best[t], x));
          const float k = ex2(ref[t] - best[t]);
          ref[t] = best[t];
          l[t] *= k;
#pragma unroll
          for (int i = 0; i < NG * 2; ++i) {
            o[t][i][0] *= k; o[t][i][1] *= k; o[t][i][2] *= k; o[t][i][3] *= k;
          }
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) l[t] = sum[t];
      // Sums of V: those of the blocks at hand by MMA, to the running ones by
      // rounded adds (the MMA truncates: 100 in a row lose 2e-6 of a long average).
      uint4 v0[JB];
      [[maybe_unused]] uint4 v1[JB];
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        const unsigned char* vr = from + j * BB + q4_v_off(HD) + c * 128 + r * 16;
        v0[j] = *reinterpret_cast<const uint4*>(vr);
        if constexpr (HD == 128) v1[j] = *reinterpret_cast<const uint4*>(vr + 512);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float d[NT][2][4];
#pragma unroll
        for (int j = 0; j < JB; ++j) {
          const uint32_t sel = g & 1 ? 0x7632u : 0x5410u;
          uint32_t x0, x1;
          if constexpr (HD == 128) {
            x0 = __byte_perm(g < 2 ? v0[j].x : v0[j].y, g < 2 ? v0[j].z : v0[j].w, sel);
            x1 = __byte_perm(g < 2 ? v1[j].x : v1[j].y, g < 2 ? v1[j].z : v1[j].w, sel);
          } else {
            x0 = __byte_perm(v0[j].x, v0[j].y, sel);
            x1 = __byte_perm(v0[j].z, v0[j].w, sel);
          }
          const uint32_t a0[4] = {unpack.low(x0), unpack.high(x0), unpack.low(x1), unpack.high(x1)};
          x0 >>= 8;
          x1 >>= 8;
          const uint32_t a1[4] = {unpack.low(x0), unpack.high(x0), unpack.low(x1), unpack.high(x1)};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint32_t q0 = pb[j][t][g % NS][0], q1 = pb[j][t][g % NS][1];
            if (j == 0) {
              mma_f16(d[t][0], a0, q0, q1, 0.f, 0.f, 0.f, 0.f);
              mma_f16(d[t][1], a1, q0, q1, 0.f, 0.f, 0.f, 0.f);
            } else {
              mma_f16(d[t][0], a0, q0, q1);
              mma_f16(d[t][1], a1, q0, q1);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            add_f32x2(o[t][2 * g][i], o[t][2 * g][i + 1], d[t][0][i], d[t][0][i + 1]);
            add_f32x2(o[t][2 * g + 1][i], o[t][2 * g + 1][i + 1], d[t][1][i], d[t][1][i + 1]);
          }
      }
    };
    for (; rel < rel_end; ++rel) {
      issue();
      __syncwarp();
      if (!dead && !mbar_wait_warp(&bar[st], phase)) {
        dead = true;
        mbar_ring_drain(bar, ST);
      }
      const int t0 = (rel + unit0) * kUnit;
      const int fl = flag[st];
      const unsigned char* at = my_ring + st * 2 * BB;
      if (++st == ST) {
        st = 0;
        phase ^= 1;
      }
      if (fl || dead) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          if (((fl & 1 || dead) && t0 < seen[t]) || (fl & 2 && t0 + kQ4Block < seen[t])) l[t] = kNaN;
      }
      if (fl < 4 && !dead) {  // (a block without a page counts as behind the end: rows that see it are NaN already)
#pragma unroll 1
        for (int j = 0; j < 2; j += JB) {
          if (fl || t0 + kUnit > min_seen)
            blocks(std::true_type{}, at + j * BB, t0 + j * kQ4Block, fl >> j);
          else
            blocks(std::false_type{}, at + j * BB, t0 + j * kQ4Block, 0);
        }
      }
      __syncwarp();  // every lane has read the stage before it is filled again
    }

    // ---- the end of the segment, or of the run
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[t] += __shfl_xor_sync(0xFFFFFFFFu, l[t], x);
    if (!CL && u0 <= seg0 && seg1 <= u1) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t * 4 + h >= n_rows) continue;
        const int row = rt * R + t * 4 + h;
        float* out = a.out + (q_first(a, s) + plan.query(row)) * a.out_stride +
                     static_cast<int64_t>(kvh * plan.G + (row - plan.query(row) * plan.G)) * HD + r;
        const float inv = l[t] == 0.f ? 0.f : 1.f / l[t];
#pragma unroll
        for (int g = 0; g < NG; ++g)
          if (g / NS == gv) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float (&d)[4] = o[t][2 * g + i];
              out[32 * g + 16 * i] = inv == 0.f && l[t] == 0.f ? 0.f : (d[0] + d[1]) * inv;
              out[32 * g + 16 * i + 8] = inv == 0.f && l[t] == 0.f ? 0.f : (d[2] + d[3]) * inv;
            }
          }
      }
    } else {
      if (!CL && lane == 0) {
        const Shared sh{seg0, seg1, q_first(a, s), n_rows, rt * R, kvh * plan.G};
        shared[warp] = sh;
        if (u == c0) shared[W] = sh;
      }
      goes_on = u0 <= seg0;  // (else it is the run's first, begun before it)
      begun |= u == c0 && seg0 < c0;
      float* to = !CL && u0 <= seg0 ? reinterpret_cast<float*>(my_ring) : parts + warp * PART;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float* mo = to + (t * 4 + h) * LD + r;
#pragma unroll
        for (int g = 0; g < NG; ++g)
          if (g / NS == gv) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float (&d)[4] = o[t][2 * g + i];
              mo[32 * g + 16 * i] = d[0] + d[1];
              mo[32 * g + 16 * i + 8] = d[2] + d[3];
            }
          }
        if (r == 0) {
          to[R * LD + t * 4 + c] = ref[t] == kNoRef && l[t] == 0.f ? -INFINITY : ref[t];
          to[R * LD + P + t * 4 + c] = l[t];
        }
      }
    }
    u = uend;
    if (!CL && u < u1) segment();
  }
  if constexpr (CL) {
    // ---- the cluster's parts into one: the CTA's warps' first, in its ring
    // (done with by all of them), then each CTA a share of the outputs
    if (u0 >= u1 && lane < P) parts[warp * PART + R * LD + lane] = -INFINITY;
    __syncthreads();
    float* mine = reinterpret_cast<float*>(ring);  // [R][HD], [P] ref, [P] sum p
    auto emit = [&](int i, float v, float ls) {
      const int hr = i / HD, row = cl_rt * R + hr;
      if (row < plan.G)
        a.out[cl_s * a.out_stride + static_cast<int64_t>(cl_kvh * plan.G + row) * HD + i % HD] = ls == 0.f ? 0.f : v / ls;
    };
    for (int i = threadIdx.x; i < R * HD; i += C::T) {
      const int hr = i / HD, d = i % HD, pr = hr * GV + d / 32 / NS;
      float top = -INFINITY, acc = 0.f, ls = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) top = fmaxf(top, parts[k * PART + R * LD + pr]);
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const float* part = parts + k * PART;
        const float pf = part[R * LD + pr];
        if (pf > -INFINITY) {
          const float f = ex2(pf - top);
          acc += f * part[hr * LD + d];
          ls += f * part[R * LD + P + pr];
        }
      }
      if (cluster == 1) {
        emit(i, acc, ls);
      } else {
        mine[i] = acc;
        if (d % (32 * NS) == 0) {
          mine[R * HD + pr] = top;
          mine[R * HD + P + pr] = ls;
        }
      }
    }
    if (cluster == 1) return;
    cluster_sync();
    const int share = R * HD / cluster, rank = blockIdx.x % cluster;
    for (int i = rank * share + threadIdx.x; i < (rank + 1) * share; i += C::T) {
      const int pr = i / HD * GV + i % HD / 32 / NS;
      float ref[8], sum[8], val[8], top = -INFINITY, acc = 0.f, ls = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < cluster) {
          ref[k] = ld_cluster(mine + R * HD + pr, k);
          sum[k] = ld_cluster(mine + R * HD + P + pr, k);
          val[k] = ld_cluster(mine + i, k);
        }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < cluster) top = fmaxf(top, ref[k]);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < cluster && ref[k] > -INFINITY) {
          const float f = ex2(ref[k] - top);
          acc += f * val[k];
          ls += f * sum[k];
        }
      emit(i, acc, ls);
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
    return;
  }
  // bit 0: the warp's run ends inside a segment that began in it; bit 1: the CTA's begins inside one
  if (lane == 0) ends[warp] = goes_on | (warp == 0 && begun ? 2 : 0);
  __syncthreads();
  unsigned last_shared = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) last_shared |= (ends[w] & 1) << w;
  const bool first_shared = ends[0] & 2;

  // ---- segments that several warps share, or that another CTA shares: the one
  // that began before the CTA's run, and those that begin in a warp's run and go on behind it
  // (four elements a thread, the segments dealt over the threads left)
  constexpr int kQuads = R * HD / 4, kDeal = C::T / kQuads > 1 ? C::T / kQuads : 1;
  for (int w = -1 + static_cast<int>(threadIdx.x) / kQuads % kDeal; w < W; w += kDeal) {
    const int w_ = max(w, 0);
    const unsigned long long w0 = c0 + w_ * plan.per;
    if (w0 >= c1) break;
    if (w < 0 ? !first_shared : !(last_shared >> w & 1)) continue;
    const Shared sh = shared[w < 0 ? W : w];
    const int last = static_cast<int>(udiv(min(sh.seg1, c1) - 1 - c0, static_cast<unsigned>(plan.per)));
    const bool whole = c0 <= sh.seg0 && sh.seg1 <= c1;
    const float* head = w >= 0 ? reinterpret_cast<const float*>(ring + w * ST * 2 * BB) : parts;
    // slot 0: a segment of the CTA's first unit; slot 1: one that begins later
    float* to = static_cast<float*>(a.scratch) +
                (static_cast<size_t>(blockIdx.x) * 2 + (sh.seg0 <= c0 ? 0 : 1)) * partial_floats(HD);
    for (int i = (kDeal > 1 ? threadIdx.x % kQuads : threadIdx.x) * 4; i < R * HD; i += (kDeal > 1 ? kQuads : C::T) * 4) {
      const int hr = i / HD, d = i % HD, pr = hr * GV + d / 32 / NS;
      float top = head[R * LD + pr];
      for (int k = w_ + 1; k <= last; ++k) top = fmaxf(top, parts[k * PART + R * LD + pr]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float ls = 0.f;
      for (int k = w_; k <= last; ++k) {
        const float* from = k == w_ ? head : parts + k * PART;
        const float pf = from[R * LD + pr];
        const float4 v = *reinterpret_cast<const float4*>(from + hr * LD + d);
        const float sum = from[R * LD + P + pr];
        if (pf > -INFINITY) {
          const float f = ex2(pf - top);
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
          ls += f * sum;
        }
      }
      if (whole) {
        if (hr < sh.n_rows) {
          const int row = sh.row0 + hr;
          float* out = a.out + (sh.token + plan.query(row)) * a.out_stride +
                       static_cast<int64_t>(sh.head0 + (row - plan.query(row) * plan.G)) * HD + d;
          out[0] = ls == 0.f ? 0.f : acc.x / ls;
          out[1] = ls == 0.f ? 0.f : acc.y / ls;
          out[2] = ls == 0.f ? 0.f : acc.z / ls;
          out[3] = ls == 0.f ? 0.f : acc.w / ls;
        }
      } else {
        *reinterpret_cast<float4*>(to + i) = acc;
        if (d % (32 * NS) == 0) {
          to[8 * HD + pr] = top;
          to[8 * HD + 8 + pr] = ls;
        }
      }
    }
  }
}

// Joins the partials of the segment that a CTA's run of units begins and does
// not end: two blocks for each run (one where a tile has one row), half the rows each.
template <int HD, int NT, int GV>
__global__ void __launch_bounds__(kCombine) k_attention_q4_join(Q4AttnArgs a) {
  using C = Cfg<HD, NT, GV>;
  constexpr int NS = C::NS, R = C::R, B = C::B, RB = R / B;
  extern __shared__ __align__(128) unsigned char sm[];
  const int run = blockIdx.x / B, row0 = blockIdx.x % B * RB;
  const Plan plan = make_plan(a, R, C::W, C::LEAD, kCtas, sm);
  const unsigned long long per = plan.per * C::W, u0 = run * per, u1 = u0 + per;
  bool mine = u1 < plan.total;  // something behind this run
  int s = 0, nb = 1;
  unsigned long long seg = 0, seg0 = 0, seg1 = 0;
  if (mine) {
    s = plan.seq_of(u1 - 1);
    nb = plan.units(s);
    seg = udiv(u1 - 1 - plan.pre[s], nb);
    seg0 = plan.pre[s] + seg * nb;
    seg1 = seg0 + nb;
    mine = seg0 >= u0 && seg1 > u1;  // else begun by an earlier run, or ended by this one
  }
  pdl_wait();
  pdl_launch_dependents();
  if (!mine) return;
  int kvh;
  const int rt = plan.tile_of(s, seg, &kvh);
  const int n_rows = plan.nq[s] * plan.G - rt * R - row0;
  if (n_rows <= 0) return;
  const int runs = static_cast<int>((seg1 - 1) / per) - run + 1;
  const float* first = static_cast<const float*>(a.scratch) +
                       (static_cast<size_t>(run) * 2 + (seg0 == u0 ? 0 : 1)) * partial_floats(HD);
  const float* rest = static_cast<const float*>(a.scratch) + static_cast<size_t>(run) * 2 * partial_floats(HD);
  auto part = [&](int k) { return k ? rest + static_cast<size_t>(k) * 2 * partial_floats(HD) : first; };
  constexpr int PB = RB * GV;
  __shared__ float wt[kCtas * PB], lsum[PB];  // each partial's weight and the sum p, for the block's column pairs
  __shared__ float4 red[kCombine];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < PB) {  // a warp per column pair
    const int pr = row0 * GV + warp;
    float ref = -INFINITY, ls = 0.f, refs[4], sums[4];  // (128 runs at once)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool on = lane + 32 * j < runs;
      refs[j] = on ? part(lane + 32 * j)[8 * HD + pr] : -INFINITY;
      sums[j] = on ? part(lane + 32 * j)[8 * HD + 8 + pr] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) ref = fmaxf(ref, refs[j]);
    for (int k = lane + 128; k < runs; k += 32) ref = fmaxf(ref, part(k)[8 * HD + pr]);
    ref = warp_max(ref);
    auto weigh = [&](int k, float pf, float sum) {
      const float w = pf > -INFINITY ? ex2(pf - ref) : 0.f;
      wt[k * PB + warp] = w;
      if (pf > -INFINITY) ls += w * sum;
    };
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 32 * j < runs) weigh(lane + 32 * j, refs[j], sums[j]);
    for (int k = lane + 128; k < runs; k += 32) weigh(k, part(k)[8 * HD + pr], part(k)[8 * HD + 8 + pr]);
    ls = warp_sum(ls);
    if (lane == 0) lsum[warp] = ls;
  }
  // four elements a thread, the partials dealt over the threads left; loaded before their weights are known
  constexpr int kQuads = RB * HD / 4, kDeal = kCombine / kQuads, kAhead = 8;
  const int i = threadIdx.x % kQuads * 4, deal = threadIdx.x / kQuads;
  const int hr = i / HD, d = i % HD, pair = hr * GV + d / 32 / NS;
  float4 ahead[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (deal + j * kDeal < runs) ahead[j] = *reinterpret_cast<const float4*>(part(deal + j * kDeal) + row0 * HD + i);
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int k, const float4& v) {
    const float w = wt[k * PB + pair];
    acc.x += w * v.x;
    acc.y += w * v.y;
    acc.z += w * v.z;
    acc.w += w * v.w;
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (deal + j * kDeal < runs) add(deal + j * kDeal, ahead[j]);
  for (int k = deal + kAhead * kDeal; k < runs; k += kDeal)
    add(k, *reinterpret_cast<const float4*>(part(k) + row0 * HD + i));
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
    const float ls = lsum[pair];
    const int row = rt * R + row0 + hr;
    float* out = a.out + (q_first(a, s) + plan.query(row)) * a.out_stride +
                 static_cast<int64_t>(kvh * plan.G + (row - plan.query(row) * plan.G)) * HD + d;
    out[0] = ls == 0.f ? 0.f : acc.x / ls;
    out[1] = ls == 0.f ? 0.f : acc.y / ls;
    out[2] = ls == 0.f ? 0.f : acc.z / ls;
    out[3] = ls == 0.f ? 0.f : acc.w / ls;
  }
}

// CTAs of a cluster for each segment, or 0 for equal runs of units.  The lengths
// are on the device: what the host knows is how many positions the table holds.
// Clusters win up to about six units a warp (us, clusters and runs; 16/8 heads of 128:
// 1 x 575 7.2 and 10.1, 1 x 8192 11.1 and 12.4, 33 ragged to 1024 11.2 and 14.2, 64 x
// 1024 24.2 and 28.8; 32/8: 33 ragged to 1024 13.3 and 17.8), runs behind that, the
// more the less equal the lengths are (16/8: 1 x 16384 16.1 and 14.6, 33 ragged to
// 4160 33.4 and 18.7).
int use_clusters(const Q4AttnArgs& a, int rows, int warps) {
  if (a.q_start) return 0;
  const int64_t segments = static_cast<int64_t>(a.c.n_seq) * a.c.n_kv * ((a.n_heads / a.c.n_kv + rows - 1) / rows);
  const int64_t units = (static_cast<int64_t>(a.c.table_stride) * a.c.page_size + kUnit - 1) / kUnit;
  int x = 8;
  while (x > 1 && segments * x > kCtas) x /= 2;
  return segments <= 4 * kCtas && units <= 6 * x * warps ? x : 0;
}

template <int HD, int NT, int GV>
cudaError_t launch(const Q4AttnArgs& a, cudaStream_t st) {
  const int clusters = use_clusters(a, Cfg<HD, NT, GV>::R, Cfg<HD, NT, GV>::W);
  using C = Cfg<HD, NT, GV>;
  const size_t plan_b = plan_bytes(a.c.n_seq), smem = C::smem + plan_b;
  static unsigned long long done = 0, done_cl = 0;
  if (clusters) {
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&k_attention_q4<HD, NT, GV, true>), C::smem, &done_cl);
    if (e != cudaSuccess) return e;
    const int segments = a.c.n_seq * a.c.n_kv * ((a.n_heads / a.c.n_kv + C::R - 1) / C::R);
    return launch_pdl_clusters(k_attention_q4<HD, NT, GV, true>, clusters, dim3(segments * clusters), C::T, C::smem, st, a,
                               clusters);
  }
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(&k_attention_q4<HD, NT, GV, false>),
                             C::smem + plan_bytes(kQ4MaxSeqs), &done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_attention_q4<HD, NT, GV, false>, dim3(kCtas), C::T, smem, st, a, 0);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_attention_q4_join<HD, NT, GV>, dim3(kCtas * C::B), kCombine, plan_b, st, a);
}

}  // namespace

size_t attention_q4_scratch_bytes(int hd) { return static_cast<size_t>(kCtas) * 2 * partial_floats(hd) * 4; }

cudaError_t launch_attention_q4(const Q4AttnArgs& args, int hd, cudaStream_t st) {
  Q4AttnArgs a = args;
  a.scale *= 1.4426950408889634f;  // scores in log2
  // rows that share a kv head; with q_start their number is on the device
  const int rows = a.q_start ? 8 : a.n_heads / a.c.n_kv;
  if (hd == 128) {
    if (rows == 1) return launch<128, 1, 4>(a, st);
    if (rows == 2) return launch<128, 1, 2>(a, st);
    if (rows <= 4) return launch<128, 1, 1>(a, st);
    return launch<128, 2, 1>(a, st);
  }
  if (rows <= 2) return launch<64, 1, 2>(a, st);
  if (rows <= 4) return launch<64, 1, 1>(a, st);
  return launch<64, 2, 1>(a, st);
}

}  // namespace tqd
