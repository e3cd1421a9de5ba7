// Products of int8 matrices with a scale for each token and each channel:
// y[j][r] = x_scale[j] w_scale[r] sum_c x[j][c] w[r][c].
//
// The sums are exact, so that their order, and how they are split, changes nothing.  The int8
// tensor instructions of this part (an m16n8k32 in 16.3 clocks an SM) have a quarter of the
// rate of f16's (an m16n8k16 in 2.0), and the fifth generation's f16 products are 2.6 times as
// fast again.  Few tokens take them all the same: memory is the bound there.  For more, codes
// become f16 operands (exact), products are exact in the f32 accumulator, and so are sums of
// up to 1024 of them (128 * 128 * 1024 = 2^24); a run of at most 1024 columns is added to a
// 32-bit whole number.
#include <cuda.h>
#include <cuda_runtime.h>

#include "tqd_device.cuh"
#include "tqd_i8.cuh"
#include "tqd_internal.h"

namespace tqd {
namespace {

constexpr int kSms = 152;

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at `p`'s place in CTA `rank` of the cluster.
__device__ __forceinline__ int ld_rank(const int* p, int rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ int4 ld_rank4(const int* p, int rank) {
  uint32_t at;
  int4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// ------------------------------------------------------------- up to 16 tokens
//
// A warp takes 16 rows; lane (g, c) = (lane / 4, lane % 4) holds sixteen bytes of rows g and g + 8 and of
// token g (and 8 + g), which are its share of two 16 x 8 x 32 int8 instructions (the columns' order within 64 does
// not matter, as long as both operands have the same).  The instruction's rate, 32 bytes of weights a clock and
// SM for eight tokens, is above what memory brings (24): nothing is converted.  Each lane copies its own
// bytes into a ring of its own, so that no barrier stands between a copy and its use: 4 steps of it, 64 KB a
// CTA and two CTAs an SM, so that 128 KB an SM are under way.  A step is 128 columns.  kw warps of a CTA and cs CTAs
// of a cluster share 16 rows: piece p of the kw cs has the steps p, p + kw cs, ...
//
// Measured (us, from a graph): 1024 x 1024 of 1 2.1, 4096 x 1024 of 1 2.9 (a launch by itself 1.0), 8192 x 8192 of 1
// 15.1 (4.4 TB/s), 151936 x 1024 of 1 29.6 (5.3 TB/s, 78 % of the measured copy rate; a plain fill of
// that many bytes reaches 5.5 TB/s).  Memory and, below 10 MB, one memory latency after another bound it.
constexpr int kFewWarps = 8;
// Eight tokens in each of kNT instructions.
template <int kNT>
struct FewCfg {
  static constexpr int lines = 2 + kNT;                     // 16-byte words of a lane and half: rows g and g + 8, tokens g, 8 + g, ...
  static constexpr int slot = 2 * lines * 32 * kFewWarps;   // of a step: [half][line][thread]
  static constexpr int depth = kNT == 1 ? 4 : 3;            // steps of the ring
};

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int kNT>
__global__ void __launch_bounds__(32 * kFewWarps, 2) k_i8_few(const I8MatmulArgs a, int kw, int cs, int groups) {
  using Cfg = FewCfg<kNT>;
  extern __shared__ uint4 few_smem[];
  __shared__ int sums[kFewWarps][4 * kNT][32];  // of the warps that share rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int share = kFewWarps / kw, part = warp % kw, rank = blockIdx.x % cs, pieces = kw * cs, piece = rank * kw + part;
  const int steps = ((a.cols + 127) / 128 + pieces - 1) / pieces;
  const int first = blockIdx.x / cs, stride = gridDim.x / cs;
  uint4* ring = few_smem + threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();

  // the next step to copy: of this CTA's row groups in turn
  int f_group = first, f_step = 0, f_slot = 0;
  auto fetch = [&]() {
    if (f_group < groups) {
      const int r = (f_group * share + warp / kw) * 16 + g, col = (f_step * pieces + piece) * 128 + c * 16;
      const int8_t* w0 = a.w + static_cast<int64_t>(min(r, a.rows - 1)) * a.cols;
      const int8_t* w1 = a.w + static_cast<int64_t>(min(r + 8, a.rows - 1)) * a.cols;
      uint4* to = ring + f_slot * Cfg::slot;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = col + k * 64;
        const uint32_t size = at < a.cols ? 16 : 0, dst = smem_addr(to + k * (Cfg::lines * 32 * kFewWarps));
        constexpr uint32_t next = 32 * kFewWarps * 16;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(w0 + (size ? at : 0)), "r"(size) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + next), "l"(w1 + (size ? at : 0)), "r"(size) : "memory");
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
          const int j = t * 8 + g;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (2 + t) * next),
                       "l"(a.x + min(j, a.n - 1) * a.x_stride + (size ? at : 0)), "r"(j < a.n ? size : 0)
                       : "memory");
        }
      }
      if (++f_step == steps) f_step = 0, f_group += stride;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (++f_slot == Cfg::depth) f_slot = 0;
  };
#pragma unroll 1
  for (int i = 0; i < Cfg::depth; ++i) fetch();
  float sx[kNT][2];  // scales of this lane's tokens, and (below) of its rows
#pragma unroll
  for (int t = 0; t < kNT; ++t)
#pragma unroll
    for (int i = 0; i < 2; ++i) sx[t][i] = __ldg(a.x_scale + min(t * 8 + 2 * c + i, a.n - 1));
  int slot = 0;
  for (int group = first; group < groups; group += stride) {
    const int r0 = (group * share + warp / kw) * 16 + g;
    const float sw[2] = {__ldg(a.w_scale + min(r0, a.rows - 1)), __ldg(a.w_scale + min(r0 + 8, a.rows - 1))};
    int total[kNT][4], other[kNT][4];
#pragma unroll
    for (int t = 0; t < kNT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[t][i] = other[t][i] = 0;
    for (int s = 0; s < steps; ++s) {
      asm volatile("cp.async.wait_group %0;" ::"n"(Cfg::depth - 1) : "memory");
      uint4 v[2][Cfg::lines];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < Cfg::lines; ++i) v[k][i] = ring[slot * Cfg::slot + (k * Cfg::lines + i) * 32 * kFewWarps];
      if (++slot == Cfg::depth) slot = 0;
      fetch();  // into the place just read
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
          mma_s8(total[t], v[k][0].x, v[k][1].x, v[k][0].y, v[k][1].y, v[k][2 + t].x, v[k][2 + t].y);
          mma_s8(other[t], v[k][0].z, v[k][1].z, v[k][0].w, v[k][1].w, v[k][2 + t].z, v[k][2 + t].w);
        }
    }
#pragma unroll
    for (int e = 0; e < 4 * kNT; ++e) total[e / 4][e % 4] += other[e / 4][e % 4];
    if (pieces > 1) {
#pragma unroll
      for (int e = 0; e < 4 * kNT; ++e) sums[warp][e][lane] = total[e / 4][e % 4];
      __syncthreads();
      if (cs > 1) {  // the CTA's sums in the place of its first warp's, then the cluster's
#pragma unroll
        for (int e = 0; e < 4 * kNT; ++e) {
          if (kw > 1 && e % kw == part) {
            int s = 0;
            for (int w = warp - part; w < warp - part + kw; ++w) s += sums[w][e][lane];
            sums[warp - part][e][lane] = s;
          }
        }
        cluster_barrier();
      }
    }
    // of the sums of 16 rows, piece p writes every (kw cs)-th
#pragma unroll
    for (int e = 0; e < 4 * kNT; ++e) {
      if (pieces > 1 && e % pieces != piece) continue;
      int s = total[e / 4][e % 4];
      if (cs > 1) {
        s = 0;
        for (int q = 0; q < cs; ++q) s += ld_rank(&sums[warp - part][e][lane], q);
      } else if (kw > 1) {
        s = 0;
        for (int w = warp - part; w < warp - part + kw; ++w) s += sums[w][e][lane];
      }
      const int r = r0 + ((e & 3) >> 1) * 8, j = (e >> 2) * 8 + 2 * c + (e & 1);
      if (r < a.rows && j < a.n) a.y[j * a.y_stride + r] = static_cast<float>(s) * sx[e >> 2][e & 1] * sw[(e & 3) >> 1];
    }
    // (no sum is overwritten, nor a CTA's memory gone, while another reads it)
    if (cs > 1) cluster_barrier();
    else if (kw > 1) __syncthreads();
  }
}

constexpr int kFewClusters[9] = {0, 304, 152, 97, 74, 58, 46, 38, 36};  // of 0 to 8 CTAs that run at once
// How many warps and CTAs share 16 rows, and the groups of rows that a CTA or cluster has at a time: what makes the
// busiest CTA's share least, counted in steps of two CTAs an SM (an SM's only CTA takes 0.6 of that, a group of rows one
// more, joining a cluster two).
void few_split(int rows, int cols, int& kw, int& cs, int& groups) {
  const int tiles = (rows + 15) / 16, pairs = (cols + 127) / 128;
  kw = cs = 1, groups = 0;
  float best = 0.f;
  for (int c = 1; c <= 8 && c <= pairs; c += c < 4 ? 1 : 2) {
    for (int k = 1; k <= kFewWarps && (k == 1 || k * c <= pairs); k *= 2) {
      const int gr = (tiles + kFewWarps / k - 1) / (kFewWarps / k), waves = (gr + kFewClusters[c] - 1) / kFewClusters[c];
      if (c > 1 && waves > 1) break;
      const int steps = (pairs + k * c - 1) / (k * c);
      const float cost = waves * (steps * (static_cast<int64_t>(gr) * c > kSms ? 1.f : 0.6f) + 1.f) + (c > 1 ? 2.f : 0.f);
      if (groups == 0 || cost < best) best = cost, kw = k, cs = c, groups = gr;
    }
  }
}

template <int kNT>
cudaError_t launch_few(const I8MatmulArgs& a, const I8Way& way, cudaStream_t st) {
  using Cfg = FewCfg<kNT>;
  constexpr int kMost = Cfg::depth * Cfg::slot * 16;
  static unsigned long long done = 0;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_i8_few<kNT>), kMost, &done);
  if (e != cudaSuccess) return e;
  const int kw = way.warps, cs = way.cluster, groups = static_cast<int>(way.tiles);
  const int clusters = groups < kFewClusters[cs] ? groups : kFewClusters[cs], pairs = (a.cols + 127) / 128;
  const int steps = (pairs + kw * cs - 1) / (kw * cs) * ((groups + clusters - 1) / clusters);
  return launch_pdl_clusters(k_i8_few<kNT>, static_cast<unsigned>(cs), dim3(static_cast<unsigned>(clusters * cs)), 32 * kFewWarps,
                             (steps < Cfg::depth ? steps : Cfg::depth) * Cfg::slot * 16, st, a, kw, cs, groups);
}

// ------------------------------------------------------------ 9 tokens and more
//
// CTAs, one per SM, make tiles of 128 rows of w by kTN tokens on the fifth-generation tensor cores.  In
// a step of K columns the rows' codes come by a tensor copy as they are, and groups of four warps, a step
// each in turn, make them f16 and put them into tensor memory as operand A (a lane is a row).  The tokens, operand
// B, are f16 in shared memory: up to 64 are made so by the same warps, more come by a bulk copy from an
// image that k_i8_image laid out in the scratch in the order of shared memory.  Other warps take the sums out of
// tensor memory after every 1024 columns and add them up as whole numbers; they write a tile's results while the next
// one's sums are made.
//
// Where there are few tiles a cluster of cs CTAs shares a tile's steps, and each adds up and writes a part of
// its tokens (1024 x 16384 of 40: 13.5 us).
// What bounds a CTA by itself is what its SM takes in: about 57 bytes a clock were the most, of which a step
// of 128 x 128 needs 48 KB, 860 clocks of which the products are 512.  So where there are many tiles a pair of CTAs makes
// 256 rows with one instruction and each brings half of the tokens: 8192 x 8192 of 2048 took 199 us with 128 x 128
// and takes 164 to 169 with pairs of 160 tokens (86 % of the measured bf16 rate), 16384 x 4096 of 4096 378 and 309 (93 %).  Tensor
// memory is what limits a pair's width: two accumulators of kTN columns and the slots of A.  192 tokens leave
// room for four slots of 64 columns only, whose steps are slower for their work (295 ns for 64 columns, 215 for 160 tokens), but 511
// tokens are three tiles of them and four of 160 (5120 x 960: 12.9 and 15.1 us).
constexpr int kBigM = 128;
constexpr int kConverters = 2;               // groups of four warps

template <int kTN, bool kPair>
struct BigCfg {
  static constexpr bool raw_tokens = kTN <= 64;
  static constexpr int K = kTN == 192 ? 64 : 128;                   // columns of a step
  static constexpr int run = 1024 / K;                       // steps that the f32 sums hold
  static constexpr int readers = kTN <= 32 ? 4 : kTN <= 128 ? 8 : 16;  // warps that read sums, 16 to 64 columns each
  static constexpr int threads = 32 * (4 + 4 * kConverters + readers);  // copies, MMAs, two idle; then these
  static constexpr uint32_t w_raw = kBigM * K;               // bytes of the rows' codes in a stage
  static constexpr int ctas = kPair ? 2 : 1;                 // that make a tile's products together
  static constexpr uint32_t image = kTN / ctas * K * 2;                 // bytes of f16 tokens in a stage
  static constexpr uint32_t raw = raw_tokens ? kTN * K : 0;       // bytes of their codes
  static constexpr uint32_t stage = w_raw + image + raw;
  static constexpr int stages = kTN == 192 ? 10 : kPair ? 6 : kTN >= 128 ? 4 : kTN == 64 ? 5 : 7;
  static constexpr int a_stages = kTN == 192 ? 4 : kPair ? 3 : stages;  // of operand A, K / 2 columns each
  static constexpr uint32_t a_col = 2 * kTN;                // behind two accumulators, in turn
  static constexpr size_t smem = stages * stage + 1024;
  static_assert(a_col + a_stages * K / 2 <= 512, "tensor memory");
  static_assert(static_cast<size_t>(kTN) * kBigM * 4 <= stages * stage, "a cluster's sums take the stages' place");
};

template <int kK>
__device__ __forceinline__ uint64_t image_desc(const void* p) {
  // core matrices of 8 tokens x 16 bytes, 128 bytes apart along the columns, kK * 16 along the tokens
  uint64_t d = static_cast<uint64_t>((smem_addr(p) & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(128 >> 4) << 16;
  d |= static_cast<uint64_t>(kK) << 32;
  return d | (1ull << 46);
}

// The products of 16 columns: operand A in tensor memory, B in shared memory; of a pair of CTAs, each with its own
// 128 rows of A and sums, and its half of B.
template <bool kPair>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// An arrival at `bar` (of a pair's CTAs, those of the mask) once the thread's products so far are over.
template <bool kPair>
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint16_t ctas = 3) {
  if (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
        "h"(ctas)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
template <bool kPair>
__device__ __forceinline__ void tmem_alloc(uint32_t* at) {
  if (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(at)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(at)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <bool kPair>
__device__ __forceinline__ void tmem_free(uint32_t at) {
  if (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(at) : "memory");
  else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(at) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t at, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at)
               : "memory");
}
// A box of K bytes a row at (col, row): 16-byte pieces turned as swizzle 128B (64B for 64) does.
__device__ __forceinline__ void copy_box(void* dst, const CUtensorMap* map, int col, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(col), "r"(row), "r"(smem_addr(bar))
      : "memory");
}
// Whether a phase is over, without waiting.
template <bool kPair>
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  if (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
  else
    asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// True in one lane of a whole warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// An arrival at the barrier, of a pair at the first CTA's.  (At its default scope: with .release.cluster
// an arrival took 1450 clocks, so 70.  What it tells of is this CTA's tensor memory and finished copies.)
template <bool kPair>
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  if (kPair) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_addr(bar)));
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(at) : "memory");
  } else {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
  }
}

struct BigArgs {
  const uint8_t* image;  // [steps][tokens, whole groups][K] f16
  const float *x_scale, *w_scale;
  float* y;
  int64_t y_stride;
  int rows, cols, n, padded, steps, row_tiles, token_tiles, cs;
};

template <int kTN, bool kPair>
__global__ void __launch_bounds__(BigCfg<kTN, kPair>::threads, 1)
    k_i8_big(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map, const BigArgs a) {
  using Cfg = BigCfg<kTN, kPair>;
  extern __shared__ uint8_t big_smem[];
  __shared__ uint64_t full[Cfg::stages], ready[Cfg::stages], empty[Cfg::stages], sums_full[2], sums_empty[2], done;
  __shared__ uint32_t tmem_at;
  __shared__ int dead_word;
  volatile int* dead = &dead_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* raw = big_smem + (1024u - (smem_addr(big_smem) & 1023u)) % 1024u;  // [stage] codes of the rows,
  uint8_t* tokens = raw + Cfg::stages * Cfg::w_raw;                             // f16 of the tokens,
  uint8_t* raw_x = tokens + Cfg::stages * Cfg::image;                        // codes of the tokens

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&ready[s], 4 * Cfg::ctas);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sums_full[i], 1);
      mbar_init(&sums_empty[i], Cfg::readers * Cfg::ctas);
    }
    mbar_init(&done, 1);
    dead_word = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc<kPair>(&tmem_at);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  if (kPair) cluster_barrier();  // the other CTA's barriers too
  else __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_at;
  // (an image's kernel begins when all before it have ended, so that what is not the image may be read at once)
  pdl_launch_dependents();
  if (Cfg::raw_tokens) pdl_wait();
  // this CTA's tiles, and its steps of each
  // (of a pair's 256 rows each has 128, and half of the tokens' image; the first one issues the products)
  const int cluster = kPair ? 2 : a.cs, rank = blockIdx.x % cluster, first = blockIdx.x / cluster, stride = gridDim.x / cluster;
  const int tiles = a.row_tiles * a.token_tiles, upper = kPair ? rank * kBigM : 0;
  const int from = kPair ? 0 : static_cast<int>(static_cast<int64_t>(a.steps) * rank / a.cs);
  const int steps = kPair ? a.steps : static_cast<int>(static_cast<int64_t>(a.steps) * (rank + 1) / a.cs) - from;

  if (warp == 0) {
    int s = 0, issued = 0;
    uint32_t phase = 0;
    bool image_there = Cfg::raw_tokens, ok = true;
    for (int tile = first; ok && tile < tiles; tile += stride) {
      const int row0 = tile / a.token_tiles * (kBigM * Cfg::ctas) + upper, j0 = tile % a.token_tiles * kTN;
      const int share = min(kTN, a.padded - j0) / Cfg::ctas, mine = j0 + (kPair ? rank * share : 0);  // tokens of the image
      const uint32_t bytes = Cfg::raw_tokens ? Cfg::raw : share * Cfg::K * 2;
      for (int k = from; k < from + steps; ++k) {
        if (issued >= Cfg::stages) ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_dead(&empty[s], phase ^ 1, dead));
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[s], Cfg::w_raw + bytes);
          copy_box(raw + s * Cfg::w_raw, &w_map, k * Cfg::K, row0, &full[s]);
          if (Cfg::raw_tokens) {
            copy_box(raw_x + s * Cfg::raw, &x_map, k * Cfg::K, j0, &full[s]);
          } else {
            if (!image_there) pdl_wait();  // the kernel before this one writes the image
            bulk_g2s(tokens + s * Cfg::image, a.image + (static_cast<int64_t>(k) * a.padded + mine) * (Cfg::K * 2), bytes, &full[s]);
          }
        }
        image_there = true;
        if (issued < Cfg::stages) ++issued;
        if (++s == Cfg::stages) s = 0, phase ^= 1;
      }
    }
    // Whatever the others do, what is still under way lands before the CTA ends: copies, and each stage's last arrival at
    // empty, which a commit makes by itself, in a pair at both CTAs.  (The oldest first: the last one comes when the
    // products end.  The readers waited for all at sums_full.  After a wait that ran out there may be none to come.)
    if (issued < Cfg::stages) s = 0, phase = 1;
    for (int i = 0; i < issued; ++i) {
      mbar_wait_warp(&full[s], phase ^ 1, kWaitLimitNs / 4);
      mbar_wait_warp(&empty[s], phase ^ 1, *dead ? 1000000ull : kWaitLimitNs / 4);
      if (++s == Cfg::stages) s = 0, phase ^= 1;
    }
  } else if (warp == 1) {
    // One thread, which looks for the next stage while this one's MMAs are issued: the tensor cores hold one or two
    // waiting instructions only, so whatever stands between two steps is time that they lack.  (The loop stands
    // inside elect.sync's branch: in one that the thread's number chooses an instruction takes 94 clocks to issue, here 9.)
    if ((!kPair || rank == 0) && elect_one()) {
      int s = 0, at = 0, run = 0;
      uint32_t phase = 0;
      bool ok = true, there = false;
      const uint64_t desc = image_desc<Cfg::K>(tokens);
      for (int tile = first; ok && tile < tiles; tile += stride) {
        const int width = min(kTN, a.padded - tile % a.token_tiles * kTN);
        const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(width >> 3) << 17) | (static_cast<uint32_t>(kBigM * Cfg::ctas >> 4) << 24);
        int left = (a.cols - from * Cfg::K) / 16;  // instructions of 16 columns (more than this CTA's where others follow)
        for (int k0 = 0; ok && k0 < steps; k0 += Cfg::run, ++run) {
          const uint32_t d = tmem + (run & 1) * kTN;
          if (run >= 2) ok = mbar_wait_or_dead<kPair>(&sums_empty[run & 1], (run / 2 - 1) & 1, dead);
          const int end = min(steps, k0 + Cfg::run);
          for (int k = k0; ok && k < end; ++k, left -= Cfg::K / 16) {
            // (ready follows full: the converting warps waited for that)
            if (!there && !mbar_wait_or_dead<kPair>(&ready[s], phase, dead)) {
              ok = false;
              break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint64_t bd = desc + static_cast<uint32_t>(s) * (Cfg::image >> 4);
            const uint32_t ad = tmem + Cfg::a_col + at * (Cfg::K / 2);
            uint64_t* over = &empty[s];
            if (++s == Cfg::stages) s = 0, phase ^= 1;
            if (++at == Cfg::a_stages) at = 0;
            there = mbar_test<kPair>(&ready[s], phase);
            if (left >= Cfg::K / 16) {
#pragma unroll
              for (int i = 0; i < Cfg::K / 16; ++i) mma_ts<kPair>(d, ad + i * 8, bd + i * 16, idesc, k > k0 || i > 0);
            } else {
              for (int i = 0; i < left; ++i) mma_ts<kPair>(d, ad + i * 8, bd + i * 16, idesc, k > k0 || i > 0);
            }
            mma_commit<kPair>(over);
          }
          if (ok) mma_commit<kPair>(&sums_full[run & 1]);
        }
      }
      mma_commit<kPair>(&done, 1);  // tensor memory is given back once every MMA is over
      mbar_wait_bounded(&done, 0, nullptr, kWaitLimitNs / 4);
    }
  } else if (warp >= 4 && warp < 4 + 4 * kConverters) {
    const int quad = warp & 3, row = quad * 32 + lane;
    constexpr int kPieces = Cfg::K / 16;  // of 16 codes
    const uint32_t turn = Cfg::K == 128 ? (row & 7) * 16 : ((row >> 1) & 3) * 16;
    const int total = (tiles - first + stride - 1) / stride * steps;  // (first < tiles)
    for (int g = warp / 4 - 1; g < total; g += kConverters) {
      const int s = g % Cfg::stages, at = g % Cfg::a_stages;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_or_dead(&full[s], (g / Cfg::stages) & 1, dead))) break;
      const uint8_t* from_w = raw + s * Cfg::w_raw + row * Cfg::K;
      uint4 w[kPieces];
#pragma unroll
      for (int c = 0; c < kPieces; ++c) w[c] = *reinterpret_cast<const uint4*>(from_w + ((c * 16) ^ turn));
      if (Cfg::raw_tokens) {
        // 16 codes a thread: token j, piece c of eight
#pragma unroll
        for (int q = quad * 32 + lane; q < kTN * 8; q += 128) {
          const int c = (q >> 3) & 7, j = (q >> 6) * 8 + (q & 7);
          const uint4 v = *reinterpret_cast<const uint4*>(raw_x + s * Cfg::raw + j * 128 + ((c * 16) ^ ((j & 7) * 16)));
          uint4 lo, hi;
          i8x4_to_f16(v.x, lo.x, lo.y);
          i8x4_to_f16(v.y, lo.z, lo.w);
          i8x4_to_f16(v.z, hi.x, hi.y);
          i8x4_to_f16(v.w, hi.z, hi.w);
          uint4* to = reinterpret_cast<uint4*>(tokens + s * Cfg::image + (j >> 3) * 2048 + c * 256 + (j & 7) * 16);
          to[0] = lo;
          to[8] = hi;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      bool there = true;
      const uint32_t operand = tmem + Cfg::a_col + at * (Cfg::K / 2) + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll
      for (int h = 0; h < kPieces / 4; ++h) {
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          i8x4_to_f16(w[h * 4 + c].x, v[c * 8], v[c * 8 + 1]);
          i8x4_to_f16(w[h * 4 + c].y, v[c * 8 + 2], v[c * 8 + 3]);
          i8x4_to_f16(w[h * 4 + c].z, v[c * 8 + 4], v[c * 8 + 5]);
          i8x4_to_f16(w[h * 4 + c].w, v[c * 8 + 6], v[c * 8 + 7]);
        }
        // (converted before the wait for the operand that stood there to be used)
        if (h == 0 && Cfg::a_stages < Cfg::stages && g >= Cfg::a_stages) {
          const int before = g - Cfg::a_stages;
          there = __all_sync(0xFFFFFFFFu, mbar_wait_or_dead(&empty[before % Cfg::stages], (before / Cfg::stages) & 1, dead));
          if (!there) break;
        }
        tmem_st32(operand + h * 32, v);
      }
      if (!there) break;  // (an operand that may be in use stays; no sums are made without this one)
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive<kPair>(&ready[s]);
    }
  } else if (warp >= 4 + 4 * kConverters) {
    constexpr int kCols = kTN / (Cfg::readers / 4);  // a warp's columns
    const int quad = warp & 3, c0 = (warp - 4 - 4 * kConverters) / 4 * kCols;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    SumsWait sums_there{sums_full, dead};
    for (int tile = first; tile < tiles; tile += stride) {
      const int row = tile / a.token_tiles * (kBigM * Cfg::ctas) + upper + quad * 32 + lane, j0 = tile % a.token_tiles * kTN;
      const int width = min(kTN, a.padded - j0);
      const float sw = row < a.rows ? a.w_scale[row] : 0.f;
      int total[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) total[i] = 0;
      bool ok = true;
      for (int k0 = 0; k0 < steps; k0 += Cfg::run) {
        const int b = sums_there.run & 1;
        ok = sums_there.next();
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
        for (int c = 0; c < kCols; c += 8) {
          if (c0 + c >= width) continue;
          uint32_t r[8];
          tmem_ld8(tmem + b * kTN + c0 + c + lanes, r);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int i = 0; i < 8; ++i) total[c + i] += __float2int_rn(__uint_as_float(r[i]));
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive<kPair>(&sums_empty[b]);
      }
      if (!kPair && a.cs > 1) {  // the stages are done with: the only tile's sums take their place, [token][row]
        int* sums = reinterpret_cast<int*>(raw);
#pragma unroll
        for (int i = 0; i < kCols; ++i) sums[(c0 + i) * kBigM + quad * 32 + lane] = total[i];
      } else {
        // (after a wait that ran out: NaN, in this tile and all that follow)
        const float w_scale = ok ? sw : __uint_as_float(0x7FC00000u);
        float* y = a.y + (j0 + c0) * a.y_stride + row;
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          const int j = j0 + c0 + i;
          if (j < a.n && row < a.rows) *y = static_cast<float>(total[i]) * __ldg(a.x_scale + j) * w_scale;
          y += a.y_stride;
        }
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  if (kPair) cluster_barrier();  // (and no thread arrives at a CTA that is gone)
  else __syncthreads();
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    tmem_free<kPair>(tmem);
  }
  if (!kPair && a.cs > 1) {
    cluster_barrier();
    const int* sums = reinterpret_cast<const int*>(raw);
    const int row0 = first / a.token_tiles * kBigM, j0 = first % a.token_tiles * kTN, width = min(kTN, a.n - j0);
    int gone = 0;  // a wait ran out in one of the CTAs
    for (int q = 0; q < a.cs; ++q) gone |= ld_rank(&dead_word, q);
    // token i of the tile by CTA i mod cs: a thread takes four rows of it
    for (int e = threadIdx.x; e < (width - rank + a.cs - 1) / a.cs * (kBigM / 4); e += Cfg::threads) {
      const int i = e / (kBigM / 4) * a.cs + rank, r = e % (kBigM / 4) * 4;
      int4 t = ld_rank4(&sums[i * kBigM + r], 0);
#pragma unroll 4
      for (int q = 1; q < a.cs; ++q) {
        const int4 o = ld_rank4(&sums[i * kBigM + r], q);
        t.x += o.x, t.y += o.y, t.z += o.z, t.w += o.w;
      }
      const float sx = gone ? __uint_as_float(0x7FC00000u) : __ldg(a.x_scale + j0 + i);
      const int v[4] = {t.x, t.y, t.z, t.w};
      float* y = a.y + (j0 + i) * a.y_stride + row0 + r;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (row0 + r + k < a.rows) y[k] = static_cast<float>(v[k]) * sx * __ldg(a.w_scale + row0 + r + k);
    }
    cluster_barrier();
  }
}

// The tokens' codes as f16 in the order of k_i8_big's shared memory: [step][8 tokens][column / 8][token][8],
// zeros past the last token and column.  A thread takes 16 codes.  (5120 x 960 of 511: 2.1 of the 12.9 us, with its launch.)
template <int kK>
__global__ void __launch_bounds__(256) k_i8_image(const int8_t* x, int64_t x_stride, int n, int cols, int padded, int steps,
                                                  uint8_t* image) {
  pdl_launch_dependents();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int j8 = static_cast<int>(at & 7), c = static_cast<int>((at >> 3) % (kK / 16));
  const int64_t rest = at / (kK / 2);  // (token group, step), the step first
  const int k = static_cast<int>(rest % steps);
  const int64_t group = rest / steps;
  if (group * 8 >= padded) return;
  const int64_t j = group * 8 + j8;
  const int col = k * kK + c * 16;
  uint4 v = make_uint4(0u, 0u, 0u, 0u), p, q;
  if (j < n && col < cols) v = __ldg(reinterpret_cast<const uint4*>(x + j * x_stride + col));
  i8x4_to_f16(v.x, p.x, p.y);
  i8x4_to_f16(v.y, p.z, p.w);
  i8x4_to_f16(v.z, q.x, q.y);
  i8x4_to_f16(v.w, q.z, q.w);
  uint4* dst = reinterpret_cast<uint4*>(image + (static_cast<int64_t>(k) * padded + group * 8) * (kK * 2) + c * 256 + j8 * 16);
  dst[0] = p;
  dst[8] = q;
}

// The map of rows of codes for boxes of box_cols (64 or 128) x box_rows.
cudaError_t map_of(const int8_t* p, int64_t stride, int rows, int cols, int box_cols, int box_rows, CUtensorMap* map) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static void* found = nullptr;  // the driver's function, the same for every device
  void* fn = __atomic_load_n(&found, __ATOMIC_RELAXED);
  if (!fn) {
    cudaDriverEntryPointQueryResult got;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &got);
    if (e != cudaSuccess) return e;
    if (got != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    __atomic_store_n(&found, fn, __ATOMIC_RELAXED);
  }
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)}, steps[2] = {1, 1};
  const CUresult r = reinterpret_cast<Encode>(fn)(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides,
                                                  box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                                  box_cols == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr int kRawMost = 64;  // tokens that k_i8_big takes as codes

// The tokens that its instructions are for: a CTA's come in sixteens, a pair's in thirty-twos.
int padded_tokens(int n) { return n <= kRawMost ? (n + 15) / 16 * 16 : (n + 31) / 32 * 32; }

template <int kTN, bool kPair = false>
cudaError_t launch_big(const I8MatmulArgs& a, int cs, cudaStream_t st) {
  using Cfg = BigCfg<kTN, kPair>;
  static unsigned long long done = 0;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_i8_big<kTN, kPair>), Cfg::smem, &done);
  if (e != cudaSuccess) return e;
  const int steps = (a.cols + Cfg::K - 1) / Cfg::K, padded = padded_tokens(a.n);
  BigArgs b{static_cast<const uint8_t*>(a.scratch), a.x_scale, a.w_scale, a.y, a.y_stride, a.rows, a.cols, a.n, padded, steps,
            (a.rows + kBigM * Cfg::ctas - 1) / (kBigM * Cfg::ctas), (a.n + kTN - 1) / kTN, cs};
  const int64_t tiles = static_cast<int64_t>(b.row_tiles) * b.token_tiles;
  CUtensorMap w_map, x_map;
  e = map_of(a.w, a.cols, a.rows, a.cols, Cfg::K, kBigM, &w_map);
  if (e == cudaSuccess && Cfg::raw_tokens) e = map_of(a.x, a.n > 1 ? a.x_stride : a.cols, a.n, a.cols, Cfg::K, kTN, &x_map);
  if (e != cudaSuccess) return e;
  constexpr int kOnce = kSms / Cfg::ctas;  // tiles that are made at once
  const unsigned grid = static_cast<unsigned>(cs > 1 ? tiles * cs : (tiles < kOnce ? tiles : kOnce) * Cfg::ctas);
  if (Cfg::raw_tokens)
    return launch_pdl_clusters(k_i8_big<kTN, kPair>, static_cast<unsigned>(kPair ? 2 : cs), dim3(grid), Cfg::threads, Cfg::smem, st, w_map, x_map, b);
  x_map = w_map;  // not read
  const int64_t threads = static_cast<int64_t>(padded / 8) * steps * (Cfg::K / 2);
  k_i8_image<Cfg::K><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, st>>>(a.x, a.x_stride, a.n, a.cols, padded, steps,
                                                                           static_cast<uint8_t*>(a.scratch));
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl_clusters(k_i8_big<kTN, kPair>, static_cast<unsigned>(kPair ? 2 : cs), dim3(grid), Cfg::threads, Cfg::smem, st, w_map, x_map, b);
}

}  // namespace

size_t i8_matmul_scratch_bytes(int rows, int cols, int n) {
  if (n <= kRawMost) return 0;
  return static_cast<size_t>(padded_tokens(n)) * ((cols + 127) / 128) * 128 * 2;
}

I8Way i8_matmul_way(int rows, int cols, int n) {
  I8Way way{0, 8, 1, 1, 0, 0};
  // Up to 8 tokens: the int8 instructions keep up with memory (151936 x 1024 of 8: 30.3 us, k_i8_big 31.0).  Up to 16 they
  // do at half the rate, which is faster where a launch and the pipeline's filling are most of the time (4096 x 1024 of 16:
  // 4.4 and 6.2 us; 5120 x 960 5.9 and 7.0; 4096 x 4096 9.6 and 9.2; 151936 x 1024 45 and 31).
  if (n <= 8 || (n <= 16 && static_cast<int64_t>(rows) * cols <= (12 << 20))) {
    if (n > 8) way.tokens = 16;
    int groups;
    few_split(rows, cols, way.warps, way.cluster, groups);
    way.tiles = groups, way.rounds = (groups + kFewClusters[way.cluster] - 1) / kFewClusters[way.cluster];
    return way;
  }
  // The width of a tile and the CTAs that share one: what takes least by these measured times in ns: 128 columns of a
  // tile, an image's kernel, a pair's beginning, a cluster's joining; a tile's beginning and end beside another's steps.
  constexpr int kWidths[6] = {16, 32, 64, 128, 160, 192}, kStep[6] = {320, 350, 430, 460, 430, 590};  // the last two: pairs
  constexpr int kClusters[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};                        // that run at once
  const int64_t row_tiles = (rows + kBigM - 1) / kBigM, steps = (cols + 127) / 128;
  int64_t best = -1;
  for (int i = 0; i < 6; ++i) {
    const bool pair = i >= 4;
    if (kWidths[i] > kRawMost && n <= kRawMost) break;  // (there is no scratch for an image)
    const int64_t tiles = (pair ? (row_tiles + 1) / 2 : row_tiles) * ((n + kWidths[i] - 1) / kWidths[i]);
    for (int c = 1; c <= (pair ? 1 : 8) && c <= steps; ++c) {
      const int once = kClusters[pair ? 2 : c];
      if (c > 1 && tiles > once) break;
      const int64_t rounds = (tiles + once - 1) / once;
      const int64_t cost = rounds * ((steps + c - 1) / c * kStep[i] + 400) + (kWidths[i] > kRawMost ? 1500 : 0) +
                           (pair ? 500 : 0) + (c > 1 ? 1800 + 8 * kWidths[i] : 0);
      if (best < 0 || cost < best) best = cost, way = I8Way{pair ? 2 : 1, kWidths[i], 1, c, tiles, rounds};
    }
  }
  return way;
}

cudaError_t launch_i8_matmul(const I8MatmulArgs& a, cudaStream_t st) {
  const I8Way way = i8_matmul_way(a.rows, a.cols, a.n);
  switch (way.tokens) {
    case 8: return launch_few<1>(a, way, st);
    case 16: return way.kind ? launch_big<16>(a, way.cluster, st) : launch_few<2>(a, way, st);
    case 32: return launch_big<32>(a, way.cluster, st);
    case 64: return launch_big<64>(a, way.cluster, st);
    case 128: return launch_big<128>(a, way.cluster, st);
    case 160: return launch_big<160, true>(a, 1, st);
    default: return launch_big<192, true>(a, 1, st);
  }
}

}  // namespace tqd
