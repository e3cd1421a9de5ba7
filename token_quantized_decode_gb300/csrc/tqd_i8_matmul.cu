// Products of int8 matrices with a scale for each token and each channel:
// y[j][r] = x_scale[j] w_scale[r] sum_c x[j][c] w[r][c].
//
// The sums are exact.  The int8 tensor instructions of this part run at a sixteenth of the
// f16 ones' rate, so codes become f16 operands (exact), products are exact in the f32
// accumulator, and so are sums of up to 1024 of them (128 * 128 * 1024 = 2^24); a run of
// at most 1024 columns is added to a 32-bit whole number.  So the order of the sums, and how
// they are split, changes nothing.
#include <cuda.h>
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

// --------------------------------------------------------------- many tokens
//
// A CTA per SM goes over tiles of 128 rows of w by kTN tokens on the fifth-generation
// tensor cores.  In a step of 64 columns the rows' codes come by a tensor copy as they are,
// four warps make them f16 and put them into tensor memory as operand A (a lane is a
// row), and the tokens' come as f16 from an image in the scratch, laid out by k_i8_image in the
// order of shared memory, so that one bulk copy brings them.  Sixteen warps take the sums out
// of tensor memory after every 16 steps (1024 columns), add them up as whole numbers, and
// write the tile's results while the next one's sums are made.
constexpr int kBigThreads = 24 * 32;  // copies, MMAs, two idle; four that convert; sixteen that read sums
constexpr int kBigM = 128, kBigK = 64, kBigRun = 16;
constexpr int kBigCtas = 152;
constexpr uint32_t kBigRaw = kBigM * kBigK;  // bytes of codes in a stage

template <int kTN>
struct BigCfg {
  static constexpr uint32_t image = kTN * kBigK * 2;  // bytes of f16 tokens in a stage
  static constexpr int stages = kTN == 256 ? 5 : kTN == 128 ? 8 : 12;
  static constexpr int sums = kTN == 256 ? 1 : 2;  // accumulators in turn
  static constexpr uint32_t a_col = sums * kTN;    // operand A's columns: 32 a stage
  static constexpr size_t smem = stages * (kBigRaw + image) + 1024;
  static_assert(a_col + stages * 32 <= 512, "tensor memory");
};

__device__ __forceinline__ uint64_t image_desc(const void* p) {
  // core matrices of 8 tokens x 16 bytes, 128 bytes apart along the columns, 1024 along the tokens
  uint64_t d = static_cast<uint64_t>((smem_addr(p) & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(128 >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  return d | (1ull << 46);
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
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
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}
// A box of 64 bytes x 128 rows at (col, row): 16-byte pieces turned as swizzle 64B does.
__device__ __forceinline__ void copy_box(void* dst, const CUtensorMap* map, int col, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(col), "r"(row), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Wait for a phase; false once any wait of the CTA ran out of time (which *dead says).
__device__ __forceinline__ bool big_wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*dead) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      *dead = 1;
      return false;
    }
  }
  return true;
}

struct BigArgs {
  const uint8_t* image;  // [steps][tokens up to a multiple of 16][64] f16
  const float *x_scale, *w_scale;
  float* y;
  int64_t y_stride;
  int rows, n, n16, steps, row_tiles, token_tiles;
};

template <int kTN>
__global__ void __launch_bounds__(kBigThreads, 1) k_i8_big(const __grid_constant__ CUtensorMap map, const BigArgs a) {
  using Cfg = BigCfg<kTN>;
  extern __shared__ uint8_t big_smem[];
  __shared__ uint64_t full[Cfg::stages], ready[Cfg::stages], empty[Cfg::stages], sums_full[2], sums_empty[2], done;
  __shared__ uint32_t tmem_at;
  __shared__ int dead_word;
  volatile int* dead = &dead_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* raw = big_smem + (1024u - (smem_addr(big_smem) & 1023u)) % 1024u;
  uint8_t* tokens = raw + Cfg::stages * kBigRaw;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&ready[s], 4);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sums_full[i], 1);
      mbar_init(&sums_empty[i], 16);
    }
    mbar_init(&done, 1);
    dead_word = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_at)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = tmem_at;
  const int tiles = a.row_tiles * a.token_tiles;

  if (warp == 0) {
    if (lane == 0) {
      int g = 0;  // steps issued
      bool image_there = false, ok = true;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        const int row0 = tile / a.token_tiles * kBigM, j0 = tile % a.token_tiles * kTN;
        const uint32_t bytes = min(kTN, a.n16 - j0) * kBigK * 2;
        for (int k = 0; k < a.steps; ++k, ++g) {
          const int s = g % Cfg::stages;
          if (g >= Cfg::stages) ok = big_wait(&empty[s], (g / Cfg::stages - 1) & 1, dead);
          if (!ok) break;
          mbar_arrive_expect_tx(&full[s], kBigRaw + bytes);
          copy_box(raw + s * kBigRaw, &map, k * kBigK, row0, &full[s]);
          if (!image_there) pdl_wait();  // the kernel before this one writes the image
          image_there = true;
          bulk_g2s(tokens + s * Cfg::image, a.image + (static_cast<int64_t>(k) * a.n16 + j0) * (kBigK * 2), bytes, &full[s]);
        }
      }
      // whatever the others do, what is still under way lands before the CTA ends
      for (int i = max(0, g - Cfg::stages); i < g; ++i)
        mbar_wait_bounded(&full[i % Cfg::stages], (i / Cfg::stages) & 1, nullptr, kWaitLimitNs / 4);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int g = 0, run = 0;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        const int width = min(kTN, a.n16 - tile % a.token_tiles * kTN);
        const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(width >> 3) << 17) | (static_cast<uint32_t>(kBigM >> 4) << 24);
        for (int k0 = 0; ok && k0 < a.steps; k0 += kBigRun, ++run) {
          const int b = run % Cfg::sums;
          if (run >= Cfg::sums) ok = big_wait(&sums_empty[b], (run / Cfg::sums - 1) & 1, dead);
          const int end = min(a.steps, k0 + kBigRun);
          for (int k = k0; ok && k < end; ++k, ++g) {
            const int s = g % Cfg::stages;
            const uint32_t phase = (g / Cfg::stages) & 1;
            ok = big_wait(&full[s], phase, dead) && big_wait(&ready[s], phase, dead);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint64_t bd = image_desc(tokens + s * Cfg::image);
#pragma unroll
            for (int i = 0; i < kBigK / 16; ++i)
              mma_ts(tmem + b * kTN, tmem + Cfg::a_col + s * 32 + i * 8, bd + i * 16, idesc, k > k0 || i > 0);
            mma_commit(&empty[s]);
          }
          if (ok) mma_commit(&sums_full[b]);
        }
      }
      mma_commit(&done);  // tensor memory is given back once every MMA is over
      mbar_wait_bounded(&done, 0, nullptr, kWaitLimitNs / 4);
    }
  } else if (warp >= 4 && warp < 8) {
    const int row = (warp - 4) * 32 + lane;
    const uint32_t turn = ((row >> 1) & 3) * 16;
    int g = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
      for (int k = 0; k < a.steps; ++k, ++g) {
        const int s = g % Cfg::stages;
        ok = __all_sync(0xFFFFFFFFu, big_wait(&full[s], (g / Cfg::stages) & 1, dead));
        if (!ok) break;
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(raw + s * kBigRaw + row * 64 + ((c * 16) ^ turn));
          i8x4_to_f16(w.x, v[c * 8], v[c * 8 + 1]);
          i8x4_to_f16(w.y, v[c * 8 + 2], v[c * 8 + 3]);
          i8x4_to_f16(w.z, v[c * 8 + 4], v[c * 8 + 5]);
          i8x4_to_f16(w.w, v[c * 8 + 6], v[c * 8 + 7]);
        }
        tmem_st32(tmem + Cfg::a_col + s * 32 + (static_cast<uint32_t>((warp - 4) * 32) << 16), v);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&ready[s]);
      }
    }
  } else if (warp >= 8) {
    constexpr int kCols = kTN / 4;  // a warp's columns: those of its quarter
    const int quad = warp & 3, c0 = (warp - 8) / 4 * kCols;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    int run = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const int row = tile / a.token_tiles * kBigM + quad * 32 + lane, j0 = tile % a.token_tiles * kTN;
      const int width = min(kTN, a.n16 - j0);
      const float sw = row < a.rows ? a.w_scale[row] : 0.f;
      int total[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) total[i] = 0;
      bool ok = true;
      for (int k0 = 0; k0 < a.steps; k0 += kBigRun, ++run) {
        const int b = run % Cfg::sums;
        ok = __all_sync(0xFFFFFFFFu, big_wait(&sums_full[b], (run / Cfg::sums) & 1, dead)) && ok;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          if (c0 + c >= width) continue;
          uint32_t r[16];
          tmem_ld16(tmem + b * kTN + c0 + c + lanes, r);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int i = 0; i < 16; ++i) total[c + i] += __float2int_rn(__uint_as_float(r[i]));
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&sums_empty[b]);
      }
      // (after a wait that ran out: NaN)
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
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// The tokens' codes as f16 in the order of k_i8_big's shared memory: [step][8 tokens][column / 8][token][8],
// zeros past the last token and column.  A thread takes 16 codes.
__global__ void __launch_bounds__(256) k_i8_image(const int8_t* x, int64_t x_stride, int n, int cols, int n16, int steps,
                                                  uint8_t* image) {
  pdl_launch_dependents();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int c = static_cast<int>(at & 3), j8 = static_cast<int>((at >> 2) & 7);
  const int64_t rest = at >> 5;  // (token group, step), the step first
  const int k = static_cast<int>(rest % steps);
  const int64_t group = rest / steps;
  if (group * 8 >= n16) return;
  const int64_t j = group * 8 + j8;
  const int col = k * kBigK + c * 16;
  uint4 v = make_uint4(0u, 0u, 0u, 0u), p, q;
  if (j < n && col < cols) v = __ldg(reinterpret_cast<const uint4*>(x + j * x_stride + col));
  i8x4_to_f16(v.x, p.x, p.y);
  i8x4_to_f16(v.y, p.z, p.w);
  i8x4_to_f16(v.z, q.x, q.y);
  i8x4_to_f16(v.w, q.z, q.w);
  uint4* dst = reinterpret_cast<uint4*>(image + (static_cast<int64_t>(k) * n16 + group * 8) * (kBigK * 2) + c * 256 + j8 * 16);
  dst[0] = p;
  dst[8] = q;
}

// The map of w for boxes of 64 columns x 128 rows.
cudaError_t map_of(const I8MatmulArgs& a, CUtensorMap* map) {
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
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.cols), static_cast<cuuint64_t>(a.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.cols)};
  const cuuint32_t box[2] = {kBigK, kBigM}, steps[2] = {1, 1};
  const CUresult r = reinterpret_cast<Encode>(fn)(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(a.w), dims, strides,
                                                  box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr int kFewMost = 32;  // tokens

template <int kTN>
cudaError_t launch_big(const I8MatmulArgs& a, cudaStream_t st) {
  static unsigned long long done = 0;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_i8_big<kTN>), BigCfg<kTN>::smem, &done);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  e = map_of(a, &map);
  if (e != cudaSuccess) return e;
  const int steps = (a.cols + kBigK - 1) / kBigK, n16 = (a.n + 15) / 16 * 16;
  const BigArgs b{static_cast<const uint8_t*>(a.scratch), a.x_scale, a.w_scale, a.y, a.y_stride, a.rows, a.n, n16, steps,
                  (a.rows + kBigM - 1) / kBigM, (a.n + kTN - 1) / kTN};
  const int64_t threads = static_cast<int64_t>(n16 / 8) * steps * 32, tiles = static_cast<int64_t>(b.row_tiles) * b.token_tiles;
  k_i8_image<<<static_cast<unsigned>((threads + 255) / 256), 256, 0, st>>>(a.x, a.x_stride, a.n, a.cols, n16, steps,
                                                                           static_cast<uint8_t*>(a.scratch));
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(k_i8_big<kTN>, dim3(static_cast<unsigned>(tiles < kBigCtas ? tiles : kBigCtas)), kBigThreads,
                    BigCfg<kTN>::smem, st, map, b);
}

}  // namespace

size_t i8_matmul_scratch_bytes(int rows, int cols, int n) {
  if (n <= kFewMost) return 0;
  return static_cast<size_t>((n + 15) / 16 * 16) * ((cols + kBigK - 1) / kBigK) * kBigK * 2;
}

cudaError_t launch_i8_matmul(const I8MatmulArgs& a, cudaStream_t st) {
  if (a.n <= 8) return launch_few<1>(a, st);
  if (a.n <= 16) return launch_few<2>(a, st);
  if (a.n <= kFewMost) return launch_few<4>(a, st);
  if (a.n <= 64) return launch_big<64>(a, st);
  if (a.n <= 128) return launch_big<128>(a, st);
  return launch_big<256>(a, st);
}

}  // namespace tqd
