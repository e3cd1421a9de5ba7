// Matrix-vector products with Q4_0 weights (4-bit codes, one f16 scale per
// 32 columns).
#include <cuda_runtime.h>

#include "tqd_internal.h"
#include "tqd_q4.cuh"

namespace tqd {
namespace {

// One thread per 32-bit word of a tile's codes or scales.  Run once per matrix when a
// model is loaded: 151936 x 1024 takes 99 us (175 MB, 1.8 TB/s; single-byte loads
// from the 18-byte blocks bound it).
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

constexpr int kMvWarps = 8;
constexpr int kMvCtas = 304;  // two per SM
constexpr int kMvThreads = 32 * kMvWarps;
// Strips of a stage, and stages of a warp's ring (nt: tiles of 8 columns).  Four
// strips a stage for few columns (151936 x 1024 of one vector 18.7 us, with two 20.1;
// 151936 x 8192 109 and 123), fewer where the staged vectors need the room.
__host__ __device__ constexpr int mv_chunk(int nt) { return nt == 4 ? 1 : nt == 1 ? 4 : 2; }
__host__ __device__ constexpr int mv_stages(int nt) { return nt == 4 ? 3 : 2; }
// Shared memory of a CTA: at most what lets two of them share an SM; the rings
// and the warps' sums, then the staged vectors.  (228 KB hold two of 113 KB, 1 KB of
// the system's and 128 bytes that are not dynamic.)
constexpr int kMvSmem = 113 * 1024 - 128;
constexpr int mv_fixed_smem(int nt) {
  return kMvWarps * (mv_stages(nt) * (mv_chunk(nt) * kQ4TileBytes + 8) + 2 * nt * 128);
}
constexpr int mv_strip_smem(int cols) { return 4 * (cols * 64 + cols / 2 * 4); }

struct MatvecQ4Args {
  const uint8_t* w;
  const float* x;
  float* y;
  int64_t xs, ys;
  int rows, groups, n;   // groups: columns / 32
  int row_tiles, strips; // of 16 rows, of 128 columns
  int slab;              // strips whose x is staged at a time
  int wk;                // warps that share a row tile's strips (1, 2, 4, 8)
  int cluster;           // CTAs of a cluster, each with a part of the strips (1, 2, 4, 8)
  int per_slot;          // row tiles of one warp (of wk warps)
};

// y = W x for up to 4 NT vectors (ONE: a single one).
//
// A tile's 16 rows are the tensor cores' 16 operand rows, its codes unpacked to
// f16 pairs of code - 8; the vectors are columns, two for each: a group of
// 32 elements is scaled by a power of two that brings its largest to 2^14
// .. 2^15 and each element split into its leading 11 bits and the rest in f16, so
// an element keeps 22 bits down to 2^-17 of its group's largest.  Each
// group's two column sums are added, scaled by the group's power of two and
// the row's f16 scale and summed over groups in f32.
// (Codes as they are, masked words that count as f16 subnormals, with 8 sum x taken off,
// save the unpacking's packed operations; but a product with a zero weight is then 8 x and
// not 0, and the tensor cores align the products of a subnormal as if it were 2^-14.
// What that loses stays where a large element meets a zero weight: 1e-4
// of the result for elements 1000 times the rest, where f32 products have 7e-7.)
//
// HBM bounds it: 4.5 bits a weight.  A weight costs 1.1 instructions of
// unpacking and 1/4 MMA lane, where unpacking to f32 and a packed FMA cost over 2;
// up to 16 vectors share them.  151936 x 1024 of one vector: 17.7 us for 88 MB (5.0
// TB/s, 73 % of a copy's rate: 5 us are the launch, the vector and the last tiles'
// sums); 16 vectors 46 us, bound by the reads of the staged vectors, the matrix
// pipe and the instructions of unpacking and sums in turn (16384 x 8192 of 16: 62
// us, 69 TFLOP/s); 1024 x 1024 5.7 us, a launch.
//
// Each warp streams its row tiles' strips, one contiguous run, through a ring of
// bulk copies of its own.  Where there are too few row tiles for the GPU's warps, or
// staging the vectors would take too long, a cluster of 2, 4 or 8 CTAs shares the
// strips (so each stages a part of the vectors) and adds its sums through
// distributed shared memory; with less than 8 row tiles the warps of a CTA share
// them too.
template <int NT, bool ONE>
__global__ void __launch_bounds__(kMvThreads, 2) k_q4_matvec(MatvecQ4Args a) {
  constexpr int NC = ONE ? 2 : 8 * NT;  // staged columns: high and low part of each vector
  constexpr int NS = 2 * NT;  // a lane's sums
  constexpr int kMvStages = mv_stages(NT), kChunk = mv_chunk(NT), kStage = kChunk * kQ4TileBytes;
  extern __shared__ __align__(128) unsigned char sm[];
  unsigned char* ring = sm;
  float* red = reinterpret_cast<float*>(ring + kMvWarps * kMvStages * kStage);  // [warps][NS][32]
  auto* bars = reinterpret_cast<uint64_t*>(red + kMvWarps * NS * 32);
  float* fs = reinterpret_cast<float*>(bars + kMvWarps * kMvStages);  // [groups of a slab][NC / 2]: the vectors' factors
  unsigned char* xs = reinterpret_cast<unsigned char*>(fs + a.slab * 4 * (NC / 2));  // [groups][NC][4][16 bytes]

  __shared__ uint4 none;  // a column of zeros
  if (ONE && threadIdx.x == 0) none = make_uint4(0u, 0u, 0u, 0u);

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r8 = lane >> 2, c = lane & 3;
  const int wk = warp % a.wk;
  const int rank = blockIdx.x % a.cluster, slots = kMvWarps / a.wk;
  const int cta0 = blockIdx.x / a.cluster * slots;  // the cluster's first slot
  const int slot = cta0 + warp / a.wk;
  const int cs0 = a.strips * rank / a.cluster, cs1 = a.strips * (rank + 1) / a.cluster;  // the CTA's strips
  const int tile0 = slot * a.per_slot, tile1 = min(tile0 + a.per_slot, a.row_tiles);
  const int v0 = blockIdx.y * 16, nv = min(a.n - v0, ONE ? 1 : 4 * NT);
  const float* x = a.x + v0 * a.xs;
  float* y = a.y + v0 * a.ys;
  const int slabs = ((a.strips + a.cluster - 1) / a.cluster + a.slab - 1) / a.slab;  // the same in every CTA

  uint64_t* bar = bars + warp * kMvStages;
  unsigned char* my_ring = ring + warp * kMvStages * kStage;
  if (lane < kMvStages) mbar_init(&bar[lane], 1);
  fence_mbar_init();
  __syncwarp();

  pdl_wait();
  pdl_launch_dependents();
  // this warp's strips of a slab
  auto share = [&](int slab, int& b, int& e) {
    const int s0 = cs0 + slab * a.slab, n = max(min(a.slab, cs1 - s0), 0);
    b = s0 + n * wk / a.wk;
    e = s0 + n * (wk + 1) / a.wk;
  };
  // the ring's next copy: slab by slab, tile by tile, strip by strip
  const uint8_t* src = nullptr;
  int left = 0, ptile = tile1 - 1, pslab = -1, pst = 0;
  bool dead = false;  // a copy that did not arrive within the wait's limit: the rows become NaN
  bool stopped = false;  // the warp knows of it
  auto issue = [&] {
    if (dead) return;
    if (left == 0) {  // the next tile, or the next slab, with strips for this warp
      int b = 0, e = 0;
      do {
        if (++ptile >= tile1) {
          ptile = tile0;
          if (++pslab >= slabs) {
            pslab = slabs;
            return;
          }
        }
        share(pslab, b, e);
        if (b == e) ptile = tile1 - 1;  // (fewer strips than warps)
      } while (b == e);
      left = e - b;
      src = a.w + (static_cast<size_t>(ptile) * a.strips + b) * kQ4TileBytes;
    }
    const int n = min(left, kChunk);
    if (lane == 0) {
      mbar_arrive_expect_tx(&bar[pst], n * kQ4TileBytes);
      bulk_g2s(my_ring + pst * kStage, src, n * kQ4TileBytes, &bar[pst]);
    }
    pst = pst + 1 == kMvStages ? 0 : pst + 1;
    src += kChunk * kQ4TileBytes;
    left -= n;
  };
  if (tile0 < tile1)
    for (int i = 0; i < kMvStages - 1; ++i) issue();

  const Unpack unpack;
  int st = 0, phase = 0;
  for (int slab = 0; slab < slabs; ++slab) {
    // ---- the slab's part of the vectors
    const int g0 = (cs0 + slab * a.slab) * 4, ng = max(min(a.slab * 4, cs1 * 4 - g0), 0);
    if (slab) __syncthreads();
    const int octs = ng * 4;
    const int real = max(min(a.groups - g0, ng), 0) * 4;
    // Octets of columns: kBatch of them loaded before the first is used.  (Whole
    // warps: octs is a multiple of 16, and a group's four octets are neighbouring lanes.)
    constexpr int kBatch = ONE ? 2 : 4;
    const bool wide = (reinterpret_cast<uintptr_t>(x) % 16 | a.xs % 4) == 0;
    for (int i0 = warp * 32; i0 < octs * (NC / 2); i0 += kBatch * kMvThreads) {
      float fs_[kBatch][8];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kMvThreads + lane, v = i / octs, o = i - v * octs;
#pragma unroll
        for (int j = 0; j < 8; ++j) fs_[k][j] = 0.f;
        if (v < nv && o < real) {
          const float* p = x + v * a.xs + static_cast<int64_t>(g0) * 32 + o * 8;
          if (wide) {
            const float4 lo4 = *reinterpret_cast<const float4*>(p), hi4 = *reinterpret_cast<const float4*>(p + 4);
            fs_[k][0] = lo4.x; fs_[k][1] = lo4.y; fs_[k][2] = lo4.z; fs_[k][3] = lo4.w;
            fs_[k][4] = hi4.x; fs_[k][5] = hi4.y; fs_[k][6] = hi4.z; fs_[k][7] = hi4.w;
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) fs_[k][j] = p[j];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kMvThreads + lane, v = i / octs, o = i - v * octs;
        if (i - lane >= octs * (NC / 2)) break;
        float (&f)[8] = fs_[k];
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
#pragma unroll
        for (int s = 1; s < 4; s <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
        const int e = static_cast<int>(__float_as_uint(m) >> 23) - 127, up = min(14 - e, 126);
        const float f1 = pow2(up / 2), f2 = pow2(up - up / 2);
        uint32_t hi[4], lo[4];  // elements j and j + 4, their leading bits and the rest
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = e > 112 ? __int_as_float(0x7FC00000) : f[j] * f1 * f2;
          const float x1 = e > 112 ? __int_as_float(0x7FC00000) : f[j + 4] * f1 * f2;
          hi[j] = pack_f16(x0, x1);
          const float2 h = unpack_f16(hi[j]);
          lo[j] = pack_f16(x0 - h.x, x1 - h.y);
        }
        if (v < NC / 2) {
          const int g = o >> 2, oc = o & 3;
          if (oc == 0) fs[g * (NC / 2) + v] = pow2(-up);
          unsigned char* d = xs + ((g * NC + 2 * v) * 4 + oc) * 16;
          *reinterpret_cast<uint4*>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(d + 64) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
    }
    __syncthreads();

    // ---- this warp's row tiles
    int b, e;
    share(slab, b, e);
    for (int k = 0; k < a.per_slot; ++k) {
      const int tile = tile0 + k;
      float acc[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = 0.f;
      if (tile < tile1) {
        for (int strip0 = b; strip0 < e; strip0 += kChunk) {
          issue();
          if (!dead) dead = !mbar_wait_bounded(&bar[st], phase, nullptr);
          const unsigned char* stage = my_ring + st * kStage;
          if (++st == kMvStages) {
            st = 0;
            phase ^= 1;
          }
#pragma unroll
          for (int u = 0; u < kChunk; ++u) {
            if (u && strip0 + u >= e) break;
            const int gl = (strip0 + u) * 4 - g0;
            const unsigned char* tl = stage + u * kQ4TileBytes;
            const uint4 w0 = *reinterpret_cast<const uint4*>(tl + lane * 16), w1 = *reinterpret_cast<const uint4*>(tl + 512 + lane * 16);
            // the operands of a group: rows r8 and r8 + 8
            auto operands = [&](int g, uint32_t (&a0)[4], uint32_t (&a1)[4]) {
              const uint32_t p = g == 0 ? w0.x : g == 1 ? w0.y : g == 2 ? w0.z : w0.w;
              const uint32_t q = g == 0 ? w1.x : g == 1 ? w1.y : g == 2 ? w1.z : w1.w;
              a0[0] = unpack.low(p);
              a0[1] = unpack.low(q);
              a0[2] = unpack.high(p);
              a0[3] = unpack.high(q);
              a1[0] = unpack.low(p >> 8);
              a1[1] = unpack.low(q >> 8);
              a1[2] = unpack.high(p >> 8);
              a1[3] = unpack.high(q >> 8);
            };
            if constexpr (ONE) {
              // the strip's four groups in the four column pairs, so that a lane takes the sums of
              // one of them, group c, and not of all four
              const unsigned char* scale = tl + kQ4TileScales + r8 * 8 + c * 2;
              const unsigned char* own = xs + (((gl + (r8 >> 1)) * 2 + (r8 & 1)) * 4 + c) * 16;
              float d[4];
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                uint32_t a0[4], a1[4];
                operands(g, a0, a1);
                const uint4 xv = *reinterpret_cast<const uint4*>(r8 >> 1 == g ? own : reinterpret_cast<const unsigned char*>(&none));
                if (g == 0)
                  mma_f16(d, a0, xv.x, xv.y, 0.f, 0.f, 0.f, 0.f);
                else
                  mma_f16(d, a0, xv.x, xv.y);
                mma_f16(d, a1, xv.z, xv.w);
              }
              const float f = fs[gl + c];
              acc[0][0] += __half2float(*reinterpret_cast<const __half*>(scale)) * (f * (d[0] + d[1]));
              acc[0][1] += __half2float(*reinterpret_cast<const __half*>(scale + 64)) * (f * (d[2] + d[3]));
              continue;
            }
            const uint2 sc0 = *reinterpret_cast<const uint2*>(tl + kQ4TileScales + r8 * 8);
            const uint2 sc1 = *reinterpret_cast<const uint2*>(tl + kQ4TileScales + 64 + r8 * 8);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t a0[4], a1[4];
              operands(g, a0, a1);
              const float2 s0 = unpack_f16(g < 2 ? sc0.x : sc0.y), s1 = unpack_f16(g < 2 ? sc1.x : sc1.y);
              const float ds0 = g & 1 ? s0.y : s0.x, ds1 = g & 1 ? s1.y : s1.x;
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                const uint4 xv = *reinterpret_cast<const uint4*>(xs + (((gl + g) * NC + t * 8 + r8) * 4 + c) * 16);
                const float f = fs[(gl + g) * (NC / 2) + t * 4 + c];
                float d[4];
                mma_f16(d, a0, xv.x, xv.y, 0.f, 0.f, 0.f, 0.f);
                mma_f16(d, a1, xv.z, xv.w);
                acc[t][0] += ds0 * (f * (d[0] + d[1]));
                acc[t][1] += ds1 * (f * (d[2] + d[3]));
              }
            }
          }
          __syncwarp();  // every lane has read the stage before it is filled again
        }
        if constexpr (ONE) {  // (the groups' sums, the same in the four lanes of a row)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            acc[0][h] += __shfl_xor_sync(0xFFFFFFFFu, acc[0][h], 1);
            acc[0][h] += __shfl_xor_sync(0xFFFFFFFFu, acc[0][h], 2);
          }
        }
        // (each lane read the timer for itself: one that ran out speaks for the warp, whose sums hold its share)
        if (__any_sync(0xFFFFFFFFu, dead)) {
          if (!stopped) mbar_ring_drain(bar, kMvStages);
          dead = stopped = true;
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = __int_as_float(0x7FC00000);
        }
      }
      auto store = [&](int of, int i, int l, float sum) {  // sum i of lane l: [4 vectors][half of the rows]
        const int v = i / 2 * 4 + (l & 3);
        const int64_t r = static_cast<int64_t>(of) * 16 + i % 2 * 8 + (l >> 2);
        if (v >= nv || r >= a.rows) return;
        float* p = y + v * a.ys + r;
        *p = slab ? *p + sum : sum;
      };
      if (a.wk * a.cluster == 1) {
        if (tile < tile1)
#pragma unroll
          for (int i = 0; i < NS; ++i) store(tile, i, lane, acc[i / 2][i % 2]);
        continue;
      }
      float* mine = red + warp * NS * 32 + lane;
#pragma unroll
      for (int i = 0; i < NS; ++i) mine[i * 32] = acc[i / 2][i % 2];
      if (a.cluster == 1)
        __syncthreads();
      else
        cluster_sync();
      // the sums of each slot's tile, dealt over the cluster's threads
      for (int i = rank * kMvThreads + threadIdx.x; i < slots * NS * 32; i += a.cluster * kMvThreads) {
        const int sl = i / (NS * 32), e2 = i % (NS * 32);
        const float* from = red + sl * a.wk * NS * 32 + e2;
        float sum = 0.f;
        for (int q = 0; q < a.cluster; ++q)
          for (int j = 0; j < a.wk; ++j)
            sum += a.cluster == 1 ? from[j * NS * 32] : ld_cluster(from + j * NS * 32, q);
        store((cta0 + sl) * a.per_slot + k, e2 / 32, e2 % 32, sum);
      }
      if (a.cluster == 1)
        __syncthreads();
      else
        cluster_sync();
    }
  }
}

template <int NT, bool ONE>
cudaError_t launch_mv(MatvecQ4Args a, cudaStream_t st) {
  constexpr int NC = ONE ? 2 : 8 * NT;
  constexpr int most = (kMvSmem - mv_fixed_smem(NT)) / mv_strip_smem(NC);  // strips whose vectors fit
  // With less than eight row tiles the warps of a CTA share a tile's strips.  The
  // cluster is the one that costs a warp the fewest instructions: about 50 for
  // each octet of columns that it stages, 110 + 60 NT a strip, 500 to add a row tile's
  // sums through distributed shared memory.
  a.wk = 1;
  while (a.wk < kMvWarps && a.row_tiles * a.wk < kMvWarps && a.wk * 2 <= a.strips) a.wk *= 2;
  const int sweep = a.n < 16 ? a.n : 16, ctas = (a.row_tiles * a.wk + kMvWarps - 1) / kMvWarps;
  int64_t least = 0;
  for (int x = 1; x <= 8 && x * a.wk <= a.strips; x *= 2) {
    const int sweeps = (a.n + 15) / 16, room = kMvCtas / (x * sweeps);  // (sweeps run side by side; at most 4)
    const int64_t rounds = (ctas + room - 1) / room, each = (a.strips + x * a.wk - 1) / (x * a.wk);
    const int64_t cost = static_cast<int64_t>(sweep) * a.strips * 6 / x + rounds * (each * (110 + 60 * NT) + (x > 1 ? 500 : 0));
    if (x == 1 || cost < least) {
      least = cost;
      a.cluster = x;
    }
  }
  const int strips = (a.strips + a.cluster - 1) / a.cluster, slabs = (strips + most - 1) / most;
  a.slab = (strips + slabs - 1) / slabs;
  const size_t smem = static_cast<size_t>(mv_fixed_smem(NT)) + static_cast<size_t>(a.slab) * mv_strip_smem(NC);
  const int slots = kMvWarps / a.wk;
  int blocks = (a.row_tiles + slots - 1) / slots;
  if (blocks > kMvCtas / a.cluster) blocks = kMvCtas / a.cluster;
  a.per_slot = (a.row_tiles + blocks * slots - 1) / (blocks * slots);
  blocks = (a.row_tiles + a.per_slot * slots - 1) / (a.per_slot * slots);
  static unsigned long long done = 0;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&k_q4_matvec<NT, ONE>), kMvSmem, &done);
  if (e != cudaSuccess) return e;
  return launch_pdl_clusters(k_q4_matvec<NT, ONE>, a.cluster, dim3(blocks * a.cluster, (a.n + 15) / 16), kMvThreads, smem,
                             st, a);
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
  MatvecQ4Args a{};
  a.w = w;
  a.x = x;
  a.y = y;
  a.xs = x_stride;
  a.ys = y_stride;
  a.rows = rows;
  a.groups = cols / 32;
  a.n = n;
  a.row_tiles = (rows + kQ4TileRows - 1) / kQ4TileRows;
  a.strips = (cols + kQ4TileCols - 1) / kQ4TileCols;
  if (n == 1) return launch_mv<1, true>(a, st);
  if (n <= 4) return launch_mv<1, false>(a, st);
  if (n <= 8) return launch_mv<2, false>(a, st);
  return launch_mv<4, false>(a, st);
}

}  // namespace tqd
