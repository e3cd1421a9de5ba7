// Log probabilities of given tokens, entropy and top alternatives, from one
// pass over the logits.
//
// Mathematics.  With m the largest logit so far, s = sum e^(x - m) and
// t = sum e^(x - m) (x - m), rescaled when m grows: log p = (x - m) - log s and
// the entropy is log s - t / s.  d = x - m is clamped to [-200, 0], which also
// settles the special values: (-inf) - m becomes a term of 0, inf - inf (NaN)
// becomes a term of 1, so infinite logits share the probability.
//
// Alternatives are ordered by a 64-bit key (the logit's bits in integer order,
// then the complement of the index), which no two tokens share, so the result
// does not depend on the order of insertion.  A block keeps a list of
// candidates in shared memory and a threshold, the k-th best logit of its
// earlier tiles: a thread compares its largest new logit with it, and on most tiles that
// is all.  The first tile's threshold is the k-th largest of the threads' own
// maxima (at least k tokens reach it, and about k do).
//
// HBM bounds it: 4 bytes a logit and about ten instructions.  A tile is 8
// logits a thread, the next one's loads issued before the current one's work.
// Few rows are cut into slices of whole tiles, one block each, whose partial
// (m, s, t) and alternatives a second kernel joins (programmatic dependent launch).
#include <cuda_runtime.h>

#include "tqd_internal.h"

namespace tqd {
namespace {

constexpr int kLT = 256;         // threads of a block
constexpr int kEach = 8;         // logits of a thread per tile
constexpr int kTile = kLT * kEach;
constexpr int kCap = 512;        // candidates a block holds
constexpr int kFull = 160;       // candidates at which it keeps the k best only
constexpr int kJoinCap = kLogprobMaxTopK * kLogprobMaxTopK;
constexpr int kMaxSlices = 256;

using Key = unsigned long long;

// 0 for NaN and -inf, which are no alternatives.
__device__ __forceinline__ Key logit_key(float x, int i) {
  if (!(x > -INFINITY)) return 0ull;
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t u = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (static_cast<Key>(u) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float key_logit(Key k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ int key_index(Key k) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k)); }

// x - m for a term of the sums, see above; m > -inf.
__device__ __forceinline__ float term(float x, float m) { return fmaxf(fminf(x - m, 0.f), -200.f); }
__device__ __forceinline__ float exp_of(float d) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d * 1.4426950408889634f));
  return y;
}

struct Sums {
  float m, s, t;
};

__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  if (r.m == -INFINITY) return a;
  const float da = term(a.m, r.m), db = term(b.m, r.m);
  const float wa = exp_of(da), wb = exp_of(db);
  r.s = wa * a.s + wb * b.s;
  r.t = wa * (a.t + a.s * da) + wb * (b.t + b.s * db);
  return r;
}

// All threads get the block's sums, joined in the same order every time.
__device__ Sums block_join(Sums v, Sums* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sums w;
    w.m = __shfl_xor_sync(0xFFFFFFFFu, v.m, o);
    w.s = __shfl_xor_sync(0xFFFFFFFFu, v.s, o);
    w.t = __shfl_xor_sync(0xFFFFFFFFu, v.t, o);
    v = threadIdx.x & o ? join(w, v) : join(v, w);
  }
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sm[0];
  for (int w = 1; w < kLT / 32; ++w) v = join(v, sm[w]);
  return v;
}

// The min(n, k) largest of keys[0..n), in order, into out; n <= 4 * kLT. keys
// and out may not overlap.  All threads call it; ends with a barrier.
__device__ void keep_best(const Key* keys, int n, int k, Key* out) {
  for (int i = threadIdx.x; i < n; i += kLT) {
    const Key mine = keys[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += keys[j] > mine;
    if (rank < k) out[rank] = mine;
  }
  __syncthreads();
}

struct RowOut {
  float m, log_s;
  __device__ float logprob(float x) const {
    return !(x > -INFINITY) ? -INFINITY : (x == m ? 0.f : x - m) - log_s;
  }
};

// The row's results from its sums and its n <= k best keys.
__device__ void write_row(const LogprobArgs& a, int64_t row, const Sums& v, const Key* best, int n) {
  const RowOut o{v.m, logf(v.s)};
  const int t = threadIdx.x;
  if (t < a.top_k) {
    const Key k = t < n ? best[t] : 0ull;
    a.top_ids[row * a.top_k + t] = k ? key_index(k) : -1;
    a.top_logprobs[row * a.top_k + t] = k ? o.logprob(key_logit(k)) : -INFINITY;
  }
  if (t == 32 && a.targets) {
    const int id = a.targets[row];
    a.logprob[row] = id < 0 || id >= a.vocab ? __int_as_float(0x7FC00000) : o.logprob(a.logits[row * a.stride + id]);
  }
  if (t == 64 && a.entropy) a.entropy[row] = v.m > -INFINITY ? o.log_s - v.t / v.s : 0.f;
}

// One slice's partial in scratch: (m, s, t, alternatives' number), top_k keys.
__host__ __device__ constexpr size_t partial_bytes(int top_k) { return 16 + static_cast<size_t>(top_k + (top_k & 1)) * 8; }

__global__ void __launch_bounds__(kLT, 4) k_logprobs(LogprobArgs a, int slices, int tiles_each) {
  __shared__ Key buf[kCap];
  __shared__ Key best[kLogprobMaxTopK];
  __shared__ __align__(16) float heads[kLT];
  __shared__ Sums sm[kLT / 32];
  __shared__ int count;
  __shared__ float floor_;
  const int tid = threadIdx.x, k = a.top_k;
  pdl_launch_dependents();
  const int64_t row = blockIdx.x / slices;
  const int slice = static_cast<int>(blockIdx.x - row * slices);
  const float* x = a.logits + row * a.stride;
  // 16-byte loads from the aligned address at or before the row; what lies outside the row is not read
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(x) >> 2) & 3);
  const int tiles = (a.vocab + off + kTile - 1) / kTile;
  const int tile0 = slice * tiles_each, tile1 = min(tile0 + tiles_each, tiles);
  if (tid == 0) {
    count = 0;
    floor_ = -INFINITY;
  }

  auto index_of = [&](int tile, int j) { return tile * kTile - off + (j >> 2) * (kLT * 4) + tid * 4 + (j & 3); };
  auto load = [&](int tile, float (&v)[kEach]) {
#pragma unroll
    for (int h = 0; h < kEach / 4; ++h) {
      const int i = index_of(tile, h * 4);
      if (i >= 0 && i + 3 < a.vocab) {
        const float4 q = __ldcs(reinterpret_cast<const float4*>(x + i));
        v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * h + j] = i + j >= 0 && i + j < a.vocab ? x[i + j] : -INFINITY;
      }
    }
  };

  Sums own{-INFINITY, 0.f, 0.f};
  float floor_r = -INFINITY;
  float nx[kEach];
  if (tile0 < tile1) load(tile0, nx);
  __syncthreads();
  for (int tile = tile0; tile < tile1; ++tile) {
    float v[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) v[j] = fmaxf(nx[j], -INFINITY);  // NaN counts as -inf
    if (tile + 1 < tile1) load(tile + 1, nx);
    float lm = v[0];
#pragma unroll
    for (int j = 1; j < kEach; ++j) lm = fmaxf(lm, v[j]);
    if (lm > own.m) {
      const float d = term(own.m, lm), w = exp_of(d);
      own.t = w * (own.t + own.s * d);
      own.s *= w;
      own.m = lm;
    }
    if (own.m > -INFINITY) {
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const float d = term(v[j], own.m), e = exp_of(d);
        own.s += e;
        own.t = fmaf(e, d, own.t);
      }
    }
    if (k == 0) continue;

    // ---- candidates
    const bool first = tile == tile0;
    float least = floor_r;
    if (first) {
      heads[tid] = lm;
      __syncthreads();
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < kLT; j += 4) {
        const float4 h = *reinterpret_cast<const float4*>(heads + j);
        rank += (h.x > lm || (h.x == lm && j < tid)) + (h.y > lm || (h.y == lm && j + 1 < tid)) +
                (h.z > lm || (h.z == lm && j + 2 < tid)) + (h.w > lm || (h.w == lm && j + 3 < tid));
      }
      if (rank == k - 1) floor_ = lm;
      __syncthreads();
      least = floor_;
    }
    bool want_merge = first;
    if (first ? lm >= least && lm > -INFINITY : lm > least) {
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (first ? v[j] >= least && v[j] > -INFINITY : v[j] > least) {
          const int p = atomicAdd(&count, 1);
          if (p < kCap) buf[p] = logit_key(v[j], index_of(tile, j));
          want_merge |= p >= kFull;
        }
    }
    if (!__syncthreads_or(want_merge) && tile + 1 < tile1) continue;

    // ---- keep the k best (all threads are here; the count is final)
    int n = count;
    if (n > kCap) {
      // More tokens passed than the list holds (many equal logits, or ascending
      // ones): the tile's own k best one by one, with the earlier list's.
      // The list before this tile held at most kFull + (a tile's last inserts),
      // and what fitted of this tile is found again, so equal keys are dropped.
      Key below = ~0ull;
      for (int r = 0; r < k; ++r) {
        Key top = 0ull;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          const Key key = logit_key(v[j], index_of(tile, j));
          if (key < below && key > top) top = key;
        }
        for (int j = tid; j < kCap; j += kLT)
          if (buf[j] < below && buf[j] > top) top = buf[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const Key w = __shfl_xor_sync(0xFFFFFFFFu, top, o);
          if (w > top) top = w;
        }
        Key* hk = reinterpret_cast<Key*>(heads);
        if ((tid & 31) == 0) hk[tid >> 5] = top;
        __syncthreads();
        top = hk[0];
        for (int w = 1; w < kLT / 32; ++w)
          if (hk[w] > top) top = hk[w];
        if (tid == 0) best[r] = top;
        below = top;
        __syncthreads();
      }
      n = k;  // (keys of 0: fewer than k above -inf, impossible with a full list)
    } else {
      keep_best(buf, n, k, best);
      n = min(n, k);
    }
    if (tid < n) buf[tid] = best[tid];
    if (tid == 0) count = n;
    floor_r = n == k ? key_logit(best[k - 1]) : -INFINITY;
    __syncthreads();
  }

  const Sums all = block_join(own, sm);
  const int n = k ? count : 0;
  if (slices == 1) {
    write_row(a, row, all, best, n);
    return;
  }
  unsigned char* part = static_cast<unsigned char*>(a.scratch) + static_cast<size_t>(blockIdx.x) * partial_bytes(k);
  if (tid == 0) *reinterpret_cast<float4*>(part) = make_float4(all.m, all.s, all.t, __int_as_float(n));
  if (tid < k) reinterpret_cast<Key*>(part + 16)[tid] = tid < n ? best[tid] : 0ull;
}

// One block per row joins its slices.
__global__ void __launch_bounds__(kLT) k_logprobs_join(LogprobArgs a, int slices) {
  __shared__ Key buf[kJoinCap];
  __shared__ Key best[kLogprobMaxTopK];
  __shared__ Key heads[kMaxSlices];
  __shared__ Sums sm[kLT / 32];
  __shared__ int count;
  __shared__ Key floor_;
  const int tid = threadIdx.x, k = a.top_k;
  const int64_t row = blockIdx.x;
  const unsigned char* part = static_cast<const unsigned char*>(a.scratch) + row * slices * partial_bytes(k);
  if (tid == 0) {
    count = 0;
    floor_ = 1ull;
  }
  pdl_wait();
  Sums own{-INFINITY, 0.f, 0.f};
  Key head = 0ull;
  if (tid < slices) {
    const float4 v = *reinterpret_cast<const float4*>(part + tid * partial_bytes(k));
    own = Sums{v.x, v.y, v.z};
    if (k) head = *reinterpret_cast<const Key*>(part + tid * partial_bytes(k) + 16);
  }
  heads[tid] = head;
  const Sums all = block_join(own, sm);  // (a barrier inside)
  int n = 0;
  if (k) {
    // the k-th largest of the slices' best: no alternative lies below it, and at most k slices hold one
    if (slices > k) {
      int rank = 0;
      for (int j = 0; j < slices; ++j) rank += heads[j] > head;
      if (tid < slices && head && rank == k - 1) floor_ = head;
      __syncthreads();
    }
    if (head >= floor_)
      for (int j = 0; j < k; ++j) {
        const Key key = reinterpret_cast<const Key*>(part + tid * partial_bytes(k) + 16)[j];
        if (key < floor_) break;
        buf[atomicAdd(&count, 1)] = key;
      }
    __syncthreads();
    keep_best(buf, count, k, best);
    n = min(count, k);
  }
  write_row(a, row, all, best, n);
}

// Slices of a row: whole tiles, so that about 152 x 4 blocks run.
int slices_of(int rows, int vocab) {
  const int tiles = (vocab + 3 + kTile - 1) / kTile;
  int want = (608 + rows - 1) / rows;
  if (want > tiles) want = tiles;
  if (want > kMaxSlices) want = kMaxSlices;
  const int each = (tiles + want - 1) / want;
  return (tiles + each - 1) / each;
}

}  // namespace

size_t logprobs_scratch_bytes(int rows, int vocab, int top_k) {
  const int s = slices_of(rows, vocab);
  return s == 1 ? 16 : static_cast<size_t>(rows) * s * partial_bytes(top_k);
}

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t st) {
  const int slices = slices_of(a.rows, a.vocab);
  const int tiles = (a.vocab + 3 + kTile - 1) / kTile;
  const int each = (tiles + slices - 1) / slices;
  k_logprobs<<<static_cast<unsigned>(a.rows) * slices, kLT, 0, st>>>(a, slices, each);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || slices == 1) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.rows);
  cfg.blockDim = dim3(kLT);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_logprobs_join, a, slices);
}

}  // namespace tqd
