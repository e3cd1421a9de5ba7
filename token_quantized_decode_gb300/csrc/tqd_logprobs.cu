// Log probabilities of given tokens, entropy and top alternatives, from one
// pass over the logits.
//
// Mathematics, in units of log2.  A thread keeps a whole number ref near its
// largest logit times log2 e and s = sum 2^(x log2 e - ref), t = sum 2^(x log2 e -
// ref) (x log2 e - ref).  x log2 e - ref is one fused operation, changes of ref are exact
// powers of two, and ref may stay up to 16 behind, so it hardly ever changes.
// With ref = rint(max log2 e) at the end: log2 p = (x log2 e - ref) - log2 s, and the
// entropy is log2 s - t / s.  The exponent is kept at -300 or more, which makes NaN
// and -inf logits terms of 0.  A row (or slice) whose largest logit is infinite
// or beyond 2^19 in magnitude is read again with terms 2^((x - max) log2 e), 1 where
// x = max: infinite logits share the probability.
//
// Alternatives are ordered by a 64-bit key (the logit's bits in integer order,
// then the complement of the index), which no two tokens share, so the result
// does not depend on the order of insertion.  A block keeps a list of
// candidates in shared memory and a threshold, the k-th best logit of the
// groups of tiles behind it: a thread compares its largest new logit with it, and on most
// tiles that is all.  The first group, and one that overflows the list, is
// read again (from L2) with a threshold of its own: the k-th largest of the threads'
// maxima over it, which at least k and, but for equal logits, at most 32 k tokens
// reach.
//
// HBM bounds it: 4 bytes a logit and about seven instructions (a fused
// multiply-add, a maximum, an exponential, two sums; half a maximum).  A tile is
// 8 logits a thread, the next one's loads issued before the current one's work.
// Few rows are cut into slices of whole tiles, one block each, whose partial
// (m, s, t) and alternatives a second kernel joins (programmatic dependent launch).
#include <cuda_runtime.h>

#include "tqd_internal.h"

namespace tqd {
namespace {

constexpr int kLT = 256;         // threads of a block
constexpr int kEach = 8;         // logits of a thread per tile
constexpr int kTile = kLT * kEach;
constexpr int kGroup = 4;        // tiles between looks at the list
constexpr int kCap = 1024;       // candidates a block holds: kGroup * kEach * kLogprobMaxTopK
constexpr int kFull = 128;       // candidates at which it keeps the k best only
static_assert(kCap == kGroup * kEach * kLogprobMaxTopK, "a group's candidates fit but for equal logits");
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

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Whether sums with largest logit m are relative to ref_of(m), or to m itself.
__device__ __forceinline__ bool by_ref(float m) { return fabsf(m) < 524288.f; }
__device__ __forceinline__ float ref_of(float m) { return rintf(m * kLog2e); }
// log2 of the largest logit's own term.
__device__ __forceinline__ float over_of(float m) { return by_ref(m) ? fmaf(m, kLog2e, -ref_of(m)) : 0.f; }
// The exponent that takes sums with largest logit a to those with b >= a > -inf.
__device__ __forceinline__ float gap(float a, float b) {
  if (a == b) return 0.f;
  const float d = by_ref(a) && by_ref(b) ? ref_of(a) - ref_of(b) : (a - b) * kLog2e - over_of(a) + over_of(b);
  return fmaxf(d, -300.f);
}

struct Sums {
  float m, s, t;  // largest logit; sums of terms, and of terms times their exponents
};

__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
  Sums r;
  r.m = fmaxf(a.m, b.m);
  if (r.m == -INFINITY) return a;
  const float da = gap(a.m, r.m), db = gap(b.m, r.m);
  const float wa = ex2(da), wb = ex2(db);
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
    int rank = 0, j = 0;
    for (; j + 4 <= n; j += 4) {
      const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(keys + j), q = *reinterpret_cast<const ulonglong2*>(keys + j + 2);
      rank += (p.x > mine) + (p.y > mine) + (q.x > mine) + (q.y > mine);
    }
    for (; j < n; ++j) rank += keys[j] > mine;
    if (rank < k) out[rank] = mine;
  }
  __syncthreads();
}

struct RowOut {
  float m, log_s;  // log_s: log sum e^(x - m)
  __device__ RowOut(const Sums& v) : m(v.m), log_s(kLn2 * (log2f(v.s) - over_of(v.m))) {}
  __device__ float logprob(float x) const {
    return !(x > -INFINITY) ? -INFINITY : (x == m ? 0.f : x - m) - log_s;
  }
};

// The row's results from its sums and its n <= k best keys.
__device__ void write_row(const LogprobArgs& a, int64_t row, const Sums& v, const Key* best, int n) {
  const RowOut o(v);
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
  if (t == 64 && a.entropy) a.entropy[row] = v.m > -INFINITY ? kLn2 * (log2f(v.s) - v.t / v.s) : 0.f;
}

// One slice's partial in scratch: (m, s, t, alternatives' number), top_k keys.
__host__ __device__ constexpr size_t partial_bytes(int top_k) { return 16 + static_cast<size_t>(top_k + (top_k & 1)) * 8; }

__global__ void __launch_bounds__(kLT, 5) k_logprobs(LogprobArgs a, int slices, int tiles_each) {
  __shared__ __align__(16) Key buf[kCap];
  __shared__ Key best[kLogprobMaxTopK];
  __shared__ __align__(16) float heads[kLT];
  __shared__ Sums sm[kLT / 32];
  __shared__ int counts[3];  // insertions of a group, of the next, of the one after
  __shared__ float floor_;
  const int tid = threadIdx.x, k = a.top_k;
  pdl_wait();
  pdl_launch_dependents();
  const unsigned row = blockIdx.x / static_cast<unsigned>(slices);
  const int slice = static_cast<int>(blockIdx.x - row * slices);
  const float* x = a.logits + static_cast<int64_t>(row) * a.stride;
  // 16-byte loads from the aligned address at or before the row; what lies outside the row is not read
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(x) >> 2) & 3);
  const int tiles = (a.vocab + off + kTile - 1) / kTile;
  const int tile0 = slice * tiles_each, tile1 = min(tile0 + tiles_each, tiles);
  if (tid < 3) counts[tid] = 0;

  auto index_of = [&](int tile, int j) { return tile * kTile - off + (j >> 2) * (kLT * 4) + tid * 4 + (j & 3); };
  const int whole0 = off ? 1 : 0, whole1 = (a.vocab + off) / kTile;  // tiles that lie inside the row
  auto load = [&](int tile, float (&v)[kEach]) {
    if (tile >= whole0 && tile < whole1) {
      const float* p = x + index_of(tile, 0);
#pragma unroll
      for (int h = 0; h < kEach / 4; ++h) {
        const float4 q = *reinterpret_cast<const float4*>(p + h * (kLT * 4));
        v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int h = 0; h < kEach; ++h) {
        const int at = index_of(tile, h);
        v[h] = at >= 0 && at < a.vocab ? x[at] : -INFINITY;
      }
    }
  };
  int held = 0, turn = 0;  // the list's length at the group's start (every thread's), and the group's counter
  auto insert = [&](float v, int i) {
    const int p = held + atomicAdd(&counts[turn], 1);
    if (p < kCap) buf[p] = logit_key(v, i);
    return p;
  };

  constexpr float kRefMin = -1048576.f;
  float ref = kRefMin, rise = -INFINITY;  // rise: a logit above it moves the reference
  float rs = 0.f, rt = 0.f, rm = -INFINITY;
  float least = INFINITY;  // the first group is read again with a threshold of its own
  float nx[kEach];
  if (tile0 < tile1) load(tile0, nx);
  __syncthreads();
  for (int group = tile0; group < tile1; group += kGroup) {
    const int end = min(group + kGroup, tile1);
    const bool first = group == tile0;
    // (the counter of the next group was last read before the barrier behind the group before this one)
    if (tid == 0) counts[turn == 2 ? 0 : turn + 1] = 0;
    float gm = -INFINITY;
    bool want = first;
    for (int tile = group; tile < end; ++tile) {
      float v[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) v[j] = nx[j];
      if (tile + 1 < tile1) load(tile + 1, nx);
      float lm = fmaxf(v[0], -INFINITY);  // (eight NaN)
#pragma unroll
      for (int j = 1; j < kEach; ++j) lm = fmaxf(lm, v[j]);
      gm = fmaxf(gm, lm);
      if (lm > rise) {
        const float nref = fminf(fmaxf(rintf(lm * kLog2e), kRefMin), -kRefMin);
        const float d = fmaxf(ref - nref, -300.f), w = ex2(d);
        rt = w * (rt + rs * d);
        rs *= w;
        ref = nref;
        rise = (nref + 16.f) * kLn2;
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const float d = fmaxf(fmaf(v[j], kLog2e, -ref), -300.f), e = ex2(d);
        rs += e;
        rt = fmaf(e, d, rt);
      }
      if (lm > least) {
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          if (v[j] > least) want |= insert(v[j], index_of(tile, j)) >= kFull;
      }
    }
    rm = fmaxf(rm, gm);
    if (k == 0) continue;
    const bool merge = __syncthreads_or(want) || end == tile1;
    int n = held + counts[turn];
    if (!merge) {
      held = n;
      turn = turn == 2 ? 0 : turn + 1;
      continue;
    }

    // ---- keep the k best
    if (first || n > kCap) {
      // The group again: the tokens that reach the k-th largest of the threads'
      // maxima, and those that the earlier list holds.  (Of this group's own
      // first insertions none are kept: they began at `held`.)
      heads[tid] = gm;
      __syncthreads();
      if (tid == 0) {
        counts[turn] = 0;
        floor_ = -INFINITY;
      }
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < kLT; j += 4) {
        const float4 h = *reinterpret_cast<const float4*>(heads + j);
        rank += (h.x > gm || (h.x == gm && j < tid)) + (h.y > gm || (h.y == gm && j + 1 < tid)) +
                (h.z > gm || (h.z == gm && j + 2 < tid)) + (h.w > gm || (h.w == gm && j + 3 < tid));
      }
      __syncthreads();
      if (rank == k - 1) floor_ = gm;
      __syncthreads();
      const float reach = floor_, above = first ? -INFINITY : least;
      if (gm >= reach && gm > above)
        for (int tile = group; tile < end; ++tile) {
          float v[kEach];
          load(tile, v);
#pragma unroll
          for (int j = 0; j < kEach; ++j)
            if (v[j] >= reach && v[j] > above) insert(v[j], index_of(tile, j));
        }
      __syncthreads();
      n = held + counts[turn];
    }
    if (n > kCap) {
      // Too many equal logits: the group's k best one by one, from it and the earlier list.
      Key below = ~0ull;
      Key* hk = reinterpret_cast<Key*>(heads);
      for (int r = 0; r < k; ++r) {
        Key top = 0ull;
        for (int tile = group; tile < end; ++tile) {
          float v[kEach];
          load(tile, v);
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            const Key key = logit_key(v[j], index_of(tile, j));
            if (key < below && key > top) top = key;
          }
        }
        for (int j = tid; j < held; j += kLT)
          if (buf[j] < below && buf[j] > top) top = buf[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const Key w = __shfl_xor_sync(0xFFFFFFFFu, top, o);
          if (w > top) top = w;
        }
        if ((tid & 31) == 0) hk[tid >> 5] = top;
        __syncthreads();
        top = hk[0];
        for (int w = 1; w < kLT / 32; ++w)
          if (hk[w] > top) top = hk[w];
        if (tid == 0) best[r] = top;
        below = top;
        __syncthreads();
      }
      n = k;  // (there are more than kCap >= k)
    } else {
      keep_best(buf, n, k, best);
      n = min(n, k);
    }
    if (tid < n) buf[tid] = best[tid];
    held = n;
    turn = turn == 2 ? 0 : turn + 1;
    least = n == k ? key_logit(best[k - 1]) : -INFINITY;
    __syncthreads();
  }

  // ---- the block's sums, relative to its own largest logit
  float bm = rm;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xFFFFFFFFu, bm, o));
  if ((tid & 31) == 0) heads[tid >> 5] = bm;
  __syncthreads();
  for (int w = 0; w < kLT / 32; ++w) bm = fmaxf(bm, heads[w]);
  Sums own{bm, 0.f, 0.f};
  if (by_ref(bm)) {
    const float d = fmaxf(ref - ref_of(bm), -300.f), w = ex2(d);
    own.t = w * (rt + rs * d);
    own.s = w * rs;
  } else if (bm > -INFINITY) {
    for (int tile = tile0; tile < tile1; ++tile) {
      float v[kEach];
      load(tile, v);
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const float d = v[j] == bm ? 0.f : fmaxf((v[j] - bm) * kLog2e, -300.f), e = ex2(d);
        own.s += e;
        own.t = fmaf(e, d, own.t);
      }
    }
  }
  const Sums all = block_join(own, sm);
  const int n = held;
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
  __shared__ __align__(16) Key buf[kJoinCap];
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
  pdl_launch_dependents();
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
  const cudaError_t e = launch_pdl(k_logprobs, dim3(static_cast<unsigned>(a.rows) * slices), kLT, 0, st, a, slices, each);
  if (e != cudaSuccess || slices == 1) return e;
  return launch_pdl(k_logprobs_join, dim3(a.rows), kLT, 0, st, a, slices);
}

}  // namespace tqd
