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
// candidates in shared memory and a threshold, the k-th best logit so far,
// brought up to date after 4, 16, 64, ... tiles (about 3 k insertions each time,
// and no other barrier while a row streams): a thread compares its largest new logit
// with it, and on most tiles that is all.  The first 4 tiles are read again (from
// L2) with the k-th largest of the threads' maxima, which at least k tokens reach
// and about k do.  A list that overflows (many equal logits, or ascending ones) is
// dropped, and at the end all threads read again what lies with the threads
// whose largest logit reaches the k-th largest; where more than 64 do, the equal
// logits are taken in order of index.
//
// HBM bounds it: 4 bytes a logit and about seven instructions (a fused
// multiply-add, a maximum, an exponential, two sums; half a maximum).  A tile
// is 8 logits a thread, the next one's loads issued before the current one's
// work.  2053 rows of 151936 take 193 us without alternatives (1.25 GB: 6.5 TB/s,
// 95 % of a copy's rate), 216 with 20 (85 %): the lists' barriers and the last
// wave of blocks.  Few rows are cut into slices of whole tiles, one block each,
// whose partial (m, s, t) and alternatives a second kernel joins (programmatic
// dependent launch): one row takes 10.8 us, two launches.
#include <cuda_runtime.h>

#include "tqd_internal.h"

namespace tqd {
namespace {

constexpr int kLT = 256;         // threads of a block
constexpr int kEach = 8;         // logits of a thread per tile
constexpr int kTile = kLT * kEach;
constexpr int kCap = 1024;       // candidates a block holds
constexpr int kFirst = 4;        // tiles before the list is first looked at
constexpr int kMost = 64;        // threads whose logits are read again
constexpr int kJoinCap = kLogprobMaxTopK * kLogprobMaxTopK;
constexpr int kMaxSlices = 256;

using Key = unsigned long long;

// An f32's bits in integer order (-0 as 0), and back.
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float bits_order(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// 0 for NaN and -inf, which are no alternatives.
__device__ __forceinline__ Key logit_key(float x, int i) {
  if (!(x > -INFINITY)) return 0ull;
  return (static_cast<Key>(order_bits(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float key_logit(Key k) { return bits_order(static_cast<uint32_t>(k >> 32)); }
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
  __shared__ int count, found, members;
  __shared__ uint8_t member[kLT];
  __shared__ uint32_t floor_;
  const int tid = threadIdx.x, lane = tid & 31, k = a.top_k;
  pdl_wait();
  pdl_launch_dependents();
  const unsigned row = blockIdx.x / static_cast<unsigned>(slices);
  const int slice = static_cast<int>(blockIdx.x - row * slices);
  const float* x = a.logits + static_cast<int64_t>(row) * a.stride;
  // 16-byte loads from the aligned address at or before the row; what lies outside the row is not read
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(x) >> 2) & 3);
  const int tiles = (a.vocab + off + kTile - 1) / kTile;
  const int tile0 = slice * tiles_each, tile1 = min(tile0 + tiles_each, tiles);
  const int whole0 = off ? 1 : 0, whole1 = (a.vocab + off) / kTile;  // tiles that lie inside the row

  // the four logits of quad `quad` of a tile (thread t holds quads t and kLT + t), and the index of the first
  auto quad_index = [&](int tile, int quad) { return tile * kTile - off + quad * 4; };
  auto load_quad = [&](int tile, int quad) {
    const int i = quad_index(tile, quad);
    if (tile >= whole0 && tile < whole1) return *reinterpret_cast<const float4*>(x + i);
    float4 q;
    q.x = i >= 0 && i < a.vocab ? x[i] : -INFINITY;
    q.y = i + 1 >= 0 && i + 1 < a.vocab ? x[i + 1] : -INFINITY;
    q.z = i + 2 >= 0 && i + 2 < a.vocab ? x[i + 2] : -INFINITY;
    q.w = i + 3 >= 0 && i + 3 < a.vocab ? x[i + 3] : -INFINITY;
    return q;
  };
  auto load = [&](int tile, float (&v)[kEach]) {
    if (tile >= whole0 && tile < whole1) {
      const float* p = x + quad_index(tile, tid);
#pragma unroll
      for (int h = 0; h < kEach / 4; ++h) {
        const float4 q = *reinterpret_cast<const float4*>(p + h * (kLT * 4));
        v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int h = 0; h < kEach / 4; ++h) {
        const float4 q = load_quad(tile, h * kLT + tid);
        v[4 * h] = q.x; v[4 * h + 1] = q.y; v[4 * h + 2] = q.z; v[4 * h + 3] = q.w;
      }
    }
  };
  auto insert = [&](float v, int i) {
    const int p = atomicAdd(&count, 1);
    if (p < kCap) buf[p] = logit_key(v, i);
  };
  auto index_of = [&](int tile, int j) { return quad_index(tile, (j >> 2) * kLT + tid) + (j & 3); };
  // The k-th largest of the threads' largest logits (in heads; this thread's is mine), -inf where fewer than k
  // are above it.  floor_ holds ~0 before.
  auto kth_head = [&](float mine) {
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < kLT; j += 4) {
      const float4 h = *reinterpret_cast<const float4*>(heads + j);
      above += h.x > mine;
      above += h.y > mine;
      above += h.z > mine;
      above += h.w > mine;
    }
    if (above < k) atomicMin(&floor_, order_bits(mine));
    __syncthreads();
    return bits_order(floor_);
  };

  // ---- one pass: sums, and the thread's largest logit
  constexpr float kRefMin = -1048576.f;
  float ref = kRefMin, rise = -INFINITY;  // rise: a logit above it moves the reference
  float rs = 0.f, rt = 0.f, rm = -INFINITY;
  float least = INFINITY;  // a logit above it is a candidate
  int check = k ? min(tile0 + kFirst, tile1) : tile1 + 1, n = 0;  // the tile before which the list is looked at; its length then
  bool over = false, first = true;
  float nx[kEach];
  if (tid == 0) {
    count = found = members = 0;
    floor_ = ~0u;
  }
  if (tile0 < tile1) load(tile0, nx);
  for (int tile = tile0; tile < tile1; ++tile) {
    float v[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) v[j] = nx[j];
    if (tile + 1 < tile1) load(tile + 1, nx);
    float lm = fmaxf(v[0], -INFINITY);  // (eight NaN)
#pragma unroll
    for (int j = 1; j < kEach; ++j) lm = fmaxf(lm, v[j]);
    rm = fmaxf(rm, lm);
    if (lm > rise) {
      const float nref = fminf(fmaxf(rintf(lm * kLog2e), kRefMin), -kRefMin);
      const float d = fmaxf(ref - nref, -300.f), w = ex2(d);
      rt = w * (rt + rs * d);
      rs *= w;
      ref = nref;
      rise = (nref + 16.f) * kLn2;
    }
    // (a tile's terms first: added one by one beside a thread's largest ones, small terms lose
    // their last bits all the same way; entropies of rows with peaks 3.3e-7 off, so 9e-8)
    float es[2] = {0.f, 0.f}, et[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const float d = fmaxf(fmaf(v[j], kLog2e, -ref), -300.f), e = ex2(d);
      es[j & 1] += e;
      et[j & 1] = fmaf(e, d, et[j & 1]);
    }
    rs += es[0] + es[1];
    rt += et[0] + et[1];
    if (lm > least) {
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (v[j] > least) insert(v[j], index_of(tile, j));
    }
    if (tile + 1 != check) continue;

    // ---- the list is brought up to date
    if (first) {  // these tiles again
      first = false;
      heads[tid] = rm;
      __syncthreads();
      const float reach = kth_head(rm);
      if (rm >= reach && rm > -INFINITY)
        for (int t = tile0; t < check; ++t) {
          float w[kEach];
          load(t, w);
#pragma unroll
          for (int j = 0; j < kEach; ++j)
            if (w[j] >= reach && w[j] > -INFINITY) insert(w[j], index_of(t, j));
        }
    }
    __syncthreads();
    n = count;
    over |= n > kCap;
    __syncthreads();
    if (over) {
      least = INFINITY;
    } else {
      keep_best(buf, n, k, best);
      n = min(n, k);
      if (tid < n) buf[tid] = best[tid];
      least = n == k ? key_logit(best[k - 1]) : -INFINITY;
    }
    if (tid == 0) count = over ? 0 : n;
    check = check == tile1 ? tile1 + 1 : min(tile0 + 4 * (check - tile0), tile1);
    __syncthreads();
  }

  // ---- the block's sums, relative to its own largest logit
  heads[tid] = rm;
  if (tid == 0) {
    count = 0;
    floor_ = ~0u;
  }
  __syncthreads();
  float bm = fmaxf(fmaxf(heads[lane], heads[lane + 32]), fmaxf(heads[lane + 64], heads[lane + 96]));
  bm = fmaxf(bm, fmaxf(fmaxf(heads[lane + 128], heads[lane + 160]), fmaxf(heads[lane + 192], heads[lane + 224])));
  bm = warp_max(bm);
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
  // (all relative to the same logit: plain sums)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    own.s += __shfl_xor_sync(0xFFFFFFFFu, own.s, o);
    own.t += __shfl_xor_sync(0xFFFFFFFFu, own.t, o);
  }
  if (lane == 0) sm[tid >> 5] = own;

  // ---- the k best, where the list overflowed
  if (over) {
    const float reach = kth_head(rm);  // -inf: fewer than k threads hold a logit above it
    const int reaching = __syncthreads_count(rm > -INFINITY && rm >= reach);
    const bool ties = reaching > kMost;
    if (rm > -INFINITY && (ties ? rm > reach : rm >= reach)) member[atomicAdd(&members, 1)] = static_cast<uint8_t>(tid);
    __syncthreads();
    const int m = members;
    const int items = (tile1 - tile0) * (kEach / 4) * m;  // quads to read again
    auto take = [&](float v, int i) {
      if (ties ? v > reach : v >= reach && v > -INFINITY) {
        const int p = atomicAdd(&count, 1);
        if (p < kCap) buf[p] = logit_key(v, i);
      }
    };
    for (int i0 = tid; i0 < items; i0 += 4 * kLT) {
      float4 q[4];
      int at[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kLT;
        q[u] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (i < items) {
          const int part = i / m, tile = tile0 + part / (kEach / 4);
          const int quad = part % (kEach / 4) * kLT + member[i - part * m];
          at[u] = quad_index(tile, quad);
          q[u] = load_quad(tile, quad);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        take(q[u].x, at[u]);
        take(q[u].y, at[u] + 1);
        take(q[u].z, at[u] + 2);
        take(q[u].w, at[u] + 3);
      }
    }
    __syncthreads();
    n = count;
    if (ties && n < k) {
      // the first k - n tokens at the threshold, in order of index: quads of a
      // tile in the threads' order, each thread's place from the counts before it
      for (int tile = tile0; tile < tile1 && n + found < k; ++tile)
        for (int h = 0; h < kEach / 4; ++h) {
          const float4 q = load_quad(tile, h * kLT + tid);
          const int mine = (q.x == reach) + (q.y == reach) + (q.z == reach) + (q.w == reach);
          int run = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, run, o);
            if (lane >= o) run += u;
          }
          if (lane == 31) heads[tid >> 5] = __int_as_float(run);
          __syncthreads();
          int place = n + found + run - mine, all = 0;
          for (int w = 0; w < kLT / 32; ++w) {
            const int c = __float_as_int(heads[w]);
            if (w < (tid >> 5)) place += c;
            all += c;
          }
          const float v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (v[j] == reach) {
              if (place < k) buf[place] = logit_key(v[j], quad_index(tile, h * kLT + tid) + j);
              ++place;
            }
          __syncthreads();
          if (tid == 0) found += all;
          __syncthreads();
        }
      n = min(n + found, k);
    }
    if (n > kCap) {
      // More than the list holds (a few threads hold most large logits): one by one.
      Key below = ~0ull;
      Key* hk = reinterpret_cast<Key*>(heads);
      for (int r = 0; r < k; ++r) {
        Key top = 0ull;
        for (int tile = tile0; tile < tile1; ++tile) {
#pragma unroll
          for (int h = 0; h < kEach / 4; ++h) {
            const float4 q = load_quad(tile, h * kLT + tid);
            const int i = quad_index(tile, h * kLT + tid);
            const Key keys[4] = {logit_key(q.x, i), logit_key(q.y, i + 1), logit_key(q.z, i + 2), logit_key(q.w, i + 3)};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (keys[j] < below && keys[j] > top) top = keys[j];
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const Key w = __shfl_xor_sync(0xFFFFFFFFu, top, o);
          if (w > top) top = w;
        }
        __syncthreads();
        if (lane == 0) hk[tid >> 5] = top;
        __syncthreads();
        top = hk[0];
        for (int w = 1; w < kLT / 32; ++w)
          if (hk[w] > top) top = hk[w];
        if (tid == 0) best[r] = top;
        below = top;
      }
      n = k;  // (there are more than kCap >= k)
      __syncthreads();
    } else {
      keep_best(buf, n, k, best);
      n = min(n, k);
    }
  } else {
    __syncthreads();
  }

  Sums all{bm, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < kLT / 32; ++w) {
    all.s += sm[w].s;
    all.t += sm[w].t;
  }
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
    const Key reach = floor_;
    for (int i0 = tid; i0 < slices * k; i0 += 4 * kLT) {
      Key key[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kLT, sl = i / k;
        key[u] = i < slices * k && heads[sl] >= reach
                     ? reinterpret_cast<const Key*>(part + sl * partial_bytes(k) + 16)[i - sl * k]
                     : 0ull;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (key[u] >= reach) buf[atomicAdd(&count, 1)] = key[u];
    }
    __syncthreads();
    keep_best(buf, count, k, best);
    n = min(count, k);
  }
  write_row(a, row, all, best, n);
}

constexpr int64_t kWave = 5 * 152;  // blocks that run at once

int tiles_of(int vocab) { return (vocab + 3 + kTile - 1) / kTile; }
int most_slices(int vocab) { return tiles_of(vocab) < kMaxSlices ? tiles_of(vocab) : kMaxSlices; }

// Slices of a row, of whole tiles: what makes the waves of 5 blocks an SM
// shortest, a block being counted as its tiles and, for its beginning, end and
// list, 8 more (2 without alternatives).  More than one only where one slice
// less leaves fewer than 4 waves of blocks.
int slices_of(int rows, int vocab, int top_k) {
  const int tiles = tiles_of(vocab), most = most_slices(vocab), fixed = top_k ? 8 : 2;
  int best = 1;
  int64_t least = -1;
  for (int s = 1; s <= most; ++s) {
    const int each = (tiles + s - 1) / s;
    const int64_t cost = (static_cast<int64_t>(rows) * s + kWave - 1) / kWave * (each + fixed);
    if (least < 0 || cost < least) {
      least = cost;
      best = s;
    }
    if (static_cast<int64_t>(rows) * s >= 4 * kWave) break;
  }
  const int each = (tiles + best - 1) / best;
  return (tiles + each - 1) / each;
}

}  // namespace

// Room for a call of these sizes and of any smaller ones.  Fewer rows are cut into more
// slices, so what a call needs does not grow with its rows; but with s > 1 slices
// rows * (s - 1) < 4 kWave, hence rows < 4 kWave and rows * s < 4 kWave + rows.
size_t logprobs_scratch_bytes(int rows, int vocab, int top_k) {
  const int most = most_slices(vocab);
  if (most == 1) return 16;
  const int64_t all = static_cast<int64_t>(rows) * most, cut = 4 * kWave + (rows < 4 * kWave ? rows : 4 * kWave);
  return static_cast<size_t>(all < cut ? all : cut) * partial_bytes(top_k);
}

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t st) {
  const int slices = slices_of(a.rows, a.vocab, a.top_k), tiles = tiles_of(a.vocab);
  const int each = (tiles + slices - 1) / slices;
  const cudaError_t e = launch_pdl(k_logprobs, dim3(static_cast<unsigned>(a.rows) * slices), kLT, 0, st, a, slices, each);
  if (e != cudaSuccess || slices == 1) return e;
  return launch_pdl(k_logprobs_join, dim3(a.rows), kLT, 0, st, a, slices);
}

}  // namespace tqd
