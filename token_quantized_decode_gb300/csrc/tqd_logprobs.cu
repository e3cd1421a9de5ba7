// Log probabilities of given tokens, entropy and top alternatives.
#include <cuda_runtime.h>

#include "tqd_internal.h"

namespace tqd {
namespace {

constexpr int kLT = 256;

// The order of alternatives: larger logit first, equal logits by ascending
// index; NaN and -inf are no alternatives (key 0).
__device__ __forceinline__ unsigned long long logit_key(float x, int i) {
  if (!(x > -INFINITY)) return 0ull;
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t u = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (static_cast<unsigned long long>(u) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
}

__device__ __forceinline__ float key_logit(unsigned long long k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

template <class T, class F>
__device__ T block_reduce(T v, F f, T* sm) {
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sm[0];
  for (int w = 1; w < kLT / 32; ++w) v = f(v, sm[w]);
  __syncthreads();
  return v;
}

// One block per row, the row read once for the maximum, once for the sums
// and once per alternative.
__global__ void __launch_bounds__(kLT) k_logprobs(LogprobArgs a) {
  __shared__ float sf[8];
  __shared__ unsigned long long sk[8];
  const int64_t row = blockIdx.x;
  const float* x = a.logits + row * a.stride;
  auto fmx = [](float p, float q) { return fmaxf(p, q); };
  auto fadd = [](float p, float q) { return p + q; };
  float m = -INFINITY;
  for (int i = threadIdx.x; i < a.vocab; i += kLT) m = fmaxf(m, x[i]);
  m = block_reduce(m, fmx, sf);
  float s = 0.f, t = 0.f;
  for (int i = threadIdx.x; i < a.vocab; i += kLT) {
    if (!(x[i] > -INFINITY)) continue;
    const float d = x[i] == m ? 0.f : fmaxf(x[i] - m, -200.f);
    const float e = expf(d);
    s += e;
    t += e * d;
  }
  s = block_reduce(s, fadd, sf);
  t = block_reduce(t, fadd, sf);
  const float log_s = logf(s);
  auto logprob = [&](float v) { return !(v > -INFINITY) ? -INFINITY : (v == m ? 0.f : v - m) - log_s; };
  if (threadIdx.x == 0) {
    if (a.targets) {
      const int id = a.targets[row];
      a.logprob[row] = id < 0 || id >= a.vocab ? __int_as_float(0x7FC00000) : logprob(x[id]);
    }
    if (a.entropy) a.entropy[row] = m > -INFINITY ? log_s - t / s : 0.f;
  }
  unsigned long long below = ~0ull;
  for (int k = 0; k < a.top_k; ++k) {
    unsigned long long best = 0;
    for (int i = threadIdx.x; i < a.vocab; i += kLT) {
      const unsigned long long key = logit_key(x[i], i);
      if (key < below && key > best) best = key;
    }
    best = block_reduce(best, [](unsigned long long p, unsigned long long q) { return p > q ? p : q; }, sk);
    if (threadIdx.x == 0) {
      a.top_ids[row * a.top_k + k] = best ? static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best)) : -1;
      a.top_logprobs[row * a.top_k + k] = best ? logprob(key_logit(best)) : -INFINITY;
    }
    below = best;
    if (!best) below = 0;
  }
}

}  // namespace

size_t logprobs_scratch_bytes(int, int, int) { return 16; }

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t st) {
  k_logprobs<<<a.rows, kLT, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace tqd
