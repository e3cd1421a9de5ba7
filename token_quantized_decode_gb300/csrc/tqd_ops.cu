// Operator entry points of libtqd: each runs one phase of the decode step on
// caller-owned device memory (contracts in tqd.h).  They exist so that every
// piece can be checked on its own, as in the inferno.rs blog's "The
// correctness ladder", rung one.
#include <cuda_runtime.h>

#include "tqd.h"
#include "tqd_internal.h"
#include "tqd_q4.cuh"

namespace tqd {

cudaError_t allow_smem(const void* kernel, size_t bytes, unsigned long long* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (__atomic_load_n(done, __ATOMIC_RELAXED) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && dev < 64) __atomic_fetch_or(done, bit, __ATOMIC_RELAXED);
  return e;
}

}  // namespace tqd

using namespace tqd;

namespace {

int32_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return TQD_OK;
  if (e == cudaErrorInvalidValue) return TQD_ERR_BAD_ARG;
  return TQD_ERR_CUDA;
}

size_t attn_scratch_floats_o(int32_t nq, int32_t hd, int32_t nch) {
  return static_cast<size_t>(nq) * nch * hd;
}
size_t attn_scratch_floats_ml(int32_t nq, int32_t nch) { return static_cast<size_t>(nq) * nch * 2; }

int32_t refuse(const char* why) {
  set_last_error(why);
  return TQD_ERR_BAD_ARG;
}

// n rows of `width` floats, `stride` floats apart (no less than width where n > 1).
struct FloatRows {
  const float* p;
  int64_t stride, width;
};

// Whether n rows of a and n rows of b share memory (rows may lie between one another's, as slices
// of one tensor's columns do).
bool overlap(const FloatRows& a, const FloatRows& b, int64_t n) {
  using Wide = __int128;  // strides and row numbers are the caller's
  const Wide d = static_cast<Wide>(reinterpret_cast<uintptr_t>(b.p)) - static_cast<Wide>(reinterpret_cast<uintptr_t>(a.p));
  const Wide wa = a.width * static_cast<Wide>(4), wb = b.width * static_cast<Wide>(4), last = n - 1;
  const Wide sa = n > 1 ? a.stride * static_cast<Wide>(4) : wa, sb = n > 1 ? b.stride * static_cast<Wide>(4) : wb;
  if (d >= last * sa + wa || -d >= last * sb + wb) return false;
  auto floor_div = [](Wide x, Wide y) { return x >= 0 ? x / y : -((-x + y - 1) / y); };
  // row i of a, from offset `at`, meets the rows of b from lo to hi
  auto meets = [&](Wide at, Wide first) {
    const Wide lo = floor_div(at - wb - d, sb) + 1, hi = -floor_div(-(at + wa - d), sb) - 1;
    return (lo > first ? lo : first) <= (hi < last ? hi : last);
  };
  if (sa == sb) return meets(0, -last);  // the same for every row but for which rows there are
  for (Wide i = 0; i <= last; ++i)
    if (meets(i * sa, 0)) return true;
  return false;
}

size_t q4_page_bytes(int32_t n_kv, int32_t hd, int32_t page_size) {
  if (n_kv <= 0 || (hd != 64 && hd != 128) || page_size <= 0 || page_size % kQ4Block || page_size > (1 << 20))
    return 0;
  return static_cast<size_t>(n_kv) * (page_size / kQ4Block) * q4_block_bytes(hd);
}

// The caller's cache descriptor as the kernels take it; TQD_OK or a refusal.
int32_t q4_cache(const tqd_kv_q4* c, Q4Cache& o) {
  if (!c || !c->pages || !c->page_table) return refuse("tqd_kv_q4: NULL cache, pages or page_table");
  const size_t pb = q4_page_bytes(c->n_kv_heads, c->head_dim, c->page_size);
  if (!pb) return refuse("tqd_kv_q4: n_kv_heads >= 1, head_dim 64 or 128, page_size a positive multiple of 16");
  if (c->n_pages <= 0 || c->n_seq <= 0 || c->table_stride <= 0)
    return refuse("tqd_kv_q4: n_pages, n_seq and table_stride must be positive");
  if (reinterpret_cast<uintptr_t>(c->pages) % 16) return refuse("tqd_kv_q4: pages must be 16-byte aligned");
  o = Q4Cache{c->pages, c->page_table, c->n_pages, c->page_size, c->n_kv_heads, c->n_seq, c->table_stride, pb};
  return TQD_OK;
}

}  // namespace

extern "C" {

int32_t tqd_op_q8_0_repack(const uint8_t* w_blocks, int64_t rows, int64_t cols, uint8_t* w_rows,
                           void* stream) {
  if (!w_blocks || !w_rows || rows <= 0 || cols <= 0 || cols % 32) return TQD_ERR_BAD_ARG;
  return status_of(
      launch_q8_repack(w_blocks, rows, cols, w_rows, 0, 1, static_cast<cudaStream_t>(stream)));
}

int32_t tqd_op_q8_0_matvec(const uint8_t* w_rows, int64_t rows, int64_t cols, const float* x,
                           float* y, void* stream) {
  if (!w_rows || !x || !y || rows <= 0 || rows > (1ll << 30) || cols <= 0 || cols % 32 ||
      matvec_cpl(0, static_cast<int>(cols)) == 0)
    return TQD_ERR_BAD_ARG;
  return status_of(launch_op_matvec(0, w_rows, q8_row_bytes(cols),
                                    static_cast<int>(rows), static_cast<int>(cols), x, y,
                                    static_cast<cudaStream_t>(stream)));
}

int32_t tqd_op_bf16_matvec(const uint16_t* w, int64_t rows, int64_t cols, const float* x, float* y,
                           void* stream) {
  if (!w || !x || !y || rows <= 0 || rows > (1ll << 30) || cols <= 0 || cols % 8 ||
      matvec_cpl(1, static_cast<int>(cols)) == 0)
    return TQD_ERR_BAD_ARG;
  return status_of(launch_op_matvec(1, reinterpret_cast<const uint8_t*>(w),
                                    static_cast<size_t>(cols) * 2, static_cast<int>(rows),
                                    static_cast<int>(cols), x, y,
                                    static_cast<cudaStream_t>(stream)));
}

int32_t tqd_op_rmsnorm(const float* x, const float* g, int32_t rows, int32_t n, float eps,
                       float* out, void* stream) {
  if (!x || !g || !out || rows <= 0 || n <= 0 || n > 12 * 1024 || rows > 65535)
    return TQD_ERR_BAD_ARG;
  return status_of(launch_op_rmsnorm(x, g, rows, n, eps, out, static_cast<cudaStream_t>(stream)));
}

int32_t tqd_op_rope_table(float theta, int32_t head_dim, int32_t max_pos, float* table,
                          void* stream) {
  if (!table || !(theta > 0.f) || head_dim <= 0 || head_dim % 2 || max_pos <= 0)
    return TQD_ERR_BAD_ARG;
  return status_of(launch_rope_table(static_cast<double>(theta), head_dim, max_pos,
                                     reinterpret_cast<float2*>(table),
                                     static_cast<cudaStream_t>(stream)));
}

int32_t tqd_op_rope(float* x, int32_t n_heads, int32_t head_dim, int32_t pos, const float* table,
                    void* stream) {
  if (!x || !table || n_heads <= 0 || pos < 0 || (head_dim != 64 && head_dim != 128))
    return TQD_ERR_BAD_ARG;
  const float2* row = reinterpret_cast<const float2*>(table) + static_cast<size_t>(pos) * (head_dim / 2);
  return status_of(launch_op_rope(x, n_heads, head_dim, row, static_cast<cudaStream_t>(stream)));
}

size_t tqd_attention_scratch_bytes(int32_t n_heads, int32_t n_kv, int32_t head_dim,
                                   int32_t n_chunks) {
  if (n_heads <= 0 || n_kv <= 0 || head_dim <= 0 || n_chunks <= 0) return 0;
  const size_t o = attn_scratch_floats_o(n_heads, head_dim, n_chunks) * 4;
  const size_t ml = attn_scratch_floats_ml(n_heads, n_chunks) * 4;
  return o + ml + static_cast<size_t>(n_kv) * 4;
}

int32_t tqd_op_attention(const float* q, const float* K, const float* V, int32_t S,
                         int32_t n_heads, int32_t n_kv, int32_t head_dim, int32_t n_chunks,
                         float* out, void* scratch, void* stream) {
  if (!q || !K || !V || !out || !scratch || S <= 0 || n_heads <= 0 || n_kv <= 0 ||
      n_heads % n_kv || n_chunks < 1 || n_chunks > 1024 || n_kv * n_chunks > (1 << 20) ||
      !attention_supported(head_dim, n_heads / n_kv))
    return TQD_ERR_BAD_ARG;
  float* po = static_cast<float*>(scratch);
  float* pml = po + attn_scratch_floats_o(n_heads, head_dim, n_chunks);
  uint32_t* cnt =
      reinterpret_cast<uint32_t*>(pml + attn_scratch_floats_ml(n_heads, n_chunks));
  return status_of(launch_op_attention(q, K, V, S, n_heads, n_kv, head_dim, n_chunks, out, po, pml,
                                       cnt, static_cast<cudaStream_t>(stream)));
}

int32_t tqd_op_wait_selftest(void* stream, uint32_t* err_bits_out) {
  if (!err_bits_out) return TQD_ERR_BAD_ARG;
  uint32_t bits = 0u;
  const cudaError_t e = run_wait_selftest(&bits, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return status_of(e);
  *err_bits_out = bits;
  return bits ? TQD_ERR_DEVICE_TIMEOUT : TQD_OK;
}

int32_t tqd_op_silu_mul(const float* g, const float* u, int64_t n, float* out, void* stream) {
  if (!g || !u || !out || n <= 0) return TQD_ERR_BAD_ARG;
  return status_of(launch_op_silu_mul(g, u, n, out, static_cast<cudaStream_t>(stream)));
}

size_t tqd_argmax_scratch_bytes(void) { return static_cast<size_t>(kOpArgmaxBlocks) * 8 + 16; }

int32_t tqd_op_argmax(const float* x, int64_t n, int32_t* idx_out, void* scratch, void* stream) {
  if (!x || !idx_out || !scratch || n <= 0 || n > 0x7FFFFFFEll) return TQD_ERR_BAD_ARG;
  float* cv = static_cast<float*>(scratch);
  int32_t* ci = reinterpret_cast<int32_t*>(cv + kOpArgmaxBlocks);
  uint32_t* cnt = reinterpret_cast<uint32_t*>(ci + kOpArgmaxBlocks);
  return status_of(launch_op_argmax(x, n, idx_out, cv, ci, cnt, static_cast<cudaStream_t>(stream)));
}

size_t tqd_sample_scratch_bytes(int32_t vocab) {
  if (vocab <= 0) return 0;
  const size_t v4 = (static_cast<size_t>(vocab) + 3) / 4 * 4;
  return 384 + 3 * 4 * v4;
}

int32_t tqd_op_sample(const float* logits, int32_t vocab, int32_t* tokens, int32_t n_inputs,
                      const tqd_sampling* sampling, void* scratch, void* stream) {
  if (!logits || !tokens || !scratch || vocab <= 0 || n_inputs < 1 || n_inputs >= 0x7FFFFFFF ||
      reinterpret_cast<uintptr_t>(scratch) % 16)
    return TQD_ERR_BAD_ARG;
  SampleArgs a{};
  bool greedy = false;
  int32_t rc = sampling_args(sampling, a, &greedy);
  if (rc) return rc;
  if (greedy) a.temperature = 0.f;
  // scratch: the sequence descriptor and its state, then the padded logits,
  // the penalised logits and the input counts ([vocab rounded up to 4] each)
  const size_t v4 = (static_cast<size_t>(vocab) + 3) / 4 * 4;
  uint8_t* base = static_cast<uint8_t*>(scratch);
  DevSeq* dseq = reinterpret_cast<DevSeq*>(base);
  DevState* dstate = reinterpret_cast<DevState*>(base + 256);
  float* lg = reinterpret_cast<float*>(base + 384);
  DevSeq h{};
  h.state = dstate;
  h.tokens = tokens;
  h.logits = lg;
  h.sz = lg + v4;
  h.scnt = reinterpret_cast<uint32_t*>(lg + 2 * v4);
  static_assert(sizeof(DevSeq) <= 256, "descriptor fits the scratch header");
  DevState st{static_cast<uint32_t>(n_inputs), 0u, 0u, 0u};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // copies from pageable host memory are staged before cudaMemcpyAsync returns
  cudaError_t e = cudaMemcpyAsync(dseq, &h, sizeof(h), cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaMemcpyAsync(dstate, &st, sizeof(st), cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaMemcpyAsync(lg, logits, 4ull * vocab, cudaMemcpyDeviceToDevice, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(h.scnt, 0, 4 * v4, s);
  if (e == cudaSuccess) e = launch_sample(dseq, 1, vocab, n_inputs, a, s);
  return status_of(e);
}

size_t tqd_kv_q4_page_bytes(int32_t n_kv_heads, int32_t head_dim, int32_t page_size) {
  return q4_page_bytes(n_kv_heads, head_dim, page_size);
}

int32_t tqd_op_kv_append_q4(const tqd_kv_q4* cache, const float* k, int64_t k_stride, const float* v,
                            int64_t v_stride, const int32_t* positions, const int32_t* seqs, int32_t n_tokens,
                            const float* rope_table, int32_t max_pos, const float* q, int64_t q_stride,
                            int32_t n_heads, float* q_out, int64_t q_out_stride, void* stream) {
  Q4Cache c;
  if (const int32_t rc = q4_cache(cache, c)) return rc;
  if (!n_tokens) return TQD_OK;
  if (!k || !v || !positions || n_tokens < 0 || (rope_table && max_pos <= 0))
    return refuse("tqd_op_kv_append_q4: NULL k, v or positions, n_tokens < 0, or a table without positions");
  if (!seqs && n_tokens > c.n_seq) return refuse("tqd_op_kv_append_q4: more tokens than sequences and no seqs");
  if (q ? n_heads <= 0 || !q_out : n_heads != 0)
    return refuse("tqd_op_kv_append_q4: q needs n_heads > 0 and q_out; without q n_heads must be 0");
  const int64_t kvw = static_cast<int64_t>(c.n_kv) * cache->head_dim, qw = static_cast<int64_t>(n_heads) * cache->head_dim;
  if (k_stride < kvw || v_stride < kvw || (q && (q_stride < qw || q_out_stride < qw)))
    return refuse("tqd_op_kv_append_q4: a row stride shorter than the row");
  if (static_cast<int64_t>(n_tokens) * c.n_kv > (1ll << 30) || kvw > (1 << 24) || qw > (1 << 24))
    return refuse("tqd_op_kv_append_q4: n_tokens * n_kv_heads above 2^30, or rows above 2^24 floats");
  if (q) {
    const FloatRows in{q, q_stride, qw}, to{q_out, q_out_stride, qw};
    const bool same = q == q_out && (q_stride == q_out_stride || n_tokens == 1);
    if ((!same && overlap(in, to, n_tokens)) || overlap(to, {k, k_stride, kvw}, n_tokens) ||
        overlap(to, {v, v_stride, kvw}, n_tokens))
      return refuse("tqd_op_kv_append_q4: q_out overlaps k, v, or q without being the same rows");
  }
  return status_of(launch_kv_append_q4(c, cache->head_dim, k, k_stride, v, v_stride, positions, seqs, n_tokens,
                                       reinterpret_cast<const float2*>(rope_table), max_pos, q, q_stride, n_heads,
                                       q_out, q_out_stride, static_cast<cudaStream_t>(stream)));
}

int32_t tqd_op_kv_read_q4(const tqd_kv_q4* cache, const int32_t* positions, const int32_t* seqs, int32_t n_tokens,
                          float* k_out, int64_t k_stride, float* v_out, int64_t v_stride, void* stream) {
  Q4Cache c;
  if (const int32_t rc = q4_cache(cache, c)) return rc;
  if (!n_tokens) return TQD_OK;
  if (!positions || (!k_out && !v_out) || n_tokens < 0)
    return refuse("tqd_op_kv_read_q4: NULL positions, no output, or n_tokens < 0");
  if (!seqs && n_tokens > c.n_seq) return refuse("tqd_op_kv_read_q4: more tokens than sequences and no seqs");
  const int64_t kvw = static_cast<int64_t>(c.n_kv) * cache->head_dim;
  if ((k_out && k_stride < kvw) || (v_out && v_stride < kvw))
    return refuse("tqd_op_kv_read_q4: a row stride shorter than the row");
  if (static_cast<int64_t>(n_tokens) * c.n_kv > (1ll << 30)) return refuse("tqd_op_kv_read_q4: n_tokens * n_kv_heads above 2^30");
  if (k_out && v_out && overlap({k_out, k_stride, kvw}, {v_out, v_stride, kvw}, n_tokens))
    return refuse("tqd_op_kv_read_q4: k_out overlaps v_out");
  return status_of(launch_kv_read_q4(c, cache->head_dim, positions, seqs, n_tokens, k_out, k_stride, v_out, v_stride,
                                     static_cast<cudaStream_t>(stream)));
}

size_t tqd_attention_q4_scratch_bytes(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 ? attention_q4_scratch_bytes(head_dim) : 0;
}

int32_t tqd_op_attention_q4(const tqd_kv_q4* cache, const float* q, int64_t q_stride, const int32_t* lens,
                            const int32_t* q_start, int32_t n_tokens, int32_t n_heads, float* out, int64_t out_stride,
                            void* scratch, void* stream) {
  Q4Cache c;
  if (const int32_t rc = q4_cache(cache, c)) return rc;
  if (!n_tokens && q_start) return TQD_OK;
  if (!q || !lens || !out || !scratch || n_tokens < 0 || n_heads <= 0 || n_heads % c.n_kv)
    return refuse("tqd_op_attention_q4: NULL pointer, n_tokens < 0, or n_heads no multiple of n_kv_heads");
  if (c.n_seq > kQ4MaxSeqs) return refuse("tqd_op_attention_q4: more than 1024 sequences");
  if (!q_start && n_tokens != c.n_seq) return refuse("tqd_op_attention_q4: without q_start one query per sequence");
  const int64_t qw = static_cast<int64_t>(n_heads) * cache->head_dim;
  if (q_stride < qw || out_stride < qw) return refuse("tqd_op_attention_q4: a row stride shorter than the row");
  if (reinterpret_cast<uintptr_t>(scratch) % 16) return refuse("tqd_op_attention_q4: scratch must be 16-byte aligned");
  if (static_cast<int64_t>(n_tokens) * n_heads > (1ll << 30))
    return refuse("tqd_op_attention_q4: n_tokens * n_heads above 2^30");
  if (overlap({q, q_stride, qw}, {out, out_stride, qw}, n_tokens)) return refuse("tqd_op_attention_q4: out overlaps q");
  const Q4AttnArgs a{c, q, out, lens, q_start, scratch, q_stride, out_stride, n_tokens, n_heads,
                     cache->head_dim == 128 ? 0.08838834764831845f : 0.125f};
  return status_of(launch_attention_q4(a, cache->head_dim, static_cast<cudaStream_t>(stream)));
}

size_t tqd_q4_0_matrix_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols % 32) return 0;
  return static_cast<size_t>((rows + kQ4TileRows - 1) / kQ4TileRows) *
         static_cast<size_t>((cols + kQ4TileCols - 1) / kQ4TileCols) * kQ4TileBytes;
}

int32_t tqd_op_q4_0_repack(const uint8_t* w_blocks, int64_t rows, int64_t cols, uint8_t* w_tiles, void* stream) {
  if (!w_blocks || !w_tiles || rows <= 0 || rows > (1ll << 30) || cols <= 0 || cols % 32 || cols > kQ4MatvecMaxCols)
    return refuse("tqd_op_q4_0_repack: NULL pointer, or cols no multiple of 32 up to 16384");
  if (tqd_q4_0_matrix_bytes(rows, cols) / kQ4TileBytes > 0x7FFFFFFFull) return refuse("tqd_op_q4_0_repack: matrix too large");
  if (reinterpret_cast<uintptr_t>(w_tiles) % 16) return refuse("tqd_op_q4_0_repack: w_tiles must be 16-byte aligned");
  return status_of(launch_q4_repack(w_blocks, rows, cols, w_tiles, static_cast<cudaStream_t>(stream)));
}

int32_t tqd_op_q4_0_matvec(const uint8_t* w_tiles, int64_t rows, int64_t cols, const float* x, int32_t n,
                           int64_t x_stride, float* y, int64_t y_stride, void* stream) {
  if (!n) return TQD_OK;
  if (!w_tiles || !x || !y || rows <= 0 || rows > (1ll << 30) || cols <= 0 || cols % 32 || cols > kQ4MatvecMaxCols ||
      n < 0 || n > kQ4MatvecMaxVectors)
    return refuse("tqd_op_q4_0_matvec: NULL pointer, cols no multiple of 32 up to 16384, or n above 64");
  if (n > 1 && (x_stride < cols || y_stride < rows)) return refuse("tqd_op_q4_0_matvec: a row stride shorter than the row");
  if (reinterpret_cast<uintptr_t>(w_tiles) % 16) return refuse("tqd_op_q4_0_matvec: w_tiles must be 16-byte aligned");
  if (overlap({x, x_stride, cols}, {y, y_stride, rows}, n)) return refuse("tqd_op_q4_0_matvec: y overlaps x");
  return status_of(launch_q4_matvec(w_tiles, static_cast<int>(rows), static_cast<int>(cols), x, n, x_stride, y, y_stride,
                                    static_cast<cudaStream_t>(stream)));
}

size_t tqd_logprobs_scratch_bytes(int32_t rows, int32_t vocab, int32_t top_k) {
  if (rows <= 0 || vocab <= 0 || vocab > (1 << 30) || top_k < 0 || top_k > kLogprobMaxTopK) return 0;
  return logprobs_scratch_bytes(rows, vocab, top_k);
}

int32_t tqd_op_logprobs(const float* logits, int64_t stride, int32_t rows, int32_t vocab, const int32_t* targets,
                        float* logprob, float* entropy, int32_t top_k, int32_t* top_ids, float* top_logprobs,
                        void* scratch, void* stream) {
  if (!rows) return TQD_OK;
  if (!logits || !scratch || rows < 0 || vocab <= 0 || vocab > (1 << 30) || stride < vocab || top_k < 0 || top_k > kLogprobMaxTopK)
    return refuse("tqd_op_logprobs: NULL logits or scratch, rows < 0, vocab outside 1 .. 2^30, stride < vocab, or top_k above 32");
  if (!targets != !logprob) return refuse("tqd_op_logprobs: targets and logprob go together");
  if (top_k ? !top_ids || !top_logprobs : !logprob && !entropy)
    return refuse("tqd_op_logprobs: top_k needs top_ids and top_logprobs; nothing else asked for");
  if (rows * static_cast<int64_t>(vocab) > (1ll << 40)) return refuse("tqd_op_logprobs: more than 2^40 logits");
  if (reinterpret_cast<uintptr_t>(scratch) % 16) return refuse("tqd_op_logprobs: scratch must be 16-byte aligned");
  const LogprobArgs a{logits, targets, logprob, entropy, top_ids, top_logprobs, scratch, stride, rows, vocab, top_k};
  return status_of(launch_logprobs(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
