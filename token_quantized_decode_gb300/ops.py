"""Operator entry points of libtqd on torch CUDA tensors (tqd_op_* in
include/tqd.h).  Each call marshals data pointers and the current stream into
one C call; outputs are written into caller-allocated tensors."""
from __future__ import annotations

from ._lib import TQDError, check, lib, tqd_kv_q4


def _s(stream):
    import torch
    return int((stream or torch.cuda.current_stream()).cuda_stream)


def tqd_op_q8_0_repack(w_blocks, rows: int, cols: int, w_rows, stream=None):
    check(lib().tqd_op_q8_0_repack(w_blocks.data_ptr(), rows, cols, w_rows.data_ptr(), _s(stream)),
          "tqd_op_q8_0_repack")


def tqd_op_q8_0_matvec(w_rows, rows: int, cols: int, x, y, stream=None):
    check(lib().tqd_op_q8_0_matvec(w_rows.data_ptr(), rows, cols, x.data_ptr(), y.data_ptr(), _s(stream)),
          "tqd_op_q8_0_matvec")


def tqd_op_bf16_matvec(w, rows: int, cols: int, x, y, stream=None):
    check(lib().tqd_op_bf16_matvec(w.data_ptr(), rows, cols, x.data_ptr(), y.data_ptr(), _s(stream)),
          "tqd_op_bf16_matvec")


def tqd_op_rmsnorm(x, g, rows: int, n: int, eps: float, out, stream=None):
    check(lib().tqd_op_rmsnorm(x.data_ptr(), g.data_ptr(), rows, n, eps, out.data_ptr(), _s(stream)),
          "tqd_op_rmsnorm")


def tqd_op_rope_table(theta: float, head_dim: int, max_pos: int, table, stream=None):
    check(lib().tqd_op_rope_table(theta, head_dim, max_pos, table.data_ptr(), _s(stream)), "tqd_op_rope_table")


def tqd_op_rope(x, n_heads: int, head_dim: int, pos: int, table, stream=None):
    check(lib().tqd_op_rope(x.data_ptr(), n_heads, head_dim, pos, table.data_ptr(), _s(stream)), "tqd_op_rope")


def tqd_attention_scratch_bytes(n_heads: int, n_kv: int, head_dim: int, n_chunks: int) -> int:
    return int(lib().tqd_attention_scratch_bytes(n_heads, n_kv, head_dim, n_chunks))


def tqd_op_attention(q, K, V, S: int, n_heads: int, n_kv: int, head_dim: int, n_chunks: int, out,
                     scratch, stream=None):
    check(lib().tqd_op_attention(q.data_ptr(), K.data_ptr(), V.data_ptr(), S, n_heads, n_kv, head_dim,
                                 n_chunks, out.data_ptr(), scratch.data_ptr(), _s(stream)),
          "tqd_op_attention")


def tqd_op_attention_noalloc(q, K, V, S: int, n_heads: int, n_kv: int, head_dim: int, n_chunks: int, out,
                             stream=None):
    """tqd_op_attention without caller scratch: the library's static device
    array holds the partials (allocates nothing per call)."""
    check(lib().tqd_op_attention_noalloc(q.data_ptr(), K.data_ptr(), V.data_ptr(), S, n_heads, n_kv, head_dim,
                                         n_chunks, out.data_ptr(), _s(stream)),
          "tqd_op_attention_noalloc")


def tqd_op_attention_noalloc_max_scratch() -> int:
    return int(lib().tqd_op_attention_noalloc_max_scratch())


def tqd_op_wait_selftest(stream=None):
    """Run the bounded-wait self-test; returns (status, error bits) without
    raising (the expected status is TQD_ERR_DEVICE_TIMEOUT)."""
    import ctypes
    bits = ctypes.c_uint32(0)
    status = lib().tqd_op_wait_selftest(_s(stream), ctypes.byref(bits))
    return int(status), int(bits.value)


def tqd_op_silu_mul(g, u, n: int, out, stream=None):
    check(lib().tqd_op_silu_mul(g.data_ptr(), u.data_ptr(), n, out.data_ptr(), _s(stream)), "tqd_op_silu_mul")


def tqd_argmax_scratch_bytes() -> int:
    return int(lib().tqd_argmax_scratch_bytes())


def tqd_op_argmax(x, n: int, idx_out, scratch, stream=None):
    check(lib().tqd_op_argmax(x.data_ptr(), n, idx_out.data_ptr(), scratch.data_ptr(), _s(stream)),
          "tqd_op_argmax")


def tqd_sample_scratch_bytes(vocab: int) -> int:
    return int(lib().tqd_sample_scratch_bytes(vocab))


def tqd_op_sample(logits, vocab: int, tokens, n_inputs: int, params, scratch, stream=None):
    """The seeded draw of tqd_sample on caller tensors: tokens[:n_inputs] are
    the inputs so far, the drawn token is written to tokens[n_inputs]."""
    import ctypes
    check(lib().tqd_op_sample(logits.data_ptr(), vocab, tokens.data_ptr(), n_inputs, ctypes.byref(params),
                              scratch.data_ptr(), _s(stream)),
          "tqd_op_sample")


# ------------------------------------------------------------------ 4-bit decode operators, log probabilities
#
# These check the tensors they are given (type, device, shape, strides) before
# the C call and refuse with TQD_ERR_BAD_ARG.

def _refuse(where, why):
    raise TQDError(1, where, why)


def _ptr(t, dtype, n, where, name):
    """Data pointer of a contiguous tensor of at least n elements on the current device."""
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous() or not t.is_cuda:
        _refuse(where, f"{name}: a contiguous CUDA tensor of {n} or more {dtype} is needed, got {tuple(t.shape)} "
                       f"{t.dtype} on {t.device}")
    _on_device(t, where, name)
    return t.data_ptr()


def _on_device(t, where, name):
    import torch
    if t.get_device() != torch.cuda.current_device():
        _refuse(where, f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _rows(t, n, width, where, name):
    """Pointer and row stride of a [n, width] f32 tensor with contiguous rows ([width] when n is 1)."""
    import torch
    shape = t.shape
    if t.dtype is not torch.float32 or not t.is_cuda or not (shape == (n, width) or (n == 1 and shape == (width,))):
        _refuse(where, f"{name}: an f32 CUDA tensor [{n}, {width}] is needed, got {tuple(shape)} {t.dtype} on {t.device}")
    if width > 1 and n and t.stride(-1) != 1:
        _refuse(where, f"{name}: the elements of a row must be contiguous")
    stride = t.stride(0) if n > 1 else width
    if stride < width:
        _refuse(where, f"{name}: rows {stride} floats apart overlap")
    _on_device(t, where, name)
    return t.data_ptr(), stride


def tqd_kv_q4_page_bytes(n_kv: int, head_dim: int, page_size: int) -> int:
    return int(lib().tqd_kv_q4_page_bytes(n_kv, head_dim, page_size))


class KVCacheQ4:
    """One layer's paged 4-bit cache: the tqd_kv_q4 descriptor and the tensors it points into."""

    def __init__(self, pages, page_table, n_kv: int, head_dim: int, page_size: int):
        import torch
        where = "kv_q4"
        page_bytes = tqd_kv_q4_page_bytes(n_kv, head_dim, page_size)
        if not page_bytes:
            _refuse(where, f"n_kv {n_kv} (>= 1), head_dim {head_dim} (64 or 128), page_size {page_size} (a multiple of 16)")
        if page_table.dim() != 2 or pages.numel() % page_bytes:
            _refuse(where, f"pages: whole pages of {page_bytes} bytes; page_table: [n_seq, pages per sequence]")
        n_seq, per_seq = page_table.shape
        p = _ptr(pages, torch.uint8, page_bytes, where, "pages")
        t = _ptr(page_table, torch.int32, 1, where, "page_table")
        self.pages, self.page_table = pages, page_table
        self.n_seq, self.n_kv, self.head_dim, self.page_size = n_seq, n_kv, head_dim, page_size
        self.struct = tqd_kv_q4(p, t, pages.numel() // page_bytes, page_size, n_kv, head_dim, n_seq, per_seq)


def kv_q4(pages, page_table, n_kv: int, head_dim: int, page_size: int) -> KVCacheQ4:
    """A 4-bit cache over pages (uint8, n_pages * tqd_kv_q4_page_bytes) and an int32 page table [n_seq, pages]."""
    return KVCacheQ4(pages, page_table, n_kv, head_dim, page_size)


def tqd_op_kv_append_q4(cache: KVCacheQ4, k, v, positions, seqs=None, table=None, q=None, q_out=None, stream=None):
    """Rotate and store k, v [n, n_kv * head_dim] at positions [n] of sequences seqs [n] (None: sequence i);
    q [n, heads * head_dim], rotated, goes to q_out.  table: tqd_op_rope_table's (None: no rotation)."""
    import ctypes

    import torch
    where = "tqd_op_kv_append_q4"
    n, kvw, f32 = positions.numel(), cache.n_kv * cache.head_dim, torch.float32
    kp, ks = _rows(k, n, kvw, where, "k")
    vp, vs = _rows(v, n, kvw, where, "v")
    qp = op = None
    qs = os_ = heads = 0
    if q is not None:
        if q_out is None or q.shape[-1] % cache.head_dim:
            _refuse(where, "q needs q_out, and whole heads")
        heads = q.shape[-1] // cache.head_dim
        qp, qs = _rows(q, n, heads * cache.head_dim, where, "q")
        op, os_ = _rows(q_out, n, heads * cache.head_dim, where, "q_out")
    check(lib().tqd_op_kv_append_q4(
        ctypes.byref(cache.struct), kp, ks, vp, vs, _ptr(positions, torch.int32, n, where, "positions"),
        None if seqs is None else _ptr(seqs, torch.int32, n, where, "seqs"), n,
        None if table is None else _ptr(table, f32, cache.head_dim, where, "table"),
        0 if table is None else table.numel() // cache.head_dim, qp, qs, heads, op, os_, _s(stream)), where)


def tqd_op_kv_read_q4(cache: KVCacheQ4, positions, seqs, k_out, v_out, stream=None):
    """The values that the cache's rows stand for, f32 [n, n_kv * head_dim] (k_out or v_out may be None)."""
    import ctypes

    import torch
    where = "tqd_op_kv_read_q4"
    n, kvw = positions.numel(), cache.n_kv * cache.head_dim
    kp, ks = (None, 0) if k_out is None else _rows(k_out, n, kvw, where, "k_out")
    vp, vs = (None, 0) if v_out is None else _rows(v_out, n, kvw, where, "v_out")
    check(lib().tqd_op_kv_read_q4(ctypes.byref(cache.struct), _ptr(positions, torch.int32, n, where, "positions"),
                                  None if seqs is None else _ptr(seqs, torch.int32, n, where, "seqs"), n, kp, ks, vp,
                                  vs, _s(stream)), where)


def tqd_attention_q4_scratch_bytes(head_dim: int) -> int:
    return int(lib().tqd_attention_q4_scratch_bytes(head_dim))


def tqd_op_attention_q4(cache: KVCacheQ4, q, lens, q_start, out, scratch, stream=None):
    """Attention of q [n, heads * head_dim] over the cache: one query per sequence (q_start None), or tokens
    q_start[s] .. q_start[s + 1] - 1 as the last positions of sequence s."""
    import ctypes

    import torch
    where = "tqd_op_attention_q4"
    if q.dim() != 2 or q.shape[1] % cache.head_dim:
        _refuse(where, "q: [n, heads * head_dim]")
    n, width = q.shape
    qp, qs = _rows(q, n, width, where, "q")
    op, os_ = _rows(out, n, width, where, "out")
    check(lib().tqd_op_attention_q4(
        ctypes.byref(cache.struct), qp, qs, _ptr(lens, torch.int32, cache.n_seq, where, "lens"),
        None if q_start is None else _ptr(q_start, torch.int32, cache.n_seq + 1, where, "q_start"), n,
        width // cache.head_dim, op, os_,
        _ptr(scratch, torch.uint8, tqd_attention_q4_scratch_bytes(cache.head_dim), where, "scratch"), _s(stream)), where)


def tqd_q4_0_matrix_bytes(rows: int, cols: int) -> int:
    return int(lib().tqd_q4_0_matrix_bytes(rows, cols))


def tqd_op_q4_0_repack(w_blocks, rows: int, cols: int, w_tiles, stream=None):
    """Q4_0 blocks (uint8, rows * cols / 32 * 18) into the tiles that the matvec reads (tqd_q4_0_matrix_bytes)."""
    import torch
    where = "tqd_op_q4_0_repack"
    if cols % 32:
        _refuse(where, "cols must be a multiple of 32")
    check(lib().tqd_op_q4_0_repack(_ptr(w_blocks, torch.uint8, rows * (cols // 32) * 18, where, "w_blocks"), rows, cols,
                                   _ptr(w_tiles, torch.uint8, tqd_q4_0_matrix_bytes(rows, cols), where, "w_tiles"),
                                   _s(stream)), where)


def tqd_op_q4_0_matvec(w_tiles, rows: int, cols: int, x, y, stream=None):
    """y [n, rows] = x [n, cols] W^T over repacked Q4_0 weights (x [cols], y [rows]: one vector), n <= 64."""
    import torch
    where = "tqd_op_q4_0_matvec"
    n = x.shape[0] if x.dim() == 2 else 1
    xp, xs = _rows(x, n, cols, where, "x")
    yp, ys = _rows(y, n, rows, where, "y")
    check(lib().tqd_op_q4_0_matvec(_ptr(w_tiles, torch.uint8, tqd_q4_0_matrix_bytes(rows, cols), where, "w_tiles"),
                                   rows, cols, xp, n, xs, yp, ys, _s(stream)), where)


def tqd_logprobs_scratch_bytes(rows: int, vocab: int, top_k: int) -> int:
    return int(lib().tqd_logprobs_scratch_bytes(rows, vocab, top_k))


def tqd_op_logprobs(logits, targets, logprob, entropy, top_ids, top_logprobs, scratch, stream=None):
    """Per row of logits [rows, vocab]: log p of targets [rows] into logprob, the entropy, and the first top_k =
    top_ids.shape[1] tokens with their log p.  targets / logprob, entropy and top_ids / top_logprobs may be None."""
    import torch
    where = "tqd_op_logprobs"
    if logits.dim() != 2:
        _refuse(where, "logits: [rows, vocab]")
    (n, v), f32, i32 = logits.shape, torch.float32, torch.int32
    lp, ls = _rows(logits, n, v, where, "logits")
    k = 0 if top_ids is None else top_ids.shape[-1]
    if k and tuple(top_ids.shape) != (n, k):
        _refuse(where, "top_ids: [rows, top_k]")
    check(lib().tqd_op_logprobs(
        lp, ls, n, v, None if targets is None else _ptr(targets, i32, n, where, "targets"),
        None if logprob is None else _ptr(logprob, f32, n, where, "logprob"),
        None if entropy is None else _ptr(entropy, f32, n, where, "entropy"), k,
        _ptr(top_ids, i32, n * k, where, "top_ids") if k else None,
        _ptr(top_logprobs, f32, n * k, where, "top_logprobs") if k else None,
        _ptr(scratch, torch.uint8, tqd_logprobs_scratch_bytes(n, v, k), where, "scratch"), _s(stream)), where)
