"""Operator entry points of libtqd on torch CUDA tensors (tqd_op_* in
include/tqd.h).  Each call marshals data pointers and the current stream into
one C call; outputs are written into caller-allocated tensors."""
from __future__ import annotations

from ctypes import byref

from ._lib import TQDError, check, lib, tqd_kv_q4


torch = None  # bound at the first call (the rest of the package does not need it)


def _bind():
    global torch, _stream_of, _device, _F32, _I32, _U8
    import torch as t
    _F32, _I32, _U8 = t.float32, t.int32, t.uint8
    # (without a GPU no tensor is on device 0, and every call is refused)
    _device = t.cuda.current_device if t.cuda.is_available() else lambda: 0
    raw = getattr(t._C, "_cuda_getCurrentRawStream", None)
    # the raw handle of the current stream: an eighth of the time that its Stream object takes to make
    _stream_of = raw if raw is not None else lambda d: int(t.cuda.current_stream(d).cuda_stream)
    torch = t


def _s(stream):
    if stream is not None:
        return int(stream.cuda_stream)
    if torch is None:
        _bind()
    return _stream_of(_device())


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


def _ptr(t, dtype, n, dev, where, name):
    """Data pointer of a contiguous tensor of at least n elements on device dev."""
    if t.dtype is dtype and t.numel() >= n and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(where, f"{name}: a contiguous {dtype} tensor of {n} or more elements on cuda:{dev} (the current CUDA "
                   f"device) is needed, got {tuple(t.shape)} {t.dtype} on {t.device}")


def _rows(t, n, width, dev, where, name):
    """Pointer and row stride of an f32 tensor [n, width] with contiguous rows ([width] when n is 1)."""
    shape = t.shape
    if t.dtype is not _F32 or t.get_device() != dev or not (shape == (n, width) or (n == 1 and shape == (width,))):
        _refuse(where, f"{name}: an f32 tensor [{n}, {width}] on cuda:{dev} (the current CUDA device) is needed, got "
                       f"{tuple(shape)} {t.dtype} on {t.device}")
    if n == 1 or not n:
        if width > 1 and n and t.stride(-1) != 1:
            _refuse(where, f"{name}: the elements of a row must be contiguous")
        return t.data_ptr(), width
    stride, one = t.stride()
    if stride < width or (one != 1 and width > 1):
        _refuse(where, f"{name}: the elements of a row must be contiguous, and rows may not overlap")
    return t.data_ptr(), stride


def tqd_kv_q4_page_bytes(n_kv: int, head_dim: int, page_size: int) -> int:
    return int(lib().tqd_kv_q4_page_bytes(n_kv, head_dim, page_size))


class KVCacheQ4:
    """One layer's paged 4-bit cache: the tqd_kv_q4 descriptor and the tensors it points into."""

    def __init__(self, pages, page_table, n_kv: int, head_dim: int, page_size: int):
        if torch is None:
            _bind()
        where = "kv_q4"
        page_bytes = tqd_kv_q4_page_bytes(n_kv, head_dim, page_size)
        if not page_bytes:
            _refuse(where, f"n_kv {n_kv} (>= 1), head_dim {head_dim} (64 or 128), page_size {page_size} (a multiple of 16)")
        if page_table.dim() != 2 or not page_table.numel() or not pages.numel() or pages.numel() % page_bytes:
            _refuse(where, f"pages: whole pages of {page_bytes} bytes; page_table: [n_seq, pages per sequence]")
        n_seq, per_seq = page_table.shape
        dev = pages.get_device()
        p = _ptr(pages, _U8, page_bytes, dev, where, "pages") if dev >= 0 else _refuse(where, "pages: a CUDA tensor")
        t = _ptr(page_table, _I32, 1, dev, where, "page_table")
        self.pages, self.page_table = pages, page_table
        self.n_seq, self.n_kv, self.head_dim, self.page_size = n_seq, n_kv, head_dim, page_size
        self.kv_width, self.device = n_kv * head_dim, dev
        self.struct = tqd_kv_q4(p, t, pages.numel() // page_bytes, page_size, n_kv, head_dim, n_seq, per_seq)
        self._ref = byref(self.struct)
        self._attention_scratch = tqd_attention_q4_scratch_bytes(head_dim)


def kv_q4(pages, page_table, n_kv: int, head_dim: int, page_size: int) -> KVCacheQ4:
    """A 4-bit cache over pages (uint8, n_pages * tqd_kv_q4_page_bytes) and an int32 page table [n_seq, pages]."""
    return KVCacheQ4(pages, page_table, n_kv, head_dim, page_size)


def _cache_device(cache, where):
    dev = _device()
    if cache.device != dev:
        _refuse(where, f"the cache is on cuda:{cache.device}, the current device is cuda:{dev}")
    return dev


def tqd_op_kv_append_q4(cache: KVCacheQ4, k, v, positions, seqs=None, table=None, q=None, q_out=None, stream=None):
    """Rotate and store k, v [n, n_kv * head_dim] at positions [n] of sequences seqs [n] (None: sequence i);
    q [n, heads * head_dim], rotated, goes to q_out.  table: tqd_op_rope_table's (None: no rotation)."""
    where = "tqd_op_kv_append_q4"
    dev = _cache_device(cache, where)
    n, kvw, hd = positions.numel(), cache.kv_width, cache.head_dim
    kp, ks = _rows(k, n, kvw, dev, where, "k")
    vp, vs = _rows(v, n, kvw, dev, where, "v")
    qp = op = sp = tp = None
    qs = os_ = heads = max_pos = 0
    if q is not None:
        width = q.shape[-1]
        heads = width // hd
        if q_out is None or width % hd or not heads:
            _refuse(where, "q needs q_out, and whole heads")
        qp, qs = _rows(q, n, width, dev, where, "q")
        op, os_ = _rows(q_out, n, width, dev, where, "q_out")
    if seqs is not None:
        sp = _ptr(seqs, _I32, n, dev, where, "seqs")
    if table is not None:
        tp, max_pos = _ptr(table, _F32, hd, dev, where, "table"), table.numel() // hd
    status = lib().tqd_op_kv_append_q4(cache._ref, kp, ks, vp, vs, _ptr(positions, _I32, n, dev, where, "positions"), sp,
                                       n, tp, max_pos, qp, qs, heads, op, os_,
                                       _stream_of(dev) if stream is None else stream.cuda_stream)
    if status:
        check(status, where)


def tqd_op_kv_read_q4(cache: KVCacheQ4, positions, seqs, k_out, v_out, stream=None):
    """The values that the cache's rows stand for, f32 [n, n_kv * head_dim] (k_out or v_out may be None)."""
    where = "tqd_op_kv_read_q4"
    dev = _cache_device(cache, where)
    n, kvw = positions.numel(), cache.kv_width
    kp, ks = (None, 0) if k_out is None else _rows(k_out, n, kvw, dev, where, "k_out")
    vp, vs = (None, 0) if v_out is None else _rows(v_out, n, kvw, dev, where, "v_out")
    sp = None if seqs is None else _ptr(seqs, _I32, n, dev, where, "seqs")
    status = lib().tqd_op_kv_read_q4(cache._ref, _ptr(positions, _I32, n, dev, where, "positions"), sp, n, kp, ks, vp, vs,
                                     _stream_of(dev) if stream is None else stream.cuda_stream)
    if status:
        check(status, where)


def tqd_attention_q4_scratch_bytes(head_dim: int) -> int:
    return int(lib().tqd_attention_q4_scratch_bytes(head_dim))


def tqd_op_attention_q4(cache: KVCacheQ4, q, lens, q_start, out, scratch, stream=None):
    """Attention of q [n, heads * head_dim] over the cache: one query per sequence (q_start None), or tokens
    q_start[s] .. q_start[s + 1] - 1 as the last positions of sequence s."""
    where = "tqd_op_attention_q4"
    dev = _cache_device(cache, where)
    if q.dim() != 2 or q.shape[1] % cache.head_dim:
        _refuse(where, "q: [n, heads * head_dim]")
    n, width = q.shape
    qp, qs = _rows(q, n, width, dev, where, "q")
    op, os_ = _rows(out, n, width, dev, where, "out")
    status = lib().tqd_op_attention_q4(
        cache._ref, qp, qs, _ptr(lens, _I32, cache.n_seq, dev, where, "lens"),
        None if q_start is None else _ptr(q_start, _I32, cache.n_seq + 1, dev, where, "q_start"), n,
        width // cache.head_dim, op, os_, _ptr(scratch, _U8, cache._attention_scratch, dev, where, "scratch"),
        _stream_of(dev) if stream is None else stream.cuda_stream)
    if status:
        check(status, where)


def tqd_q4_0_matrix_bytes(rows: int, cols: int) -> int:
    return int(lib().tqd_q4_0_matrix_bytes(rows, cols))


def tqd_op_q4_0_repack(w_blocks, rows: int, cols: int, w_tiles, stream=None):
    """Q4_0 blocks (uint8, rows * cols / 32 * 18) into the tiles that the matvec reads (tqd_q4_0_matrix_bytes)."""
    where = "tqd_op_q4_0_repack"
    if torch is None:
        _bind()
    dev = _device()
    if cols % 32:
        _refuse(where, "cols must be a multiple of 32")
    check(lib().tqd_op_q4_0_repack(_ptr(w_blocks, _U8, rows * (cols // 32) * 18, dev, where, "w_blocks"), rows, cols,
                                   _ptr(w_tiles, _U8, tqd_q4_0_matrix_bytes(rows, cols), dev, where, "w_tiles"),
                                   _s(stream)), where)


def tqd_op_q4_0_matvec(w_tiles, rows: int, cols: int, x, y, stream=None):
    """y [n, rows] = x [n, cols] W^T over repacked Q4_0 weights (x [cols], y [rows]: one vector), n <= 64."""
    where = "tqd_op_q4_0_matvec"
    if torch is None:
        _bind()
    dev = _device()
    n = x.shape[0] if x.dim() == 2 else 1
    xp, xs = _rows(x, n, cols, dev, where, "x")
    yp, ys = _rows(y, n, rows, dev, where, "y")
    tile_bytes = (rows + 15) // 16 * ((cols + 127) // 128) * 1152  # tqd_q4_0_matrix_bytes
    status = lib().tqd_op_q4_0_matvec(_ptr(w_tiles, _U8, tile_bytes, dev, where, "w_tiles"), rows, cols, xp, n, xs, yp,
                                      ys, _stream_of(dev) if stream is None else stream.cuda_stream)
    if status:
        check(status, where)


def tqd_logprobs_scratch_bytes(rows: int, vocab: int, top_k: int) -> int:
    return int(lib().tqd_logprobs_scratch_bytes(rows, vocab, top_k))


def tqd_op_logprobs(logits, targets, logprob, entropy, top_ids, top_logprobs, scratch, stream=None):
    """Per row of logits [rows, vocab]: log p of targets [rows] into logprob, the entropy, and the first top_k =
    top_ids.shape[1] tokens with their log p.  targets / logprob, entropy and top_ids / top_logprobs may be None."""
    where = "tqd_op_logprobs"
    if torch is None:
        _bind()
    dev = _device()
    if logits.dim() != 2:
        _refuse(where, "logits: [rows, vocab]")
    n, v = logits.shape
    lp, ls = _rows(logits, n, v, dev, where, "logits")
    tp = op = ep = ip = kp = None
    k = 0
    if targets is not None:
        tp = _ptr(targets, _I32, n, dev, where, "targets")
    if logprob is not None:
        op = _ptr(logprob, _F32, n, dev, where, "logprob")
    if entropy is not None:
        ep = _ptr(entropy, _F32, n, dev, where, "entropy")
    if top_ids is not None and top_ids.shape[-1]:
        k = top_ids.shape[-1]
        if top_ids.shape != (n, k) or top_logprobs is None or top_logprobs.shape != (n, k):
            _refuse(where, "top_ids and top_logprobs: [rows, top_k] both")
        ip = _ptr(top_ids, _I32, n * k, dev, where, "top_ids")
        kp = _ptr(top_logprobs, _F32, n * k, dev, where, "top_logprobs")
    elif top_ids is None and top_logprobs is not None:
        _refuse(where, "top_logprobs needs top_ids")
    L = lib()
    status = L.tqd_op_logprobs(
        lp, ls, n, v, tp, op, ep, k, ip, kp,
        _ptr(scratch, _U8, L.tqd_logprobs_scratch_bytes(n, v, k), dev, where, "scratch"),
        _stream_of(dev) if stream is None else stream.cuda_stream)
    if status:
        check(status, where)
