"""The 4-bit operators without a GPU: the oracle's formats against their
definition, and every refusal that the C ABI and the tensor wrappers make
before anything is launched."""
import ctypes

import numpy as np
import pytest

from oracle import q4
from token_quantized_decode_gb300 import _lib, ops
from token_quantized_decode_gb300 import build as tqd_build
from tests.test_abi import _c_layout

BAD = _lib.TQD_ERR_BAD_ARG


@pytest.fixture(scope="module")
def L():
    tqd_build.build()
    return _lib.lib()


# ------------------------------------------------------------------ the oracle

def test_quantiser_is_within_half_a_step():
    y = np.random.default_rng(1).normal(size=(50, 128)) * np.logspace(-3, 3, 50)[:, None]
    codes, scales = q4.quantise_groups(y)
    assert codes.min() >= 1 and codes.max() <= 15
    a = np.abs(y.reshape(50, 4, 32)).max(-1)
    # half a step of max / 7, and 7 times the scale's f16 rounding (2^-11 relative, 2^-25 absolute below 2^-14)
    bound = a / 14 + 7 * np.maximum(a / 7 * 2.0**-11, 2.0**-25)
    err = np.abs(q4.group_values(codes, scales) - y).reshape(50, 4, 32).max(-1)
    assert np.all(err <= bound)


def test_quantiser_special_groups():
    y = np.zeros((5, 32))
    y[1, 3], y[2, 4], y[3, 5], y[4, 6] = np.nan, np.inf, 1e6, 3.0
    codes, scales = q4.quantise_groups(y)
    assert np.all(codes[0] == 8) and scales[0, 0] == 0
    assert np.all(np.isnan(scales[1:4, 0])) and codes[4, 6] == 15


@pytest.mark.parametrize("hd", [64, 128])
def test_block_layout_is_a_bijection_and_round_trips(hd):
    rng = np.random.default_rng(hd)
    page, n_kv = 32, 3
    pages = np.zeros((2, q4.page_bytes(n_kv, hd, page)), dtype=np.uint8)
    used = np.zeros((18 * hd, 2), dtype=int)
    for b in range(16):
        (kb, ksh), (vb, vsh), ksb, vsb = q4._nibble_places(b, hd)
        for at, sh in ((kb, ksh), (vb, vsh)):
            np.add.at(used, (at, sh // 4), 1)
        for at in (ksb, vsb):
            used[at] += 1
            used[at + 1] += 1
    assert np.all(used == 1)  # every nibble of a block has one owner
    rows = {}
    for p in range(2):
        for h in range(n_kv):
            for t in range(page):
                kc, ks = q4.quantise_groups(rng.normal(size=hd))
                vc, vs = q4.quantise_groups(rng.normal(size=hd))
                q4.store_row(pages, p, h, t, page, kc, ks, vc, vs)
                rows[p, h, t] = q4.group_values(kc, ks), q4.group_values(vc, vs)
    for (p, h, t), (k, v) in rows.items():
        gk, gv, _, _ = q4.load_row(pages, p, h, t, page, hd)
        assert np.array_equal(gk, k) and np.array_equal(gv, v)


def test_oracle_logprobs_special_rows():
    inf = np.inf
    lp, h, ids, tops, *_ = q4.logprobs([1.0, inf, 2.0, inf], 3, 3)
    assert lp == -np.log(2) and np.isclose(h, np.log(2)) and list(ids) == [1, 3, 2] and tops[2] == -inf
    lp, h, ids, tops, *_ = q4.logprobs([np.nan, -inf], 0, 2)
    assert lp == -inf and h == 0 and list(ids) == [-1, -1]
    lp, h, ids, *_ = q4.logprobs([0.5, np.nan, 0.5], 2, 3)
    assert np.isclose(lp, -np.log(2)) and list(ids) == [0, 2, -1]


# ------------------------------------------------------------------ sizes and refusals

def test_sizes(L):
    assert L.tqd_kv_q4_page_bytes(8, 128, 16) == 8 * 2304
    assert L.tqd_kv_q4_page_bytes(5, 64, 64) == 5 * 4 * 1152
    for bad in ((0, 128, 16), (8, 96, 16), (8, 128, 0), (8, 128, 24), (8, 128, -16), (8, 128, 1 << 21)):
        assert L.tqd_kv_q4_page_bytes(*bad) == 0
    assert L.tqd_q4_0_matrix_bytes(16, 128) == 1152
    assert L.tqd_q4_0_matrix_bytes(17, 160) == 4 * 1152
    assert L.tqd_q4_0_matrix_bytes(0, 128) == L.tqd_q4_0_matrix_bytes(16, 100) == 0
    assert L.tqd_attention_q4_scratch_bytes(128) > 0 and L.tqd_attention_q4_scratch_bytes(96) == 0
    assert L.tqd_logprobs_scratch_bytes(1, 100, 32) > 0
    assert L.tqd_logprobs_scratch_bytes(1, 100, 33) == L.tqd_logprobs_scratch_bytes(0, 100, 1) == 0


@pytest.mark.parametrize("vocab", [1, 1000, 2045, 2046, 9001, 151936, 1 << 20])
def test_a_logprob_scratch_serves_every_smaller_call(L, vocab):
    """The size never falls as rows, vocabulary or alternatives grow (a program keeps one for its largest batch)."""
    rows = sorted({1, 2, 3, 7, 8, 9, 40, 41, 512, 700, 759, 760, 761, 1000, 1519, 1520, 2053, 3039, 3040, 3041, 6080,
                   6081, 100000, *range(10, 400, 13)})
    sizes = {k: [L.tqd_logprobs_scratch_bytes(r, vocab, k) for r in rows] for k in (0, 1, 2, 5, 20, 31, 32)}
    for a in sizes.values():
        assert a == sorted(a)
    for a, b in zip(list(sizes.values()), list(sizes.values())[1:]):
        assert all(x <= y for x, y in zip(a, b))
    for r in (1, 8, 512, 760, 2053):
        by_vocab = [L.tqd_logprobs_scratch_bytes(r, v, 20) for v in (1, 2045, 2046, 4094, 9001, 49152, 151936, 1 << 20)]
        assert by_vocab == sorted(by_vocab)


def test_cache_struct_matches_the_header():
    cls = _lib.tqd_kv_q4
    fields = [f[0] for f in cls._fields_]
    size, offsets = _c_layout("tqd_kv_q4", fields)
    assert ctypes.sizeof(cls) == size and [getattr(cls, f).offset for f in fields] == offsets


def cache(**over):
    f = dict(pages=0x1000, page_table=0x2000, n_pages=4, page_size=16, n_kv_heads=2, head_dim=64, n_seq=3,
             table_stride=2)
    f.update(over)
    return ctypes.byref(_lib.tqd_kv_q4(*[f[n] for n, _ in _lib.tqd_kv_q4._fields_]))


BAD_CACHES = [dict(pages=0), dict(page_table=0), dict(n_pages=0), dict(page_size=8), dict(page_size=40),
              dict(n_kv_heads=0), dict(head_dim=96), dict(n_seq=0), dict(table_stride=0), dict(pages=0x1008)]

P = 0x3000  # a pointer that a refused call never reads


@pytest.mark.parametrize("over", BAD_CACHES)
def test_bad_caches_are_refused(L, over):
    c = cache(**over)
    assert L.tqd_op_kv_append_q4(c, P, 128, P, 128, P, P, 1, None, 0, None, 0, 0, None, 0, None) == BAD
    assert L.tqd_op_kv_read_q4(c, P, P, 1, P, 128, P, 128, None) == BAD
    assert L.tqd_op_attention_q4(c, P, 256, P, P, 1, 4, P, 256, P, None) == BAD
    assert L.tqd_last_error()


def test_append_refusals(L):
    good = dict(c=cache(), k=P, ks=128, v=P, vs=128, pos=P, seqs=P, n=2, rope=P, max_pos=8, q=P, qs=256, heads=4,
                out=P, os=256, st=None)
    for bad in (dict(c=None), dict(k=None), dict(v=None), dict(pos=None), dict(n=-1), dict(max_pos=0), dict(ks=127),
                dict(vs=0), dict(out=None), dict(heads=0), dict(heads=-1), dict(q=None), dict(qs=255), dict(os=255),
                dict(seqs=None, n=4), dict(n=1 << 30, heads=1 << 20, qs=1 << 40, os=1 << 40)):
        assert L.tqd_op_kv_append_q4(*{**good, **bad}.values()) == BAD, bad
    assert L.tqd_op_kv_append_q4(*{**good, "n": 0, "k": None}.values()) == 0  # nothing to do


def test_read_refusals(L):
    good = dict(c=cache(), pos=P, seqs=P, n=2, k=P, ks=128, v=P, vs=128, st=None)
    for bad in (dict(c=None), dict(pos=None), dict(k=None, v=None), dict(n=-1), dict(ks=1), dict(vs=127),
                dict(seqs=None, n=4)):
        assert L.tqd_op_kv_read_q4(*{**good, **bad}.values()) == BAD, bad
    assert L.tqd_op_kv_read_q4(*{**good, "n": 0}.values()) == 0


def test_attention_refusals(L):
    good = dict(c=cache(), q=P, qs=256, lens=P, start=P, n=5, heads=4, out=P, os=256, scratch=P, st=None)
    for bad in (dict(c=None), dict(q=None), dict(lens=None), dict(out=None), dict(scratch=None), dict(n=-1),
                dict(heads=0), dict(heads=3), dict(qs=255), dict(os=255), dict(scratch=0x3008), dict(start=None),
                dict(start=None, n=0), dict(c=cache(n_seq=1025)), dict(n=1 << 30, heads=4)):
        assert L.tqd_op_attention_q4(*{**good, **bad}.values()) == BAD, bad
    assert L.tqd_op_attention_q4(*{**good, "n": 0, "q": None}.values()) == 0


def test_matvec_refusals(L):
    good = dict(w=P, rows=20, cols=96, x=P, n=2, xs=96, y=P, ys=20, st=None)
    for bad in (dict(w=None), dict(x=None), dict(y=None), dict(rows=0), dict(rows=(1 << 30) + 1), dict(cols=0),
                dict(cols=100), dict(cols=16416), dict(n=-1), dict(n=65), dict(xs=95), dict(ys=19), dict(w=0x3008)):
        assert L.tqd_op_q4_0_matvec(*{**good, **bad}.values()) == BAD, bad
    assert L.tqd_op_q4_0_matvec(*{**good, "n": 0, "x": None}.values()) == 0
    for bad in ((None, 16, 128, P), (P, 16, 128, None), (P, 0, 128, P), (P, 16, 100, P), (P, 16, 16416, P),
                (P, 16, 128, 0x3008), (P, 1 << 30, 16384, P)):
        assert L.tqd_op_q4_0_repack(*bad, None) == BAD, bad


def test_overlapping_rows_are_refused(L):
    """Outputs that would be read as inputs while they are written."""
    f = lambda i: P + 4 * i  # noqa: E731
    app = dict(c=cache(), k=f(256), ks=512, v=f(384), vs=512, pos=P, seqs=P, n=3, rope=None, max_pos=0, q=f(0), qs=512,
               heads=4, out=f(0), os=512, st=None)
    for bad in (dict(out=f(1)), dict(out=f(512)), dict(os=511), dict(out=f(128)), dict(out=f(300)), dict(out=f(512 + 256)),
                dict(out=f(100000), k=f(100000 + 255)), dict(out=f(4000), os=1024, v=f(4000 + 2048 - 127))):
        assert L.tqd_op_kv_append_q4(*{**app, **bad}.values()) == BAD, bad
        assert b"overlap" in L.tqd_last_error()
    assert L.tqd_op_kv_read_q4(cache(), P, P, 3, f(0), 128, f(127), 128, None) == BAD
    att = dict(c=cache(), q=f(0), qs=512, lens=P, start=P, n=4, heads=4, out=f(0), os=512, scratch=P, st=None)
    for bad in (dict(), dict(out=f(255)), dict(out=f(512 * 3)), dict(out=f(512 * 3 + 255)), dict(out=f(-255)),
                dict(out=f(300), os=600), dict(out=f(260), os=256), dict(n=1 << 20, out=f(512 * (1 << 19) + 3))):
        assert L.tqd_op_attention_q4(*{**att, **bad}.values()) == BAD, bad
        assert b"overlap" in L.tqd_last_error(), bad
    mv = dict(w=P, rows=20, cols=96, x=f(0), n=2, xs=96, y=f(0), ys=20, st=None)
    for bad in (dict(), dict(y=f(95)), dict(y=f(191)), dict(y=f(-39)), dict(n=1, y=f(95), xs=0, ys=0)):
        assert L.tqd_op_q4_0_matvec(*{**mv, **bad}.values()) == BAD, bad
        assert b"overlap" in L.tqd_last_error(), bad


def _meet(a, sa, wa, b, sb, wb, n):
    rows = lambda p, s, w: {(p + s * i + j) for i in range(n) for j in range(w)}  # noqa: E731
    return bool(rows(a, sa, wa) & rows(b, sb, wb))


def test_overlaps_of_rows_of_any_stride_are_found(L):
    """Against sets of addresses.  (Rows that lie between one another's without an overlap are taken: a call with them
    would launch, so they are tested with memory behind them.)"""
    rng = np.random.default_rng(0)
    c = cache(n_kv_heads=1, n_seq=8)
    hits = 0
    for _ in range(3000):
        n, sk, sv = int(rng.integers(1, 6)), int(rng.integers(64, 300)), int(rng.integers(64, 300))
        if rng.random() < 0.4:
            sv = sk
        at = int(rng.integers(-1400, 1400))
        if _meet(0, sk, 64, at, sv, 64, n):
            hits += 1
            assert L.tqd_op_kv_read_q4(c, P, P, n, P + 65536, sk, P + 65536 + 4 * at, sv, None) == BAD
            assert b"overlap" in L.tqd_last_error()
    assert hits > 500


def test_logprob_refusals(L):
    good = dict(x=P, stride=100, rows=2, vocab=100, t=P, lp=P, ent=P, k=3, ids=P, tops=P, scratch=P, st=None)
    for bad in (dict(x=None), dict(stride=99), dict(rows=-1), dict(vocab=0), dict(t=None), dict(lp=None), dict(k=-1),
                dict(k=33), dict(ids=None), dict(tops=None), dict(scratch=None), dict(scratch=0x3008),
                dict(k=0, t=None, lp=None, ent=None)):
        assert L.tqd_op_logprobs(*{**good, **bad}.values()) == BAD, bad
    assert L.tqd_op_logprobs(*{**good, "rows": 0, "x": None}.values()) == 0


def test_wrappers_refuse_tensors_of_the_wrong_kind():
    torch = pytest.importorskip("torch")
    tqd_build.build()
    f = torch.zeros(4, 128)
    with pytest.raises(_lib.TQDError, match="CUDA"):
        ops.tqd_op_logprobs(f, None, None, torch.zeros(4), None, None, torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(_lib.TQDError, match="CUDA"):
        ops.tqd_op_q4_0_matvec(torch.zeros(1152, dtype=torch.uint8), 16, 128, torch.zeros(128), torch.zeros(16))
    with pytest.raises(_lib.TQDError, match="CUDA"):
        ops.kv_q4(torch.zeros(2 * 1152, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32), 2, 64, 16)
    with pytest.raises(_lib.TQDError, match="page_size"):
        ops.kv_q4(torch.zeros(2 * 1152, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32), 2, 64, 24)
