"""Rows of 8-bit codes, their products and the rotation of many rows, without a
GPU: the oracle against the definitions, and every refusal that the C ABI and the
tensor wrappers make before anything is launched."""
import ctypes
import importlib.util
import os
import subprocess

import numpy as np
import pytest

from oracle import i8
from token_quantized_decode_gb300 import _lib, ops
from token_quantized_decode_gb300 import build as tqd_build
from tests.test_abi import _c_layout

BAD = _lib.TQD_ERR_BAD_ARG
P = 0x3000  # a pointer that a refused call never reads


@pytest.fixture(scope="module")
def L():
    tqd_build.build()
    return _lib.lib()


def f(i):
    return P + 4 * i


def test_calls_that_the_module_does_not_take(L):
    """The compiled module answers None, and raises nothing, for whatever is not a call on the current device's tensors."""
    torch = pytest.importorskip("torch")
    ops._bind()
    call = ops._call
    x, q, s = torch.zeros(2, 32), torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2)
    for f in (call.rows_i8, call.rmsnorm_i8, call.silu_mul_i8, call.rows_i8_read, call.i8_matmul, call.rope_rows):
        for args in ((), (None,) * 4, (1, "a", 2.0, None), (x, q, s, None), (q, s, x, None), (x, x, q, s, None), (x, x, q, s, 3),
                     (x, None, s, 1e-6, None, q, s, None), (q, s, q, s, x, None, None), (x, s, x, 32, 32, False, x, None),
                     (x, s, x, 0, 1 << 80, None, x, "stream")):
            assert f(*args) is None


def test_kinds_of_scaling_are_the_package_s():
    import token_quantized_decode_gb300 as tqd
    names = ("TQD_ROPE_UNSCALED", "TQD_ROPE_LINEAR", "TQD_ROPE_BY_ROTATIONS", "TQD_ROPE_BY_INDEX")
    assert [getattr(tqd, name) for name in names] == [0, 1, 2, 3] and set(names) <= set(tqd.__all__)
    s = ops.rope_scaling(tqd.TQD_ROPE_LINEAR, factor=4.0)
    assert (s.kind, s.factor, s.attention_factor) == (1, 4.0, 1.0)


# ------------------------------------------------------------------ the oracle

def test_codes_are_within_half_a_step():
    y = np.random.default_rng(1).normal(size=(40, 300)) * np.logspace(-6, 6, 40)[:, None]
    q, s = i8.rows(y)
    assert np.all(np.abs(q * s[:, None] - y) <= s[:, None] * (0.5 + 1e-9)) and np.all(np.abs(q).max(1) == 127)


def test_codes_of_ties_and_special_rows():
    y = np.zeros((6, 5))
    y[0] = [127, 0.5, 1.5, -2.5, 126.5]
    y[1, 2], y[2, 3], y[3, 0] = np.nan, np.inf, 1e39
    y[4] = [1e-300, 0, 0, 0, -1e-300]
    q, s = i8.rows(y)
    assert list(q[0]) == [127, 0, 2, -2, 126] and s[0] == 1
    assert np.all(np.isnan(s[1:4])) and not q[1:4].any() and list(q[4]) == [127, 0, 0, 0, -127] and s[5] == 0


def test_codes_of_products_at_exact_borders():
    """Ties that a quotient in 64 bits does not see: |h| = k j, j up to 254, times g of 24 bits."""
    rng = np.random.default_rng(3)
    j = np.arange(-254, 255)
    k, g = rng.integers(20000, 33000, size=(40, 1)) * 2 + 1, rng.integers(2**22, 2**23, size=(40, 1)) * 2 + 1
    q, _ = i8.rows((k * j * g).astype(np.float64))  # 48 bits: exact
    assert np.array_equal(q, np.broadcast_to(np.rint(j / 2), q.shape))


def test_the_norms_scale_makes_rows_of_unit_mean_square():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(3, 4096)).astype(np.float32) * np.float32(7)
    h, q, s = i8.norm_rows(x, None, np.ones(4096, dtype=np.float32), 0.0)
    y = q * s[:, None]
    # each element is off by at most half a step
    assert np.array_equal(h, x) and np.all(np.abs(np.sqrt((y * y).mean(1)) - 1) <= s)


@pytest.mark.parametrize("d,inter", [(64, False), (64, True), (24, False)])
def test_rotation_keeps_norms_and_adds_angles(d, inter):
    t = i8.rope_table(1e6, d, 100)
    x = np.random.default_rng(d).normal(size=(7, 3 * 64))
    pos = np.arange(7) * 5
    y, _ = i8.rope_rows(x, 3, pos, t, inter)
    assert np.allclose(np.linalg.norm(y.reshape(7, 3, 64), axis=-1), np.linalg.norm(x.reshape(7, 3, 64), axis=-1))
    z, _ = i8.rope_rows(y, 3, pos + 2, t, inter)
    assert np.allclose(z, i8.rope_rows(x, 3, 2 * pos + 2, t, inter)[0])
    assert np.array_equal(y.reshape(7, 3, 64)[..., d:], x.reshape(7, 3, 64)[..., d:])


def test_scaled_tables_at_their_ends():
    base = i8.rope_table(1e4, 64, 50)
    lin = i8.rope_table(1e4, 64, 50, 1, 4.0)
    assert np.allclose(lin[::4][:12], base[:12])
    for kind in (2, 3):
        t = i8.rope_table(1e4, 64, 50, kind, 4.0, 4096)
        assert np.allclose(t[:, 0], base[:, 0]) and np.allclose(t[:, -1], lin[:, -1])
        assert np.allclose(i8.rope_table(1e4, 64, 50, kind, 4.0, 4096, attention=1.5), 1.5 * t)


# ------------------------------------------------------------------ refusals of the C ABI

def refused(L, fn, good, bads, text=None):
    for bad in bads:
        assert getattr(L, fn)(*{**good, **bad}.values()) == BAD, bad
        said = L.tqd_last_error()
        assert fn.encode() in said, bad
        if text:
            assert text in said, (bad, said)


ROWS = dict(x=f(0), xs=100, rows=3, n=100, q=f(4000), qs=112, scale=f(8000), st=None)
NORM = dict(x=f(0), xs=100, add=f(1000), adds=100, g=f(2000), rows=3, n=100, eps=1e-6, sum=f(3000), ss=100, q=f(4000), qs=112,
            scale=f(8000), st=None)
SILU = dict(g=f(0), gs=200, u=f(100), us=200, rows=3, n=100, q=f(4000), qs=112, scale=f(8000), st=None)
READ = dict(q=f(4000), qs=112, scale=f(8000), rows=3, n=100, out=f(0), os=100, st=None)
MUL = dict(w=f(0), ws=f(2000), rows=20, cols=96, x=f(4000), xs=96, xsc=f(5000), n=3, y=f(6000), ys=20, scratch=f(8000), st=None)
ROPE = dict(x=f(0), xs=256, pos=f(2000), n=3, heads=4, hd=64, table=f(4000), mp=10, rot=64, inter=0, out=f(8000), os=256, st=None)


def test_no_rows_launch_nothing(L):
    assert L.tqd_op_rows_i8(*{**ROWS, "rows": 0, "x": None}.values()) == 0
    assert L.tqd_op_rmsnorm_i8(*{**NORM, "rows": 0, "x": None}.values()) == 0
    assert L.tqd_op_silu_mul_i8(*{**SILU, "rows": 0}.values()) == 0
    assert L.tqd_op_rows_i8_read(*{**READ, "rows": 0}.values()) == 0
    assert L.tqd_op_i8_matmul(*{**MUL, "n": 0, "x": None}.values()) == 0
    assert L.tqd_op_rope_rows(*{**ROPE, "n": 0}.values()) == 0


def test_row_refusals(L):
    sizes = [dict(rows=-1), dict(rows=(1 << 28) + 1), dict(n=0), dict(n=-4), dict(n=16385, xs=20000, qs=20000)]
    refused(L, "tqd_op_rows_i8", ROWS, [dict(x=None), dict(q=None), dict(scale=None), dict(xs=99), dict(qs=99)] + sizes[:4])
    refused(L, "tqd_op_rows_i8", ROWS, [dict(q=f(0)), dict(q=f(299)), dict(scale=f(150)), dict(scale=f(4000)), dict(q=f(7999))],
            b"overlap")
    refused(L, "tqd_op_rmsnorm_i8", NORM, [dict(x=None), dict(g=None), dict(q=None), dict(scale=None), dict(adds=99),
                                           dict(ss=99), dict(xs=1), dict(qs=2), dict(eps=-1.0), dict(eps=float("nan")),
                                           dict(eps=float("inf"))] + sizes[:4])
    refused(L, "tqd_op_rmsnorm_i8", NORM, [dict(sum=f(1)), dict(sum=f(0), ss=104), dict(sum=f(1050)), dict(sum=f(2050)), dict(q=f(3010)),
                                           dict(q=f(0)), dict(q=f(1100)), dict(q=f(2010)), dict(scale=f(3100)), dict(scale=f(1)),
                                           dict(scale=f(4010)), dict(scale=f(2099))], b"overlap")
    refused(L, "tqd_op_silu_mul_i8", SILU, [dict(g=None), dict(u=None), dict(q=None), dict(scale=None), dict(gs=99), dict(us=99),
                                            dict(qs=99)] + sizes[:4])
    refused(L, "tqd_op_silu_mul_i8", SILU, [dict(q=f(0)), dict(q=f(590)), dict(scale=f(300)), dict(scale=f(4001))], b"overlap")
    refused(L, "tqd_op_rows_i8_read", READ, [dict(q=None), dict(scale=None), dict(out=None), dict(qs=99), dict(os=99)] + sizes[:4])
    refused(L, "tqd_op_rows_i8_read", READ, [dict(out=f(4000)), dict(out=f(3710)), dict(out=f(7990))], b"overlap")


def test_product_sizes_and_refusals(L):
    size = L.tqd_i8_matmul_scratch_bytes
    for bad in ((0, 96, 3), (-1, 96, 3), (20, 0, 3), (20, 100, 3), (20, 16416, 3), (20, 96, 0), (20, 96, (1 << 20) + 1),
                ((1 << 24) + 1, 96, 3)):
        assert size(*bad) == 0
    refused(L, "tqd_op_i8_matmul", MUL, [dict(w=None), dict(ws=None), dict(x=None), dict(xsc=None), dict(y=None), dict(rows=0),
                                         dict(rows=(1 << 24) + 1), dict(cols=0), dict(cols=100), dict(cols=16416), dict(n=-1),
                                         dict(n=(1 << 20) + 1), dict(xs=95), dict(xs=104), dict(ys=19), dict(w=f(1)), dict(x=f(4001))])
    refused(L, "tqd_op_i8_matmul", MUL, [dict(y=f(0)), dict(y=f(479)), dict(y=f(2019)), dict(y=f(4071)), dict(y=f(5001))], b"overlap")


def test_the_products_sizes_take_every_way(L):
    """Whatever kernel, width, sharing of columns and number of rounds a size can lead to, some size of the GPU tests leads to."""
    pytest.importorskip("torch")
    from tests import test_gpu_i8 as gpu

    def kind(rows, cols, n):
        kernel, tokens, warps, cluster, tiles, rounds = ops.tqd_i8_matmul_way(rows, cols, n)
        assert tiles >= 1 and rounds >= 1 and 1 <= cluster <= 8 and warps in (1, 2, 4, 8)
        return kernel, tokens, warps > 1, cluster > 1, rounds > 1
    rows = [1, 17, 100, 240, 300, 700, 1300, 2100, 4096, 5120, 9800, 14000, 20000, 30000, 39000, 40000, 60000, 100000, 151936, 400000]
    cols = [32, 64, 96, 160, 256, 416, 640, 960, 1024, 1824, 2560, 4096, 8192, 16384]
    tokens = [1, 4, 8, 9, 12, 16, 17, 30, 32, 33, 64, 65, 100, 128, 150, 170, 185, 256, 304, 511, 700, 1000, 1500, 2048, 2436, 3323, 4096]
    ways = {kind(r, c, n) for r in rows for c in cols for n in tokens}
    assert len(ways) == 26
    assert ways == {kind(*size) for size in gpu.PRODUCTS + gpu.WAYS + gpu.MORE_WAYS}


def test_ways_of_refused_products(L):
    way = (ctypes.c_int64 * 6)()
    for bad in ((0, 96, 3), (20, 100, 3), (20, 16416, 3), (20, 96, 0), (20, 96, (1 << 20) + 1), ((1 << 24) + 1, 96, 3)):
        assert L.tqd_i8_matmul_way(*bad, way) == BAD and b"tqd_i8_matmul_way" in L.tqd_last_error()
    assert L.tqd_i8_matmul_way(20, 96, 3, None) == BAD
    assert L.tqd_i8_matmul_way(1 << 24, 16384, 1 << 20, way) == 0


@pytest.mark.parametrize("cols", [32, 96, 1024, 16384])
def test_a_product_scratch_serves_every_smaller_call(L, cols):
    """The size never falls as rows, columns or tokens grow (a program keeps one for its largest batch)."""
    size = L.tqd_i8_matmul_scratch_bytes
    ns = sorted({1, 2, 8, 9, 16, 17, 31, 32, 33, 48, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 2048, 4097, 1 << 20})
    rs = [1, 15, 16, 17, 127, 128, 129, 960, 1024, 4096, 5120, 8192, 151936, 1 << 24]
    for r in rs:
        got = [size(r, cols, n) for n in ns]
        assert got == sorted(got)
    for n in ns:
        got = [size(r, cols, n) for r in rs]
        assert got == sorted(got)
        by_cols = [size(4096, c, n) for c in (32, 64, 96, 128, 960, 1024, 2560, 8192, 16384)]
        assert by_cols == sorted(by_cols)


def test_rotation_refusals(L):
    refused(L, "tqd_op_rope_rows", ROPE, [dict(x=None), dict(pos=None), dict(table=None), dict(out=None), dict(n=-1), dict(mp=0),
                                          dict(heads=0), dict(hd=0), dict(rot=0), dict(rot=63), dict(rot=66), dict(inter=2),
                                          dict(heads=1025, xs=65600, os=65600), dict(xs=255), dict(os=255), dict(table=f(4000) + 4)])
    refused(L, "tqd_op_rope_rows", ROPE, [dict(out=f(1)), dict(out=f(0), os=260), dict(out=f(760)), dict(out=f(2000)), dict(out=f(4600))],
            b"overlap")
    sc = lambda **k: ctypes.byref(_lib.tqd_rope_scaling(*{**dict(kind=2, factor=4.0, original_len=100, low=1.0, high=32.0,  # noqa: E731
                                                                 attention=1.0), **k}.values()))
    good = dict(theta=1e6, rot=64, mp=10, sc=None, table=P, st=None)
    nan = float("nan")
    refused(L, "tqd_op_rope_table_scaled", good,
            [dict(theta=0.0), dict(theta=nan), dict(theta=float("inf")), dict(rot=0), dict(rot=3), dict(rot=65538), dict(mp=0), dict(table=None)]
            + [dict(sc=sc(**k)) for k in (dict(kind=4), dict(kind=-1), dict(factor=0.0), dict(factor=nan), dict(original_len=0),
                                          dict(low=0.0), dict(high=1.0), dict(high=nan), dict(attention=0.0), dict(attention=nan),
                                          dict(kind=1, factor=-1.0))] + [dict(theta=1.0, sc=sc(kind=3))])


def test_scaling_struct_matches_the_header():
    cls = _lib.tqd_rope_scaling
    fields = [x[0] for x in cls._fields_]
    size, offsets = _c_layout("tqd_rope_scaling", fields)
    assert ctypes.sizeof(cls) == size and [getattr(cls, x).offset for x in fields] == offsets


# ------------------------------------------------------------------ refusals of the tensor wrappers

def test_wrappers_refuse_tensors_that_are_not_on_the_device(L):
    torch = pytest.importorskip("torch")
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t)  # noqa: E731
    q, s = z(2, 32, t=torch.int8), z(2)
    calls = [lambda: ops.tqd_op_rows_i8(z(2, 32), q, s), lambda: ops.tqd_op_rmsnorm_i8(z(2, 32), None, z(32), 1e-6, None, q, s),
             lambda: ops.tqd_op_silu_mul_i8(z(2, 32), z(2, 32), q, s), lambda: ops.tqd_op_rows_i8_read(q, s, z(2, 32)),
             lambda: ops.tqd_op_i8_matmul(z(4, 32, t=torch.int8), z(4), q, s, z(2, 4)),
             lambda: ops.tqd_op_i8_matmul(z(4, 64, t=torch.int8), z(4), q, s, z(2, 4)),
             lambda: ops.tqd_op_rope_rows(z(2, 64), z(2, t=torch.int32), z(9, 16, 2), 32, 32, False, z(2, 64)),
             lambda: ops.tqd_op_rope_rows(z(2, 64), z(2, t=torch.int32), z(9, 16, 2), 48, 32, False, z(2, 64)),
             lambda: ops.tqd_op_rope_table_scaled(1e6, 64, 4, None, z(4, 32, 2)),
             lambda: ops.tqd_op_rows_i8(z(2, 32, 1), q, s)]
    for call in calls:
        with pytest.raises(_lib.TQDError) as e:
            call()
        assert e.value.status == BAD


@pytest.fixture
def without_the_call_module(monkeypatch):
    """The tensor wrappers as they are where the compiled module cannot be had."""
    pytest.importorskip("torch")

    def hide(path):
        monkeypatch.setattr(_lib, "CALL_PATH", str(path))
        ops._bind()
    yield hide
    monkeypatch.undo()
    ops._bind()


@pytest.mark.parametrize("what", ["absent", "not a library"])
def test_wrappers_go_on_without_the_call_module(L, without_the_call_module, tmp_path, what):
    """The checks in Python are complete: neither the operators that have a call in the module nor the others need it."""
    torch = pytest.importorskip("torch")
    path = tmp_path / "_tqd_call.so"
    if what == "absent":
        without_the_call_module(path)
    else:
        path.write_bytes(b"no library")
        with pytest.warns(RuntimeWarning, match="call module"):
            without_the_call_module(path)
    test_wrappers_refuse_tensors_that_are_not_on_the_device(L)
    x = torch.zeros(2, 64)
    for call in (lambda: ops.tqd_op_q4_0_matvec(torch.zeros(10, dtype=torch.uint8), 2, 64, x, x),
                 lambda: ops.tqd_op_logprobs(x, torch.zeros(2, dtype=torch.int32), x, x, None, None, x)):
        with pytest.raises(_lib.TQDError) as e:
            call()
        assert e.value.status == BAD


@pytest.mark.parametrize("made_for", [None, "torch 1.0 cpython-39-x86_64-linux-gnu"])
def test_a_call_module_for_another_torch_is_not_loaded(L, without_the_call_module, tmp_path, made_for):
    """It would read tensors' sizes and pointers at that torch's offsets."""
    path = tmp_path / "_tqd_call.so"
    path.write_bytes(open(tqd_build.CALL, "rb").read())
    if made_for:
        (tmp_path / "_tqd_call.so.for").write_text(made_for)
    with pytest.warns(RuntimeWarning, match="built for " + (made_for or "nothing")):
        without_the_call_module(path)
    test_wrappers_refuse_tensors_that_are_not_on_the_device(L)
    (tmp_path / "_tqd_call.so.for").write_text(open(tqd_build.CALL_FOR).read())
    without_the_call_module(path)
    assert hasattr(ops._call, "bind")


def test_a_call_module_for_another_torch_is_built_again(L, monkeypatch, tmp_path):
    """Whatever the files' times say."""
    pytest.importorskip("torch")
    assert tqd_build._newest()
    other = tmp_path / "for"
    other.write_text("torch 1.0 cpython-39-x86_64-linux-gnu")
    monkeypatch.setattr(tqd_build, "CALL_FOR", str(other))
    assert not tqd_build._newest()


def test_a_call_module_that_does_not_load_is_left_out(L, without_the_call_module, tmp_path):
    path = tmp_path / "_tqd_call.so"
    path.write_bytes(b"no library")
    (tmp_path / "_tqd_call.so.for").write_text(open(tqd_build.CALL_FOR).read())
    with pytest.warns(RuntimeWarning, match="does not load"):
        without_the_call_module(path)
    test_wrappers_refuse_tensors_that_are_not_on_the_device(L)


@pytest.fixture
def pretended_build(monkeypatch, tmp_path):
    """build() into a folder of its own with compilers that only write their outputs; g++ answers what `answers` says."""
    pytest.importorskip("torch")
    ran, answers = [], {"g++": 0}
    for name in ("LIB", "CALL", "CALL_FOR"):
        monkeypatch.setattr(tqd_build, name, str(tmp_path / getattr(tqd_build, name).rsplit("/", 1)[1]))
    monkeypatch.setattr(tqd_build, "BUILD", str(tmp_path))

    def run(cmd, **kw):
        name = cmd[0].rsplit("/", 1)[-1]
        ran.append(name)
        code = answers.get(name, 0)
        if not code:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, code, "", "no such header" if code else "")
    monkeypatch.setattr(tqd_build.subprocess, "run", run)
    return ran, answers


def test_the_library_is_built_where_the_call_module_is_not(pretended_build):
    """Its compiler's errors are told, and leave the library and the wrappers' way in Python; the next build tries the module
    alone."""
    ran, answers = pretended_build
    answers["g++"] = 1
    with pytest.warns(RuntimeWarning, match="no such header"):
        assert os.path.exists(tqd_build.build())
    assert not os.path.exists(tqd_build.CALL) and "nvcc" in ran
    ran.clear()
    answers["g++"] = 0
    tqd_build.build()
    assert ran == ["g++"] and os.path.exists(tqd_build.CALL)
    ran.clear()
    tqd_build.build()
    assert ran == []


def test_a_torch_without_cuda_has_no_call_module(pretended_build, monkeypatch, tmp_path):
    """There is no libc10_cuda to link it with."""
    ran, _ = pretended_build
    (tmp_path / "torch").mkdir()
    (tmp_path / "torch" / "__init__.py").write_text("")
    (tmp_path / "torch" / "version.py").write_text("__version__ = '2.0+cpu'")
    spec = importlib.util.spec_from_file_location("torch", tmp_path / "torch" / "__init__.py", submodule_search_locations=[str(tmp_path / "torch")])
    monkeypatch.setattr(tqd_build.util, "find_spec", lambda name: spec)
    assert os.path.exists(tqd_build.build()) and "g++" not in ran
    ran.clear()
    tqd_build.build()
    assert ran == []
