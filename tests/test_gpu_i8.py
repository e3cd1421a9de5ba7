"""Rows of 8-bit codes, their products and the rotation of many rows on the GPU,
against the 64-bit oracle (oracle/i8.py).

Tolerances, fixed before the first run.  u = 2^-24 is f32's half step.
 * codes: equal.  The norm's sum: equal to the f32 sum.  Values read back: equal to one f32 product.
 * a scale of rows as they are: one quotient: u.  Of silu(gate) up: expf 4 u, 1 + e, the quotient, the product
   and / 127 u each: 8 u.  Of the norm: the sum of squares (chains of at most 32 terms a thread, 5 steps in a
   warp, 16 warps: 53 u), / n and + eps 2 u, halved by the root; the root, its reciprocal, the product with the
   largest h g (itself rounded), / 127: 5 u: 33 u.  Rows done in 64 bits: u.
 * a product: equal to the stated roundings of the exact sum.
 * a table: cos and sin to u of the attention factor, and 1e-9 for the angle in 64 bits.
 * a rotated element: two products and a sum: 2 u (|a cos| + |b sin|).
"""
import numpy as np
import pytest

import oracle.i8 as i8
import oracle.q4 as q4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0**-24
FULL = 77  # what bytes that no call may write hold


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import token_quantized_decode_gb300 as tqd
    return tqd.ops


@pytest.fixture(scope="module")
def TQDError():
    import token_quantized_decode_gb300 as tqd
    return tqd.TQDError


def dev(a, pad=0, lead=0):
    """A device copy of rows a [n, w] inside rows `pad` elements longer, the first `lead` elements in."""
    t = torch.from_numpy(np.ascontiguousarray(a))
    if not pad and not lead:
        return t.cuda()
    n, w = t.shape
    room = torch.full((n * (w + pad) + lead,), FULL, dtype=t.dtype, device="cuda")
    rows = room[lead:].view(n, w + pad)[:, :w]
    rows.copy_(t)
    return rows


def i32(a):
    return dev(np.asarray(a, dtype=np.int32))


def codes_room(n, w, pad=0, lead=0):
    return dev(np.full((n, w), FULL, dtype=np.int8), pad, lead)


def check_rows(q, scale, want_q, want_scale, tol):
    assert np.array_equal(q.cpu().numpy(), want_q)
    s = scale.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(s), np.isnan(want_scale))
    fine = ~np.isnan(s)
    # (2^-150: half a step of the smallest f32)
    assert np.all(np.abs(s - want_scale)[fine] <= tol * want_scale[fine] + 2.0**-150)


# widths in warps and blocks, whole groups of four and not, the borders of every variant
SHAPES = [(1, 1), (1, 4), (3, 31), (5, 33), (1, 1024), (7, 960), (2, 1025), (2, 2048), (3, 2049), (2, 4096), (2, 4099), (2, 8192),
          (2, 8200), (1, 16384), (2, 16383), (1500, 1000), (1100, 64), (1029, 7), (1025, 1024), (203, 4096)]
# (row padding, first element) of the f32 rows, of the codes
PLACES = [((0, 0), (0, 0)), ((4, 4), (16, 0)), ((3, 0), (5, 0)), ((0, 1), (0, 1))]


@pytest.mark.parametrize("n,w", SHAPES)
@pytest.mark.parametrize("place", PLACES)
def test_rows(ops, n, w, place):
    rng = np.random.default_rng(n * 7 + w)
    x = (rng.normal(size=(n, w)) * np.exp(rng.normal(size=(n, 1)))).astype(np.float32)
    q, s = codes_room(n, w, *place[1]), torch.empty(n, device="cuda")
    ops.tqd_op_rows_i8(dev(x, *place[0]), q, s)
    check_rows(q, s, *i8.rows(x), U)
    if place[1][0]:  # what lies between the rows is left alone
        assert bool((torch.as_strided(q, (n, place[1][0]), (w + place[1][0], 1), q.storage_offset() + w) == FULL).all())
    out = dev(np.zeros((n, w), dtype=np.float32), *place[0])
    ops.tqd_op_rows_i8_read(q, s, out)
    assert np.array_equal(out.cpu().numpy(), q.cpu().numpy().astype(np.float32) * s.cpu().numpy()[:, None])


@pytest.mark.parametrize("n,w", SHAPES)
@pytest.mark.parametrize("place", PLACES)
def test_silu(ops, n, w, place):
    rng = np.random.default_rng(n * 11 + w)
    gu = (rng.normal(size=(n, 2 * w)) * 2).astype(np.float32)
    d = dev(gu, *place[0])  # gate and up as slices of one projection's rows
    q, s = codes_room(n, w, *place[1]), torch.empty(n, device="cuda")
    ops.tqd_op_silu_mul_i8(d[:, :w], d[:, w:], q, s)
    check_rows(q, s, *i8.silu_rows(gu[:, :w], gu[:, w:]), 8 * U)


@pytest.mark.parametrize("n,w", SHAPES)
@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("form", ["plain", "add", "keep", "into x", "into add"])
def test_norm(ops, n, w, place, form):
    rng = np.random.default_rng(n * 13 + w)
    x = rng.normal(size=(n, w)).astype(np.float32)
    add = None if form == "plain" else (rng.normal(size=(n, w)) * 0.3).astype(np.float32)
    g = (1 + 0.1 * rng.normal(size=w)).astype(np.float32)
    q, s = codes_room(n, w, *place[1]), torch.empty(n, device="cuda")
    dx, da = dev(x, *place[0]), None if add is None else dev(add, *place[0])
    kept = {"plain": None, "add": None, "keep": dev(np.zeros_like(x), *place[0]), "into x": dx, "into add": da}[form]
    ops.tqd_op_rmsnorm_i8(dx, da, dev(g), 1e-6, kept, q, s)
    h, want_q, want_s = i8.norm_rows(x, add, g, 1e-6)
    check_rows(q, s, want_q, want_s, 33 * U)
    if kept is not None:
        assert np.array_equal(kept.cpu().numpy(), h)


def special_rows(w):
    """Rows at the ends of f32, without values, with ties: [n, w]."""
    rng = np.random.default_rng(w)
    x = rng.normal(size=(16, w)).astype(np.float32)
    x[0] = 0
    x[1, w // 2], x[2, 0], x[3, w - 1] = np.nan, np.inf, -np.inf
    x[4] *= np.float32(1e-42)
    x[5] *= np.float32(1e-30)
    x[6] *= np.float32(1e25)
    x[7] *= np.float32(5e37)
    x[8] = np.float32(3e38)
    x[9] = 0
    x[9, w // 3] = np.float32(1e-45)
    x[10] = np.round(x[10] * 20) + np.float32(0.5)  # ties with a largest value of 127
    x[10, 0] = 127
    x[11] = -x[10]
    x[12, 1:] *= np.float32(1e-20)
    x[12, 0] = 1
    x[13] = np.float32(-1)
    x[14] *= np.float32(1e-20)
    return x


@pytest.mark.parametrize("w", [5, 128, 1024, 3000, 12288])
@pytest.mark.parametrize("many", [1, 80])
def test_special_rows(ops, w, many):
    x = np.tile(special_rows(w), (many, 1))
    n = x.shape[0]
    q, s = codes_room(n, w), torch.empty(n, device="cuda")
    ops.tqd_op_rows_i8(dev(x), q, s)
    check_rows(q, s, *i8.rows(x), U)
    out = torch.empty(n, w, device="cuda")
    ops.tqd_op_rows_i8_read(q, s, out)
    assert bool(out[1:4].isnan().all()) and not bool(out[0].any())
    for eps in (0.0, 1e-6):
        for g in (np.ones(w), np.linspace(-2, 2, w), np.full(w, 1e-25), np.full(w, 1e20), np.zeros(w)):
            g = g.astype(np.float32)
            kept = torch.empty(n, w, device="cuda")
            ops.tqd_op_rmsnorm_i8(dev(x), dev(x[::-1].copy()), dev(g), eps, kept, q, s)
            h, want_q, want_s = i8.norm_rows(x, x[::-1], g, eps)
            check_rows(q, s, want_q, want_s, 33 * U)
            assert np.array_equal(kept.cpu().numpy(), h, equal_nan=True)
    ops.tqd_op_silu_mul_i8(dev(x), dev(np.roll(x, 1, 0)), q, s)
    check_rows(q, s, *i8.silu_rows(x, np.roll(x, 1, 0)), 8 * U)
    ops.tqd_op_silu_mul_i8(dev(x), dev(np.ones_like(x)), q, s)
    check_rows(q, s, *i8.silu_rows(x, np.ones_like(x)), 8 * U)
    # gates far below zero: e^-z passes f32, then f64
    for z in (-60.0, -87.5, -100.0, -700.0, -750.0):
        y = np.full_like(x, z) + np.linspace(0, 1, w, dtype=np.float32)
        ops.tqd_op_silu_mul_i8(dev(y), dev(np.full_like(x, 1e30)), q, s)
        check_rows(q, s, *i8.silu_rows(y, np.full_like(x, 1e30)), 8 * U)


def test_quotients_next_to_borders(ops):
    """Every element within 2^-20 of a border between two codes."""
    rng = np.random.default_rng(5)
    n, w = 64, 2048
    m = np.abs(rng.normal(size=(n, 1))) + 0.5
    c = rng.integers(-126, 126, size=(n, w)) + 0.5
    x = (c * m / 127 * (1 + rng.integers(-8, 9, size=(n, w)) * 2.0**-23)).astype(np.float32)
    x[:, 7] = m[:, 0]
    q, s = codes_room(n, w), torch.empty(n, device="cuda")
    ops.tqd_op_rows_i8(dev(x), q, s)
    check_rows(q, s, *i8.rows(x), U)
    g = np.exp2(rng.integers(-1, 2, size=w)).astype(np.float32)
    ops.tqd_op_rmsnorm_i8(dev((x / g).astype(np.float32)), None, dev(g), 1e-5, None, q, s)
    check_rows(q, s, *i8.norm_rows((x / g).astype(np.float32), None, g, 1e-5)[1:], 33 * U)


def border_codes(y, most):
    """rint(127 y / most), ties to even, of whole numbers (Python's, of any size)."""
    t = 254 * y + most  # 2 most (127 y / most + 1 / 2)
    low = t // (2 * most)
    return low - ((t % (2 * most) == 0) & (low % 2 == 1))


@pytest.mark.parametrize("w", [100, 509, 1018, 4072])
@pytest.mark.parametrize("shift", [0, -90])
@pytest.mark.parametrize("part", [1.0, 0.04])
def test_norms_at_exact_borders(ops, w, shift, part):
    """Products h g of 48 bits whose quotient is a border exactly, or beside it by less than 64 bits tell: h = k j with |j| up
    to 254.  (Shifted by 2^-90 the row is done in 64 bits as a whole; where all odd j stay there are more than are noted.)"""
    rng = np.random.default_rng(w)
    n = 64
    k = rng.integers(20000, 33000, size=(n, 1)) * 2 + 1
    j = rng.permutation(np.resize(np.arange(-254, 255), w))
    j = np.where(rng.random(w) < part, j, j // 2 * 2)
    j[w // 2] = 254
    h = (k * j).astype(np.int64)
    one = int(rng.integers(2**22, 2**23)) * 2 + 1
    for g in (np.full(w, one), one + 2 * rng.integers(-1, 2, size=w)):
        g[w // 2] = one
        y = h.astype(object) * g.astype(object)
        want = border_codes(y, np.abs(y).max(1, keepdims=True)).astype(np.int8)
        x = np.ldexp(h.astype(np.float64), shift).astype(np.float32)
        q, s = codes_room(n, w), torch.empty(n, device="cuda")
        ops.tqd_op_rmsnorm_i8(dev(x), None, dev(np.ldexp(g.astype(np.float64), -23).astype(np.float32)), 1e-6, None, q, s)
        assert np.array_equal(q.cpu().numpy(), want)


@pytest.mark.parametrize("w", [40, 300, 2048, 5000])
def test_gates_far_below_zero(ops, w):
    """Their silu is nothing, however large they are and whatever they meet in up."""
    rng = np.random.default_rng(w)
    gate, up = rng.normal(size=(8, w)).astype(np.float32), rng.normal(size=(8, w)).astype(np.float32)
    for r, far in enumerate((-87.5, -104.0, -1e9, -6e10, -7e10, -1e30, -1e35, -3e38)):
        gate[r, rng.integers(0, w, size=3)] = far
        up[r, ::7] *= np.float32(2.0 ** (30 if r < 4 else 3))
    q, s = codes_room(8, w), torch.empty(8, device="cuda")
    ops.tqd_op_silu_mul_i8(dev(gate), dev(up), q, s)
    check_rows(q, s, *i8.silu_rows(gate, up), 8 * U)


@pytest.mark.parametrize("w", [5, 64, 300, 1000, 2048, 4096, 8192, 12288])
def test_gates_of_zero(ops, w):
    """Rows of zeros whatever their up values are, but for products that f32 does not hold."""
    rng = np.random.default_rng(w)
    gate, up = np.zeros((8, w), dtype=np.float32), rng.normal(size=(8, w)).astype(np.float32)
    gate[1], gate[2, ::2], up[2, 1::2] = -0.0, 1.0, 0.0
    up[2, ::2] = 0
    gate[3, w // 2], up[3, w // 2] = 1e-30, 1e-30
    gate[4, w - 1], up[4, w - 1] = 1e-3, 1.0
    up[5, 0] = np.inf
    up[6, w - 1] = np.nan
    q, s = codes_room(8, w), torch.empty(8, device="cuda")
    ops.tqd_op_silu_mul_i8(dev(gate), dev(up), q, s)
    check_rows(q, s, *i8.silu_rows(gate, up), 8 * U)


@pytest.mark.parametrize("n,w", [(700, 300), (64, 2048), (40, 5000)])
def test_rows_with_more_borders_than_are_kept(ops, n, w):
    """Products next to borders throughout: more of them than a group of rows has room to note."""
    rng = np.random.default_rng(w)
    m = np.abs(rng.normal(size=(n, 1))) + 0.5
    c = rng.integers(-126, 126, size=(n, w)) + 0.5
    up = (c * m / 127 / 64 * (1 + rng.integers(-8, 9, size=(n, w)) * 2.0**-23)).astype(np.float32)
    up[:, 7] = m[:, 0] / 64
    gate = np.full((n, w), 64, dtype=np.float32)  # silu(64) = 64 to 2^-80
    q, s = codes_room(n, w), torch.empty(n, device="cuda")
    ops.tqd_op_silu_mul_i8(dev(gate), dev(up), q, s)
    check_rows(q, s, *i8.silu_rows(gate, up), 8 * U)
    ops.tqd_op_rmsnorm_i8(dev(up), None, dev(np.ones(w, dtype=np.float32)), 1e-9, None, q, s)
    check_rows(q, s, *i8.norm_rows(up, None, np.ones(w, dtype=np.float32), 1e-9)[1:], 33 * U)


@pytest.mark.parametrize("n,w", [(700, 300), (64, 2048), (40, 5000)])
def test_a_row_is_the_same_beside_any_others(ops, n, w):
    """Rows whose elements are all as large, so that most have no room in a block's list: codes and scales are those of
    the row by itself."""
    rng = np.random.default_rng(w)
    x = (np.exp(rng.normal(size=(n, 1))) * np.sign(rng.normal(size=(n, w)))).astype(np.float32)
    up, g = np.full((n, w), 1.3, dtype=np.float32), np.ones(w, dtype=np.float32)
    x[::9] = rng.normal(size=x[::9].shape)
    dx, du, dg = dev(x), dev(up), dev(g)
    calls = (lambda i, q, s: ops.tqd_op_rmsnorm_i8(dx[i], None, dg, 1e-6, None, q, s), lambda i, q, s: ops.tqd_op_silu_mul_i8(dx[i], du[i], q, s))
    for call in calls:
        q, s = codes_room(n, w), torch.empty(n, device="cuda")
        one_q, one_s = codes_room(n, w), torch.empty(n, device="cuda")
        call(slice(0, n), q, s)
        for i in range(n):
            call(slice(i, i + 1), one_q[i:i + 1], one_s[i:i + 1])
        assert torch.equal(q, one_q) and torch.equal(s, one_s)


@pytest.mark.parametrize("w,alone", [(300, 4256), (2048, 760), (5000, 304)])
def test_borders_that_64_bits_hardly_tell_beside_any_rows(ops, w, alone):
    """SwiGLU products within 2^-41 of a border, where the value that an element is settled by decides: in rows whose block has
    listed other rows' elements up to its last place before, and by themselves.  (alone: the rows that blocks begin with.)"""
    rng = np.random.default_rng(w)
    g0, u0 = np.float64(8), np.float64(np.float32(0.3))
    silu = lambda g: g / (1 + np.exp(-g))  # noqa: E731
    most = silu(g0) * u0
    n = 12_000_000
    # (e^-g halfway between two powers of two, where a series in what is left is at its worst)
    g = -np.log(2) * (rng.integers(0, 6, size=n) + 0.5 + rng.uniform(-0.03, 0.03, size=n))
    g = g.astype(np.float32).astype(np.float64)
    border = (rng.integers(1, 126, size=n) + 0.5) * most / 127
    u = -(border / silu(g)).astype(np.float32).astype(np.float64)
    near = np.nonzero(np.abs(-silu(g) * u / border - 1) < 2.0**-41)[0]
    assert near.size > 100
    gate, up = (rng.normal(size=(2, alone, w)) * 0.3).astype(np.float32)
    gate[:, 3], up[:, 3] = g0, u0
    for i, k in enumerate(near):
        r, c = i % alone, 4 + i // alone
        gate[r, c], up[r, c] = g[k], u[k]
    q, s = codes_room(alone, w), torch.empty(alone, device="cuda")
    ops.tqd_op_silu_mul_i8(dev(gate), dev(up), q, s)
    full = np.concatenate([np.full((alone, w), 1.5, dtype=np.float32), gate]), np.concatenate([np.full((alone, w), 2, dtype=np.float32), up])
    both, scale = codes_room(2 * alone, w), torch.empty(2 * alone, device="cuda")
    ops.tqd_op_silu_mul_i8(dev(full[0]), dev(full[1]), both, scale)
    assert torch.equal(both[alone:], q) and torch.equal(scale[alone:], s)
    assert bool((both[:alone] == 127).all())
    # (all codes but those at the borders are the exact ones)
    differ = np.nonzero(q.cpu().numpy() != i8.silu_rows(gate, up)[0])
    assert set(zip(*(d.tolist() for d in differ))) <= {(i % alone, 4 + i // alone) for i in range(near.size)}


@pytest.mark.parametrize("n,w", [(100000, 40), (30000, 260), (12000, 1100)])
def test_many_rows_a_block(ops, n, w):
    """Blocks that go over more rows than they keep notes of at once."""
    rng = np.random.default_rng(n)
    x, z = rng.normal(size=(2, n, w)).astype(np.float32)
    q, s = codes_room(n, w), torch.empty(n, device="cuda")
    ops.tqd_op_silu_mul_i8(dev(x), dev(z), q, s)
    check_rows(q, s, *i8.silu_rows(x, z), 8 * U)
    g = (1 + 0.1 * rng.normal(size=w)).astype(np.float32)
    dx = dev(x)
    ops.tqd_op_rmsnorm_i8(dx, dev(z), dev(g), 1e-6, dx, q, s)
    h, want_q, want_s = i8.norm_rows(x, z, g, 1e-6)
    check_rows(q, s, want_q, want_s, 33 * U)
    assert np.array_equal(dx.cpu().numpy(), h)
    ops.tqd_op_rows_i8(dev(z), q, s)
    check_rows(q, s, *i8.rows(z), U)
    out = torch.empty(n, w, device="cuda")
    ops.tqd_op_rows_i8_read(q, s, out)
    assert np.array_equal(out.cpu().numpy(), q.cpu().numpy().astype(np.float32) * s.cpu().numpy()[:, None])


# ------------------------------------------------------------------ products

PRODUCTS = [(1, 32, 1), (17, 64, 3), (16, 96, 8), (129, 160, 9), (300, 1056, 17), (1000, 2080, 33), (128, 16384, 2),
            (50, 8192, 65), (257, 4096, 128), (640, 992, 300), (1300, 64, 600), (33, 16384, 40), (4096, 1024, 1), (2500, 1024, 16),
            (127, 1024, 255), (385, 1536, 257), (5120, 960, 31), (9000, 128, 5), (20000, 32, 70), (1, 16384, 513), (2050, 2016, 1000)]


def run_product(ops, w, ws, x, xs, place=(0, 0), scratch=None):
    rows, cols = w.shape
    n = x.shape[0]
    y = dev(np.full((n, rows), FULL, dtype=np.float32), *place)
    if scratch is None:
        scratch = torch.full((ops.tqd_i8_matmul_scratch_bytes(rows, cols, n),), 0xFF, dtype=torch.uint8, device="cuda")
    ops.tqd_op_i8_matmul(dev(w), dev(ws), x if isinstance(x, torch.Tensor) else dev(x), dev(xs), y, scratch)
    return y


def scales(rng, n):
    return np.exp(rng.normal(size=n)).astype(np.float32)


@pytest.mark.parametrize("rows,cols,n", PRODUCTS)
def test_product_is_the_exact_sum(ops, rows, cols, n):
    rng = np.random.default_rng(rows + cols + n)
    w = rng.integers(-128, 128, size=(rows, cols)).astype(np.int8)
    x = rng.integers(-128, 128, size=(n, cols)).astype(np.int8)
    ws, xs = scales(rng, rows), scales(rng, n)
    y = run_product(ops, w, ws, x, xs, place=(3, 1))
    assert np.array_equal(y.cpu().numpy(), i8.matmul(w, ws, x, xs)[1])
    assert bool((torch.as_strided(y, (n, 3), (rows + 3, 1), 1 + rows) == FULL).all())


# Sizes at which each way of making a product is taken: tiles of 16 to 128 tokens with and without clusters, and pairs of
# CTAs, with rows and tokens that end inside a tile, a pair whose second half has no rows, and a pair of few tokens.
WAYS = [(30000, 512, 10), (9000, 2048, 12), (20000, 640, 30), (20000, 640, 64), (6000, 96, 700), (40000, 64, 170), (4000, 4096, 100),
        (13000, 1056, 330), (20100, 32, 1000), (20097, 1056, 161), (26112, 160, 1016), (40000, 2080, 150), (38912, 1024, 304), (5000, 992, 511),
        (40000, 2080, 185), (1000, 8192, 300), (4090, 4096, 250), (12000, 1984, 1500), (260, 16384, 90), (3900, 2080, 600)]


@pytest.mark.parametrize("rows,cols,n", WAYS)
def test_every_way_of_a_product(ops, rows, cols, n):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + n)
    draw = lambda *s: torch.randint(-128, 128, s, dtype=torch.int8, device="cuda", generator=g)  # noqa: E731
    w, x = draw(rows, cols), draw(n, cols)
    w[::5], x[::7] = 127, -128  # sums of one sign past 2^24
    w[2::5], x[3::7] = -128, 127
    ws, xs = torch.rand(rows, device="cuda", generator=g), torch.rand(n, device="cuda", generator=g)
    y = torch.full((n, rows + 3), float(FULL), device="cuda")
    scratch = torch.full((ops.tqd_i8_matmul_scratch_bytes(rows, cols, n),), 0xFF, dtype=torch.uint8, device="cuda")
    ops.tqd_op_i8_matmul(w, ws, x, xs, y[:, :rows], scratch)
    want = (x.double() @ w.double().T).float() * xs[:, None] * ws  # exact in f64
    assert torch.equal(y[:, :rows], want) and bool((y[:, rows:] == FULL).all())


# More of the ways: int8 instructions with several groups of rows one after another (a ring that goes on from one to the next), by warps
# that share columns and by single ones, and what else tests/test_i8_cpu.py asks for.  Rows that end inside a group.
MORE_WAYS = [(50000, 64, 1), (38970, 32, 8), (151936, 1024, 3), (151930, 96, 5), (60001, 1024, 8), (39901, 416, 2), (100003, 640, 7),
             (40000, 256, 16), (39580, 32, 9), (150007, 64, 13), (60009, 192, 10), (9800, 1824, 4), (300, 64, 12), (2100, 32, 16),
             (100, 64, 2500), (240, 96, 2436), (261, 8192, 13)]


@pytest.mark.parametrize("rows,cols,n", MORE_WAYS)
def test_more_ways_of_a_product(ops, rows, cols, n):
    test_every_way_of_a_product(ops, rows, cols, n)


@pytest.mark.parametrize("rows,cols,n", [(40, 16384, 3), (130, 16384, 200), (130, 4096, 40), (260, 8192, 12), (16, 1056, 20)])
def test_product_of_the_largest_codes(ops, rows, cols, n):
    """Sums far past 2^24, of one sign, of both, and with one odd term: a sum that was rounded on the way differs."""
    rng = np.random.default_rng(rows)
    w = np.full((rows, cols), -128, dtype=np.int8)
    x = np.full((n, cols), -128, dtype=np.int8)
    w[1::3], x[1::3] = 127, 127
    w[2::3, ::2], x[2::3, 1::2] = 127, 127
    w[np.arange(rows), rng.integers(0, cols, size=rows)] = 1
    x[np.arange(n), rng.integers(0, cols, size=n)] = 3
    s, want = i8.matmul(w, np.ones(rows), x, np.ones(n))
    assert np.abs(s).max() > 2**24
    y = run_product(ops, w, np.ones(rows, dtype=np.float32), x, np.ones(n, dtype=np.float32))
    assert np.array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("n", [1, 5, 40, 130])
def test_product_of_rows_that_stand_for_nan(ops, n):
    rng = np.random.default_rng(n)
    w = rng.integers(-127, 128, size=(70, 96)).astype(np.int8)
    x = rng.integers(-127, 128, size=(n, 96)).astype(np.int8)
    ws, xs = scales(rng, 70), scales(rng, n)
    ws[3], ws[9], xs[n // 2], x[n // 2] = np.nan, 0, np.nan, 0
    y = run_product(ops, w, ws, x, xs)
    assert np.array_equal(y.cpu().numpy(), i8.matmul(w, ws, x, xs)[1], equal_nan=True)


@pytest.mark.parametrize("n", [1, 7, 16, 33, 200])
def test_product_of_strided_rows(ops, n):
    """Tokens' rows inside longer ones (other bytes between them), beginning anywhere on 16 bytes."""
    rng = np.random.default_rng(n)
    w = rng.integers(-127, 128, size=(150, 224)).astype(np.int8)
    x = rng.integers(-127, 128, size=(n, 224)).astype(np.int8)
    ws, xs = scales(rng, 150), scales(rng, n)
    want = i8.matmul(w, ws, x, xs)[1]
    for pad, lead in ((16, 16), (48, 0), (0, 32)):
        assert np.array_equal(run_product(ops, w, ws, dev(x, pad, lead), xs).cpu().numpy(), want)


def test_product_of_sliced_codes(ops):
    """Codes and scales as the row operators make them, padded to 16 bytes."""
    rng = np.random.default_rng(3)
    x = rng.normal(size=(70, 2 * 992)).astype(np.float32)
    w = rng.normal(size=(200, 992)).astype(np.float32)
    qx, sx = codes_room(70, 992, 32), torch.empty(70, device="cuda")
    qw, sw = codes_room(200, 992), torch.empty(200, device="cuda")
    d = dev(x)
    ops.tqd_op_silu_mul_i8(d[:, :992], d[:, 992:], qx, sx)
    ops.tqd_op_rows_i8(dev(w), qw, sw)
    y = torch.empty(70, 200, device="cuda")
    scratch = torch.empty(ops.tqd_i8_matmul_scratch_bytes(200, 992, 70), dtype=torch.uint8, device="cuda")
    ops.tqd_op_i8_matmul(qw, sw, qx, sx, y, scratch)
    assert np.array_equal(y.cpu().numpy(), i8.matmul(qw.cpu().numpy(), sw.cpu().numpy(), qx.cpu().numpy(), sx.cpu().numpy())[1])


@pytest.mark.parametrize("rows,cols,n", [(4096, 1024, 1), (640, 2048, 40), (1000, 960, 300), (20000, 128, 200), (1000, 2048, 12),
                                         (1000, 8192, 300)])
def test_products_on_two_streams_and_in_graphs(ops, rows, cols, n):
    """Calls on two streams at once, each with its scratch, and a captured call replayed on new codes."""
    rng = np.random.default_rng(n)
    w = rng.integers(-127, 128, size=(rows, cols)).astype(np.int8)
    ws = scales(rng, rows)
    X = [rng.integers(-127, 128, size=(n, cols)).astype(np.int8) for _ in range(3)]
    xs = scales(rng, n)
    want = [i8.matmul(w, ws, x, xs)[1] for x in X]
    dw, dws, dxs, dX = dev(w), dev(ws), dev(xs), [dev(x) for x in X]
    room = lambda: torch.empty(ops.tqd_i8_matmul_scratch_bytes(rows, cols, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    streams, scratch, Y = [torch.cuda.Stream() for _ in range(2)], [room(), room()], [torch.zeros(n, rows, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            ops.tqd_op_i8_matmul(dw, dws, dX[i], dxs, Y[i], scratch[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert np.array_equal(Y[i].cpu().numpy(), want[i])
    x, graphs, outs = dX[0].clone(), [], []
    for _ in range(2):  # two graphs that share a scratch
        y = torch.zeros(n, rows, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.tqd_op_i8_matmul(dw, dws, x, dxs, y, scratch[0])
        graphs.append(g)
        outs.append(y)
    for k in (1, 2, 0):
        x.copy_(dX[k])
        for g, y in zip(graphs, outs):
            y.zero_()
            g.replay()
            assert np.array_equal(y.cpu().numpy(), want[k])


@pytest.mark.parametrize("rows,cols,n", [(8192, 512, 400), (40000, 64, 170), (5000, 992, 511), (1000, 2048, 12), (20000, 640, 64)])
def test_products_one_after_another(ops, rows, cols, n):
    """Many short products in a row, with row operators between them: a CTA's shared memory serves the next kernel as soon as it
    is given up."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    draw = lambda *s: torch.randint(-128, 128, s, dtype=torch.int8, device="cuda", generator=g)  # noqa: E731
    w, X = draw(rows, cols), [draw(n, cols) for _ in range(4)]
    ws, xs = torch.rand(rows, device="cuda", generator=g), torch.rand(n, device="cuda", generator=g)
    want = [(x.double() @ w.double().T).float() * xs[:, None] * ws for x in X]
    scratch = torch.empty(ops.tqd_i8_matmul_scratch_bytes(rows, cols, n), dtype=torch.uint8, device="cuda")
    Y = [torch.zeros(n, rows, device="cuda") for _ in X]
    rows_x = torch.randn(n, cols, device="cuda", generator=g)
    q, s = torch.empty(n, cols, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    for k in range(100):
        ops.tqd_op_i8_matmul(w, ws, X[k % 4], xs, Y[k % 4], scratch)
        if k % 3 == 0:
            ops.tqd_op_rows_i8(rows_x, q, s)
    assert all(torch.equal(y, v) for y, v in zip(Y, want))


def test_nothing_is_believed_after_a_wait_that_ran_out(ops):
    """A product's readers wait for two barriers in turn: two runs after the one that never came the parity is that of a
    phase that is over, and a tile that nobody made would be written as numbers."""
    status, bits = ops.tqd_op_wait_selftest()
    assert status != 0 and not bits & 8


# ------------------------------------------------------------------ rotation

@pytest.mark.parametrize("kind,factor,original,low,high,att", [(0, 1.0, 0, 1.0, 32.0, 1.0), (1, 4.0, 0, 1.0, 32.0, 1.0),
                                                               (2, 8.0, 8192, 1.0, 4.0, 1.0), (2, 4.0, 32768, 1.0, 32.0, 1.1386),
                                                               (3, 4.0, 32768, 1.0, 32.0, 1.1386), (3, 2.0, 64, 1.0, 32.0, 1.0)])
@pytest.mark.parametrize("theta,d,n", [(1e6, 128, 9001), (1e5, 64, 131072), (1e4, 20, 300), (5e5, 2, 3)])
def test_tables(ops, kind, factor, original, low, high, att, theta, d, n):
    t = torch.empty(n, d // 2, 2, device="cuda")
    ops.tqd_op_rope_table_scaled(theta, d, n, ops.rope_scaling(kind, factor, original, low, high, att), t)
    want = i8.rope_table(theta, d, n, kind, factor, original, low, high, att)
    assert np.all(np.abs(t.cpu().numpy() - want) <= U * att + 1e-9)
    if kind == 0 and d in (64, 128):
        u = torch.empty(n, d // 2, 2, device="cuda")
        ops.tqd_op_rope_table(theta, d, n, u)
        assert torch.equal(t, u)
        ops.tqd_op_rope_table_scaled(theta, d, n, None, u)
        assert torch.equal(t, u)


ROPES = [(1, 1, 2, 2), (3, 5, 64, 64), (16, 24, 128, 128), (7, 3, 80, 80), (33, 9, 128, 96), (5, 2, 96, 24), (4, 4, 64, 30),
         (2, 1, 6, 4), (40, 40, 256, 64), (3, 256, 256, 256), (1030, 2, 16, 8), (2, 70, 33, 14)]


@pytest.mark.parametrize("n,heads,hd,d", ROPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("pad,lead", [(0, 0), (64, 4), (3, 0), (0, 1)])
def test_rope_rows(ops, n, heads, hd, d, inter, pad, lead):
    rng = np.random.default_rng(n + heads + hd + d)
    top = 500
    x = rng.normal(size=(n, heads * hd)).astype(np.float32)
    pos = rng.integers(0, top, size=n)
    t = torch.empty(top, d // 2, 2, device="cuda")
    ops.tqd_op_rope_table_scaled(1e6, d, top, None, t)
    want, size = i8.rope_rows(x, heads, pos, t.cpu().numpy().astype(np.float64), inter)
    dx, out = dev(x, pad, lead), dev(np.full_like(x, np.nan), pad, lead)
    ops.tqd_op_rope_rows(dx, i32(pos), t, hd, d, inter, out)
    got = out.cpu().numpy()
    assert np.all(np.abs(got - want) <= 2 * U * size)
    assert np.array_equal(dx.cpu().numpy(), x)
    # the same in place, with tokens that are padding left as they are
    skip = rng.random(n) < 0.3
    far = np.where(skip, rng.choice([-1, -2**31, top, 2**31 - 1], size=n), pos)
    ops.tqd_op_rope_rows(dx, i32(far), t, hd, d, inter, dx)
    assert np.array_equal(dx.cpu().numpy(), np.where(skip[:, None], x, got))
    if pad:
        assert bool((torch.as_strided(dx, (n, pad), (heads * hd + pad, 1), lead + heads * hd) == FULL).all())


def test_rotation_of_as_many_tokens_as_an_int_counts(ops):
    """2^31 - 1 tokens, most of them padding: rows, positions and blocks past 32 bits, in place."""
    n = 2**31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    x = torch.ones(n, 2, device="cuda")
    pos = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 1, 255, 256, 2**30 - 1, 2**30, n - 256, n - 255, n - 2, n - 1], device="cuda")
    pos[at] = 1
    t = torch.empty(2, 1, 2, device="cuda")
    ops.tqd_op_rope_table_scaled(1e4, 2, 2, None, t)
    want, _ = i8.rope_rows(np.ones((1, 2)), 1, np.array([1]), t.cpu().numpy().astype(np.float64), False)
    ops.tqd_op_rope_rows(x, pos, t, 2, 2, False, x)
    assert np.all(np.abs(x[at].cpu().numpy() - want) <= 2 * U * 2)
    x[at] = 1
    assert bool((x.view(-1)[:2**31] == 1).all()) and bool((x.view(-1)[2**31:] == 1).all())


def test_rope_rows_agrees_with_the_rotation_of_one_token(ops):
    x = torch.randn(1, 16 * 128, device="cuda")
    t = torch.empty(50, 64, 2, device="cuda")
    ops.tqd_op_rope_table(1e6, 128, 50, t)
    one, rows = x.clone(), x.clone()
    ops.tqd_op_rope(one, 16, 128, 41, t)
    ops.tqd_op_rope_rows(rows, i32([41]), t, 128, 128, False, rows)
    # a fused and a separate rounding of one of two products
    assert bool(((one - rows).abs() <= 2 * U * (x.abs().view(1, 16, 2, 64).sum(2, keepdim=True).expand(1, 16, 2, 64).reshape(1, -1))).all())


# ------------------------------------------------------------------ together

class Layer:
    """One decoder layer over 8-bit rows and a paged 4-bit cache, each step checked on what the one before gave."""

    def __init__(self, ops, rng, H, heads, kv, hd, inner, n, page=16, top=128):
        self.ops, self.H, self.heads, self.kv, self.hd, self.inner, self.n = ops, H, heads, kv, hd, inner, n
        qw, kvw = heads * hd, kv * hd
        self.host = {}
        for name, r, c in (("qkv", qw + 2 * kvw, H), ("o", H, qw), ("gu", 2 * inner, H), ("down", H, inner)):
            w = torch.from_numpy(rng.normal(size=(r, c)).astype(np.float32) / np.sqrt(c).astype(np.float32)).cuda()
            q, s = torch.empty(r, c, dtype=torch.int8, device="cuda"), torch.empty(r, device="cuda")
            ops.tqd_op_rows_i8(w, q, s)
            self.host[name] = (q, s)
        self.g = [dev((1 + 0.1 * rng.normal(size=H)).astype(np.float32)) for _ in range(2)]
        self.table = torch.empty(top, hd // 2, 2, device="cuda")
        ops.tqd_op_rope_table_scaled(1e6, hd, top, ops.rope_scaling(2, 4.0, 32), self.table)
        per = top // page
        self.cache = ops.kv_q4(torch.zeros(n * per, ops.tqd_kv_q4_page_bytes(kv, hd, page), dtype=torch.uint8, device="cuda"),
                               torch.arange(n * per, dtype=torch.int32, device="cuda").view(n, per), kv, hd, page)
        f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        self.h, self.delta, self.qkv, self.att, self.gu = f(n, H), f(n, H), f(n, qw + 2 * kvw), f(n, qw), f(n, 2 * inner)
        self.codes = {w: (torch.zeros(n, w, dtype=torch.int8, device="cuda"), f(n)) for w in {H, qw, inner}}
        self.scratch = torch.zeros(max(1, max(ops.tqd_i8_matmul_scratch_bytes(*q.shape, n) for q, _ in self.host.values())),
                                   dtype=torch.uint8, device="cuda")
        self.room = torch.zeros(ops.tqd_attention_q4_scratch_bytes(hd), dtype=torch.uint8, device="cuda")
        self.lens = i32(np.arange(n) % 5)

    def product(self, name, x, y):
        self.ops.tqd_op_i8_matmul(*self.host[name], *x, y, self.scratch)

    def step(self, watch=lambda *a: None):
        ops, H, hd, inner = self.ops, self.H, self.hd, self.inner
        qw, kvw = self.heads * hd, self.kv * hd
        a, o, d = self.codes[H], self.codes[qw], self.codes[inner]
        ops.tqd_op_rmsnorm_i8(self.h, None, self.g[0], 1e-6, None, *a)
        watch("norm", self.h, a)
        self.product("qkv", a, self.qkv)
        watch("qkv", a, self.qkv)
        q, k, v = self.qkv.split([qw, kvw, kvw], 1)
        before = self.qkv.clone()
        ops.tqd_op_rope_rows(self.qkv[:, :qw + kvw], self.lens, self.table, hd, hd, False, self.qkv[:, :qw + kvw])
        watch("rope", before, self.qkv)
        ops.tqd_op_kv_append_q4(self.cache, k, v, self.lens)
        self.lens += 1
        ops.tqd_op_attention_q4(self.cache, q, self.lens, None, self.att, self.room)
        ops.tqd_op_rows_i8(self.att, *o)
        watch("rows", self.att, o)
        self.product("o", o, self.delta)
        watch("o", o, self.delta)
        before = self.h.clone()
        ops.tqd_op_rmsnorm_i8(self.h, self.delta, self.g[1], 1e-6, self.h, *a)
        watch("norm2", before, a)
        self.product("gu", a, self.gu)
        ops.tqd_op_silu_mul_i8(self.gu[:, :inner], self.gu[:, inner:], *d)
        watch("silu", self.gu, d)
        self.product("down", d, self.delta)
        watch("down", d, self.delta)
        self.h += self.delta


@pytest.mark.parametrize("H,heads,kv,hd,inner,n", [(256, 4, 2, 64, 768, 3), (960, 15, 5, 64, 2560, 1), (1024, 16, 8, 128, 2048, 37)])
def test_a_layer_of_8_bit_steps(ops, H, heads, kv, hd, inner, n):
    rng = np.random.default_rng(H)
    layer = Layer(ops, rng, H, heads, kv, hd, inner, n)
    x0 = rng.normal(size=(n, H)).astype(np.float32)
    layer.h.copy_(dev(x0))
    np_ = lambda t: t.cpu().numpy()  # noqa: E731
    seen = []

    def watch(name, x, y):
        seen.append(name)
        if name in layer.host:
            w, ws = layer.host[name]
            assert np.array_equal(np_(y), i8.matmul(np_(w), np_(ws), np_(x[0]), np_(x[1]))[1])
        elif name == "rope":
            w = (heads + kv) * hd
            want, size = i8.rope_rows(np_(x)[:, :w], heads + kv, np_(layer.lens), np_(layer.table).astype(np.float64), False)
            assert np.all(np.abs(np_(y)[:, :w] - want) <= 2 * U * size) and torch.equal(x[:, w:], y[:, w:])
        elif name == "rows":
            check_rows(*y, *i8.rows(np_(x)), U)
        elif name == "silu":
            check_rows(*y, *i8.silu_rows(np_(x)[:, :inner], np_(x)[:, inner:]), 8 * U)
        else:
            second = name == "norm2"
            h, q, s = i8.norm_rows(np_(x), np_(layer.delta) if second else None, np_(layer.g[second]), 1e-6)
            check_rows(*y, q, s, 33 * U)
            assert np.array_equal(np_(layer.h), h)

    layer.step(watch)
    assert len(seen) == 8
    # the attention of the step, over the rows that the cache holds
    S, qw = n, heads * hd
    q = np_(layer.qkv)[:, :qw].reshape(n, heads, hd).astype(np.float64)
    lens = np_(layer.lens)
    K, V = torch.empty(n, kv * hd, device="cuda"), torch.empty(n, kv * hd, device="cuda")
    ops.tqd_op_kv_read_q4(layer.cache, i32(lens - 1), None, K, V)
    first = np.nonzero(lens == 1)[0]  # sequences of one position: its value
    for s in first:
        v = np_(V)[s].reshape(kv, hd).repeat(heads // kv, 0)
        assert np.all(np.abs(np_(layer.att)[s].reshape(heads, hd) - v) <= 2.0**-18 * np.abs(v).max())
    # two more steps, then the same three as a replayed graph
    want = [layer.h.clone()]
    for _ in range(2):
        layer.step()
        want.append(layer.h.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    layer.lens.copy_(i32(np.arange(n) % 5))
    layer.cache.pages.zero_()
    layer.h.copy_(dev(x0))
    for k in range(3):
        graph.replay()
        assert torch.equal(layer.h, want[k])


# ------------------------------------------------------------------ refusals that need a device

def test_refusals_of_tensors(ops, TQDError):
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    q, s = b(4, 64), f(4)
    t = f(9, 16, 2)
    calls = [lambda: ops.tqd_op_rows_i8(f(4, 64).double(), q, s), lambda: ops.tqd_op_rows_i8(f(4, 64), b(4, 63), s),
             lambda: ops.tqd_op_rows_i8(f(4, 64), q, f(3)), lambda: ops.tqd_op_rows_i8(f(64, 4).T, q, s),
             lambda: ops.tqd_op_rows_i8(f(4, 64), q.cpu(), s), lambda: ops.tqd_op_rows_i8(f(2, 2, 64), q, s),
             lambda: ops.tqd_op_rmsnorm_i8(f(4, 64), f(4, 63), f(64), 1e-6, None, q, s),
             lambda: ops.tqd_op_rmsnorm_i8(f(4, 64), None, f(63), 1e-6, None, q, s),
             lambda: ops.tqd_op_silu_mul_i8(f(4, 64), f(5, 64), q, s),
             lambda: ops.tqd_op_rows_i8_read(q, s, f(4, 32)), lambda: ops.tqd_op_rows_i8_read(q.float(), s, f(4, 64)),
             lambda: ops.tqd_op_i8_matmul(b(8, 32), f(8), q, s, f(4, 8)), lambda: ops.tqd_op_i8_matmul(b(8, 64), f(7), q, s, f(4, 8)),
             lambda: ops.tqd_op_i8_matmul(b(8, 64), f(8), q, s, f(4, 9)), lambda: ops.tqd_op_i8_matmul(b(8, 64).T, f(64), b(4, 8), s, f(4, 64)),
             lambda: ops.tqd_op_i8_matmul(b(600, 64), f(600), b(300, 64), f(300), f(300, 600), b(1).view(torch.uint8)),
             lambda: ops.tqd_op_rope_rows(f(2, 64), i32([1, 2]), t, 32, 30, False, f(2, 64)),
             lambda: ops.tqd_op_rope_rows(f(2, 64), i32([1]), t, 32, 32, False, f(2, 64)),
             lambda: ops.tqd_op_rope_rows(f(2, 64), i32([1, 2]), t, 48, 32, False, f(2, 64)),
             lambda: ops.tqd_op_rope_rows(f(2, 64), i32([1, 2]).long(), t, 32, 32, False, f(2, 64))]
    for i, call in enumerate(calls):
        if i == 15 and not ops.tqd_i8_matmul_scratch_bytes(600, 64, 300):
            continue  # no scratch is needed there
        with pytest.raises(TQDError):
            call()
    torch.cuda.synchronize()


def test_common_calls_are_the_module_s(ops):
    """The compiled module makes the calls of tensors as they come, in strided rows and on a given stream too, and leaves
    derived classes and refusals to the checks in Python."""
    ops._bind()
    call, f = ops._call, lambda *s: torch.ones(*s, device="cuda")
    c = lambda *s: torch.ones(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    pos, side = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x, wide, q, s, room = f(3, 64), f(3, 128)[:, :64], c(3, 64), f(3), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for x in (x, wide):
        for st in (None, side):
            assert call.rows_i8(x, q, s, st) is True
            assert call.rmsnorm_i8(x, None, f(64), 1e-6, None, q, s, st) is True
            assert call.rmsnorm_i8(x, x, f(64), 1e-6, x, q, s, st) is True
            assert call.silu_mul_i8(x, x, q, s, st) is True
            assert call.rows_i8_read(q, s, x, st) is True
            assert call.i8_matmul(c(64, 64), f(64), q, s, x, None, st) is True
            assert call.i8_matmul(c(64, 64), f(64), c(70, 64), f(70), f(70, 64), room, st) is True
            assert call.rope_rows(x, pos, f(5, 32), 32, 32, False, x, st) is True
    assert call.rows_i8(f(64), c(1, 64), f(1), None) is True
    torch.cuda.synchronize()

    class Derived(torch.Tensor):
        pass
    assert call.rows_i8(f(3, 64).as_subclass(Derived), q, s, None) is None
    assert call.rows_i8(f(64, 3).t(), q, s, None) is None and call.rows_i8(f(1, 64).expand(3, 64), q, s, None) is None
    assert call.i8_matmul(c(64, 64), f(64), c(70, 64), f(70), f(70, 64), None, None) is None
    assert call.i8_matmul(c(64, 64), f(64), c(70, 64), f(70), f(70, 64), room[:100], None) is None
    assert call.rows_i8(x, q, f(2), None) is None and call.rows_i8(x.double(), q, s, None) is None
    torch.cuda.synchronize()


def test_calls_without_the_call_module(ops, monkeypatch, tmp_path):
    """What the module makes and what the checks in Python make is the same, to the bit."""
    from token_quantized_decode_gb300 import _lib
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    f = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, add, gain, w, table, pos = f(70, 96), f(70, 96), f(96), f(40, 96), f(9, 32), torch.arange(70, dtype=torch.int32, device="cuda") % 11

    def calls():
        c = lambda n, w: (torch.zeros(n, w, dtype=torch.int8, device="cuda"), torch.zeros(n, device="cuda"))  # noqa: E731
        wq, a, b, s, y, back = c(40, 96), c(70, 96), c(70, 96), torch.zeros(70, 96, device="cuda"), torch.zeros(70, 40, device="cuda"), f(70, 96)
        ops.tqd_op_rows_i8(w, *wq)
        ops.tqd_op_rmsnorm_i8(x, add, gain, 1e-6, s, *a)
        ops.tqd_op_silu_mul_i8(x, add, *b)
        ops.tqd_op_rows_i8_read(*b, back)
        ops.tqd_op_i8_matmul(*wq, *a, y, torch.zeros(ops.tqd_i8_matmul_scratch_bytes(40, 96, 70), dtype=torch.uint8, device="cuda"))
        out = x.clone()
        ops.tqd_op_rope_rows(out, pos, table, 48, 32, True, out)
        return [*wq, *a, *b, s, y, back, out]
    ops._bind()
    fast = calls()
    monkeypatch.setattr(_lib, "CALL_PATH", str(tmp_path / "none.so"))
    ops._bind()
    try:
        slow = calls()
    finally:
        monkeypatch.undo()
        ops._bind()
    assert all(torch.equal(a, b) for a, b in zip(fast, slow))


def test_empty_calls(ops):
    e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    q, s = e(0, 64, t=torch.int8), e(0)
    ops.tqd_op_rows_i8(e(0, 64), q, s)
    ops.tqd_op_rmsnorm_i8(e(0, 64), e(0, 64), e(64), 1e-6, e(0, 64), q, s)
    ops.tqd_op_silu_mul_i8(e(0, 64), e(0, 64), q, s)
    ops.tqd_op_rows_i8_read(q, s, e(0, 64))
    ops.tqd_op_i8_matmul(e(8, 64, t=torch.int8), e(8), q, s, e(0, 8))
    ops.tqd_op_rope_rows(e(0, 64), e(0, t=torch.int32), e(3, 16, 2), 32, 32, False, e(0, 64))
    torch.cuda.synchronize()
