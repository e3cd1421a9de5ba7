"""The 4-bit decode operators and the log probabilities on the GPU, against
the 64-bit oracle (oracle/q4.py).

Tolerances, fixed before the first run.  u = 2^-24 is f32's half step.
 * stored codes and scales: equal, byte for byte; a rotated query: one rounded
   product, one rounded sum: 2 u (|x0| + |x1|).
 * a sum of products with 4-bit codes is taken over the codes 0..15 as they are,
   its terms of size T = 15 * scale * |x|; operands carry 22 bits (4 u), the sums
   are f32.  Rounding errors of the terms are independent, so the sum's error
   is taken as 16 u * sqrt(sum T^2) + 4 u * |sum| (six deviations of 2 u, and the
   final roundings), where a systematic error (a lost position, a wrong code or
   scale) is of the size of a term.
 * a weight of the softmax: the error of its score, and 8 u for exp2 and the
   split.  So an output: 15 * max(v scale) * (2 * score error + 16 u).
 * log p = d - log s, d = x - max: 4 u (1 + |log p| + |d|); the sum s: 4 u (its
   terms 2 u (1 + |d|) each, weighted by p); entropy: 4 u (2 + H + E|d| + E d^2).
"""
import math

import numpy as np
import pytest

import oracle.q4 as q4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0**-24


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


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def i32(a):
    return dev(np.asarray(a, dtype=np.int32))


def rope_table(ops, hd, n, theta=1e6):
    t = torch.empty(n, hd // 2, 2, device="cuda")
    ops.tqd_op_rope_table(theta, hd, n, t)
    return t


class Host:
    """A cache on the host: pages as bytes, a shuffled table, and the rows that were stored."""

    def __init__(self, rng, n_seq, n_kv, hd, page, positions, spare=1, room=0):
        self.hd, self.n_kv, self.page, self.n_seq = hd, n_kv, page, n_seq
        self.per_seq = max(1, -(-positions // page))
        self.n_pages = n_seq * self.per_seq + spare
        self.table = rng.permutation(self.n_pages)[:n_seq * self.per_seq].reshape(n_seq, -1).astype(np.int32)
        # room: positions that the table has beyond, without pages (the attention goes by the table's size)
        self.table = np.concatenate([self.table, np.full((n_seq, -(-room // page)), -1, dtype=np.int32)], 1)
        # bytes that no call wrote: any codes, scales that are NaN
        self.pages = np.full((self.n_pages, q4.page_bytes(n_kv, hd, page)), 0xFF, dtype=np.uint8)

    def store(self, s, pos, k, v):
        """k, v [n_kv, hd]: coded and stored; returns the values they stand for."""
        kc, ks = q4.quantise_groups(k)
        vc, vs = q4.quantise_groups(v)
        for h in range(self.n_kv):
            q4.store_row(self.pages, self.table[s, pos // self.page], h, pos % self.page, self.page, kc[h], ks[h],
                         vc[h], vs[h])
        return q4.group_values(kc, ks), q4.group_values(vc, vs)

    def fill(self, rng, lens, k_gain=1.0):
        """Random rows for every sequence; self.K[s], self.V[s] [len, n_kv, hd]."""
        self.K, self.V = [], []
        for s, n in enumerate(lens):
            rows = [self.store(s, p, rng.normal(size=(self.n_kv, self.hd)) * k_gain,
                               rng.normal(size=(self.n_kv, self.hd))) for p in range(n)]
            self.K.append(np.array([r[0] for r in rows]).reshape(n, self.n_kv, self.hd))
            self.V.append(np.array([r[1] for r in rows]).reshape(n, self.n_kv, self.hd))

    def device(self, ops):
        return ops.kv_q4(dev(self.pages), dev(self.table), self.n_kv, self.hd, self.page)


# ------------------------------------------------------------------ append and read

@pytest.mark.parametrize("heads,n_kv,hd,page", [(16, 8, 128, 16), (15, 5, 64, 64), (4, 2, 64, 32), (7, 1, 128, 256)])
@pytest.mark.parametrize("gain", [1.0, 1e-6, 300.0])
def test_append_stores_the_oracles_bytes(ops, heads, n_kv, hd, page, gain):
    rng = np.random.default_rng(heads * hd)
    n, n_seq, top = 203, 3, 300
    host = Host(rng, n_seq, n_kv, hd, page, top)
    cache = host.device(ops)
    seqs = np.sort(rng.integers(0, n_seq, size=n))
    pos = np.zeros(n, dtype=np.int64)
    for s in range(n_seq):
        m = int((seqs == s).sum())
        pos[seqs == s] = rng.permutation(top)[:m]
    width = (heads + 2 * n_kv) * hd
    fused = (rng.normal(size=(n, width + 3)) * gain).astype(np.float32)  # rows of a fused projection, odd stride
    table = rope_table(ops, hd, top)
    d = dev(fused)
    q_out = torch.full((n, heads * hd), float("nan"), device="cuda")
    ops.tqd_op_kv_append_q4(cache, d[:, heads * hd:(heads + n_kv) * hd], d[:, (heads + n_kv) * hd:width], i32(pos),
                            i32(seqs), table, d[:, :heads * hd], q_out)
    x = fused[:, :width].reshape(n, -1, hd).astype(np.float64)
    t = table.cpu().numpy()
    rq, rk = q4.rotate(x[:, :heads], pos, t), q4.rotate(x[:, heads:heads + n_kv], pos, t)
    K = np.zeros((n, n_kv, hd))
    V = np.zeros((n, n_kv, hd))
    for i in range(n):
        K[i], V[i] = host.store(seqs[i], int(pos[i]), rk[i], x[i, heads + n_kv:])
    assert np.array_equal(cache.pages.cpu().numpy(), host.pages)  # and nothing else was touched
    size = np.abs(x[:, :heads].reshape(n, heads, 2, -1)).sum(2, keepdims=True).repeat(2, 2).reshape(n, heads, hd)
    assert np.all(np.abs(q_out.cpu().numpy().reshape(n, heads, hd) - rq) <= 2 * U * size)
    k_out, v_out = torch.empty(n, n_kv * hd, device="cuda"), torch.empty(n, n_kv * hd, device="cuda")
    ops.tqd_op_kv_read_q4(cache, i32(pos), i32(seqs), k_out, v_out)
    assert np.array_equal(k_out.cpu().numpy().astype(np.float64), K.reshape(n, -1))
    assert np.array_equal(v_out.cpu().numpy().astype(np.float64), V.reshape(n, -1))


@pytest.mark.parametrize("heads,n_kv,hd", [(16, 8, 128), (15, 5, 64), (40, 2, 64), (7, 1, 128)])
def test_append_rows_on_any_boundary(ops, heads, n_kv, hd):
    """The same rows on 16-byte boundaries and off them: the same bytes and the same queries."""
    rng = np.random.default_rng(heads + 2 * hd)
    n, width = 37, (heads + 2 * n_kv) * hd
    rows = rng.normal(size=(n, width)).astype(np.float32)
    pos = np.arange(n)
    table = rope_table(ops, hd, n)
    got = []
    for stride, start in ((width, 0), (width + 4, 4), (width + 1, 0), (width + 4, 1), (width + 2, 2)):
        d = torch.zeros(n, stride + start, device="cuda")[:, start:start + width]
        d.copy_(dev(rows))
        host = Host(np.random.default_rng(1), 1, n_kv, hd, 16, n)
        cache = host.device(ops)
        q = d[:, :heads * hd]
        ops.tqd_op_kv_append_q4(cache, d[:, heads * hd:(heads + n_kv) * hd], d[:, (heads + n_kv) * hd:], i32(pos),
                                i32(np.zeros(n)), table, q, q)  # in place
        got.append((cache.pages.cpu().numpy(), q.cpu().numpy()))
    for pages, q in got[1:]:
        assert np.array_equal(pages, got[0][0]) and np.array_equal(q, got[0][1])


def test_append_codes_values_next_to_a_border_exactly(ops):
    """Elements at (k + 1/2) / 7 of the largest and one f32 step to either side, and rotated keys whose
    exact value lies within f32 rounding of such a border."""
    rng = np.random.default_rng(3)
    n, hd, page = 4096, 64, 16
    host = Host(rng, 1, 1, hd, page, n, spare=0)
    cache = host.device(ops)
    a = rng.uniform(0.5, 2.0, size=(n, 2, 1)).astype(np.float32)
    k = rng.integers(-7, 7, size=(n, 2, 32)) + 0.5
    y = (a.astype(np.float64) * k / 7).astype(np.float32)
    y = np.where(rng.random(y.shape) < 0.3, np.nextafter(y, np.float32(np.inf)), y)
    y = np.where(rng.random(y.shape) < 0.3, np.nextafter(y, np.float32(-np.inf)), y)
    y[:, :, 7] = a[:, :, 0]
    v = y.reshape(n, hd).astype(np.float32)
    # keys that a rotation brings next to such values: the borders rotated back
    table = rope_table(ops, hd, n)
    t = table.cpu().numpy().astype(np.float64)
    pos = np.arange(n)
    c, s = t[:, :, 0], t[:, :, 1]
    y64 = v.astype(np.float64)
    kx = np.concatenate([y64[:, :32] * c + y64[:, 32:] * s, y64[:, 32:] * c - y64[:, :32] * s], 1).astype(np.float32)
    ops.tqd_op_kv_append_q4(cache, dev(kx), dev(v), i32(pos), i32(np.zeros(n)), table)
    rk = q4.rotate(kx[:, None].astype(np.float64), pos, table.cpu().numpy())
    for i in range(n):
        host.store(0, i, rk[i], v[i][None])
    assert np.array_equal(cache.pages.cpu().numpy(), host.pages)


def test_append_scales_next_to_the_end_of_f16(ops):
    """Rotated keys whose f32 rotation passes the largest scale (max / 7 = 65520) while the exact one does not, or the
    other way round: by cancelling from far larger elements, or by lying within f32 rounding of it."""
    rng = np.random.default_rng(29)
    n, hd, page = 4096, 64, 16
    host = Host(rng, 1, 1, hd, page, n, spare=0)
    cache = host.device(ops)
    table = rope_table(ops, hd, n)
    t = table.cpu().numpy().astype(np.float64)
    pos = np.arange(n)
    c, s = t[:, :, 0], t[:, :, 1]
    y = rng.normal(size=(n, hd)) * 1e4
    i = rng.integers(0, 32, size=n)
    far = rng.random(n) < 0.6
    # one pair of a token: its first element becomes small or next to the end, the second large
    y[pos, i] = np.where(far, 0.0, 7 * 65520.0 * (1 + rng.uniform(-3, 3, size=n) * 2.0**-24)) * rng.choice([-1, 1], n)
    y[pos, i + 32] = np.where(far, 10.0 ** rng.uniform(11.5, 14, size=n), rng.choice([0.0, 4e5], n)) * rng.choice([-1, 1], n)
    k = np.concatenate([y[:, :32] * c + y[:, 32:] * s, y[:, 32:] * c - y[:, :32] * s], 1).astype(np.float32)
    v = rng.normal(size=(n, hd)).astype(np.float32)
    v[:, 5] = (7 * 65520.0 * (1 + rng.integers(-3, 4, size=n) * 2.0**-24)).astype(np.float32)
    ops.tqd_op_kv_append_q4(cache, dev(k), dev(v), i32(pos), i32(np.zeros(n)), table)
    rk = q4.rotate(k[:, None].astype(np.float64), pos, table.cpu().numpy())
    for p in range(n):
        host.store(0, p, rk[p], v[p][None])
    got, want = cache.pages.cpu().numpy(), host.pages
    assert np.array_equal(got, want), int((got != want).any(1).sum())


def test_append_without_rotation_padding_and_pages_outside_the_pool(ops):
    rng = np.random.default_rng(5)
    hd, n_kv, page = 128, 2, 16
    host = Host(rng, 4, n_kv, hd, page, 32)
    host.table[2, 1] = -1
    host.table[3, 0] = host.n_pages
    cache = host.device(ops)
    seqs = [0, 1, -1, 4, 0, 2, 2, 3, 1, 0]
    pos = [0, 31, 3, 3, -1, 16, 15, 5, 32, 1 << 30]
    n = len(seqs)
    k, v = rng.normal(size=(2, n, n_kv * hd)).astype(np.float32)
    k[5 + 1, 3] = np.nan          # sequence 2, position 15
    v[1, 130] = np.inf            # sequence 1, position 31
    ops.tqd_op_kv_append_q4(cache, dev(k), dev(v), i32(pos), i32(seqs))
    for i in (0, 1, 6):
        host.store(seqs[i], pos[i], k[i].reshape(n_kv, hd), v[i].reshape(n_kv, hd))
    assert np.array_equal(cache.pages.cpu().numpy(), host.pages)
    out_k, out_v = torch.zeros(n, n_kv * hd, device="cuda"), torch.zeros(n, n_kv * hd, device="cuda")
    ops.tqd_op_kv_read_q4(cache, i32(pos), i32(seqs), out_k, out_v)
    outside = [2, 3, 4, 5, 7, 8, 9]
    assert torch.isnan(out_k[outside]).all() and torch.isnan(out_v[outside]).all()
    assert torch.isnan(out_k[6, :32]).all() and torch.isfinite(out_k[6, 32:]).all()
    assert torch.isnan(out_v[1, 128:160]).all() and torch.isfinite(out_v[1, :128]).all()
    # padding leaves its query row alone, a page outside the pool does not
    table = rope_table(ops, hd, 20)
    q = torch.randn(n, hd, device="cuda")
    q_out = torch.full_like(q, -5.0)
    ops.tqd_op_kv_append_q4(cache, dev(k), dev(v), i32(pos), i32(seqs), table, q, q_out)
    left = [bool((q_out[i] == -5.0).all()) for i in range(n)]
    assert left == [not (0 <= s < 4 and 0 <= p < 20) for s, p in zip(seqs, pos)]
    # in place, without seqs: token i of sequence i
    want = q_out[[0]].clone()
    ops.tqd_op_kv_append_q4(cache, dev(k[:1]), dev(v[:1]), i32([0]), None, table, q[:1], q[:1])
    assert torch.equal(q[:1], want)


def test_a_pool_beyond_four_gigabytes(ops):
    hd, n_kv, page = 128, 8, 256
    pb = ops.tqd_kv_q4_page_bytes(n_kv, hd, page)
    n_pages = (9 << 30) // (2 * pb) + 2  # 4.5 GB
    pages = torch.zeros(n_pages, pb, dtype=torch.uint8, device="cuda")
    table = i32([[n_pages - 1, 0, n_pages // 2, n_pages - 2]])
    cache = ops.kv_q4(pages, table, n_kv, hd, page)
    rng = np.random.default_rng(9)
    n = 4 * page
    k, v = rng.normal(size=(2, n, n_kv * hd)).astype(np.float32)
    ops.tqd_op_kv_append_q4(cache, dev(k), dev(v), i32(np.arange(n)), i32(np.zeros(n)))
    ko, vo = torch.empty(n, n_kv * hd, device="cuda"), torch.empty(n, n_kv * hd, device="cuda")
    ops.tqd_op_kv_read_q4(cache, i32(np.arange(n)), i32(np.zeros(n)), ko, vo)
    kc, ks = q4.quantise_groups(k)
    vc, vs = q4.quantise_groups(v)
    K, V = q4.group_values(kc, ks), q4.group_values(vc, vs)
    assert np.array_equal(ko.cpu().numpy(), K) and np.array_equal(vo.cpu().numpy(), V)
    assert int(pages[[n_pages - 1, 0, n_pages // 2, n_pages - 2]].count_nonzero()) > 3 * pb
    q = rng.normal(size=(1, 16 * hd)).astype(np.float32)
    out = attend(ops, cache, q, [n])
    check_attention(out, q, [K.reshape(n, n_kv, hd)], [V.reshape(n, n_kv, hd)], [n], [1], hd)


# ------------------------------------------------------------------ attention

def attend(ops, cache, q, lens, q_start=None, dirty=0xFF, fill=float("nan")):
    scratch = torch.full((ops.tqd_attention_q4_scratch_bytes(cache.head_dim),), dirty, dtype=torch.uint8, device="cuda")
    qd = q if torch.is_tensor(q) else dev(q)
    out = torch.full(tuple(qd.shape), fill, device="cuda")
    ops.tqd_op_attention_q4(cache, qd, i32(lens), None if q_start is None else i32(q_start), out, scratch)
    return out.cpu().numpy().astype(np.float64)


def attention_tolerance(q, K, V, hd):
    """Per head: see the file's head.  15 * scale is at most 15 / 7 of a group's largest value."""
    heads, n_kv = q.shape[0], K.shape[1]
    step = lambda x: np.abs(x.reshape(len(x), n_kv, -1, 32)).max(-1, keepdims=True) / 7  # noqa: E731
    sk = np.broadcast_to(step(K), K.reshape(len(K), n_kv, -1, 32).shape).reshape(K.shape)
    out = np.zeros(heads)
    for h in range(heads):
        g = h // (heads // n_kv)
        terms = np.sqrt(((15 * sk[:, g] * q[h]) ** 2).sum(-1)).max() / math.sqrt(hd)
        score = np.abs(K[:, g] @ q[h]).max() / math.sqrt(hd)
        out[h] = 15 * step(V)[:, g].max() * (2 * (16 * U * terms + 4 * U * score) + 16 * U)
    return out


def check_attention(got, q, K, V, lens, nq, hd):
    t = 0
    for s, (n, m) in enumerate(zip(lens, nq)):
        for i in range(m):
            qi = q[t].reshape(-1, hd).astype(np.float64)
            seen = n - m + i + 1
            want = q4.attention(qi, K[s], V[s], seen)
            g = got[t].reshape(-1, hd)
            t += 1
            if seen <= 0:
                assert np.array_equal(g, want)
                continue
            tol = attention_tolerance(qi, K[s][:seen], V[s][:seen], hd)[:, None]
            err = np.abs(g - want)
            assert np.all(err <= tol), (s, i, n, float((err / tol).max()))


HEADS = [(2, 2, 64), (16, 8, 128), (15, 5, 64), (4, 1, 128), (10, 2, 128), (8, 1, 64), (12, 1, 128), (40, 2, 64)]


@pytest.mark.parametrize("heads,n_kv,hd", HEADS)
@pytest.mark.parametrize("page", [16, 64])
def test_attention_ragged_lengths(ops, heads, n_kv, hd, page):
    rng = np.random.default_rng(heads + hd + page)
    lens = [1, 0, 2, 15, 16, 17, 31, 33, 64, 100, 257, 0, 513]
    host = Host(rng, len(lens), n_kv, hd, page, max(lens))
    host.fill(rng, lens)
    q = rng.normal(size=(len(lens), heads * hd)).astype(np.float32)
    got = attend(ops, host.device(ops), q, lens)
    check_attention(got, q, host.K, host.V, lens, [1] * len(lens), hd)


@pytest.mark.parametrize("heads,n_kv,hd", HEADS)
@pytest.mark.parametrize("room", [0, 100000])
def test_attention_by_clusters_and_by_runs(ops, heads, n_kv, hd, room):
    """The same lengths with a short page table (a cluster for each row tile) and a long one (equal runs)."""
    rng = np.random.default_rng(heads * 7 + hd)
    lens = [0, 700, 1, 33, 64, 1023, 480]
    host = Host(rng, len(lens), n_kv, hd, 32, max(lens), room=room)
    host.fill(rng, lens)
    q = rng.normal(size=(len(lens), heads * hd)).astype(np.float32)
    got = attend(ops, host.device(ops), q, lens)
    check_attention(got, q, host.K, host.V, lens, [1] * len(lens), hd)


def test_attention_pages_outside_the_pool_by_runs(ops):
    rng = np.random.default_rng(25)
    hd, page = 128, 16
    host = Host(rng, 4, 2, hd, page, 96, room=50000)
    host.fill(rng, [90, 90, 90, 96])
    host.table[1, 3] = -7
    host.table[2, 5] = host.n_pages
    q = rng.normal(size=(4, 4 * hd)).astype(np.float32)
    got = attend(ops, host.device(ops), q, [90, 90, 90, 97])
    assert np.all(np.isnan(got[1:]))
    check_attention(got[:1], q[:1], host.K[:1], host.V[:1], [90], [1], hd)
    got = attend(ops, host.device(ops), q, [90, 48, 80, 96])
    check_attention(got, q, host.K, host.V, [90, 48, 80, 96], [1] * 4, hd)
    got = attend(ops, host.device(ops), q, [90, 48, 2**31 - 1, -2**31])
    check_attention(got[:2], q[:2], host.K[:2], host.V[:2], [90, 48], [1] * 2, hd)
    assert np.all(np.isnan(got[2])) and np.all(got[3] == 0)


def test_attention_lengths_of_any_size(ops):
    """Lengths up to int32's ends, over a short table and with several queries: the queries that see no position
    past the table keep their values."""
    rng = np.random.default_rng(26)
    hd, page = 64, 16
    host = Host(rng, 3, 1, hd, page, 32)
    host.fill(rng, [32, 32, 32])
    q = rng.normal(size=(12, 2 * hd)).astype(np.float32)
    got = attend(ops, host.device(ops), q[:3], [2**31 - 1, 20, -2**31])
    assert np.all(np.isnan(got[0])) and np.all(got[2] == 0)
    check_attention(got[1:2], q[1:2], host.K[1:2], host.V[1:2], [20], [1], hd)
    # sequence 1's queries are positions 29 .. 33 of 34, of which 32 are in the table
    got = attend(ops, host.device(ops), q, [32, 34, 2**31 - 1], [0, 4, 9, 12])
    check_attention(got[:4], q[:4], host.K[:1], host.V[:1], [32], [4], hd)
    check_attention(got[4:7], q[4:7], [host.K[1]], [host.V[1]], [32], [3], hd)
    assert np.all(np.isnan(got[7:]))


@pytest.mark.parametrize("heads,n_kv,hd", [(16, 8, 128), (15, 5, 64), (4, 1, 128), (12, 1, 128)])
def test_attention_of_several_queries(ops, heads, n_kv, hd):
    rng = np.random.default_rng(heads * 3 + hd)
    lens = [5, 1, 300, 40, 0, 129, 33, 16]
    nq = [5, 1, 16, 0, 3, 129, 40, 2]  # all of a prompt, none, more than are cached
    host = Host(rng, len(lens), n_kv, hd, 32, max(lens))
    host.fill(rng, lens)
    n = sum(nq)
    start = np.concatenate([[0], np.cumsum(nq)])
    q = rng.normal(size=(n + 2, heads * hd)).astype(np.float32)
    got = attend(ops, host.device(ops), q, lens, start, fill=7.0)
    check_attention(got, q, host.K, host.V, lens, nq, hd)
    assert np.all(got[n:] == 7.0)  # rows behind the last sequence


@pytest.mark.parametrize("hd", [64, 128])
def test_attention_picks_each_position(ops, hd):
    """A query that matches one position's key almost alone: the output is that position's value, for every
    position up to the last, and never one behind it."""
    rng = np.random.default_rng(hd)
    n, n_kv = 67, 1
    host = Host(rng, 1, n_kv, hd, 16, n + 13)
    keys = rng.choice([-1.0, 1.0], size=(n + 13, hd)) * 7
    vals = rng.normal(size=(n + 13, hd))
    rows = [host.store(0, p, keys[p][None], vals[p][None]) for p in range(n + 13)]
    cache = host.device(ops)
    for p in range(n):
        out = attend(ops, cache, (keys[p] * 3).astype(np.float32)[None], [n])[0]
        want = q4.attention((keys[p] * 3)[None], np.array([r[0] for r in rows]), np.array([r[1] for r in rows]), n)[0]
        assert np.max(np.abs(out - want)) < 1e-4 and np.max(np.abs(want - rows[p][1][0])) < 1e-3, p
    out = attend(ops, cache, (keys[n] * 3).astype(np.float32)[None], [n])[0]
    assert np.max(np.abs(out - rows[n][1][0])) > 0.1


@pytest.mark.parametrize("heads,n_kv,hd", [(16, 8, 128), (15, 5, 64)])
def test_attention_long(ops, heads, n_kv, hd):
    """4160 positions with values of very unequal size and a peaked softmax."""
    rng = np.random.default_rng(11)
    n, page = 4160, 64
    host = Host(rng, 1, n_kv, hd, page, n)
    size = 10.0 ** rng.uniform(-4, 1, size=n)
    rows = [host.store(0, p, rng.normal(size=(n_kv, hd)) * (3.0 if p % 5 else 0.1),
                       rng.normal(size=(n_kv, hd)) * size[p]) for p in range(n)]
    K, V = np.array([r[0] for r in rows]), np.array([r[1] for r in rows])
    q = rng.normal(size=(1, heads * hd)).astype(np.float32)
    check_attention(attend(ops, host.device(ops), q, [n]), q, [K], [V], [n], [1], hd)


def test_attention_small_values_next_to_large_ones(ops):
    """Weights over many octaves: the tail of the softmax keeps its mass, and values of one head 2^30 apart."""
    rng = np.random.default_rng(12)
    hd, n = 128, 1500
    host = Host(rng, 1, 1, hd, 16, n)
    key = rng.normal(size=hd)
    rows = []
    for p in range(n):
        far = 1.0 if p == 700 else 0.2
        gain = 2.0**-12 if p < 400 else (2.0**12 if p == 1200 else 1.0)
        rows.append(host.store(0, p, key[None] * far, rng.normal(size=(1, hd)) * gain))
    K, V = np.array([r[0] for r in rows]), np.array([r[1] for r in rows])
    q = np.stack([key * 1.2, key * 0.0, -key], 0).reshape(1, -1).astype(np.float32)
    check_attention(attend(ops, host.device(ops), q, [n]), q, [K], [V], [n], [1], hd)


def check_weighted(got, q, K, V, hd):
    """got [heads, hd] against 64 bits with the terms that an element's sum has: the error of a weight (the file's head:
    2 * its score's error + 16 u) times sum_i p_i 7 scale_i over the element's own group."""
    heads, n_kv = q.shape[0], K.shape[1]
    for h in range(heads):
        k, v = K[:, h // (heads // n_kv)], V[:, h // (heads // n_kv)]
        sk = np.repeat(np.abs(k.reshape(len(k), -1, 32)).max(-1) / 7, 32, axis=1)
        sv = np.repeat(np.abs(v.reshape(len(v), -1, 32)).max(-1) / 7, 32, axis=1)
        s = k @ q[h] / math.sqrt(hd)
        p = np.exp(s - s.max())
        p /= p.sum()
        score = 16 * U * np.sqrt(((15 * sk * q[h]) ** 2).sum(-1)).max() / math.sqrt(hd) + 4 * U * np.abs(s).max()
        tol = p @ (7 * sv) * (2 * score + 16 * U) + 1e-30
        err = np.abs(got[h] - p @ v)
        assert np.all(err <= tol), (h, float((err / tol).max()))


@pytest.mark.parametrize("heads,n_kv,hd", [(1, 1, 64), (1, 1, 128), (2, 1, 128), (4, 1, 128), (8, 1, 128), (3, 1, 64),
                                           (8, 1, 64)])
@pytest.mark.parametrize("room", [0, 100000])
@pytest.mark.parametrize("large", [0, 40, 299])
def test_attention_large_values_of_no_weight(ops, heads, n_kv, hd, room, large):
    """A position with values 2^24 times the others' that the queries hardly see (weights of 2^-60): the others keep
    their accuracy, wherever it lies.  And the other way round: the position that has nearly all the weight has values
    2^-20 of the others', or none (scale 0)."""
    rng = np.random.default_rng(heads + hd + large)
    n = 300
    key = rng.choice([-1.0, 1.0], size=hd)
    cases = [(-1.0, 2.0**24, 2.0**-12), (1.0, 2.0**-20, 1.0), (1.0, 0.0, 1.0)]
    host = Host(rng, len(cases), n_kv, hd, 16, n, room=room)
    K, V = [], []
    for s, (sign, gain, base) in enumerate(cases):
        rows = []
        for p in range(n):
            k = key * sign if p == large else rng.normal(size=hd) * 0.1
            v = rng.normal(size=hd) * base * (gain if p == large else 1.0)
            rows.append(host.store(s, p, k[None], v[None]))
        K.append(np.array([r[0] for r in rows]))
        V.append(np.array([r[1] for r in rows]))
    q = np.concatenate([np.tile(key * 41.6 / math.sqrt(hd), heads)[None] * (1.0 if s == 0 else 0.5)
                        for s in range(len(cases))]).astype(np.float32)
    got = attend(ops, host.device(ops), q, [n] * len(cases))
    for s in range(len(cases)):
        check_weighted(got[s].reshape(heads, hd), q[s].reshape(heads, hd).astype(np.float64), K[s], V[s], hd)


@pytest.mark.parametrize("heads,hd", [(1, 64), (1, 128), (2, 128), (4, 128), (8, 128), (3, 64), (8, 64)])
@pytest.mark.parametrize("ratio", [1, 30, 1000])
def test_attention_large_query_elements_that_meet_zero_keys(ops, heads, hd, ratio):
    """One element of each group of a query is far larger than the rest, and every key is 0 there (code 8): what the
    rest keeps beside it is what the header states, 2^-22 of the largest of the group.  A score's tolerance: its
    products' 16 u sqrt(sum T^2) + 4 u |sum|, four times the root sum square of |k| 2^-22 max|q|, and the tensor cores'
    truncation of a group's 32 low parts times codes, 2^-20 max|q| scale.  A weight's: twice that and 16 u."""
    rng = np.random.default_rng(heads + hd + ratio)
    n = 400
    host = Host(rng, 1, 1, hd, 16, n)
    at = 32 * np.arange(hd // 32) + rng.integers(0, 32, size=hd // 32)
    keys = rng.normal(size=(n, hd))
    keys[:, at] = 0
    rows = [host.store(0, p, keys[p][None], rng.normal(size=(1, hd))) for p in range(n)]
    K, V = np.array([r[0][0] for r in rows]), np.array([r[1][0] for r in rows])
    q = rng.normal(size=(heads, hd)).astype(np.float32)
    q[:, at] = ratio * rng.uniform(0.7, 1.4, size=(heads, at.size)) * rng.choice([-1, 1], size=(heads, at.size))
    got = attend(ops, host.device(ops), q.reshape(1, -1), [n]).reshape(heads, hd)
    step = lambda x: np.abs(x.reshape(n, -1, 32)).max(-1) / 7  # noqa: E731
    for h in range(heads):
        x = q[h].astype(np.float64)
        top = np.abs(x.reshape(-1, 32)).max(-1)
        s = K @ x / math.sqrt(hd)
        hold = 4 * np.sqrt(((K * np.repeat(top, 32) * 2.0**-22) ** 2).sum(-1)) + 2.0**-20 * step(K) @ top
        score = (16 * U * np.sqrt(((K * x) ** 2).sum(-1)) + hold) / math.sqrt(hd) + 4 * U * np.abs(s)
        p = np.exp(s - s.max())
        p /= p.sum()
        tol = (p * (2 * score.max() + 16 * U)) @ (7 * np.repeat(step(V), 32, axis=1))
        err = np.abs(got[h] - p @ V)
        assert np.all(err <= tol), (h, float((err / tol).max()))


@pytest.mark.parametrize("heads,hd", [(1, 64), (1, 128), (2, 128), (4, 128), (8, 128), (8, 64)])
@pytest.mark.parametrize("octaves", [8, 16, 24])
def test_attention_groups_of_very_unequal_values(ops, heads, hd, octaves):
    """The groups of 32 of one head's values differ by 2^8 to 2^24: a group far below the largest keeps what the header
    states, each product of weight and scale to 2^-22 of itself or 2^-37 of the head's largest product (times codes up
    to 8, with random signs: four times the root of their number)."""
    rng = np.random.default_rng(heads + hd + octaves)
    n = 500
    host = Host(rng, 1, 1, hd, 16, n)
    gain = np.repeat(2.0 ** (12 - octaves * np.arange(hd // 32) / (hd // 32 - 1)), 32)
    rows = [host.store(0, p, rng.normal(size=(1, hd)), rng.normal(size=(1, hd)) * gain) for p in range(n)]
    K, V = np.array([r[0][0] for r in rows]), np.array([r[1][0] for r in rows])
    q = rng.normal(size=(heads, hd)).astype(np.float32)
    got = attend(ops, host.device(ops), q.reshape(1, -1), [n]).reshape(heads, hd)
    step = lambda x: np.repeat(np.abs(x.reshape(n, -1, 32)).max(-1) / 7, 32, axis=1)  # noqa: E731
    for h in range(heads):
        x = q[h].astype(np.float64)
        s = K @ x / math.sqrt(hd)
        p = np.exp(s - s.max())
        p /= p.sum()
        score = 16 * U * np.sqrt(((15 * step(K) * x) ** 2).sum(-1)).max() / math.sqrt(hd) + 4 * U * np.abs(s).max()
        tol = p @ (7 * step(V)) * (2 * score + 16 * U) + 4 * math.sqrt(n) * 8 * 2.0**-37 * (p[:, None] * step(V)).max()
        err = np.abs(got[h] - p @ V)
        assert np.all(err <= tol), (h, float((err / tol).max()))


def test_attention_scales_of_either_sign(ops):
    """Pages that a program wrote itself: any finite f16 is a scale, and a negative one can be the largest by far."""
    rng = np.random.default_rng(27)
    n_kv, n = 2, 150
    for hd, heads in ((64, 2), (128, 4), (128, 8), (64, 16)):
        host = Host(rng, 1, n_kv, hd, 16, n)
        K, V = [], []
        for p in range(n):
            kc, ks = q4.quantise_groups(rng.normal(size=(n_kv, hd)))
            vc, vs = q4.quantise_groups(rng.normal(size=(n_kv, hd)) * 2.0 ** (p // 8))
            ks, vs = -ks if p % 3 == 0 else ks, -vs if p % 8 else vs
            for h in range(n_kv):
                q4.store_row(host.pages, host.table[0, p // 16], h, p % 16, 16, kc[h], ks[h], vc[h], vs[h])
            K.append(q4.group_values(kc, ks))
            V.append(q4.group_values(vc, vs))
        for scale in (1.0, -1.0):
            q = rng.normal(size=(1, heads * hd)).astype(np.float32) * np.float32(scale)
            cache = host.device(ops)
            for visible in (40, 136):
                check_attention(attend(ops, cache, q, [visible]), q, [np.array(K)], [np.array(V)], [visible], [1], hd)
            # from 2^18 * 1.75 a group's scale passes f16 and stands for NaN
            got = attend(ops, cache, q, [n]).reshape(heads, hd)
            want = q4.attention(q[0].reshape(heads, hd).astype(np.float64), np.array(K), np.array(V), n)
            assert np.any(np.isnan(want)) and np.all(np.isnan(got[np.isnan(want)]))


def test_attention_extreme_queries(ops):
    """Queries of any f32 size: tiny ones weigh all positions alike, huge ones pick the largest score."""
    rng = np.random.default_rng(13)
    hd, n = 64, 50
    host = Host(rng, 1, 1, hd, 16, n)
    host.fill(rng, [n])
    cache = host.device(ops)
    q = rng.normal(size=(3, hd))
    got = attend(ops, cache, np.stack([q[0] * 1e-30, q[1] * 1e20, q[2] * 0], 0).astype(np.float32).reshape(1, -1), [n])
    got = got.reshape(3, hd)
    mean, vmax = host.V[0][:, 0].mean(0), np.abs(host.V[0]).max()
    assert np.max(np.abs(got[0] - mean)) < 1e-5 * vmax and np.max(np.abs(got[2] - mean)) < 1e-5 * vmax
    top = np.argmax(host.K[0][:, 0] @ q[1].astype(np.float32))
    assert np.max(np.abs(got[1] - host.V[0][top, 0])) < 1e-5 * vmax


@pytest.mark.parametrize("heads,hd", [(1, 128), (2, 128), (4, 128), (8, 128), (2, 64), (8, 64)])
@pytest.mark.parametrize("room", [0, 100000])
def test_attention_scores_far_below_and_above_zero(ops, heads, hd, room):
    """Scores of one sign up to 1e34: the largest one takes all the weight, the one nearest to zero where all are
    negative; also where the first positions score 1e30 less than later ones, and the other way round."""
    rng = np.random.default_rng(heads + hd)
    n = 200
    host = Host(rng, 2, 1, hd, 16, n, room=room)
    key = rng.choice([-1.0, 1.0], size=hd)
    size = np.stack([rng.permutation(np.linspace(1, 6, n)), np.where(np.arange(n) < 90, 1.0, 5.0) + rng.permutation(n) / n])
    rows = [[host.store(s, p, (key * size[s, p])[None], rng.normal(size=(1, hd))) for p in range(n)] for s in range(2)]
    cache = host.device(ops)
    for gain in (1e5, -1e5, 1e20, -1e20, 3e32, -3e32):
        q = np.tile(key, (2, heads)) * gain * rng.uniform(0.5, 1, size=(2, heads)).repeat(hd, 1)
        got = attend(ops, cache, q.astype(np.float32), [n, n]).reshape(2, heads, hd)
        for s in range(2):
            K = np.array([r[0][0] for r in rows[s]])
            score = K @ key * (1 if gain > 0 else -1)
            top = np.flatnonzero(score == score.max())
            want = np.mean([rows[s][p][1][0] for p in top], 0)
            assert np.all(np.abs(got[s] - want) <= 1e-5), (gain, s)


@pytest.mark.parametrize("heads", [1, 4, 8])
def test_attention_nan_keys_and_values(ops, heads):
    """A NaN in a position reaches the queries that see it and no other; NaN scales behind the end reach none."""
    rng = np.random.default_rng(14)
    hd, n, nq = 128, 45, 30
    host = Host(rng, 2, 1, hd, 16, n + 5)
    host.fill(rng, [n, n])
    bad = rng.normal(size=(1, hd))
    bad[0, 40] = np.nan
    for p in range(n, n + 5):
        host.store(0, p, bad, bad)
    host.store(0, 30, bad, host.V[0][30])
    host.store(1, 30, host.K[1][30], bad)
    q = rng.normal(size=(2 * nq, heads * hd)).astype(np.float32)
    got = attend(ops, host.device(ops), q, [n, n], [0, nq, 2 * nq])
    for s in range(2):
        for i in range(nq):
            seen = n - nq + i + 1
            g = got[s * nq + i].reshape(heads, hd)
            if seen <= 30:
                want = q4.attention(q[s * nq + i].reshape(heads, hd).astype(np.float64), host.K[s], host.V[s], seen)
                assert np.max(np.abs(g - want)) < 1e-4
            elif s == 0:
                assert np.all(np.isnan(g))
            else:
                assert np.all(np.isnan(g[:, 32:64])) and np.all(np.isfinite(g[:, :32])) and np.all(np.isfinite(g[:, 64:]))


def test_attention_pages_outside_the_pool_and_lengths_past_the_table(ops):
    rng = np.random.default_rng(15)
    hd, page = 64, 16
    lens = [40, 40, 40, 70, 40]
    host = Host(rng, 5, 2, hd, page, 48)
    host.fill(rng, [40, 40, 40, 48, 40])
    host.table[1, 1] = -1
    host.table[2, 2] = host.n_pages
    q = rng.normal(size=(5, 4 * hd)).astype(np.float32)
    got = attend(ops, host.device(ops), q, lens)
    assert np.all(np.isnan(got[1:4]))
    keep = [0, 4]
    check_attention(got[keep], q[keep], [host.K[s] for s in keep], [host.V[s] for s in keep], [40, 40], [1, 1], hd)
    # a bad page behind the end is not looked at; negative lengths are empty
    got = attend(ops, host.device(ops), q, [40, 16, 32, 48, -3])
    keep = [0, 1, 2, 3]
    check_attention(got[keep], q[keep], [host.K[s] for s in keep], [host.V[s] for s in keep], [40, 16, 32, 48],
                    [1] * 4, hd)
    assert np.all(got[4] == 0)


def test_attention_strides_streams_graphs_and_a_shared_scratch(ops):
    rng = np.random.default_rng(16)
    hd, heads, n_kv = 128, 16, 8
    lens = [300, 20, 0, 150]
    host = Host(rng, 4, n_kv, hd, 16, 512)
    host.fill(rng, lens)
    cache = host.device(ops)
    wide = torch.randn(4, heads * hd + 8, device="cuda")
    q = wide[:, 4:4 + heads * hd]
    scratch = torch.full((ops.tqd_attention_q4_scratch_bytes(hd),), 0x7F, dtype=torch.uint8, device="cuda")
    out_wide = torch.full((4, heads * hd + 3), 9.0, device="cuda")
    out = out_wide[:, 1:1 + heads * hd]
    ld = i32(lens)
    ops.tqd_op_attention_q4(cache, q, ld, None, out, scratch)
    ref = out.clone()
    assert torch.all(out_wide[:, 0] == 9.0) and torch.all(out_wide[:, -2:] == 9.0)
    check_attention(ref.cpu().numpy(), q.cpu().numpy(), host.K, host.V, lens, [1] * 4, hd)
    # another stream, and twice on it; the result is the same to the bit
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out2 = torch.empty(4, heads * hd, device="cuda")
    torch.cuda.synchronize()
    for _ in range(2):
        ops.tqd_op_attention_q4(cache, q, ld, None, out2, scratch, stream=st)
    st.synchronize()
    assert torch.equal(out2, ref)
    # two graphs over one scratch: the tile's queries, and the decode step; lengths read when replayed
    q3 = torch.randn(9, heads * hd, device="cuda")
    start = i32([0, 3, 4, 4, 9])
    ops.tqd_op_attention_q4(cache, q3, ld, start, torch.empty_like(q3), scratch)
    torch.cuda.synchronize()
    o1, o2 = torch.zeros_like(out2), torch.zeros_like(q3)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        ops.tqd_op_attention_q4(cache, q, ld, None, o1, scratch)
    with torch.cuda.graph(g2):
        ops.tqd_op_attention_q4(cache, q3, ld, start, o2, scratch)
    for new in ([300, 20, 0, 150], [100, 1, 0, 7], [300, 20, 0, 150]):
        ld.copy_(torch.tensor(new, dtype=torch.int32))
        for _ in range(2):
            g1.replay()
            g2.replay()
        torch.cuda.synchronize()
        check_attention(o1.cpu().numpy(), q.cpu().numpy(), host.K, host.V, new, [1] * 4, hd)
        check_attention(o2.cpu().numpy(), q3.cpu().numpy(), host.K, host.V, new, [3, 1, 0, 5], hd)
    assert torch.equal(o1, ref)


@pytest.mark.parametrize("heads,n_kv,hd", [(16, 8, 128), (15, 5, 64), (4, 1, 128), (8, 1, 64), (2, 2, 128)])
@pytest.mark.parametrize("many", [False, True])
def test_attention_of_short_sequences_by_runs(ops, heads, n_kv, hd, many):
    """A long page table over many sequences of a few positions, and one long one among them: a warp's run takes
    several whole segments, ends before the positions of one, or begins at its first."""
    rng = np.random.default_rng(heads + hd + many)
    lens = [int(x) for x in rng.integers(0, 4, size=240 if many else 7)]
    lens[3] = 700
    lens[-1] = 33
    host = Host(rng, len(lens), n_kv, hd, 16, max(lens), room=100000)
    host.fill(rng, lens)
    q = rng.normal(size=(len(lens), heads * hd)).astype(np.float32)
    got = attend(ops, host.device(ops), q, lens)
    check_attention(got, q, host.K, host.V, lens, [1] * len(lens), hd)


def test_attention_many_sequences(ops):
    rng = np.random.default_rng(17)
    hd, heads, n_kv, n_seq = 64, 4, 2, 1024
    lens = (rng.integers(0, 40, size=n_seq) * (rng.random(n_seq) < 0.8)).tolist()
    lens[1000] = 700
    host = Host(rng, n_seq, n_kv, hd, 16, max(lens))
    host.fill(rng, lens)
    q = rng.normal(size=(n_seq, heads * hd)).astype(np.float32)
    got = attend(ops, host.device(ops), q, lens)
    check_attention(got, q, host.K, host.V, lens, [1] * n_seq, hd)


def random_blocks(g, n, hd):
    """n cache blocks [n, 18 * hd] of any codes, with scales of either size: K's 0.05 .. 0.15, V's 0.01 .. 1."""
    b = torch.randint(0, 256, (n, 18 * hd), generator=g, device="cuda", dtype=torch.uint8)
    ks = 0.05 + 0.1 * torch.rand(n, hd // 2, generator=g, device="cuda")
    vs = 10.0 ** (-2 * torch.rand(n, hd // 2, generator=g, device="cuda"))
    b[:, 8 * hd:9 * hd] = ks.half().view(torch.uint8)
    b[:, 17 * hd:] = vs.half().view(torch.uint8)
    return b


def block_values(b, hd):
    """K and V values f64 [n, 16, hd] of blocks [n, 18 * hd]."""
    def f16(at):
        at = torch.from_numpy(at).cuda()
        return torch.stack([b[:, at], b[:, at + 1]], -1).view(torch.float16)[..., 0].double().repeat_interleave(32, 1)
    K, V = [], []
    for p in range(16):
        (kb, ksh), (vb, vsh), ksb, vsb = q4._nibble_places(p, hd)
        for out, at, sh, sc in ((K, kb, ksh, ksb), (V, vb, vsh, vsb)):
            code = (b[:, torch.from_numpy(at).cuda()].int() >> torch.from_numpy(sh).cuda().int()) & 15
            out.append((code - 8).double() * f16(sc))
    return torch.stack(K, 1), torch.stack(V, 1)


@pytest.mark.parametrize("heads,n_kv,hd,n_seq,length,nq", [
    (8, 1, 128, 1, 131067, 1), (8, 1, 64, 1, 131067, 1), (8, 1, 128, 1, 131067, 3), (4, 1, 128, 1, 131072, 1),
    (2, 1, 128, 1, 130000, 1), (1, 1, 128, 1, 131041, 1), (3, 1, 64, 1, 131072, 2),
    (32, 8, 128, 64, 8190, 1), (64, 8, 128, 64, 8190, 1), (32, 8, 64, 64, 8190, 1), (16, 8, 128, 64, 8190, 2),
    (32, 4, 64, 64, 8190, 3)])
def test_attention_of_long_runs(ops, heads, n_kv, hd, n_seq, length, nq):
    """A warp's run of more than 32 units (its pages are looked up 32 at a time), and segments that over 250 CTAs
    share.  Pages are filled on the device and shared by the sequences; some heads are compared."""
    g = torch.Generator(device="cuda")
    g.manual_seed(heads * 1000 + hd + length + nq)
    page, G = 64, heads // n_kv
    n_pages = 2100 if n_seq == 1 else 600
    blocks = random_blocks(g, n_pages * n_kv * (page // 16), hd)
    per_seq = -(-length // page)
    table = torch.stack([torch.randperm(n_pages, generator=g, device="cuda")[:per_seq] for _ in range(n_seq)]).to(torch.int32)
    cache = ops.kv_q4(blocks.view(n_pages, -1), table.contiguous(), n_kv, hd, page)
    lens = [length - 3 * (s % 7) for s in range(n_seq)]
    q = torch.randn(n_seq * nq, heads * hd, generator=g, device="cuda") * (3.0 if nq == 1 else 1.0)
    start = None if nq == 1 else [nq * s for s in range(n_seq + 1)]
    got = torch.from_numpy(attend(ops, cache, q, lens, start)).cuda()
    rng = np.random.default_rng(length)
    for s in {0, n_seq - 1, *rng.integers(0, n_seq, size=3).tolist()}:
        h = int(rng.integers(n_kv))
        at = (table[s].long()[:, None] * n_kv + h) * (page // 16) + torch.arange(page // 16, device="cuda")
        k, v = block_values(blocks[at.reshape(-1)], hd)
        k, v = k.reshape(-1, hd), v.reshape(-1, hd)
        for i in range(nq):
            seen = lens[s] - nq + i + 1
            K, V = k[:seen], v[:seen]
            size = lambda x: x.abs().view(seen, -1, 32).amax(-1).repeat_interleave(32, 1)  # noqa: E731
            for row in range(G):
                at0 = (h * G + row) * hd
                qr = q[s * nq + i, at0:at0 + hd].double()
                sc = K @ qr / math.sqrt(hd)
                p = torch.softmax(sc, 0)
                # the tolerance of check_weighted
                score = 16 * U * (15 / 7 * size(K) * qr).square().sum(-1).sqrt().max() / math.sqrt(hd) + 4 * U * sc.abs().max()
                tol = (p @ size(V)) * (2 * score + 16 * U)
                err = (got[s * nq + i, at0:at0 + hd] - p @ V).abs()
                assert bool((err <= tol).all()), (s, h, i, row, float((err / tol).max()))


# ------------------------------------------------------------------ matvec

def q4_matrix(rng, rows, cols, sigma=0.02):
    codes = np.clip(np.rint(rng.normal(size=(rows, cols)) * 3) + 8, 0, 15).astype(np.uint8)
    d = (sigma / 3 * rng.uniform(0.5, 1.5, size=(rows, cols // 32)) * rng.choice([-1, 1], size=(rows, cols // 32)))
    return codes, d.astype(np.float16)


def tiles_of(ops, codes, d):
    rows, cols = codes.shape
    t = torch.full((ops.tqd_q4_0_matrix_bytes(rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    ops.tqd_op_q4_0_repack(dev(q4.q4_0_blocks(codes, d)), rows, cols, t)
    return t


@pytest.mark.parametrize("rows,cols", [(1, 32), (16, 128), (17, 160), (33, 416)])
def test_q4_repack_layout(ops, rows, cols):
    codes, d = q4_matrix(np.random.default_rng(rows), rows, cols)
    assert np.array_equal(tiles_of(ops, codes, d).cpu().numpy(), q4.q4_0_tiles(codes, d))


def check_matvec(got, codes, d, x):
    w = q4.q4_0_values(codes, d)
    want = x.astype(np.float64) @ w.T
    step = np.repeat(np.abs(d.astype(np.float64)), 32, axis=1)
    terms = np.sqrt((x.astype(np.float64) ** 2) @ (15 * step.T) ** 2)
    tol = 16 * U * terms + 4 * U * np.abs(want) + 1e-37
    err = np.abs(got - want)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("rows,cols", [(1, 32), (15, 64), (16, 128), (17, 160), (100, 2080), (1024, 1024), (2560, 960),
                                       (4099, 416), (40, 16384), (515, 4096), (20000, 256)])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9, 16])
def test_q4_matvec(ops, rows, cols, n):
    rng = np.random.default_rng(rows + cols)
    codes, d = q4_matrix(rng, rows, cols)
    x = rng.normal(size=(n, cols)).astype(np.float32)
    x[:, ::31] *= 50
    t = tiles_of(ops, codes, d)
    y = torch.full((n, rows), float("nan"), device="cuda")
    ops.tqd_op_q4_0_matvec(t, rows, cols, dev(x), y)
    check_matvec(y.cpu().numpy(), codes, d, x)


@pytest.mark.parametrize("rows,cols", [(9713, 160), (9729, 32), (9744, 1184), (9760, 2080)])
@pytest.mark.parametrize("n", [9, 16, 30])
def test_q4_matvec_many_rows(ops, rows, cols, n):
    """Row tiles in twos: an odd number of them, a last one in part, one strip and several slabs."""
    rng = np.random.default_rng(rows + cols)
    codes, d = q4_matrix(rng, rows, cols)
    x = rng.normal(size=(n, cols)).astype(np.float32)
    y = torch.full((n + 1, rows), 3.0, device="cuda")
    ops.tqd_op_q4_0_matvec(tiles_of(ops, codes, d), rows, cols, dev(x), y[:n])
    check_matvec(y[:n].cpu().numpy(), codes, d, x)
    assert bool((y[n] == 3.0).all())


@pytest.mark.parametrize("n", [17, 33, 64])
def test_q4_matvec_more_vectors_than_a_sweep(ops, n):
    rng = np.random.default_rng(n)
    rows, cols = 270, 672
    codes, d = q4_matrix(rng, rows, cols)
    x = rng.normal(size=(n, cols + 5)).astype(np.float32)
    t = tiles_of(ops, codes, d)
    y = torch.full((n, rows + 3), 5.0, device="cuda")
    ops.tqd_op_q4_0_matvec(t, rows, cols, dev(x)[:, 3:3 + cols], y[:, 1:1 + rows])
    check_matvec(y[:, 1:1 + rows].cpu().numpy(), codes, d, x[:, 3:3 + cols])
    assert torch.all(y[:, 0] == 5.0) and torch.all(y[:, 1 + rows:] == 5.0)


def test_q4_matvec_integers_are_exact(ops):
    """Power-of-two scales and small whole x: every product and sum is exact in f32."""
    rng = np.random.default_rng(2)
    rows, cols = 300, 1024
    codes = rng.integers(0, 16, size=(rows, cols)).astype(np.uint8)
    d = (2.0 ** rng.integers(-3, 4, size=(rows, cols // 32))).astype(np.float16)
    x = rng.integers(-8, 9, size=(3, cols)).astype(np.float32)
    y = torch.empty(3, rows, device="cuda")
    ops.tqd_op_q4_0_matvec(tiles_of(ops, codes, d), rows, cols, dev(x), y)
    assert np.array_equal(y.cpu().numpy(), x.astype(np.float64) @ q4.q4_0_values(codes, d).T)


def test_q4_matvec_extremes(ops):
    """x of any f32 size, zero vectors, NaN and infinities, and scales at f16's ends."""
    rng = np.random.default_rng(4)
    rows, cols = 40, 256
    codes, d = q4_matrix(rng, rows, cols)
    d[3, 2], d[4, :] = np.float16(6e-8), np.float16(65504)
    t = tiles_of(ops, codes, d)
    x = rng.normal(size=(6, cols)).astype(np.float32)
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] = 0
    x[3] = 0
    x[3, 200] = -3e-38
    x[4, 10] = np.nan
    x[5, 11] = np.inf
    y = torch.empty(6, rows, device="cuda")
    ops.tqd_op_q4_0_matvec(t, rows, cols, dev(x), y)
    y = y.cpu().numpy()
    check_matvec(y[:3], codes, d, x[:3])
    want = x[3].astype(np.float64) @ q4.q4_0_values(codes, d).T
    assert np.all(np.abs(y[3] - want) <= 1e-3 * np.abs(want) + 3e-45) and np.all(y[2] == 0)
    assert np.all(np.isnan(y[4])) and not np.any(np.isfinite(y[5]))
    d[7, 1] = np.nan
    y = torch.empty(1, rows, device="cuda")
    ops.tqd_op_q4_0_matvec(tiles_of(ops, codes, d), rows, cols, dev(x[2:3] + 1), y)
    y = y.cpu().numpy()[0]
    assert np.isnan(y[7]) and np.all(np.isfinite(np.delete(y, 7)))


@pytest.mark.parametrize("ratio", [1, 20, 100, 1000, 5000, 2**20])
@pytest.mark.parametrize("n", [1, 3, 8, 16])
def test_q4_matvec_large_elements_that_meet_zero_weights(ops, ratio, n):
    """One element of each group of 32 is far larger than the rest and its weights are 0 (code 8), so that nothing of
    the result hides what the rest lost beside it.  Terms of the tolerance are the products themselves, |w x|: f32's
    16 u sqrt(sum T^2) + 4 u |sum| (the file's head), and an element off by up to 2^-40 of its group's largest (four
    times the root sum square)."""
    rng = np.random.default_rng(ratio + n)
    rows, cols = 2000, 1024
    codes, d = q4_matrix(rng, rows, cols)
    x = rng.normal(size=(n, cols)).astype(np.float32)
    at = 32 * np.arange(cols // 32) + rng.integers(0, 32, size=cols // 32)
    x[:, at] = (ratio * rng.uniform(0.7, 1.4, size=(n, at.size)) * rng.choice([-1, 1], size=(n, at.size)))
    codes[:, at] = 8
    y = torch.empty(n, rows, device="cuda")
    ops.tqd_op_q4_0_matvec(tiles_of(ops, codes, d), rows, cols, dev(x), y)
    w, x64 = q4.q4_0_values(codes, d), x.astype(np.float64)
    want = x64 @ w.T
    top = np.repeat(np.abs(x64).reshape(n, -1, 32).max(-1), 32, axis=1)
    off = 4 * np.sqrt((top * 2.0**-40) ** 2 @ (w**2).T)
    tol = 16 * U * np.sqrt((x64**2) @ (w**2).T) + 4 * U * np.abs(want) + off
    err = np.abs(y.cpu().numpy() - want)
    assert np.all(err <= tol), float((err / tol).max())


def test_q4_matvec_groups_of_every_shape(ops):
    """Groups of equal elements, at the ends of an octave, of one large element and 31 small ones, all codes 0, all 15
    and mixed: sums at their longest, and terms of very unequal size."""
    rng = np.random.default_rng(77)
    cols = 256
    top = np.float32(2.0) - np.float32(2.0**-23)
    groups = [np.full(32, top), np.full(32, 1.0), np.full(32, top) * rng.choice([-1, 1], 32),
              np.r_[top, np.full(31, 2.0**-5)], np.r_[1.0, np.full(31, 2.0**-12 * 1.7)],
              np.r_[top, np.full(31, 2.0**-20 * 1.3)], np.full(32, 2.0**-40 * 1.1), np.r_[-top, np.full(31, top)]]
    x = np.concatenate(groups).astype(np.float32)
    x = np.stack([x, x * np.float32(1 / 3), -x * np.float32(1.7)])
    codes = np.concatenate([np.zeros((3, cols)), np.full((3, cols), 15), rng.choice([0, 15], size=(26, cols)),
                            rng.integers(0, 16, size=(8, cols))]).astype(np.uint8)
    d = np.exp2(rng.integers(-3, 4, size=(40, cols // 32))).astype(np.float16)
    y = torch.empty(3, 40, device="cuda")
    ops.tqd_op_q4_0_matvec(tiles_of(ops, codes, d), 40, cols, dev(x), y)
    w, x64 = q4.q4_0_values(codes, d), x.astype(np.float64)
    want = x64 @ w.T
    tol = 16 * U * np.sqrt((x64**2) @ (w**2).T) + 4 * U * np.abs(want)
    err = np.abs(y.cpu().numpy() - want)
    assert np.all(err <= tol), float((err / tol).max())


def test_q4_matvec_in_a_graph_and_on_a_stream(ops):
    rng = np.random.default_rng(6)
    rows, cols = 1000, 1056
    codes, d = q4_matrix(rng, rows, cols)
    t = tiles_of(ops, codes, d)
    x = torch.randn(3, cols, device="cuda")
    y = torch.empty(3, rows, device="cuda")
    ops.tqd_op_q4_0_matvec(t, rows, cols, x, y)
    ref = y.clone()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y2 = torch.empty_like(y)
    torch.cuda.synchronize()
    ops.tqd_op_q4_0_matvec(t, rows, cols, x, y2, stream=st)
    st.synchronize()
    assert torch.equal(y2, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.tqd_op_q4_0_matvec(t, rows, cols, x, y)
    x.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, 2 * ref)


# ------------------------------------------------------------------ log probabilities

def run_logprobs(ops, x, targets, k, pad=0):
    n, v = x.shape
    wide = np.full((n, v + pad), 99.0, dtype=np.float32)
    wide[:, :v] = x
    logits = dev(wide)[:, :v]
    lp, ent = torch.full((n,), 9.0, device="cuda"), torch.full((n,), 9.0, device="cuda")
    ids = torch.full((n, k), 77, dtype=torch.int32, device="cuda")
    tops = torch.full((n, k), 9.0, device="cuda")
    scratch = torch.full((ops.tqd_logprobs_scratch_bytes(n, v, k),), 0xFF, dtype=torch.uint8, device="cuda")
    ops.tqd_op_logprobs(logits, i32(targets), lp, ent, ids if k else None, tops if k else None, scratch)
    return [t.cpu().numpy() for t in (lp, ent, ids, tops)]


def check_logprobs(ops, x, targets, k, pad=0):
    lp, ent, ids, tops = run_logprobs(ops, x, targets, k, pad)
    for r in range(len(x)):
        a, h, i, t, e1, e2 = q4.logprobs(x[r], targets[r], k)
        sum_err = 4 * U * (1 + e1)

        def near(got, want):
            if not math.isfinite(want):
                return (math.isnan(got) and math.isnan(want)) or got == want
            return abs(got - want) <= 4 * U * (1 + 3 * abs(want)) + sum_err
        assert near(float(lp[r]), a), (r, lp[r], a)
        assert abs(float(ent[r]) - h) <= 4 * U * (2 + h + e1 + e2) + sum_err, (r, ent[r], h)
        assert np.array_equal(ids[r], i), (r, ids[r], i)
        for got, want in zip(tops[r], t):
            assert near(float(got), float(want)), (r, got, want)


@pytest.mark.parametrize("n,v,k,pad", [(1, 1, 3, 0), (3, 5, 5, 2), (2, 31, 32, 1), (5, 1000, 20, 0), (4, 4096, 1, 3),
                                       (3, 8193, 32, 0), (2, 151936, 20, 1), (1, 151936, 5, 0), (400, 2049, 8, 0),
                                       (700, 333, 32, 5), (2, 49152, 0, 0), (1, 262147, 32, 0), (310, 9001, 31, 0)])
def test_logprobs(ops, n, v, k, pad):
    rng = np.random.default_rng(n + v)
    x = (rng.normal(size=(n, v)) * 3).astype(np.float32)
    peaks = rng.integers(0, v, size=(n, 4))
    np.put_along_axis(x, peaks, (8 + 4 * rng.random((n, 4))).astype(np.float32), 1)
    targets = np.where(rng.random(n) < 0.5, peaks[:, 0], rng.integers(0, v, size=n))
    check_logprobs(ops, x, targets, k, pad)


@pytest.mark.parametrize("v", [40, 3000, 20011, 151936])
def test_logprobs_ties_masks_and_order(ops, v):
    """Rows whose alternatives are hard to find: all equal, few values, ascending, descending, masked, empty."""
    rng = np.random.default_rng(v)
    asc = np.sort(rng.normal(size=v)).astype(np.float32)
    few = rng.integers(-3, 4, size=v).astype(np.float32)
    masked = np.where(rng.random(v) < 0.999, -np.inf, rng.normal(size=v)).astype(np.float32)
    one = np.full(v, -np.inf, dtype=np.float32)
    one[v - 1] = -5.0
    nan = rng.normal(size=v).astype(np.float32)
    nan[::3] = np.nan
    end = rng.normal(size=v).astype(np.float32)
    end[-20:] += 50
    zeros = np.where(rng.random(v) < 0.5, -0.0, 0.0).astype(np.float32)
    lowest = np.full(v, np.finfo(np.float32).min, dtype=np.float32)
    lowest[7] = 1.0
    x = np.stack([np.zeros(v, np.float32), few, asc, asc[::-1], masked, np.full(v, -np.inf, np.float32), one, nan,
                  np.full(v, np.nan, np.float32), end, zeros, lowest, np.full(v, np.finfo(np.float32).min, np.float32),
                  few * 1e30])
    targets = rng.integers(0, v, size=len(x))
    targets[6], targets[3] = v - 1, 0
    check_logprobs(ops, x, targets, 32)
    check_logprobs(ops, x, targets, 7, pad=1)


def hard_rows(rng, v, off, k):
    """Rows whose alternatives a block finds on each of its paths when it streams a whole row; off: how far the row
    lies past a 16-byte boundary.  Thread t of a block holds the logits i with (i + off) / 4 % 256 == t."""
    thread = (np.arange(v) + off) // 4 % 256
    rows = {"random": rng.normal(size=v) * 2}
    rows["ascending"] = np.sort(rng.normal(size=v))          # a list that overflows after its first look
    rows["descending"] = rows["ascending"][::-1]
    rows["equal"] = np.zeros(v)
    rows["last"] = rng.normal(size=v)                        # the best lie in the last tile
    rows["last"][-40:] += 30
    rows["late"] = rng.normal(size=v)                        # and behind the second look
    rows["late"][v * 3 // 5:v * 3 // 5 + 50] += 30
    rows["few"] = rng.integers(-3, 4, size=v)
    rows["steps"] = np.floor(np.arange(v) / 777.0)           # ascending in groups of equal ones
    # fewer threads than alternatives hold thousands of values above what all others have in common
    rows["columns"] = np.where(np.isin(thread, rng.permutation(256)[:15]), rng.uniform(1, 2, size=v), 0.0)
    # and one thread less than alternatives, 30 threads of equal values behind them, the rest below
    pick = rng.permutation(256)
    rows["two levels"] = np.where(np.isin(thread, pick[:k - 1]), rng.uniform(10, 11, size=v), rng.uniform(-9, -8, size=v))
    rows["two levels"] = np.where(np.isin(thread, pick[k - 1:k + 29]), 5.0, rows["two levels"])
    rows["masked"] = np.where(rng.random(v) < 0.9, -np.inf, rng.normal(size=v))
    rows["ten"] = np.full(v, -np.inf)
    rows["ten"][rng.permutation(v)[:10]] = rng.normal(size=10)
    rows["infinite"] = np.sort(rng.normal(size=v))
    rows["infinite"][[v // 3, v - 5]] = np.inf
    return {k: np.asarray(r, dtype=np.float32) for k, r in rows.items()}


@pytest.mark.parametrize("v,pad", [(151936, 0), (40961, 1), (200003, 2)])
@pytest.mark.parametrize("k", [20, 32])
def test_logprobs_of_rows_streamed_whole(ops, v, pad, k):
    """760 rows are a block each (20 to 98 tiles): candidates above a threshold, lists looked at after 4, 16 and 64
    tiles and at the end, lists that overflow between looks, and what is read again then."""
    rng = np.random.default_rng(v + k)
    n = 760
    wide = torch.randn(n, v + pad, device="cuda") * 2
    picked = {}
    for i, where in enumerate((0, 300, 301, 302, 303)):      # at every place of a 16-byte boundary
        off = where * (v + pad) % 4
        for j, (name, row) in enumerate(hard_rows(rng, v, off, k).items()):
            r = where + 20 * j if i == 0 else where + 4 * (j + 1) + 4 * 13 * (i - 1)
            while r in picked or r * (v + pad) % 4 != off:
                r += 1
            picked[r] = name, row
            wide[r, :v] = dev(row)
    logits = wide[:, :v]
    targets = rng.integers(0, v, size=n)
    lp, ent = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    ids, tops = torch.empty(n, k, dtype=torch.int32, device="cuda"), torch.empty(n, k, device="cuda")
    scratch = torch.full((ops.tqd_logprobs_scratch_bytes(n, v, k),), 0xFF, dtype=torch.uint8, device="cuda")
    ops.tqd_op_logprobs(logits, i32(targets), lp, ent, ids, tops, scratch)
    picked |= {r: ("plain", logits[r].cpu().numpy()) for r in (5, 758, 759)}
    for r, (name, row) in picked.items():
        a, h, i, t, e1, e2 = q4.logprobs(row, targets[r], k)
        near = lambda got, want: got == want if not math.isfinite(want) else (  # noqa: E731
            abs(got - want) <= 4 * U * (1 + 3 * abs(want)) + 4 * U * (1 + e1))
        assert np.array_equal(ids[r].cpu().numpy(), i), (r, name)
        assert near(float(lp[r]), a) and all(map(near, tops[r].tolist(), t.tolist())), (r, name)
        assert abs(float(ent[r]) - h) <= 4 * U * (2 + h + e1 + e2) + 4 * U * (1 + e1), (r, name, float(ent[r]), h)


@pytest.mark.parametrize("peaks", [False, True])
def test_logprobs_entropy_keeps_f32(ops, peaks):
    """The entropy of long rows, (log2 s - t / s) ln 2 with s = sum 2^d and t = sum d 2^d, d relative to the largest
    logit: four f32 roundings of log2 s, t / s and twice their difference, each u / sqrt(3) of its value in the root
    mean square.  Over 760 rows the error's root mean square stays below three times theirs, which leaves the sums
    of 151936 terms two of the three: small terms may not be lost one by one beside large ones."""
    n, v = 760, 151936
    g = torch.Generator(device="cuda")
    g.manual_seed(8 + peaks)
    x = 2 * torch.randn(n, v, generator=g, device="cuda")
    if peaks:
        x.scatter_add_(1, torch.randint(0, v, (n, 8), generator=g, device="cuda"),
                       6 + 6 * torch.rand(n, 8, generator=g, device="cuda"))
    ent = torch.empty(n, device="cuda")
    scratch = torch.empty(ops.tqd_logprobs_scratch_bytes(n, v, 0), dtype=torch.uint8, device="cuda")
    ops.tqd_op_logprobs(x, None, None, ent, None, None, scratch)
    parts = []
    for rows, got in zip(x.split(38), ent.split(38)):
        d = (rows.double() - rows.double().amax(1, keepdim=True)) / math.log(2)
        e = torch.exp2(d)
        a, b = torch.log2(e.sum(1)), (e * d).sum(1) / e.sum(1)
        h = (a - b) * math.log(2)
        scale = U / math.sqrt(3) * math.log(2) * torch.sqrt(a**2 + b**2 + 2 * (a - b) ** 2)
        parts.append((got.double() - h) / scale)
    rms = float(torch.cat(parts).square().mean().sqrt())
    assert rms <= 3, rms


def test_logprobs_infinite_logits_and_targets_outside(ops):
    x = np.random.default_rng(1).normal(size=(4, 5000)).astype(np.float32)
    x[0, [17, 4000]] = np.inf
    x[1, 4999] = np.inf
    x[2, 5] = 88.0
    check_logprobs(ops, x, np.array([17, 3, -1, 5000]), 4)
    check_logprobs(ops, x, np.array([4, 4999, 1 << 30, -(1 << 31)]), 32)


def test_logprobs_parts_can_be_left_out(ops):
    x = torch.randn(3, 7000, device="cuda")
    scratch = torch.empty(ops.tqd_logprobs_scratch_bytes(3, 7000, 5), dtype=torch.uint8, device="cuda")
    full = [torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), torch.empty(3, 5, dtype=torch.int32, device="cuda"),
            torch.empty(3, 5, device="cuda")]
    t = i32([1, 2, 3])
    ops.tqd_op_logprobs(x, t, *full, scratch)
    got = [torch.empty_like(f) for f in full]
    ops.tqd_op_logprobs(x, None, None, None, got[2], got[3], scratch)
    ops.tqd_op_logprobs(x, t, got[0], None, None, None, scratch)
    ops.tqd_op_logprobs(x, None, None, got[1], None, None, scratch)
    assert torch.equal(got[2], full[2])
    for g, f in zip(got, full):
        assert torch.allclose(g.float(), f.float(), rtol=1e-6, atol=1e-6)


def test_logprobs_repeat_to_the_bit_and_in_a_graph(ops):
    n, v, k = 3, 151936, 20
    x = torch.randn(n, v, device="cuda") * 4
    t = i32([5, 6, 7])
    scratch = torch.empty(ops.tqd_logprobs_scratch_bytes(n, v, k), dtype=torch.uint8, device="cuda")
    make = lambda: [torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"),  # noqa: E731
                    torch.zeros(n, k, dtype=torch.int32, device="cuda"), torch.zeros(n, k, device="cuda")]
    a, b = make(), make()
    ops.tqd_op_logprobs(x, t, *a, scratch)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.tqd_op_logprobs(x, t, *b, scratch)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_logprobs_with_the_scratch_of_a_larger_call(ops):
    """One scratch, sized for the largest batch, serves calls of fewer rows, which are cut into more slices; what
    lies behind it stays as it was."""
    rng = np.random.default_rng(31)
    v, k, rows = 20011, 20, 2053
    size, guard = ops.tqd_logprobs_scratch_bytes(rows, v, k), 4 << 20
    mem = torch.full((size + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    x = (rng.normal(size=(rows, v)) * 3).astype(np.float32)
    d, targets = dev(x), rng.integers(0, v, size=rows)
    for n in (1, 8, 40, 333, 700, rows):
        lp, ent = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        ids, tops = torch.empty(n, k, dtype=torch.int32, device="cuda"), torch.empty(n, k, device="cuda")
        ops.tqd_op_logprobs(d[:n], i32(targets[:n]), lp, ent, ids, tops, mem[:size])
        for r in {0, n // 2, n - 1}:
            a, h, i, t, e1, e2 = q4.logprobs(x[r], targets[r], k)
            tol = 4 * U * (1 + e1)
            assert abs(float(lp[r]) - a) <= 4 * U * (1 + 3 * abs(a)) + tol
            assert abs(float(ent[r]) - h) <= 4 * U * (2 + h + e1 + e2) + tol
            assert np.array_equal(ids[r].cpu().numpy(), i)
            assert np.all(np.abs(tops[r].cpu().numpy() - t) <= 4 * U * (1 + 3 * np.abs(t)) + tol)
    assert bool((mem[size:] == 0x5A).all())


def test_lanes_of_a_warp_agree_about_a_wait_that_runs_out_in_some(ops):
    """A phase that completes between two lanes' limits: the attention and the products go on with whole warps."""
    status, bits = ops.tqd_op_wait_selftest()
    assert status != 0 and not bits & 4


# ------------------------------------------------------------------ refusals of the wrappers

def test_wrapper_refusals(ops, TQDError):
    pages = torch.zeros(4 * ops.tqd_kv_q4_page_bytes(2, 64, 16), dtype=torch.uint8, device="cuda")
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    cache = ops.kv_q4(pages, table, 2, 64, 16)
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    pos = i32([0, 1])
    scratch = torch.zeros(ops.tqd_attention_q4_scratch_bytes(64), dtype=torch.uint8, device="cuda")
    bad = [
        lambda: ops.kv_q4(pages[:-1], table, 2, 64, 16),
        lambda: ops.kv_q4(pages[1:1 + 1152 * 2], table, 2, 64, 16) and ops.tqd_op_kv_append_q4(
            ops.kv_q4(pages[1:1 + 1152 * 2], table, 2, 64, 16), f(2, 128), f(2, 128), pos),
        lambda: ops.kv_q4(pages, table.long(), 2, 64, 16),
        lambda: ops.kv_q4(pages, table[:, :1], 2, 64, 16),
        lambda: ops.tqd_op_kv_append_q4(cache, f(2, 64), f(2, 128), pos),
        lambda: ops.tqd_op_kv_append_q4(cache, f(2, 128).half(), f(2, 128), pos),
        lambda: ops.tqd_op_kv_append_q4(cache, f(2, 128), f(2, 256)[:, ::2], pos),
        lambda: ops.tqd_op_kv_append_q4(cache, f(2, 128), f(2, 128), pos, pos.long()),
        lambda: ops.tqd_op_kv_append_q4(cache, f(2, 128), f(2, 128), pos, None, None, f(2, 128)),
        lambda: ops.tqd_op_kv_append_q4(cache, f(3, 128), f(3, 128), i32([0, 1, 2])),
        lambda: ops.tqd_op_kv_read_q4(cache, pos, None, None, None),
        lambda: ops.tqd_op_attention_q4(cache, f(2, 192), pos, None, f(2, 192), scratch),
        lambda: ops.tqd_op_attention_q4(cache, f(3, 128), pos, None, f(3, 128), scratch),
        lambda: ops.tqd_op_attention_q4(cache, f(2, 128), pos[:1], None, f(2, 128), scratch),
        lambda: ops.tqd_op_attention_q4(cache, f(2, 128), pos, pos, f(2, 128), scratch),
        lambda: ops.tqd_op_attention_q4(cache, f(2, 128), pos, None, f(2, 128), scratch[:-1]),
        lambda: ops.tqd_op_attention_q4(cache, f(2, 128), pos, None, f(1, 128).expand(2, 128), scratch),
        lambda: ops.tqd_op_q4_0_matvec(pages, 16, 100, f(100), f(16)),
        lambda: ops.tqd_op_q4_0_matvec(pages[:1152], 17, 128, f(128), f(17)),
        lambda: ops.tqd_op_q4_0_matvec(pages, 16, 128, f(65, 128), f(65, 16)),
        lambda: ops.tqd_op_q4_0_repack(pages[:18], 2, 32, pages),
        lambda: ops.tqd_op_logprobs(f(2, 100), pos, f(2), None, None, None, scratch[:1]),
        lambda: ops.tqd_op_logprobs(f(2, 100), pos, None, None, None, None, scratch),
        lambda: ops.tqd_op_logprobs(f(2, 100), None, None, None, torch.zeros(2, 33, dtype=torch.int32, device="cuda"),
                                    f(2, 33), scratch),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(TQDError) as ei:
            call()
        assert ei.value.name == "TQD_ERR_BAD_ARG", i
    # calls with no rows
    e = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    ops.tqd_op_kv_append_q4(cache, e(0, 128), e(0, 128), none)
    ops.tqd_op_attention_q4(cache, e(0, 128), pos, i32([0, 0, 0]), e(0, 128), scratch)
    ops.tqd_op_q4_0_matvec(pages, 16, 128, e(0, 128), e(0, 16))
    ops.tqd_op_logprobs(e(0, 100), none, e(0), None, None, None, scratch)


def test_rows_between_one_anothers(ops, TQDError):
    """Outputs as slices of one buffer with strides of any kind: read where they do not overlap, refused where they do."""
    rng = np.random.default_rng(33)
    host = Host(rng, 1, 1, 64, 16, 16)
    host.fill(rng, [8])
    cache = host.device(ops)
    taken = 0
    for _ in range(400):
        n, sk, sv = int(rng.integers(1, 6)), int(rng.integers(64, 300)), int(rng.integers(64, 300))
        if rng.random() < 0.5:
            sv = sk
        at = int(rng.integers(-1400, 1400))
        buf = torch.full((6000,), 7.0, device="cuda")
        k, v = buf.as_strided((n, 64), (sk, 1), 2000), buf.as_strided((n, 64), (sv, 1), 2000 + at)
        mine = [{2000 + o + s * i + j for i in range(n) for j in range(64)} for o, s in ((0, sk), (at, sv))]
        pos = i32(np.arange(n))
        seqs = i32(np.zeros(n))
        if mine[0] & mine[1]:
            with pytest.raises(TQDError, match="overlap"):
                ops.tqd_op_kv_read_q4(cache, pos, seqs, k, v)
            continue
        taken += 1
        ops.tqd_op_kv_read_q4(cache, pos, seqs, k, v)
        assert np.array_equal(k.cpu().numpy(), host.K[0][:n, 0]) and np.array_equal(v.cpu().numpy(), host.V[0][:n, 0])
        assert int((buf != 7.0).sum()) <= 128 * n
    assert taken > 100
    x = torch.randn(4, 160, device="cuda")  # x and y side by side in one tensor
    t = tiles_of(ops, *q4_matrix(rng, 32, 96))
    ops.tqd_op_q4_0_matvec(t, 32, 96, x[:, :96], x[:, 100:132])
    with pytest.raises(TQDError, match="overlap"):
        ops.tqd_op_q4_0_matvec(t, 32, 96, x[:, :96], x[:, 95:127])


def test_logprob_alternatives_go_together(ops, TQDError):
    """top_logprobs of another shape than top_ids would be filled with another stride, and alone with nothing."""
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    x, ids = f(2, 100), torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    scratch = torch.zeros(ops.tqd_logprobs_scratch_bytes(2, 100, 5), dtype=torch.uint8, device="cuda")
    for top_ids, tops in ((ids, f(2, 10)), (ids, f(10)), (ids, f(3, 5)), (ids, None), (None, f(2, 5))):
        with pytest.raises(TQDError, match="top_"):
            ops.tqd_op_logprobs(x, None, None, f(2), top_ids, tops, scratch)
    ops.tqd_op_logprobs(x, None, None, f(2), ids, f(2, 5), scratch)
    ops.tqd_op_logprobs(x, None, None, f(2), ids[:, :0], f(2, 0), scratch)


# ------------------------------------------------------------------ a decode step of them together

def test_a_decode_step_in_four_bits(ops):
    """Projections, append, attention, output projection, lm_head and log probabilities, for a prompt given as
    one tile and then single tokens, three sequences with different lengths."""
    rng = np.random.default_rng(21)
    hidden, heads, n_kv, hd, vocab, n_seq, page = 256, 4, 2, 64, 1000, 3, 16
    qw, kvw = heads * hd, n_kv * hd
    mats = {n: q4_matrix(rng, r, c, 0.06) for n, (r, c) in
            {"qkv": (qw + 2 * kvw, hidden), "o": (hidden, qw), "head": (vocab, hidden)}.items()}
    tiles = {n: tiles_of(ops, *m) for n, m in mats.items()}
    w = {n: q4.q4_0_values(*m) for n, m in mats.items()}
    table = rope_table(ops, hd, 128)
    th = table.cpu().numpy()
    host = Host(rng, n_seq, n_kv, hd, page, 64)
    cache = host.device(ops)
    scratch = torch.empty(ops.tqd_attention_q4_scratch_bytes(hd), dtype=torch.uint8, device="cuda")
    lscratch = torch.empty(ops.tqd_logprobs_scratch_bytes(64, vocab, 5), dtype=torch.uint8, device="cuda")
    lens = [0] * n_seq
    K, V = [[] for _ in range(n_seq)], [[] for _ in range(n_seq)]
    for nq in ([17, 5, 1], [1, 1, 1], [1, 1, 1], [2, 3, 1]):
        n = sum(nq)
        seqs = np.repeat(np.arange(n_seq), nq)
        pos = np.concatenate([np.arange(lens[s], lens[s] + nq[s]) for s in range(n_seq)])
        lens = [a + b for a, b in zip(lens, nq)]
        x = rng.normal(size=(n, hidden)).astype(np.float32)
        xd, qkv = dev(x), torch.empty(n, qw + 2 * kvw, device="cuda")
        q, att = torch.empty(n, qw, device="cuda"), torch.empty(n, qw, device="cuda")
        h, logits = torch.empty(n, hidden, device="cuda"), torch.empty(n, vocab, device="cuda")
        ops.tqd_op_q4_0_matvec(tiles["qkv"], qw + 2 * kvw, hidden, xd, qkv)
        ops.tqd_op_kv_append_q4(cache, qkv[:, qw:qw + kvw], qkv[:, qw + kvw:], i32(pos), i32(seqs), table,
                                qkv[:, :qw], q)
        single = nq == [1] * n_seq
        start = None if single else i32(np.concatenate([[0], np.cumsum(nq)]))
        ops.tqd_op_attention_q4(cache, q, i32(lens), start, att, scratch)
        ops.tqd_op_q4_0_matvec(tiles["o"], hidden, qw, att, h)
        ops.tqd_op_q4_0_matvec(tiles["head"], vocab, hidden, h, logits)
        lp, ent = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        ids, tops = torch.empty(n, 5, dtype=torch.int32, device="cuda"), torch.empty(n, 5, device="cuda")
        targets = rng.integers(0, vocab, size=n)
        ops.tqd_op_logprobs(logits, i32(targets), lp, ent, ids, tops, lscratch)
        # the oracle, on the device's projections where a code is decided (a value next to a border may fall either way)
        f = qkv.cpu().numpy().astype(np.float64).reshape(n, -1, hd)
        assert np.max(np.abs(f.reshape(n, -1) - x.astype(np.float64) @ w["qkv"].T)) < 1e-5
        rq, rk = q4.rotate(f[:, :heads], pos, th), q4.rotate(f[:, heads:heads + n_kv], pos, th)
        for i in range(n):
            kk, vv = host.store(seqs[i], int(pos[i]), rk[i], f[i, heads + n_kv:])
            K[seqs[i]].append(kk)
            V[seqs[i]].append(vv)
        assert np.array_equal(cache.pages.cpu().numpy(), host.pages)
        want = np.stack([q4.attention(rq[i], np.array(K[seqs[i]]), np.array(V[seqs[i]]), pos[i] + 1).reshape(-1)
                         for i in range(n)])
        final = want @ w["o"].T @ w["head"].T
        assert np.max(np.abs(logits.cpu().numpy() - final)) < 1e-4 * max(1.0, np.abs(final).max())
        for i in range(n):
            a, ent_w, id_w, top_w, *_ = q4.logprobs(logits[i].cpu().numpy(), targets[i], 5)
            assert abs(float(lp[i]) - a) < 1e-5 and abs(float(ent[i]) - ent_w) < 1e-5
            assert np.array_equal(ids[i].cpu().numpy(), id_w) and np.max(np.abs(tops[i].cpu().numpy() - top_w)) < 1e-5


def test_a_captured_decode_step_repeats_the_eager_one(ops):
    """The whole step as one graph, replayed with positions, lengths and inputs that change on the device, beside the
    same calls made one by one on a copy of the cache: the same bits, over steps that cross pages and blocks."""
    rng = np.random.default_rng(34)
    hidden, heads, n_kv, hd, vocab, n_seq, page, k = 256, 8, 2, 64, 3001, 5, 16, 6
    qw, kvw = heads * hd, n_kv * hd
    tiles = {n: tiles_of(ops, *q4_matrix(rng, r, c, 0.06)) for n, (r, c) in
             {"qkv": (qw + 2 * kvw, hidden), "o": (hidden, qw), "head": (vocab, hidden)}.items()}
    table = rope_table(ops, hd, 128)
    first = [0, 13, 31, 3, 70]
    host = Host(rng, n_seq, n_kv, hd, page, 112)
    host.fill(rng, first)

    class Step:
        def __init__(self):
            e = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
            self.cache = host.device(ops)
            self.scratch = torch.zeros(ops.tqd_attention_q4_scratch_bytes(hd), dtype=torch.uint8, device="cuda")
            self.lscratch = torch.zeros(ops.tqd_logprobs_scratch_bytes(n_seq, vocab, k), dtype=torch.uint8, device="cuda")
            self.x, self.qkv, self.att = e(n_seq, hidden), e(n_seq, qw + 2 * kvw), e(n_seq, qw)
            self.h, self.logits = e(n_seq, hidden), e(n_seq, vocab)
            self.lp, self.ent, self.tops = e(n_seq), e(n_seq), e(n_seq, k)
            self.ids = torch.zeros(n_seq, k, dtype=torch.int32, device="cuda")
            self.pos, self.lens, self.targets = i32(first), i32([f + 1 for f in first]), i32([1, 2, 3, 4, 5])

        def run(self):
            q, kk, v = self.qkv.split([qw, kvw, kvw], 1)
            ops.tqd_op_q4_0_matvec(tiles["qkv"], qw + 2 * kvw, hidden, self.x, self.qkv)
            ops.tqd_op_kv_append_q4(self.cache, kk, v, self.pos, None, table, q, q)
            ops.tqd_op_attention_q4(self.cache, q, self.lens, None, self.att, self.scratch)
            ops.tqd_op_q4_0_matvec(tiles["o"], hidden, qw, self.att, self.h)
            ops.tqd_op_q4_0_matvec(tiles["head"], vocab, hidden, self.h, self.logits)
            ops.tqd_op_logprobs(self.logits, self.targets, self.lp, self.ent, self.ids, self.tops, self.lscratch)

        def advance(self, x):
            self.x.copy_(x)
            self.pos += 1
            self.lens += 1

        def results(self):
            return [t.clone() for t in (self.cache.pages, self.qkv, self.att, self.logits, self.lp, self.ent, self.ids,
                                        self.tops)]

    eager, captured = Step(), Step()
    warm = Step()  # (every kernel once before the capture)
    warm.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.run()
    for step in range(40):
        x = torch.randn(n_seq, hidden, device="cuda")
        for s in (eager, captured):
            if step:
                s.advance(x)
            else:
                s.x.copy_(x)
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.results(), captured.results()):
            assert torch.equal(a, b), step
    assert bool(torch.isfinite(eager.logits).all()) and eager.lens.tolist() == [f + 40 for f in first]
