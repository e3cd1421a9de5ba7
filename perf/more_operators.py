"""Cases of the operators on rows of 8-bit codes: quantising rows, the RMSNorm and the SwiGLU product that end in
such rows, the matrix product of two such matrices, and the rotation of many tokens' heads.  For each: what it
takes in, its plain form in elementary torch operations, its definition in 64 bits, and the calls of the library.

8-bit rows (also described in include/tqd.h).  A row y is held as one f32 scale, max|y| / 127, and a code for each
element, rint(127 y / max|y|) of the exact values (ties to even), so an element stands for code * scale.

Rotation.  The first rotary_dim elements of a head are turned in pairs by angles position * f_i, f_i =
theta^(-2 i / rotary_dim): elements i and i + rotary_dim / 2, or 2 i and 2 i + 1 (interleaved).  For contexts
longer than those of training, f_i is divided by a factor, either throughout (linear) or where a pair turns too
seldom over the original length (by rotations), and cos and sin carry an attention factor.
"""
import math

import torch

own = False

THETA = 1e6
EPS = 1e-6


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the norm before a projection of one decode step, with the residual's addition (hidden size of the benchmark)
        {"name": "norm 1 x 1024", "op": "norm", "n": 1, "width": 1024, "add": True},
        # a long prompt's rows at a wider model
        {"name": "norm 4099 x 4096", "op": "norm", "n": 4099, "width": 4096, "add": True},
        # the attention's output at batch 1 (16 heads of 128), before the output projection
        {"name": "rows 1 x 2048", "op": "rows", "n": 1, "width": 2048},
        # the same for a long prompt
        {"name": "rows 8191 x 2048", "op": "rows", "n": 8191, "width": 2048},
        # SwiGLU of a decode batch (15/5 heads model's feed-forward), before the down projection
        {"name": "silu 16 x 2560", "op": "silu", "n": 16, "width": 2560},
        # a prompt's at a wide feed-forward
        {"name": "silu 2053 x 8192", "op": "silu", "n": 2053, "width": 8192},
        # the q, k, v projection of one decode step (16/8 heads of 128): latency
        {"name": "product 4096 x 1024 of 1", "op": "product", "rows": 4096, "cols": 1024, "n": 1},
        # the lm_head of a decode batch: bandwidth
        {"name": "product 151936 x 1024 of 16", "op": "product", "rows": 151936, "cols": 1024, "n": 16},
        # gate and up rows for a prompt of 511 tokens, columns that end inside a tile
        {"name": "product 5120 x 960 of 511", "op": "product", "rows": 5120, "cols": 960, "n": 511},
        # a large projection of a long prompt: compute
        {"name": "product 8192 x 8192 of 2048", "op": "product", "rows": 8192, "cols": 8192, "n": 2048},
        # a decode batch's q and k heads inside fused rows (16/8 heads of 128)
        {"name": "rope 16 x 24 heads", "op": "rope", "n": 16, "heads": 24, "head_dim": 128, "rotary_dim": 128,
         "interleaved": False, "scaling": "none", "positions": 4096},
        # a long prompt's, part of the head in neighbouring pairs, at far positions
        {"name": "rope 8191 x 20 heads, 96 of 128", "op": "rope", "n": 8191, "heads": 20, "head_dim": 128,
         "rotary_dim": 96, "interleaved": True, "scaling": "rotations", "positions": 131072},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rows", "silu", "product", "product", "product", "rope"])
    if op in ("norm", "rows", "silu"):
        width = _log(rng, 16, 12288)
        if rng.random() < 0.6:  # most models' widths are multiples of 32
            width = max(32, width // 32 * 32)
        case = {"op": op, "n": _log(rng, 1, min(8192, (1 << 24) // width)), "width": width}
        return case | ({"add": rng.random() < 0.7} if op == "norm" else {})
    if op == "product":
        cols = 32 * _log(rng, 1, 512)
        rows = _log(rng, 1, min(151936, (1 << 28) // cols))
        return {"op": op, "rows": rows, "cols": cols, "n": _log(rng, 1, min(4096, (1 << 37) // (rows * cols), (1 << 27) // rows))}
    head_dim = rng.choice([64, 64, 80, 96, 128, 128, 256])
    rotary = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4, head_dim * 3 // 4])
    heads = rng.choice([1, 2, 6, 9, 20, 24, 40])
    return {"op": op, "n": _log(rng, 1, min(8192, (1 << 24) // (heads * head_dim))), "heads": heads, "head_dim": head_dim,
            "rotary_dim": rotary, "interleaved": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "rotations"]),
            "positions": _log(rng, 64, 131072)}


def work(case):
    op, n = case["op"], case["n"]
    if op == "product":
        r, c = case["rows"], case["cols"]
        return {"bytes": r * c + n * c + 4 * (r + n) + 4 * n * r, "flops": 2 * r * c * n}
    if op == "rope":
        w = case["heads"] * case["head_dim"]
        return {"bytes": n * (8 * w + 4 * case["rotary_dim"] + 4), "flops": 3 * n * case["heads"] * case["rotary_dim"]}
    w = case["width"]
    inputs = {"rows": 4, "silu": 8, "norm": 4 + 8 * case.get("add", False)}[op]  # the norm's sum is an output too
    # the codes and scales, and the values they stand for
    return {"bytes": n * w * (inputs + 1 + 4) + 4 * n + (4 * w if op == "norm" else 0),
            "flops": n * w * {"rows": 4, "silu": 9, "norm": 7}[op]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _codes(y):
    """Codes int8 and f32 scales of the rows of y."""
    m = y.abs().amax(1, keepdim=True)
    q = torch.round(y * (127 / torch.where(m > 0, m, torch.ones_like(m))))
    return q.to(torch.int8), (m / 127).squeeze(1)


def _frequencies(case):
    """Angles per position, the attention factor: host numbers."""
    d, kind = case["rotary_dim"], case["scaling"]
    f = [THETA ** (-2.0 * i / d) for i in range(d // 2)]
    if kind == "none":
        return f, 1.0
    factor, original = 4.0, max(16, case["positions"] // 4)
    if kind == "linear":
        return [x / factor for x in f], 1.0
    # pairs that turn more than 32 times over the original length keep their angle, those that turn less than
    # once have it divided, those between are mixed
    out = []
    for x in f:
        keep = min(1.0, max(0.0, (original * x / (2 * math.pi) - 1.0) / 31.0))
        out.append(x * (keep + (1 - keep) / factor))
    return out, 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    g = _gen(seed)
    op, n = case["op"], case["n"]
    st = {"case": dict(case)}
    if op == "product":
        rows, cols = case["rows"], case["cols"]
        x = _randn(g, n, cols)
        x[:, ::97] *= 8.0  # activations have a few large channels
        st["x"], st["x_scale"] = _codes(x)
        st["w"] = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
        st["w_scale"] = torch.empty(rows, device="cuda")
        step = max(1, (1 << 24) // cols)
        for r in range(0, rows, step):
            m = min(step, rows - r)
            st["w"][r:r + m], st["w_scale"][r:r + m] = _codes(_randn(g, m, cols) * 0.02)
        st["y"] = torch.empty(n, rows, device="cuda")
        return st
    if op == "rope":
        w, d, P = case["heads"] * case["head_dim"], case["rotary_dim"], case["positions"]
        f, attention = _frequencies(case)
        angle = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * torch.tensor(f, device="cuda", dtype=torch.float64)
        st["table"] = (torch.stack([angle.cos(), angle.sin()], -1) * attention).float()
        # q and k heads at the front of fused rows, whose last sixth are v's
        fused = _randn(g, n, w + max(1, case["heads"] // 5) * case["head_dim"])
        st["x"] = fused[:, :w]
        st["positions"] = torch.randint(0, P, (n,), generator=g, device="cuda").to(torch.int32)
        st["out"] = torch.empty(n, w, device="cuda")
        return st
    w = case["width"]
    st |= {"q": torch.empty(n, -(-w // 16) * 16, dtype=torch.int8, device="cuda")[:, :w],
           "scale": torch.empty(n, device="cuda"), "values": torch.empty(n, w, device="cuda")}
    if op == "silu":
        gu = _randn(g, n, 2 * w) * 1.5  # one projection's rows: gate, then up
        st |= {"gate": gu[:, :w], "up": gu[:, w:]}
        return st
    x = _randn(g, n, w) * torch.exp(0.5 * _randn(g, n, 1))
    x[:, ::61] *= 6.0
    st["x"] = x
    if op == "norm":
        st |= {"g": 1.0 + 0.1 * _randn(g, w)}
        if case["add"]:
            st |= {"add": _randn(g, n, w) * 0.5, "sum": torch.empty(n, w, device="cuda")}
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _own[st["case"]["op"]](st)
    return _plain[st["case"]["op"]](st)


def _held(y):
    """Values that rows y (64 bits: a code is decided by the side of a border its value lies on) are held as."""
    m = y.abs().amax(1, keepdim=True)
    q = torch.round(127 * y / torch.where(m > 0, m, torch.ones_like(m)))
    return q.float() * (m / 127).float()


def _plain_rows(st):
    return _held(st["x"].double())


def _plain_norm(st):
    x = st["x"]
    if st["case"]["add"]:
        x = x + st["add"]
    d = x.double()
    t = d * st["g"].double()  # 1 / rms multiplies the row's scale alone
    m = t.abs().amax(1, keepdim=True)
    q = torch.round(127 * t / torch.where(m > 0, m, torch.ones_like(m)))
    scale = m / torch.sqrt((d * d).mean(1, keepdim=True) + EPS) / 127
    values = q.float() * scale.float()
    return {"values": values, "sum": x} if st["case"]["add"] else {"values": values}


def _plain_silu(st):
    g = st["gate"].double()
    return _held(g / (1 + torch.exp(-g)) * st["up"].double())


def _plain_product(st):
    return (st["x"].float() @ st["w"].float().T) * st["x_scale"][:, None] * st["w_scale"]


def _plain_rope(st):
    c = st["case"]
    n, d = c["n"], c["rotary_dim"]
    x = st["x"].reshape(n, c["heads"], c["head_dim"])
    cs = st["table"][st["positions"].long()][:, None]
    cos, sin = cs[..., 0], cs[..., 1]
    if c["interleaved"]:
        a, b = x[..., 0:d:2], x[..., 1:d:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : d // 2], x[..., d // 2:d]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., d:]], -1).reshape(n, -1)


_plain = {"rows": _plain_rows, "norm": _plain_norm, "silu": _plain_silu, "product": _plain_product, "rope": _plain_rope}


# ------------------------------------------------------------------ the library's calls

def _ops():
    import token_quantized_decode_gb300 as tqd
    return tqd.ops


def _read(ops, st):
    ops.tqd_op_rows_i8_read(st["q"], st["scale"], st["values"])
    return st["values"]


def _own_rows(st):
    ops = _ops()
    ops.tqd_op_rows_i8(st["x"], st["q"], st["scale"])
    return _read(ops, st)


def _own_norm(st):
    ops = _ops()
    if not st["case"]["add"]:
        ops.tqd_op_rmsnorm_i8(st["x"], None, st["g"], EPS, None, st["q"], st["scale"])
        return {"values": _read(ops, st)}
    ops.tqd_op_rmsnorm_i8(st["x"], st["add"], st["g"], EPS, st["sum"], st["q"], st["scale"])
    return {"values": _read(ops, st), "sum": st["sum"]}


def _own_silu(st):
    ops = _ops()
    ops.tqd_op_silu_mul_i8(st["gate"], st["up"], st["q"], st["scale"])
    return _read(ops, st)


def _own_product(st):
    ops = _ops()
    if "scratch" not in st:  # what a program keeps beside its weights
        c = st["case"]
        st["scratch"] = torch.empty(ops.tqd_i8_matmul_scratch_bytes(c["rows"], c["cols"], c["n"]), dtype=torch.uint8, device="cuda")
    ops.tqd_op_i8_matmul(st["w"], st["w_scale"], st["x"], st["x_scale"], st["y"], st["scratch"])
    return st["y"]


def _own_rope(st):
    c = st["case"]
    _ops().tqd_op_rope_rows(st["x"], st["positions"], st["table"], c["head_dim"], c["rotary_dim"], c["interleaved"], st["out"])
    return st["out"]


_own = {"rows": _own_rows, "norm": _own_norm, "silu": _own_silu, "product": _own_product, "rope": _own_rope}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    return _exact[case["op"]](prepare(case, seed))


def _nearest(y):
    """(codes, largest magnitude) of each row of y."""
    most = torch.maximum(y.max(1).values, -y.min(1).values)[:, None]
    t = 127 * y / most.masked_fill(most == 0, 1.0)
    low = torch.floor(t)
    up = (t - low > 0.5) | ((t - low == 0.5) & (low % 2 != 0))
    return low + up, most


def _exact_rows(st):
    codes, most = _nearest(st["x"].double())
    return codes * (most / 127)


def _exact_norm(st):
    h = st["x"] + st["add"] if st["case"]["add"] else st["x"]  # the sum is kept in f32: what is normed is what is kept
    h = h.double()
    codes, most = _nearest(h * st["g"].double()[None])
    rms = torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / h.shape[1] + EPS)
    out = {"values": codes * (most / (127 * rms))}
    if st["case"]["add"]:
        out["sum"] = st["x"].double() + st["add"].double()
    return out


def _exact_silu(st):
    codes, most = _nearest(st["gate"].double() * torch.special.expit(st["gate"].double()) * st["up"].double())
    return codes * (most / 127)


def _exact_product(st):
    w, x = st["w"], st["x"].double()
    y = torch.empty(x.shape[0], w.shape[0], dtype=torch.float64, device=w.device)
    step = max(1, (1 << 26) // w.shape[1])
    for r in range(0, w.shape[0], step):
        y[:, r:r + step] = torch.einsum("nc,rc->nr", x, w[r:r + step].double())
    return y.mul_(st["x_scale"].double()[:, None]).mul_(st["w_scale"].double()[None])


def _exact_rope(st):
    c = st["case"]
    n, d = c["n"], c["rotary_dim"]
    f, attention = _frequencies(c)
    angle = st["positions"].double()[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda")[None]
    turn = torch.polar(torch.full_like(angle, attention), angle)[:, None]
    out = st["x"].double().reshape(n, c["heads"], c["head_dim"]).clone()
    at = torch.arange(d // 2, device="cuda")
    first, second = (2 * at, 2 * at + 1) if c["interleaved"] else (at, at + d // 2)
    z = torch.complex(out[..., first], out[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out.reshape(n, -1)


_exact = {"rows": _exact_rows, "norm": _exact_norm, "silu": _exact_silu, "product": _exact_product, "rope": _exact_rope}
