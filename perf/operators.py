"""Cases of the 4-bit decode operators and of the log probabilities: what they
take in, their plain form in elementary torch operations, their definition in
64 bits, and the calls of the library's operators.

Formats (also described in include/tqd.h):

Q4 cache.  A page holds page_size positions of every kv head, a head's part
first [page_size / 16] blocks of 16 positions.  A block is the K codes, the K
scales (f16 [16][hd / 32]), the V codes, the V scales.  A group is 32
consecutive elements of one head's row: scale = f16(max|y| / 7), code =
rint(7 y / max|y|) + 8, value (code - 8) * scale.

Q4_0 weights.  18-byte blocks of 32 consecutive weights of a row: f16 scale,
then 16 bytes, byte j holding element j in its low nibble and element j + 16
in its high one; value (nibble - 8) * scale.
"""
import math
import random

import torch

own = False

THETA = 1e6


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one sequence's decode step (the benchmark's model: 16/8 heads of 128)
        {"name": "append 1 token", "op": "append", "n": 1, "n_seq": 1, "heads": 16, "kv_heads": 8, "head_dim": 128,
         "page": 16, "history": 639},
        # a batched decode step over far positions (15/5 heads of 64), an odd batch
        {"name": "append 61 sequences", "op": "append", "n": 61, "n_seq": 61, "heads": 15, "kv_heads": 5,
         "head_dim": 64, "page": 64, "history": 131000},
        # prompts of three sequences appended together, ends inside pages
        {"name": "append 5003 of a prompt", "op": "append", "n": 5003, "n_seq": 3, "heads": 16, "kv_heads": 8,
         "head_dim": 128, "page": 32, "history": 100},
        # batch 1 at the benchmark's mid position
        {"name": "attend 1 x 575", "op": "attend", "n_seq": 1, "len": 575, "ragged": False, "queries": 1, "heads": 16,
         "kv_heads": 8, "head_dim": 128, "page": 16},
        # a serving batch of unequal sequences, one slot empty
        {"name": "attend 33 ragged to 4160", "op": "attend", "n_seq": 33, "len": 4160, "ragged": True, "queries": 1,
         "heads": 16, "kv_heads": 8, "head_dim": 128, "page": 64},
        # one long context, four query heads per kv head
        {"name": "attend 1 x 131071", "op": "attend", "n_seq": 1, "len": 131071, "ragged": False, "queries": 1,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 256},
        # prefill tiles: up to 16 positions of each sequence at once, three heads of 64 per kv head
        {"name": "attend tiles of 16 queries", "op": "attend", "n_seq": 9, "len": 2048, "ragged": True, "queries": 16,
         "heads": 15, "kv_heads": 5, "head_dim": 64, "page": 32},
        # the smallest projection: latency
        {"name": "matvec 1024 x 1024", "op": "matvec", "rows": 1024, "cols": 1024, "n": 1},
        # the lm_head at batch 1
        {"name": "matvec 151936 x 1024", "op": "matvec", "rows": 151936, "cols": 1024, "n": 1},
        # gate and up rows for a batch of 16, columns that end inside a tile
        {"name": "matvec 5120 x 960 of 16", "op": "matvec", "rows": 5120, "cols": 960, "n": 16},
        # one generated token's log probabilities
        {"name": "logprobs 1 x 151936", "op": "logprobs", "n": 1, "vocab": 151936, "top_k": 5, "masked": False},
        # scoring a prompt
        {"name": "logprobs 2053 x 151936", "op": "logprobs", "n": 2053, "vocab": 151936, "top_k": 20, "masked": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# (query heads, kv heads, head size) of the decoder configurations and of grouped and ungrouped relatives
_HEADS = [(16, 8, 128), (15, 5, 64), (4, 2, 64), (8, 1, 128), (32, 8, 128), (8, 8, 64), (12, 2, 128)]


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "matvec", "logprobs"])
    if op in ("append", "attend"):
        heads, kv_heads, hd = rng.choice(_HEADS)
        page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        n = _log(rng, 1, 8192)
        return {"op": op, "n": n, "n_seq": _log(rng, 1, min(n, 256)), "heads": heads, "kv_heads": kv_heads,
                "head_dim": hd, "page": page, "history": _log(rng, 1, 100000)}
    if op == "attend":
        n_seq = _log(rng, 1, 128)
        length = _log(rng, 1, min(131072, (1 << 19) // n_seq))
        most = min(64, (1 << 21) // (n_seq * length))
        queries = rng.choice([1, 1, _log(rng, 2, most)]) if most > 2 else 1
        return {"op": op, "n_seq": n_seq, "len": length, "ragged": rng.random() < 0.7, "queries": queries,
                "heads": heads, "kv_heads": kv_heads, "head_dim": hd, "page": page}
    if op == "matvec":
        cols = 32 * _log(rng, 1, 512)
        return {"op": op, "rows": _log(rng, 1, min(151936, (1 << 28) // cols)), "cols": cols, "n": _log(rng, 1, 64)}
    vocab = _log(rng, 32, 200000)
    return {"op": op, "n": _log(rng, 1, min(4096, (1 << 28) // vocab)), "vocab": vocab, "top_k": rng.randint(0, 32),
            "masked": rng.random() < 0.4}


def _queries(case):
    """Query tokens of each sequence (host numbers, the same for every seed)."""
    if case["queries"] == 1:
        return [1] * case["n_seq"]
    r = random.Random(case["n_seq"] * 7919 + case["queries"])
    return [case["queries"]] + [r.randint(1, case["queries"]) for _ in range(case["n_seq"] - 1)]


def _lens(case):
    """Cached positions of each sequence (host numbers, the same for every seed)."""
    if not case["ragged"]:
        return [case["len"]] * case["n_seq"]
    r = random.Random(case["n_seq"] * 104729 + case["len"])
    lens = [case["len"]] + [_log(r, 1, case["len"]) for _ in range(case["n_seq"] - 1)]
    if case["n_seq"] > 2:
        lens[case["n_seq"] // 2] = 0  # an empty slot of the batch
    return lens


def work(case):
    op = case["op"]
    if op == "append":
        n, hd, qw, kvw = case["n"], case["head_dim"], case["heads"] * case["head_dim"], case["kv_heads"] * case["head_dim"]
        moved = n * (4 * (qw + 2 * kvw) + 4 * hd + 8) + n * (4 * qw + 2 * kvw * 9 // 16 + 2 * kvw * 4)
        return {"bytes": moved, "flops": n * (3 * (qw + kvw) + 3 * 2 * kvw)}
    if op == "attend":
        hd, heads, kv = case["head_dim"], case["heads"], case["kv_heads"]
        bytes_, flops = 0, 0
        for length, nq in zip(_lens(case), _queries(case)):
            bytes_ += length * kv * hd * 9 // 8 + nq * heads * hd * 8
            seen = sum(max(0, length - nq + i + 1) for i in range(nq))
            flops += 4 * seen * heads * hd
        return {"bytes": bytes_, "flops": flops}
    if op == "matvec":
        r, c, n = case["rows"], case["cols"], case["n"]
        return {"bytes": r * (c // 32) * 18 + 4 * n * (r + c), "flops": 2 * r * c * n}
    n, v, k = case["n"], case["vocab"], case["top_k"]
    return {"bytes": n * (4 * v + 4 + 8 + 8 * k), "flops": 5 * n * v}


# ------------------------------------------------------------------ formats

def _quantise(y):
    """y [..., hd] -> codes uint8 [..., hd] (1..15), scales f16 [..., hd / 32].  In 64 bits: a code is decided by
    the side of a border its value lies on."""
    g = y.double().unflatten(-1, (-1, 32))
    a = g.abs().amax(-1, keepdim=True)
    q = torch.round(g * 7 / torch.where(a > 0, a, 1.0))
    return (q + 8).to(torch.uint8).flatten(-2), (a.squeeze(-1) / 7).half()


def _values(codes, scales):
    return ((codes.float() - 8).unflatten(-1, (-1, 32)) * scales.float().unsqueeze(-1)).flatten(-2)


def _pack_blocks(kc, ks, vc, vs):
    """Codes [B, 16, hd] and scales [B, 16, hd / 32] of whole 16-position blocks -> bytes [B, block]."""
    B, _, hd = kc.shape
    ng = hd // 32
    k = kc.view(B, 4, 2, 2, ng, 4, 4, 2)                     # position a, e, o; group, octet c, byte, nibble
    k = k[..., 0] | (k[..., 1] << 4)
    k = k.permute(0, 2, 1, 3, 5, 4, 6).reshape(B, -1)        # e, a, o, c, group, byte
    v = vc.view(B, 4, 2, 2, ng, 2, 2, 8)                     # a, e, o; group, octet pair, octet, n
    v = v[..., 0, :] | (v[..., 1, :] << 4)                   # a, e, o, group, pair, n
    order = (0, 2, 1, 6, 3, 4, 5) if hd == 128 else (0, 1, 6, 2, 3, 4, 5)
    v = v.permute(*order).reshape(B, -1)
    f16 = lambda s: s.contiguous().view(B, -1).view(torch.uint8)  # noqa: E731
    return torch.cat([k, f16(ks), v, f16(vs)], 1)


def _unpack_blocks(b, hd):
    """bytes [B, block] -> K and V values f32 [B, 16, hd]."""
    B, ng = b.shape[0], hd // 32
    nk, ns = 8 * hd, 32 * ng
    k, ks, v, vs = b.split([nk, ns, nk, ns], 1)
    k = k.reshape(B, 2, 4, 2, 4, ng, 4).permute(0, 2, 1, 3, 5, 4, 6)      # a, e, o, group, c, byte
    kc = torch.stack([k & 15, k >> 4], -1).reshape(B, 16, hd)
    if hd == 128:
        v = v.reshape(B, 2, 4, 8, 2, ng, 2).permute(0, 2, 1, 4, 5, 6, 3)  # from e, a, n, o, group, pair
    else:
        v = v.reshape(B, 4, 8, 2, 2, ng, 2).permute(0, 1, 3, 4, 5, 6, 2)  # from a, n, e, o, group, pair
    vc = torch.stack([v & 15, v >> 4], -2).reshape(B, 16, hd)             # octet before n
    f16 = lambda s: s.contiguous().view(torch.float16).view(B, 16, ng)    # noqa: E731
    return _values(kc, f16(ks)), _values(vc, f16(vs))


def _row_places(tb, hd):
    """Byte offsets of a block position's K codes [.., hd / 2], K scales, V codes, V scales, as bytes (each
    scale two), for positions-in-block tb [n]: the bytes' order is that of _row_bytes."""
    dev, ng = tb.device, hd // 32
    a, e, o = tb >> 2, (tb >> 1) & 1, tb & 1
    ar = lambda n: torch.arange(n, device=dev)  # noqa: E731
    c, g, by = torch.meshgrid(ar(4), ar(ng), ar(4), indexing="ij")
    k = (e * 8 + a * 2 + o)[:, None] * (hd // 2) + (c * 4 * ng + g * 4 + by).reshape(-1)[None]
    ks = 8 * hd + tb[:, None] * (2 * ng) + ar(2 * ng)[None]
    v0 = 8 * hd + 32 * ng
    n, b = torch.meshgrid(ar(8), ar(2 * ng), indexing="ij")
    n, b = n.reshape(-1)[None], b.reshape(-1)[None]
    if hd == 128:
        v = v0 + e[:, None] * 512 + a[:, None] * 128 + n * 16 + o[:, None] * 8 + b
    else:
        v = v0 + a[:, None] * 128 + n * 16 + (tb & 3)[:, None] * 4 + b
    vs = v0 + 8 * hd + tb[:, None] * (2 * ng) + ar(2 * ng)[None]
    return torch.cat([k, ks, v, vs], 1)


def _row_bytes(kc, ks, vc, vs):
    """Codes [n, kv, hd], scales [n, kv, hd / 32] -> bytes [n, kv, hd * 9 / 8] in the order of _row_places."""
    n, kv, hd = kc.shape
    ng = hd // 32
    k = kc.view(n, kv, ng, 4, 4, 2)
    k = (k[..., 0] | (k[..., 1] << 4)).permute(0, 1, 3, 2, 4).reshape(n, kv, -1)
    v = vc.view(n, kv, ng, 2, 2, 8)
    v = (v[..., 0, :] | (v[..., 1, :] << 4)).permute(0, 1, 4, 2, 3).reshape(n, kv, -1)
    f16 = lambda s: s.contiguous().view(torch.uint8)  # noqa: E731
    return torch.cat([k, f16(ks), v, f16(vs)], 2)


def _page_bytes(kv, hd, page):
    return kv * page * hd * 9 // 8


def _pack_weights(codes, d):
    """Q4_0 codes uint8 [rows, cols] and scales f16 [rows, cols / 32] -> (blocks [rows, cols / 32 * 18], tiles).
    Tiles: [ceil(rows / 16)][ceil(cols / 128)] of 1152 bytes: for half h (rows h * 8 + r) and lane (r, c) 16
    bytes, the 8 codes 8c .. 8c + 7 of each of the four groups, then f16 scales [16][4]; padding has scale 0."""
    rows, cols = codes.shape
    blk = codes.view(rows, cols // 32, 2, 16)
    blocks = torch.cat([d.view(torch.uint8).view(rows, -1, 2), blk[:, :, 0] | (blk[:, :, 1] << 4)], 2)
    rt, st = -(-rows // 16), -(-cols // 128)
    pc = torch.full((rt * 16, st * 128), 8, dtype=torch.uint8, device=codes.device)
    pc[:rows, :cols] = codes
    pd = torch.zeros(rt * 16, st * 4, dtype=torch.float16, device=codes.device)
    pd[:rows, : cols // 32] = d
    t = pc.view(rt, 2, 8, st, 4, 4, 4, 2)  # tile, half, r, strip, group, c, byte, nibble
    t = (t[..., 0] | (t[..., 1] << 4)).permute(0, 3, 1, 2, 5, 4, 6).reshape(rt, st, 1024)
    s = pd.view(rt, 16, st, 4).permute(0, 2, 1, 3).contiguous().view(torch.uint8).view(rt, st, 128)
    return blocks.reshape(rows, -1).contiguous(), torch.cat([t, s], 2).contiguous()


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _page_table(g, n_seq, per_seq):
    """Pages of the sequences in no order, and how many the pool has."""
    n = n_seq * per_seq
    t = torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(n_seq, per_seq)
    return t.contiguous(), n


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op == "append":
        n, n_seq, hd, page = case["n"], case["n_seq"], case["head_dim"], case["page"]
        qw, kvw = case["heads"] * hd, case["kv_heads"] * hd
        # the fused projections' rows: q, k (a few strong channels, as keys have), v
        qkv = _randn(g, n, qw + 2 * kvw)
        strong = torch.ones(qw + 2 * kvw, device="cuda")
        strong[qw:qw + kvw:17] = 6.0
        qkv *= strong
        r = random.Random(seed)
        starts = [r.randint(0, case["history"]) for _ in range(n_seq)]
        counts = [n // n_seq + (s < n % n_seq) for s in range(n_seq)]
        seqs = torch.repeat_interleave(torch.arange(n_seq), torch.tensor(counts))
        first = torch.tensor([sum(counts[:s]) for s in range(n_seq)])
        pos = torch.tensor(starts)[seqs] + torch.arange(n) - first[seqs]
        top = case["history"] + max(counts) + 1
        per_seq = -(-top // page)
        # a sequence's first pages are not touched here: the pool holds the pages from the first written one on
        table = torch.full((n_seq, per_seq), -1, dtype=torch.int32)
        used = torch.unique(seqs * per_seq + pos // page)
        order = torch.randperm(len(used), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        table.view(-1)[used] = order
        angle = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
            torch.tensor(THETA, device="cuda", dtype=torch.float64), -torch.arange(hd // 2, device="cuda", dtype=torch.float64) / (hd // 2))
        st |= {"qkv": qkv, "positions": pos.to(torch.int32).cuda(), "seqs": seqs.to(torch.int32).cuda(),
               "page_table": table.cuda(), "rope": torch.stack([angle.cos(), angle.sin()], -1).float().contiguous(),
               "pages": torch.zeros(len(used), _page_bytes(case["kv_heads"], hd, page), dtype=torch.uint8, device="cuda"),
               "q_out": torch.empty(n, qw, device="cuda"), "k_out": torch.empty(n, kvw, device="cuda"),
               "v_out": torch.empty(n, kvw, device="cuda")}
    elif op == "attend":
        n_seq, hd, page, kv = case["n_seq"], case["head_dim"], case["page"], case["kv_heads"]
        lens, queries = _lens(case), _queries(case)
        per_seq = max(1, -(-max(lens) // page))
        table, n_pages = _page_table(g, n_seq, per_seq)
        blocks = n_pages * kv * (page // 16)
        pages = torch.empty(blocks, 18 * hd, dtype=torch.uint8, device="cuda")
        gain = torch.ones(hd, device="cuda")
        gain[::17] = 4.0  # strong key channels
        step = 1 << 16
        for b in range(0, blocks, step):
            m = min(step, blocks - b)
            kc, ks = _quantise(_randn(g, m, 16, hd) * gain)
            vc, vs = _quantise(_randn(g, m, 16, hd))
            pages[b:b + m] = _pack_blocks(kc, ks, vc, vs)
        start = [0]
        for q in queries:
            start.append(start[-1] + q)
        n = start[-1]
        st |= {"pages": pages.view(n_pages, -1), "page_table": table, "lens": torch.tensor(lens, dtype=torch.int32).cuda(),
               "q_start": torch.tensor(start, dtype=torch.int32).cuda() if case["queries"] > 1 else None,
               "max_len": max(lens), "max_queries": max(queries), "n": n,
               "q": _randn(g, n, case["heads"] * hd) * 1.2, "out": torch.empty(n, case["heads"] * hd, device="cuda")}
    elif op == "matvec":
        rows, cols = case["rows"], case["cols"]
        w = _randn(g, rows, cols).view(rows, -1, 32) * 0.02
        at = w.abs().argmax(-1, keepdim=True)
        d = (w.gather(-1, at) / -8).half()  # the largest weight takes code 0
        inv = torch.where(d != 0, 1 / d.float(), torch.zeros((), device="cuda"))
        codes = (torch.round(w * inv) + 8).clamp(0, 15).to(torch.uint8).view(rows, cols)
        del w, at
        blocks, tiles = _pack_weights(codes, d.squeeze(-1).contiguous())
        x = _randn(g, case["n"], cols)
        x[:, ::97] *= 20.0  # activations have a few large channels
        st |= {"w_blocks": blocks, "w_tiles": tiles, "x": x, "y": torch.empty(case["n"], rows, device="cuda")}
    else:
        n, v, k = case["n"], case["vocab"], case["top_k"]
        x = _randn(g, n, v) * 2.0
        m = min(8, v)
        peaks = torch.randint(0, v, (n, m), generator=g, device="cuda")
        x.scatter_add_(1, peaks, 6.0 + 6.0 * torch.rand(n, m, generator=g, device="cuda"))
        if case["masked"]:  # a grammar's mask: most tokens not allowed, in one row none
            x.masked_fill_(torch.rand(n, v, generator=g, device="cuda") < 0.7, -math.inf)
            x[n // 2] = -math.inf
        st |= {"logits": x, "targets": peaks[:, 0].to(torch.int32).contiguous(),
               "logprob": torch.empty(n, device="cuda"), "entropy": torch.empty(n, device="cuda"),
               "top_ids": torch.empty(n, k, dtype=torch.int32, device="cuda"),
               "top_logprobs": torch.empty(n, k, device="cuda")}
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _own[st["case"]["op"]](st)
    return _plain[st["case"]["op"]](st)


def _rotate(x, cos, sin):
    half = x.shape[-1] // 2
    x0, x1 = x[..., :half], x[..., half:]
    return torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)


def _plain_append(st):
    c = st["case"]
    n, hd, kv, page = c["n"], c["head_dim"], c["kv_heads"], c["page"]
    qw, kvw = c["heads"] * hd, kv * hd
    q, k, v = st["qkv"].split([qw, kvw, kvw], 1)
    pos, seqs = st["positions"].long(), st["seqs"].long()
    cs = st["rope"][pos][:, None]
    q = _rotate(q.view(n, -1, hd), cs[..., 0], cs[..., 1])
    kc, ks = _quantise(_rotate(k.view(n, kv, hd).double(), cs[..., 0], cs[..., 1]))
    vc, vs = _quantise(v.reshape(n, kv, hd))
    place = _row_places(pos % 16, hd)[:, None] + ((pos % page) // 16 * (18 * hd))[:, None, None]
    place = place + (torch.arange(kv, device=pos.device) * (page * hd * 9 // 8))[None, :, None]
    place = place + (st["page_table"][seqs, pos // page].long() * st["pages"].shape[1])[:, None, None]
    st["pages"].view(-1)[place] = _row_bytes(kc, ks, vc, vs)
    return {"q": q.reshape(n, qw), "k": _values(kc, ks).reshape(n, kvw), "v": _values(vc, vs).reshape(n, kvw)}


def _plain_attend(st):
    c = st["case"]
    S, hd, kv, page, heads = c["n_seq"], c["head_dim"], c["kv_heads"], c["page"], c["heads"]
    G, L, Q = heads // kv, st["max_len"], st["max_queries"]
    if L == 0:
        return torch.zeros_like(st["q"])
    got = st["pages"].view(-1, kv, page // 16, 18 * hd)[st["page_table"].long()]  # [S, pages, kv, blocks, bytes]
    got = got.transpose(1, 2).reshape(-1, 18 * hd)
    k, v = _unpack_blocks(got, hd)
    k, v = k.view(S, kv, -1, hd), v.view(S, kv, -1, hd)
    T = k.shape[2]
    start = st["q_start"].long() if st["q_start"] is not None else torch.arange(S + 1, device=k.device)
    nq = start[1:] - start[:-1]
    i = torch.arange(Q, device=k.device)
    row = (start[:-1, None] + torch.minimum(i[None], nq[:, None] - 1))       # [S, Q]
    q = st["q"][row].view(S, Q, kv, G, hd).permute(0, 2, 1, 3, 4).reshape(S, kv, Q * G, hd)
    s = q @ k.transpose(-1, -2) * (1.0 / math.sqrt(hd))
    last = st["lens"].long()[:, None] - nq[:, None] + i[None]                # a query's own position
    seen = torch.arange(T, device=k.device)[None, None] <= last[:, :, None]  # [S, Q, T]
    seen = seen.repeat_interleave(G, 1)[:, None]
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(l == 0, torch.ones_like(l), l)
    o = o.view(S, kv, Q, G, hd).permute(0, 2, 1, 3, 4).reshape(S, Q, heads * hd)
    return o[i[None] < nq[:, None]]


def _plain_matvec(st):
    rows, cols = st["case"]["rows"], st["case"]["cols"]
    b = st["w_blocks"].view(rows, cols // 32, 18)
    d = b[:, :, :2].contiguous().view(torch.float16).float()
    w = torch.cat([b[:, :, 2:] & 15, b[:, :, 2:] >> 4], 2).float() - 8
    return st["x"] @ (w * d).view(rows, cols).T


def _plain_logprobs(st):
    x, k = st["logits"], st["case"]["top_k"]
    n, v = x.shape
    x = torch.where(x == x, x, torch.full_like(x, -math.inf))
    m = x.amax(1, keepdim=True)
    some = m > -math.inf
    d = torch.where(x > -math.inf, x - torch.where(some, m, torch.zeros_like(m)), torch.full_like(x, -math.inf))
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    t = torch.where(e > 0, e * d, torch.zeros_like(d)).sum(1, keepdim=True)
    log_s = torch.log(s)
    none = torch.full_like(m, -math.inf)
    at = st["targets"].long()[:, None]
    logprob = torch.where(some, d.gather(1, at) - log_s, none)
    entropy = torch.where(some, log_s - t / s, torch.zeros_like(m))
    if k == 0:
        return {"logprob": logprob[:, 0], "entropy": entropy[:, 0]}
    # descending by value, equal values by ascending index: one whole-number key
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits)
    key = key * (1 << 31) + ((1 << 31) - 1 - torch.arange(v, device=x.device))
    ids = torch.topk(key, min(k, v), 1).indices
    lp = torch.where(some, d.gather(1, ids) - log_s, none)
    ids = torch.where(lp > -math.inf, ids, torch.full_like(ids, -1))
    pad = k - ids.shape[1]
    ids = torch.nn.functional.pad(ids, (0, pad), value=-1)
    lp = torch.nn.functional.pad(lp, (0, pad), value=-math.inf)
    return {"logprob": logprob[:, 0], "entropy": entropy[:, 0], "top_ids": ids.int(), "top_logprobs": lp}


_plain = {"append": _plain_append, "attend": _plain_attend, "matvec": _plain_matvec, "logprobs": _plain_logprobs}


# ------------------------------------------------------------------ the library's calls

def _ops():
    import token_quantized_decode_gb300 as tqd
    return tqd.ops


def _cache(st, ops):
    """The cache's descriptor and the scratch a program keeps beside it."""
    if "cache" not in st:
        c = st["case"]
        st["cache"] = ops.kv_q4(st["pages"], st["page_table"], c["kv_heads"], c["head_dim"], c["page"])
        if c["op"] == "attend":
            st["scratch"] = torch.empty(ops.tqd_attention_q4_scratch_bytes(c["head_dim"]), dtype=torch.uint8, device="cuda")
    return st["cache"]


def _own_append(st):
    ops, c = _ops(), st["case"]
    cache = _cache(st, ops)
    qw, kvw = c["heads"] * c["head_dim"], c["kv_heads"] * c["head_dim"]
    q, k, v = st["qkv"].split([qw, kvw, kvw], 1)
    ops.tqd_op_kv_append_q4(cache, k, v, st["positions"], st["seqs"], st["rope"], q, st["q_out"])
    ops.tqd_op_kv_read_q4(cache, st["positions"], st["seqs"], st["k_out"], st["v_out"])
    return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}


def _own_attend(st):
    ops = _ops()
    cache = _cache(st, ops)
    ops.tqd_op_attention_q4(cache, st["q"], st["lens"], st["q_start"], st["out"], st["scratch"])
    return st["out"]


def _own_matvec(st):
    ops, c = _ops(), st["case"]
    ops.tqd_op_q4_0_matvec(st["w_tiles"], c["rows"], c["cols"], st["x"], st["y"])
    return st["y"]


def _own_logprobs(st):
    ops = _ops()
    k = st["case"]["top_k"]
    if "scratch" not in st:
        n, v = st["logits"].shape
        st["scratch"] = torch.empty(ops.tqd_logprobs_scratch_bytes(n, v, k), dtype=torch.uint8, device="cuda")
    ops.tqd_op_logprobs(st["logits"], st["targets"], st["logprob"], st["entropy"], st["top_ids"], st["top_logprobs"],
                        st["scratch"])
    out = {"logprob": st["logprob"], "entropy": st["entropy"]}
    return out | ({"top_ids": st["top_ids"], "top_logprobs": st["top_logprobs"]} if k else {})


_own = {"append": _own_append, "attend": _own_attend, "matvec": _own_matvec, "logprobs": _own_logprobs}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    return _exact[case["op"]](prepare(case, seed))


def _exact_append(st):
    c = st["case"]
    n, hd, kv, heads = c["n"], c["head_dim"], c["kv_heads"], c["heads"]
    x = st["qkv"].double().view(n, heads + 2 * kv, hd)
    cs = st["rope"].double()[st["positions"].long()]
    z = torch.complex(cs[:, None, :, 0], cs[:, None, :, 1])
    r = torch.complex(x[:, : heads + kv, : hd // 2].contiguous(), x[:, : heads + kv, hd // 2:].contiguous()) * z
    r = torch.cat([r.real, r.imag], 2)
    def held(y):
        b = y.reshape(-1, 32)
        most = b.abs().max(1).values[:, None]
        q = torch.round(7 * b / torch.where(most > 0, most, torch.ones_like(most)))
        return (q * (most / 7).half().double()).view(n, kv * hd)
    return {"q": r[:, :heads].reshape(n, -1), "k": held(r[:, heads:]), "v": held(x[:, heads + kv:])}


def _exact_attend(st):
    c = st["case"]
    hd, kv, page, heads = c["head_dim"], c["kv_heads"], c["page"], c["heads"]
    G, ng, out = heads // kv, hd // 32, []
    dev = st["q"].device
    d = torch.arange(hd, device=dev)
    g, j = d // 32, d % 32
    pool, q0 = st["pages"], 0
    per_head = page * hd * 9 // 8
    block = 18 * hd
    for s, (length, nq) in enumerate(zip(_lens(c), _queries(c))):
        q = st["q"][q0:q0 + nq].double().view(nq, heads, hd)
        q0 += nq
        o = torch.zeros(nq, heads, hd, dtype=torch.float64, device=dev)
        if length:
            t = torch.arange(length, device=dev)
            b = t % 16
            base = (t % page) // 16 * block
            krow = ((b >> 1) & 1) * 8 + (b >> 2) * 2 + (b & 1)
            kat = base[:, None] + krow[:, None] * (hd // 2) + (j // 8 * 4 * ng + g * 4 + j % 8 // 2)[None]
            ksat = base[:, None] + 8 * hd + 2 * (b[:, None] * ng + torch.arange(ng, device=dev)[None])
            v0, nib = 8 * hd + 32 * ng, 4 * g + j // 8
            if hd == 128:
                vat = v0 + (b % 4 // 2 * 512 + b // 4 * 128 + b % 2 * 8)[:, None] + (d % 8 * 16 + nib // 2)[None]
            else:
                vat = v0 + (b // 4 * 128 + b % 4 * 4)[:, None] + (d % 8 * 16 + nib // 2)[None]
            vat = vat + base[:, None]
            vsat = ksat + v0
            of_page = st["page_table"][s].long()[t // page]
            last = length - nq + torch.arange(nq, device=dev)
            hidden = t[None] > last[:, None]
            for h in range(kv):
                head = lambda at: pool[of_page[:, None], h * per_head + at]  # noqa: E731
                def scale(at):
                    lo, hi = head(at).int(), head(at + 1).int()
                    return (lo | (hi << 8)).to(torch.int16).view(torch.float16).double().repeat_interleave(32, 1)
                K = (((head(kat).int() >> (4 * (j % 2))[None]) & 15) - 8).double() * scale(ksat)
                V = (((head(vat).int() >> (4 * (nib % 2))[None]) & 15) - 8).double() * scale(vsat)
                sc = torch.einsum("qgd,td->qgt", q[:, h * G:(h + 1) * G], K) / math.sqrt(hd)
                sc = sc.masked_fill(hidden[:, None], -math.inf)
                top = sc.max(-1, keepdim=True).values
                w = torch.exp(sc - top.clamp(min=-1e300))
                sums = w.sum(-1, keepdim=True)
                o[:, h * G:(h + 1) * G] = torch.einsum("qgt,td->qgd", w, V) / torch.where(sums > 0, sums, torch.ones_like(sums))
        out.append(o.view(nq, -1))
    return torch.cat(out)


def _exact_matvec(st):
    rows, cols = st["case"]["rows"], st["case"]["cols"]
    x, out = st["x"].double(), []
    for r in range(0, rows, 8192):  # rows at a time: 64-bit weights take room
        b = st["w_blocks"][r:r + 8192].view(-1, 18).int()
        d = (b[:, 0] | (b[:, 1] << 8)).to(torch.int16).view(torch.float16).double()
        at = torch.arange(32, device=b.device)
        w = ((b[:, 2 + at % 16] >> (4 * (at // 16))[None]) & 15).double() - 8
        out.append((w * d[:, None]).view(-1, cols) @ x.T)
    return torch.cat(out).T.contiguous()


def _exact_logprobs(st):
    k, none = st["case"]["top_k"], -math.inf
    lp, ent, ids, tops = [], [], [], []
    for x, target in zip(st["logits"].split(256), st["targets"].split(256)):
        x = x.double()
        x = torch.where(torch.isnan(x), torch.full_like(x, none), x)
        lse = torch.logsumexp(x, 1, keepdim=True)
        y = torch.where(x == none, torch.full_like(x, none), x - lse)  # log p
        lp.append(y.gather(1, target.long()[:, None])[:, 0])
        p = torch.exp(y)
        ent.append(-(torch.where(p > 0, p * y, torch.zeros_like(y))).sum(1))
        if k:
            order = torch.sort(x, stable=True, dim=1, descending=True)
            i = order.indices[:, :k]
            z = y.gather(1, i)
            i = torch.where(z == none, torch.full_like(i, -1), i)
            pad = k - i.shape[1]
            ids.append(torch.nn.functional.pad(i, (0, pad), value=-1).int())
            tops.append(torch.nn.functional.pad(z, (0, pad), value=none))
    out = {"logprob": torch.cat(lp), "entropy": torch.cat(ent)}
    return out | ({"top_ids": torch.cat(ids), "top_logprobs": torch.cat(tops)} if k else {})


_exact = {"append": _exact_append, "attend": _exact_attend, "matvec": _exact_matvec, "logprobs": _exact_logprobs}
