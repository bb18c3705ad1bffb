"""Measured cases of drafting on the microscaled paged cache: appending rows with the rotation of their positions on the
way, the tree of a draft, attention over a tree, and keeping the path that was accepted.

The cache holds keys and values in pages of 16 tokens, as E2M1 (4-bit) or E4M3 (8-bit) elements with one power-of-two
scale per token, head and 32 channels. A page of one head is one record:
  key codes      [16 tokens][D bits_k / 8 bytes], channel order, low nibble first
  value codes    [4 token groups][16 lanes][4 tokens][D / 16 channels]: lane n holds channels n D / 16 ...
  key scales     [16 tokens][D / 32 bytes]
  value scales   [4 token groups][D / 32 blocks][4 tokens]
A scale byte s stands for 2^(s - 127), 255 for NaN.

A sequence's rows in a call are its last tokens. Of a draft, row i names its parent among the sequence's rows (-1: it
follows the last token before the draft); bit j of its mask says that it sees row j, itself and its ancestors.
"""
import math
import random

import torch

own = False

DEV = "cuda"
PAGE = 16
TOP = {4: 6.0, 8: 448.0}     # largest element
OVER = {4: 7.0, 8: 464.0}    # from here on an element would round past the largest
BYTE_TOP = {4: 252, 8: 246}  # largest scale byte whose largest element is finite in bf16
BYTE_LOW = 15                # smallest: every element stays a normal bf16 number


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # one layer of a served batch's decode step: a token a sequence rotated, written and read back (smallest calls)
        {"name": "rope step 64", "op": "rope", "layers": 1, "H": 8, "G": 4, "D": 128, "dtype": "bf16", "bk": 4, "bv": 4,
         "n": 64, "rows_min": 1, "rows_max": 1, "past_min": 100, "past_max": 4000, "fused": True, "pattern": 21,
         "style": "half", "rot": 128, "theta": 5e5, "axes": 1, "given": False},
        # one layer of a ragged batch of prompts, slices of one projection, keys in 8 bits, positions up to 100000
        {"name": "rope prompts k8v4", "op": "rope", "layers": 1, "H": 8, "G": 4, "D": 128, "dtype": "bf16", "bk": 8, "bv": 4,
         "n": 16, "rows_min": 100, "rows_max": 2000, "past_min": 0, "past_max": 300, "fused": True, "pattern": 22,
         "style": "half", "rot": 128, "theta": 5e5, "axes": 1, "given": True},
        # a video's patches among text: time, height and width, fp32, short heads of which half is rotated
        {"name": "rope video fp32 d64", "op": "rope", "layers": 1, "H": 3, "G": 2, "D": 64, "dtype": "fp32", "bk": 8, "bv": 8,
         "n": 2, "rows_min": 1500, "rows_max": 2700, "past_min": 5, "past_max": 50, "fused": True, "pattern": 23,
         "style": "half", "rot": 32, "theta": 1e4, "axes": 3, "given": True},
        # a whole cache of keys without rotation [L, H, T, D] brought into pages, neighbouring channels paired
        {"name": "rope cache 32x8x4096", "op": "rope", "layers": 32, "H": 8, "G": 0, "D": 128, "dtype": "bf16", "bk": 4, "bv": 4,
         "n": 1, "rows_min": 4096, "rows_max": 4096, "past_min": 0, "past_max": 0, "fused": False, "pattern": 24,
         "style": "interleaved", "rot": 128, "theta": 5e5, "axes": 1, "given": False},
        # the trees of a served batch, once a step
        {"name": "tree 64 x 60", "op": "tree", "n": 64, "rows_min": 20, "rows_max": 60, "past_min": 100, "past_max": 4000, "pattern": 25},
        # long drafts (a copied passage with branches), many words a mask
        {"name": "tree 16 x 1000", "op": "tree", "n": 16, "rows_min": 300, "rows_max": 1000, "past_min": 0, "past_max": 4000, "pattern": 26},
        # a short draft of one conversation, fp32, short heads: latency
        {"name": "attn tree 1 x 7 fp32 d64", "op": "attn", "H": 3, "G": 2, "D": 64, "dtype": "fp32", "bk": 8, "bv": 8,
         "n": 1, "rows_min": 7, "rows_max": 7, "past_min": 501, "past_max": 501, "pattern": 27},
        # a served batch, ragged lengths of the framework's paged workload, up to 16 drafted tokens a sequence
        {"name": "attn tree 64 x 16 ragged", "op": "attn", "H": 8, "G": 4, "D": 128, "dtype": "bf16", "bk": 4, "bv": 4,
         "n": 64, "rows_min": 5, "rows_max": 16, "past_min": 511, "past_max": 8175, "pattern": 28},
        # large trees, 64 query heads, keys in 8 bits: matrix products bound it
        {"name": "attn tree 16 x 60 k8v4", "op": "attn", "H": 8, "G": 8, "D": 128, "dtype": "bf16", "bk": 8, "bv": 4,
         "n": 16, "rows_min": 40, "rows_max": 60, "past_min": 3000, "past_max": 4036, "pattern": 29},
        # drafts of a batch behind one system prompt
        {"name": "attn tree 32 x 25 shared", "op": "attn", "H": 8, "G": 4, "D": 128, "dtype": "bf16", "bk": 4, "bv": 4,
         "n": 32, "rows_min": 10, "rows_max": 25, "past_min": 8192, "past_max": 8700, "prefix": 512, "pattern": 30},
        # the end of a step: drafts of all layers written, the accepted path of each kept, the last tokens read
        {"name": "keep 64 x 8", "op": "keep", "layers": 32, "H": 8, "D": 128, "dtype": "bf16", "bk": 4, "bv": 4,
         "n": 64, "rows_min": 4, "rows_max": 8, "past_min": 100, "past_max": 1000, "pattern": 31},
        # one long draft, 8 bits, fp32, short heads
        {"name": "keep 1 x 300 fp32 d64", "op": "keep", "layers": 2, "H": 5, "D": 64, "dtype": "fp32", "bk": 8, "bv": 8,
         "n": 1, "rows_min": 300, "rows_max": 300, "past_min": 777, "past_max": 777, "pattern": 32},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "attn", "attn", "attn", "keep"])
    pattern = rng.randrange(1 << 30)
    if op == "tree":
        n, hi = _log(rng, 1, 128), _log(rng, 1, 1000)
        return {"op": op, "n": n, "rows_min": max(1, hi // rng.randint(1, 5)), "rows_max": hi, "past_min": 0,
                "past_max": _log(rng, 1, 10000), "pattern": pattern}
    c = {"op": op, "H": rng.randint(1, 8), "D": rng.choice([64, 128, 128]), "dtype": rng.choice(["bf16", "bf16", "fp32"]),
         "bk": rng.choice([4, 8]), "bv": rng.choice([4, 8]), "pattern": pattern}
    if op == "rope":
        n = _log(rng, 1, 128)
        hi = _log(rng, 1, max(1, min(8192, 30000 // n)))
        layers = rng.choice([1, 1, 2, 4]) if n == 1 else 1
        axes = rng.choice([1, 1, 2, 3, 4])
        return {**c, "layers": layers, "G": rng.choice([0, 1, 2, 4, 8]) if layers == 1 else 0, "n": n,
                "rows_min": max(1, hi // rng.randint(1, 8)), "rows_max": hi, "past_min": 0, "past_max": rng.randint(0, 200),
                "fused": layers == 1 and rng.random() < 0.7, "style": rng.choice(["half", "interleaved"]),
                "rot": rng.choice([c["D"], c["D"], c["D"] // 2, 16 * rng.randint(1, c["D"] // 16)]),
                "theta": rng.choice([1e4, 5e5]), "axes": axes, "given": axes > 1 or rng.random() < 0.5}
    if op == "keep":
        n, layers = _log(rng, 1, 64), rng.randint(1, 8)
        hi = _log(rng, 1, max(1, min(300, 2000 // n)))
        return {**c, "layers": layers, "n": n, "rows_min": max(1, hi // rng.randint(1, 4)), "rows_max": hi, "past_min": 16, "past_max": 500}
    G = rng.choice([1, 2, 3, 4, 6, 8, 16])
    n, hi = _log(rng, 1, 64), _log(rng, 1, 100)
    most = _log(rng, 8, max(8, min(65536, 200000 // n)))
    least = most // rng.randint(1, 10)
    if rng.random() < 0.3:  # now and then a sequence, or its draft, is still inside the prefix
        pages = _log(rng, 1, 512)
        least, most = min(least, 300), min(most, 1500) + PAGE * pages
        least += PAGE * pages if rng.random() < 0.9 else 0
        least = min(least, most)
        c["prefix"] = pages
    while n > 1 and n * hi * G * c["H"] * (most + hi) > 2.5e8:
        n -= 1
    while hi > 1 and n * hi * G * c["H"] * (most + hi) > 2.5e8:
        hi -= 1 + hi // 16
    return {**c, "G": G, "n": n, "rows_min": max(1, hi // rng.randint(1, 3)), "rows_max": hi, "past_min": least, "past_max": most}


def _lens(case):
    """(rows, length after them) of each sequence: whole numbers that the case fixes."""
    r = random.Random(case["pattern"])
    rows = [r.randint(case["rows_min"], case["rows_max"]) for _ in range(case["n"])]
    past = [r.randint(case["past_min"], case["past_max"]) for _ in range(case["n"])]
    return rows, [a + b for a, b in zip(rows, past)]


def _record(case):
    D = case["D"]
    kc, vc, sc = PAGE * D * case["bk"] // 8, PAGE * D * case["bv"] // 8, PAGE * D // 32
    return kc, vc, sc, kc + vc + 2 * sc


TAIL = 8  # tokens of each sequence that are read after keeping


def work(case):
    rows, lens = _lens(case)
    t = sum(rows)
    words = -(-case["rows_max"] // 32)
    if case["op"] == "tree":
        return {"bytes": t * (8 + 4 * words) + 8 * case["n"], "flops": 0}
    H, D = case["H"], case["D"]
    e = 2 if case["dtype"] == "bf16" else 4
    token = D * (case["bk"] + case["bv"]) // 8 + D // 16  # bytes of a cached token of one head
    if case["op"] == "rope":
        v, q = t * H * case["layers"], t * H * case["G"]
        return {"bytes": v * 2 * (2 * D * e + token) + q * 2 * D * e + (4 * t * case["axes"] if case["given"] else 0),
                "flops": v * (2 * D * 4 + 3 * case["rot"]) + q * 3 * case["rot"]}
    if case["op"] == "keep":  # drafts in, codes out; the path's codes (about three tokens) moved; the tail read
        v, x = t * H * case["layers"], case["n"] * H * case["layers"]
        return {"bytes": v * (2 * D * e + token) + x * (3 * 2 * token + TAIL * (token + 2 * D * e)), "flops": v * 2 * D * 4}
    p = PAGE * case.get("prefix", 0)
    tokens = p + sum(max(0, ln - p) for ln in lens)
    q = t * H * case["G"]
    seen = sum(n * (ln - n + 1) for n, ln in zip(rows, lens))
    return {"bytes": tokens * H * token + q * (2 * D * e + 4) + 4 * words * t, "flops": 4 * D * H * case["G"] * seen}


# --------------------------------------------------------------------- inputs

def _power(e, dtype=torch.float32):
    """2^e of whole numbers e in [-126, 127], exactly."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32).to(dtype)


def _quantise(x, b):
    """(elements as numbers, scale bytes) of x [..., D] in blocks of 32: in x's own type, fp32 or fp64."""
    y = x.unflatten(-1, (-1, 32))
    a = y.abs().amax(-1, keepdim=True)
    m, k = torch.frexp(a)
    lead, base = (0.875, 2) if b == 4 else (0.90625, 8)
    s = (k.to(torch.int32) - 1 - base + (m >= lead) + 127).clamp(BYTE_LOW, BYTE_TOP[b])
    s = torch.where(a > 0, s, torch.full_like(s, BYTE_LOW))
    u = (y * _power(127 - s, y.dtype)).clamp(-TOP[b], TOP[b])
    low, bits = (0, 1) if b == 4 else (-6, 3)
    step = _power((torch.frexp(u)[1].to(torch.int32) - 1).clamp_min(low) - bits, y.dtype)
    u = torch.round(u / step) * step
    u = torch.where(y == 0, torch.zeros_like(u), u)
    fine = torch.isfinite(a)
    return torch.where(fine, u, torch.zeros_like(u)).float(), torch.where(fine, s, torch.full_like(s, 255))


def _values(u, s, dtype):
    """What elements u [..., nb, 32] under scale bytes s [..., nb, 1] stand for."""
    x = u * _power(s.clamp(max=254) - 127)
    return torch.where(s == 255, torch.full_like(x, float("nan")), x).flatten(-2).to(dtype)


def _codes(u, b):
    """Element numbers -> 8-bit codes (4 bits: one code a byte)."""
    if b == 8:
        return u.to(torch.float8_e4m3fn).view(torch.uint8)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=u.device)
    return (torch.bucketize(u.abs(), grid) + 8 * (u < 0)).to(torch.uint8)


def _pages(k, v, case):
    """k, v [pages, H, 16, D] fp32 -> records [pages, H, record] uint8."""
    P, H, _, D = k.shape
    out = []
    for x, b, key in ((k, case["bk"], True), (v, case["bv"], False)):
        u, s = _quantise(x, b)
        c = _codes(u.flatten(-2), b)
        if not key:
            c = c.view(P, H, 4, 4, 16, D // 16).transpose(3, 4).contiguous()
        if b == 4:
            c = c.unflatten(-1, (-1, 2))
            c = c[..., 0] | (c[..., 1] << 4)
        s = s.view(P, H, 16, D // 32).to(torch.uint8)
        if not key:
            s = s.view(P, H, 4, 4, D // 32).transpose(3, 4)
        out.append((c.reshape(P, H, -1), s.reshape(P, H, -1)))
    return torch.cat([out[0][0], out[1][0], out[0][1], out[1][1]], -1)


def _axis(case):
    """Axis of each rotated pair: two stretches, three in turn, four stretches."""
    p = case["rot"] // 2
    return [j % 3 if case["axes"] == 3 else j * case["axes"] // p for j in range(p)]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, lens = _lens(case)
    n, t, most = case["n"], sum(rows), max(rows)
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    i32 = dict(dtype=torch.int32, device=DEV)
    st = {"case": case, "rows": t, "max_rows": most, "max_len": max(lens), "shared": case.get("prefix", 0),
          "kv_lens": torch.tensor(lens, **i32), "row_start": torch.tensor(starts, **i32)}
    need = [-(-x // PAGE) for x in lens]
    shared = st["shared"]
    width = max(max(need), shared) + 1
    pool_pages = shared + sum(max(0, x - shared) for x in need) + 3
    host = torch.randperm(pool_pages, generator=g, device=DEV).tolist()
    head, at, table = host[:shared], shared, []
    for x in need:
        row = (head + host[at:at + max(0, x - shared)])[:width]
        at += max(0, x - shared)
        table.append(row + [0] * (width - len(row)))
    st["page_table"] = torch.tensor(table, **i32)
    if case["op"] != "rope":  # most rows follow a recent one, some branch off further back
        i = torch.cat([torch.arange(r) for r in rows]).to(DEV)
        back = torch.rand(t, generator=g, device=DEV) ** 3 * 12
        st["parents"] = (i - 1 - back.to(torch.int64)).clamp_min(-1).to(torch.int32)
    if case["op"] == "tree":
        st["pool"] = torch.zeros(1, 1, 1, 16 * 64 * 2 + 64, dtype=torch.uint8, device=DEV)  # trees do not touch it
        return st
    H, D, L = case["H"], case["D"], case.get("layers", 1)
    dt = st["dtype"] = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    gain = torch.exp(0.6 * torch.randn(2, H, 1, D, generator=g, device=DEV))  # channels differ in loudness, keys and values apart
    rec = _record(case)[3]
    if case["op"] == "rope":
        Hq = H * case["G"]
        st["pool"] = torch.zeros(L, pool_pages, H, rec, dtype=torch.uint8, device=DEV)
        if case["fused"]:  # slices of one projection's output, as a model's layer has them
            qkv = torch.randn(t, Hq + 2 * H, D, generator=g, device=DEV)
            qkv[:, Hq:] *= gain.transpose(1, 2).reshape(1, 2 * H, D)
            qkv = qkv.to(dt)
            st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        else:
            st["q"] = torch.randn(t, Hq, D, generator=g, device=DEV).to(dt)
            st["k"] = (torch.randn(L, H, t, D, generator=g, device=DEV) * gain[0]).to(dt)
            st["v"] = (torch.randn(L, H, t, D, generator=g, device=DEV) * gain[1]).to(dt)
        p = case["rot"] // 2
        st["freqs"] = torch.tensor([case["theta"] ** (-j / p) for j in range(p)], dtype=torch.float64, device=DEV)
        st["axis"] = _axis(case)
        if case["given"]:  # text counts on, pictures of 24 x 36 patches count time, height and width
            r = torch.arange(t, device=DEV)
            if case["axes"] == 1:
                pos = (r * 37 + int(torch.randint(0, 1000, (1,), generator=g, device=DEV))) % 100000
            else:
                first = int(torch.randint(0, 5000, (1,), generator=g, device=DEV))
                pos = torch.stack([r // 864, r // 36 % 24, r % 36, r % 7])[:case["axes"]] + first
            st["positions"] = pos.to(torch.int32).reshape(case["axes"], t)
        else:
            st["positions"] = None
        return st
    m, _ = _tree(st["parents"], st)
    st["masks"] = m
    if case["op"] == "keep":
        st["pool"] = torch.zeros(L, pool_pages, H, rec, dtype=torch.uint8, device=DEV)
        st["k"] = (torch.randn(L, H, t, D, generator=g, device=DEV) * gain[0]).to(dt)
        st["v"] = (torch.randn(L, H, t, D, generator=g, device=DEV) * gain[1]).to(dt)
        u = torch.rand(n, generator=g, device=DEV) ** 2  # the first nodes are the likely ones; -1: no draft was right
        st["nodes"] = ((u * (torch.tensor(rows, device=DEV) + 1)).floor() - 1).to(torch.int32)
        return st
    pool = torch.empty(1, pool_pages, H, rec, dtype=torch.uint8, device=DEV)
    for a in range(0, pool_pages, 4096):
        m = min(4096, pool_pages - a)
        kv = torch.randn(2, m, H, PAGE, D, generator=g, device=DEV) * gain[:, None]
        pool[0, a:a + m] = _pages(kv[0].to(dt).float(), kv[1].to(dt).float(), case)
    st["pool"] = pool
    st["q"] = torch.randn(t, H * case["G"], D, generator=g, device=DEV).to(dt)
    st["scale"] = 1.0 / math.sqrt(D)
    return st


# ------------------------------------------------------------------ the calls

def _cache(st):
    """The handles that a user's program makes once for its cache and batch."""
    if "cache" not in st:
        from tensor_compression_amd import kvtc
        c = st["case"]
        cfg = {"layers": c.get("layers", 1), "kv_heads": c.get("H", 1), "head_dim": c.get("D", 64),
               "dtype": kvtc.FP32 if c.get("dtype") == "fp32" else kvtc.BF16, "bits_k": c.get("bk", 8), "bits_v": c.get("bv", 8)}
        st["cache"] = cache = kvtc.MxCache(cfg, st["pool"].shape[1], pool=st["pool"])
        st["batch"] = cache.batch(st["page_table"], st["kv_lens"], st["row_start"], total_rows=st["rows"],
                                  max_rows=st["max_rows"], max_len=st["max_len"])
        if c["op"] == "rope":
            st["rope"] = kvtc.MxRope(st["freqs"], kvtc.ROPE_HALF if c["style"] == "half" else kvtc.ROPE_INTERLEAVED, st["axis"])
            shape = (st["rows"], c["H"], c["D"]) if c["fused"] else (c["layers"], c["H"], st["rows"], c["D"])
            st["out"] = [torch.empty(shape, dtype=st["dtype"], device=DEV) for _ in range(2)]
            st["q_out"] = torch.empty(st["q"].shape, dtype=st["dtype"], device=DEV)
        elif c["op"] == "tree":
            st["out"] = [torch.empty(st["rows"], -(-st["max_rows"] // 32), dtype=torch.int32, device=DEV),
                         torch.empty(st["rows"], dtype=torch.int32, device=DEV)]
        elif c["op"] == "keep":
            n = c["n"]
            st["lens"] = torch.empty(n, dtype=torch.int32, device=DEV)
            st["tail"] = cache.batch(st["page_table"], st["lens"], TAIL * torch.arange(n + 1, dtype=torch.int32, device=DEV),
                                     total_rows=TAIL * n, max_rows=TAIL, max_len=st["max_len"])
            st["out"] = [torch.empty(c["layers"], c["H"], TAIL * n, c["D"], dtype=st["dtype"], device=DEV) for _ in range(2)]
        else:
            st["out"] = [torch.empty_like(st["q"]), torch.empty(st["q"].shape[:2], dtype=torch.float32, device=DEV)]
            st["ws"] = cache.workspace_tree(st["batch"], c["H"] * c["G"], shared_pages=st["shared"])
    return st["cache"], st["batch"]


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        cache, batch = _cache(state)
        if op == "rope":
            q = cache.write_rope(batch, state["k"], state["v"], state["rope"], positions=state["positions"],
                                 q=state["q"] if c["G"] else None, out=state["q_out"] if c["G"] else None)
            k, v = cache.read(batch, *state["out"])
            return (k, v, q) if c["G"] else (k, v)
        if op == "tree":
            return cache.tree(batch, state["parents"], masks=state["out"][0], positions=state["out"][1])
        if op == "keep":
            cache.write(batch, state["k"], state["v"])
            cache.keep(batch, state["nodes"], state["masks"], lens_out=state["lens"])
            return (state["lens"], *cache.read(state["tail"], *state["out"]))
        return cache.attention_tree(batch, state["q"], state["masks"], shared_pages=state["shared"], scale=state["scale"],
                                    out=state["out"][0], lse=state["out"][1], ws=state["ws"])
    if op == "rope":
        return _plain_rope(state)
    if op == "tree":
        return _tree(state["parents"], state)
    return _plain_keep(state) if op == "keep" else _plain_attention(state)


# --------------------------------------------------------------- plain forms

def _rows_of(st):
    """Sequence of each row, and its index there."""
    t = torch.arange(st["rows"], dtype=torch.int32, device=DEV)
    z = torch.searchsorted(st["row_start"][1:], t, right=True)
    return z, t - st["row_start"][z]


def _turn(x, cos, sin, rot, half):
    """x [..., D] with its first `rot` channels rotated by cos, sin [..., rot / 2], in their type."""
    a = x[..., :rot].to(cos.dtype)
    a = a.unflatten(-1, (2, -1)).transpose(-1, -2) if half else a.unflatten(-1, (-1, 2))
    a = torch.stack([a[..., 0] * cos - a[..., 1] * sin, a[..., 0] * sin + a[..., 1] * cos], -1)
    a = (a.transpose(-1, -2) if half else a).flatten(-2)
    return torch.cat([a, x[..., rot:].to(cos.dtype)], -1)


def _plain_rope(st):
    c = st["case"]
    pos = st["positions"]
    if pos is None:
        z, i = _rows_of(st)
        pos = (st["kv_lens"][z] - st["row_start"][z + 1] + st["row_start"][z] + i)[None]
    # angles in 64 bits, and the keys too up to their elements: those may lie next to a border
    ang = pos.double()[torch.tensor(st["axis"], device=DEV)].T * st["freqs"]  # [rows, pairs]
    cos, sin = torch.cos(ang), torch.sin(ang)
    half = c["style"] == "half"
    if c["fused"]:
        cos, sin = cos[:, None], sin[:, None]
    k = _values(*_quantise(_turn(st["k"], cos, sin, c["rot"], half), c["bk"]), st["dtype"])
    v = _values(*_quantise(st["v"].float(), c["bv"]), st["dtype"])
    if not c["G"]:
        return k, v
    if not c["fused"]:
        cos, sin = cos[:, None], sin[:, None]
    return k, v, _turn(st["q"], cos.float(), sin.float(), c["rot"], half).to(st["dtype"])


def _tree(parents, st):
    """Masks [rows, words] and positions [rows] of the rows' trees."""
    R, n = st["max_rows"], st["kv_lens"].numel()
    z, i = _rows_of(st)
    W = -(-R // 32)
    up = torch.zeros(n, 32 * W, 32 * W, device=DEV)  # paths of at most 2^k steps
    up[z, i, i] = 1.0
    up[z, i, parents.clamp_min(0)] = torch.where(parents >= 0, 1.0, (i == 0).float())
    for _ in range((R - 1).bit_length()):
        up = (torch.matmul(up, up) > 0).float()
    up = up[z, i]  # [rows, 32 W]
    bits = up.view(-1, W, 32).to(torch.int64) << torch.arange(32, device=DEV)
    word = bits.sum(-1)
    masks = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
    base = st["kv_lens"] - st["row_start"][1:] + st["row_start"][:-1]
    return masks, base[z] + up.sum(-1).to(torch.int32) - 1


def _bits(masks, R):
    """masks [..., words] -> truth values [..., R]."""
    j = torch.arange(R, device=DEV)
    return (masks[..., j // 32] >> (j % 32)) & 1 > 0


def _plain_keep(st):
    c = st["case"]
    n, R = c["n"], st["max_rows"]
    first = st["row_start"][:-1]
    base = st["kv_lens"] - st["row_start"][1:] + first
    node = st["nodes"]
    on = _bits(st["masks"][(first + node.clamp_min(0)).long()], R) & (node >= 0)[:, None]
    lens = base + on.sum(-1).to(torch.int32)
    # the tail's tokens: kept rows in their order, before them what lay there (nothing was written: zeros)
    order = torch.argsort(torch.where(on, 0, 1), dim=-1, stable=True)
    k = lens[:, None] - TAIL + torch.arange(TAIL, device=DEV) - base[:, None]  # index among the kept
    row = (first[:, None] + order.gather(1, k.clamp(0, R - 1))).clamp(max=st["rows"] - 1)
    out = []
    for x, b in ((st["k"], c["bk"]), (st["v"], c["bv"])):
        y = _values(*_quantise(x[:, :, row.reshape(-1)].float(), b), st["dtype"])
        out.append(torch.where((k >= 0).reshape(-1)[:, None], y, torch.zeros_like(y)))
    return lens, out[0], out[1]


def _elements(b):
    if b == 4:
        half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
        return torch.cat([half, -half])
    return torch.arange(256, device=DEV).to(torch.uint8).view(torch.float8_e4m3fn).float()


def _tokens(pool, table, case):
    """k, v [n, H, tokens, D] fp32 of the pages table [n, pages]."""
    rec = pool[table].transpose(1, 2)  # [n, H, pages, record]
    D = case["D"]
    kc, vc, sc, _ = _record(case)
    lead = rec.shape[:-1]
    out = []
    for b, key, c, s in ((case["bk"], True, rec[..., :kc], rec[..., kc + vc:kc + vc + sc]),
                         (case["bv"], False, rec[..., kc:kc + vc], rec[..., kc + vc + sc:])):
        if b == 4:
            c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
        if not key:
            c = c.reshape(*lead, 4, 16, 4, D // 16).transpose(-3, -2)
            s = s.reshape(*lead, 4, D // 32, 4).transpose(-2, -1)
        u = _elements(b)[c.reshape(*lead, 16, D // 32, 32).int()]
        out.append(_values(u, s.reshape(*lead, 16, D // 32, 1).int(), torch.float32).flatten(2, 3))
    return out


def _plain_attention(st):
    c = st["case"]
    H, G, D, n = c["H"], c["G"], c["D"], c["n"]
    R, sp = st["max_rows"], st["shared"]
    i = torch.arange(R, device=DEV)
    at = (st["row_start"][:-1, None] + i).clamp(max=st["rows"] - 1)
    q = st["q"].float()[at].view(n, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(n, H, R * G, D)
    pages = -(-st["max_len"] // PAGE)
    k, v = _tokens(st["pool"][0], st["page_table"][:, sp:max(pages, sp)], c)
    s = torch.matmul(q, k.transpose(2, 3))
    if sp:  # the prefix once, for the rows of all sequences together
        pk, pv = _tokens(st["pool"][0], st["page_table"][:1, :sp], c)
        qp = q.transpose(0, 1).reshape(H, n * R * G, D)
        s0 = torch.matmul(qp, pk[0].transpose(1, 2)).view(H, n, R * G, sp * PAGE).transpose(0, 1)
        s = torch.cat([s0, s], -1)
    T = s.shape[-1]
    j = torch.arange(T, device=DEV) - (st["kv_lens"] - st["row_start"][1:] + st["row_start"][:-1])[:, None]  # [n, T]: draft row
    seen = _bits(st["masks"][at], R).gather(2, j.clamp(0, R - 1)[:, None].expand(n, R, T))
    seen = (j < 0)[:, None] | (seen & (j < (st["row_start"][1:] - st["row_start"][:-1])[:, None])[:, None])
    s = (s * st["scale"]).masked_fill(~seen.repeat_interleave(G, 1)[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    vz = torch.where((sp * PAGE + torch.arange(v.shape[2], device=DEV) < st["kv_lens"][:, None])[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p[..., sp * PAGE:], vz)
    if sp:
        pp = p[..., :sp * PAGE].transpose(0, 1).reshape(H, n * R * G, sp * PAGE)
        o = o + torch.matmul(pp, pv[0]).view(H, n, R * G, D).transpose(0, 1)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + torch.log(l))[..., 0]
    z, r = _rows_of(st)
    o = o.view(n, H, R, G, D)[z, :, r].reshape(st["rows"], H * G, D)
    lse = lse.view(n, H, R, G)[z, :, r].reshape(st["rows"], H * G)
    return o.to(st["dtype"]), lse


# ------------------------------------------------------------------ in 64 bits

def _grid64(b):
    """Magnitudes in the order of their codes."""
    if b == 4:
        return torch.tensor([(m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)) for e in range(4) for m in range(2)], dtype=torch.float64, device=DEV)
    return torch.tensor([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127], dtype=torch.float64, device=DEV)


def _exact_values(x, b):
    grid = _grid64(b)
    mid = (grid[1:] + grid[:-1]) / 2
    y = x.double().unflatten(-1, (-1, 32))
    a = y.abs().amax(-1, keepdim=True)
    e = torch.frexp(a / OVER[b])[1]  # the smallest e with a < OVER 2^e
    e = torch.where(a > 0, e, torch.full_like(e, -1000)).clamp(BYTE_LOW - 127, BYTE_TOP[b] - 127)
    scale = torch.exp2(e.double())
    u = (y / scale).abs()
    lo, hi = torch.bucketize(u, mid), torch.bucketize(u, mid, right=True)
    near = torch.where(lo % 2 == 0, lo, hi)  # a tie goes to the even code
    out = torch.copysign(grid[near], y) * scale
    return torch.where(torch.isfinite(a), out, torch.full_like(out, math.nan)).flatten(-2)


def _exact_turn(x, turn, case):
    """x [..., rows, D] by the unit numbers turn [rows, pairs]: a pair of channels as one complex number."""
    rot, p = case["rot"], case["rot"] // 2
    j = torch.arange(p, device=DEV)
    one, two = (j, j + p) if case["style"] == "half" else (2 * j, 2 * j + 1)
    y = x.double().clone()
    w = torch.complex(y[..., one], y[..., two]) * turn
    y[..., one], y[..., two] = w.real, w.imag
    return y


def _exact_rope(st):
    c = st["case"]
    rows, lens = _lens(c)
    if st["positions"] is None:
        pos = torch.tensor([ln - n + i for n, ln in zip(rows, lens) for i in range(n)], dtype=torch.float64, device=DEV)[None]
    else:
        pos = st["positions"].double()
    ang = torch.stack([pos[a] * f for a, f in zip(st["axis"], st["freqs"])], -1)
    turn = torch.polar(torch.ones_like(ang), ang)
    if c["fused"]:  # [rows, heads, D] -> [heads, rows, D] and back
        k = _exact_values(_exact_turn(st["k"].transpose(0, 1), turn, c), c["bk"]).transpose(0, 1).contiguous()
        v = _exact_values(st["v"], c["bv"])
    else:
        k = torch.stack([_exact_values(_exact_turn(st["k"][l], turn, c), c["bk"]) for l in range(c["layers"])])
        v = torch.stack([_exact_values(st["v"][l], c["bv"]) for l in range(c["layers"])])
    return (k, v, _exact_turn(st["q"].transpose(0, 1), turn, c).transpose(0, 1).contiguous()) if c["G"] else (k, v)


def _paths(st):
    """Rows that each row sees, from the parents alone."""
    rows, _ = _lens(st["case"])
    parents, at, out = st["parents"].tolist(), 0, []
    for n in rows:
        seen = []
        for i in range(n):
            p = parents[at + i]
            seen.append((seen[p] if p >= 0 else []) + [i])
        out.append(seen)
        at += n
    return out


def _exact_token(case, key):
    """Byte offset, nibble shift and scale offset of (token, channel) within a record."""
    D = case["D"]
    kc, vc, sc, _ = _record(case)
    b = case["bk"] if key else case["bv"]
    at, sh, so = [], [], []
    for r in range(PAGE):
        for j in range(D):
            u = D // 16
            e = r * D + j if key else ((r // 4) * 16 + j // u) * 4 * u + (r % 4) * u + j % u
            at.append((0 if key else kc) + e * b // 8)
            sh.append(4 * (e % 2) if b == 4 else 0)
            so.append(kc + vc + r * (D // 32) + j // 32 if key else kc + vc + sc + ((r // 4) * (D // 32) + j // 32) * 4 + r % 4)
    return [torch.tensor(x, device=DEV) for x in (at, sh, so)]


def _exact_unpack(rec, case, key, places):
    """rec [pages, record] of one head -> [pages 16, D] in 64 bits."""
    b = case["bk"] if key else case["bv"]
    at, sh, so = places
    code = rec[:, at].int() >> sh
    mag = code & (7 if b == 4 else 127)
    sign = 1 - 2 * ((code >> (b - 1)) & 1)
    grid = torch.cat([_grid64(b), torch.full((1,), math.nan, dtype=torch.float64, device=DEV)])
    byte = rec[:, so].int()
    x = sign * grid[mag] * torch.exp2((byte - 127).double())
    return torch.where(byte == 255, torch.full_like(x, math.nan), x).view(-1, case["D"])


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    rows, lens = _lens(case)
    paths = _paths(st)
    if case["op"] == "tree":  # whole numbers
        words = -(-st["max_rows"] // 32)
        bits = [sum(1 << j for j in p) for seen in paths for p in seen]
        masks = [[((b >> (32 * w)) & 0xFFFFFFFF ^ 0x80000000) - 0x80000000 for w in range(words)] for b in bits]
        pos = [ln - n + len(p) - 1 for n, ln, seen in zip(rows, lens, paths) for p in seen]
        return torch.tensor(masks, dtype=torch.int32), torch.tensor(pos, dtype=torch.int32)
    H, D = case["H"], case["D"]
    if case["op"] == "keep":
        nodes, new, at = st["nodes"].tolist(), [], 0
        out = [torch.zeros(case["layers"], H, TAIL * case["n"], D, dtype=torch.float64, device=DEV) for _ in range(2)]
        for z, (n, ln) in enumerate(zip(rows, lens)):
            kept = paths[z][nodes[z]] if nodes[z] >= 0 else []
            new.append(ln - n + len(kept))
            m = min(len(kept), TAIL)
            if m:
                take = torch.tensor([at + j for j in kept[-m:]], device=DEV)
                for o, x, b in ((out[0], st["k"], case["bk"]), (out[1], st["v"], case["bv"])):
                    o[:, :, TAIL * (z + 1) - m:TAIL * (z + 1)] = _exact_values(x[:, :, take], b)
            at += n
        return torch.tensor(new, dtype=torch.int32), out[0], out[1]
    G = case["G"]
    o = torch.zeros(st["rows"], H * G, D, dtype=torch.float64, device=DEV)
    lse = torch.full((st["rows"], H * G), -math.inf, dtype=torch.float64, device=DEV)
    table = st["page_table"].tolist()
    places = [_exact_token(case, key) for key in (True, False)]
    see, at = [], 0
    for n, ln, seen in zip(rows, lens, paths):
        s = torch.zeros(n, n, dtype=torch.bool)
        for i, p in enumerate(seen):
            s[i, p] = True
        see.append(torch.cat([torch.ones(n, ln - n, dtype=torch.bool), s], 1)[:, None].to(DEV))
    for h in range(H):
        at = 0
        for z, (n, ln) in enumerate(zip(rows, lens)):
            own_pages = table[0][:st["shared"]] + table[z][st["shared"]:]
            pages = torch.tensor(own_pages[: -(-ln // PAGE)], device=DEV, dtype=torch.int64)
            k, v = (_exact_unpack(st["pool"][0, pages, h], case, key, w)[:ln] for key, w in zip((True, False), places))
            s = (st["q"][at:at + n, h * G:(h + 1) * G].reshape(n * G, D).double() @ k.T).view(n, G, ln) * st["scale"]
            s = torch.where(see[z], s, torch.full_like(s, -math.inf))
            x = torch.logsumexp(s, -1)
            o[at:at + n, h * G:(h + 1) * G] = (torch.exp(s - x[..., None]).view(n * G, ln) @ v).view(n, G, D)
            lse[at:at + n, h * G:(h + 1) * G] = x
            at += n
    return o, lse
