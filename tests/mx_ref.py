"""Plain 64-bit implementation of the microscaled paged cache (test
infrastructure): quantisation, record layout, reading, attention."""
import numpy as np

PAGE = 16
OVER = {4: 7.0, 8: 464.0}
TOP = {4: 6.0, 8: 448.0}
E_MAX = {4: 125, 8: 119}
E_MIN = -112


def grid(b):
    """Element magnitudes in code order."""
    if b == 4:
        return np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    return np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:127])


def quantise(x, b):
    """x [..., 32 k] float64 -> (codes uint8 [...], scale bytes uint8 [..., k])."""
    x = np.asarray(x, np.float64)
    y = x.reshape(*x.shape[:-1], -1, 32)
    a = np.abs(y).max(-1)
    fine = np.isfinite(y).all(-1)
    a = np.where(fine, a, 1.0)
    e = np.full(a.shape, E_MIN)
    for cand in range(E_MAX[b], E_MIN - 1, -1):  # the smallest e with a < OVER 2^e
        e = np.where(a < OVER[b] * 2.0 ** cand, cand, e)
    e = np.where(a >= OVER[b] * 2.0 ** E_MAX[b], E_MAX[b], e)
    u = np.minimum(np.abs(np.where(fine[..., None], y, 0.0)) / 2.0 ** e[..., None], TOP[b])
    g = grid(b)
    i = np.clip(np.searchsorted(g, u, side="right") - 1, 0, len(g) - 2)
    lo, hi = u - g[i], g[i + 1] - u
    code = np.where((hi < lo) | ((hi == lo) & (i % 2 == 1)), i + 1, i)
    code = code | np.where(np.signbit(y), 1 << (b - 1), 0)
    code = np.where(fine[..., None], code, 0)
    return code.reshape(x.shape).astype(np.uint8), np.where(fine, e + 127, 255).astype(np.uint8)


def values(code, s, b):
    """What codes [..., 32 k] under scale bytes [..., k] stand for."""
    g = grid(b)
    g = np.concatenate([g, [np.nan]]) if b == 8 else g
    sign = 1.0 - 2.0 * (code >> (b - 1))
    x = (sign * g[code & ((1 << (b - 1)) - 1)]).reshape(*code.shape[:-1], -1, 32)
    s = s.astype(np.int64)[..., None]
    return np.where(s == 255, np.nan, x * 2.0 ** (s - 127.0)).reshape(code.shape)


def record_bytes(D, bk, bv):
    return PAGE * D * (bk + bv) // 8 + PAGE * D // 16


def places(D, bk, bv, kv):
    """(byte, shift) of every (token, channel) and the byte of every (token,
    block) of a record: keys (kv 0) or values (kv 1)."""
    b, other = (bk, bv) if kv == 0 else (bv, bk)
    C = D // 16
    t, c = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
    el = t * D + c if kv == 0 else ((t // 4 * 16 + c // C) * 4 + t % 4) * C + c % C
    base = 0 if kv == 0 else PAGE * D * bk // 8
    t2, j = np.meshgrid(np.arange(PAGE), np.arange(D // 32), indexing="ij")
    so = t2 * (D // 32) + j if kv == 0 else (t2 // 4 * (D // 32) + j) * 4 + t2 % 4
    sbase = PAGE * D * (bk + bv) // 8 + (PAGE * D // 32 if kv else 0)
    return base + el * b // 8, (el % 2) * 4 if b == 4 else el * 0, sbase + so


def put(rec, tok, kv, code, s, b, where):
    """Write token `tok` (0..15) of one record (uint8 [record]) in place."""
    at, sh, so = where
    if b == 8:
        rec[at[tok]] = code
    else:  # two codes a byte, never of different tokens
        assert np.array_equal(at[tok, 0::2], at[tok, 1::2])
        rec[at[tok, 0::2]] = code[0::2] | (code[1::2] << 4)
    rec[so[tok]] = s


def write(pool, table, lens, starts, k, v, D, bk, bv):
    """pool uint8 [pages, H, record] in place; k, v [rows, H, D] float64."""
    H = pool.shape[1]
    q = [quantise(x, b) for x, b in ((k, bk), (v, bv))]
    where = [places(D, bk, bv, kv) for kv in (0, 1)]
    for z, ln in enumerate(lens):
        n = starts[z + 1] - starts[z]
        for i in range(n):
            pos = ln - n + i
            if pos < 0:
                continue
            pg = table[z][pos // PAGE]
            for h in range(H):
                for kv in (0, 1):
                    code, s = q[kv]
                    put(pool[pg, h], pos % PAGE, kv, code[starts[z] + i, h], s[starts[z] + i, h], (bk, bv)[kv], where[kv])


def unpack(pool, D, bk, bv):
    """pool uint8 [pages, H, record] -> k, v [pages, H, 16, D] float64."""
    out = []
    for kv, b in ((0, bk), (1, bv)):
        at, sh, so = places(D, bk, bv, kv)
        code = (pool[..., at] >> sh.astype(np.uint8)) & (0xF if b == 4 else 0xFF)
        out.append(values(code, pool[..., so], b))
    return out


def tokens(kp, vp, pages, n):
    """k, v [H, n, D] of a sequence from unpacked pages."""
    f = lambda x: x[pages].transpose(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[-1])[:, :n]  # noqa: E731
    return f(kp), f(vp)


def attention(kp, vp, table, lens, starts, q, scale, causal):
    """q [rows, Hq, D] float64 -> (out, lse, mass, spread): mass = sum p |v|
    per output, spread = the largest scale sum |q k| over attended tokens."""
    rows, Hq, D = q.shape
    H = kp.shape[1]
    G = Hq // H
    out, lse = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
    mass, spread = np.zeros((rows, Hq, D)), np.zeros((rows, Hq))
    with np.errstate(invalid="ignore"):
        for z, ln in enumerate(lens):
            n = starts[z + 1] - starts[z]
            if n == 0 or ln == 0:
                continue
            k, v = tokens(kp, vp, table[z][: -(-ln // PAGE)], ln)
            for i in range(n):
                lim = ln - n + i + 1 if causal else ln
                if lim <= 0:
                    continue
                r = starts[z] + i
                for h in range(Hq):
                    kk, vv = k[h // G, :lim], v[h // G, :lim]
                    s = scale * (kk @ q[r, h])
                    m = s.max()
                    p = np.exp(s - m)
                    lse[r, h] = m + np.log(p.sum())
                    p /= p.sum()
                    out[r, h] = p @ vv
                    mass[r, h] = p @ np.abs(vv)
                    spread[r, h] = (scale * (np.abs(kk) @ np.abs(q[r, h]))).max()
    return out, lse, mass, spread


# ---- rotation, drafts


def rotate(x, pos, freqs, axis, half):
    """x [..., rows, heads, D] float64, pos [axes][rows] -> rotated: the pairs
    of the first 2 len(freqs) channels by pos[axis[j]] freqs[j]."""
    x = np.array(x, np.float64)
    p = len(freqs)
    with np.errstate(invalid="ignore", over="ignore"):
        for j in range(p):
            a, b = (j, j + p) if half else (2 * j, 2 * j + 1)
            ang = np.asarray(pos[axis[j]], np.float64) * freqs[j]
            c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
            u, v = x[..., a].copy(), x[..., b].copy()
            x[..., a], x[..., b] = u * c - v * s, u * s + v * c
    return x


def tree(parents):
    """Sorted rows that each row of a draft sees: itself and its ancestors."""
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else []) + [i])
    return seen


def mask_words(seen, words):
    """Rows seen -> int32 words [rows][words]."""
    out = np.zeros((len(seen), words), np.uint32)
    for i, rows in enumerate(seen):
        for j in rows:
            out[i, j // 32] |= np.uint32(1 << (j % 32))
    return out.view(np.int32)


def attention_seen(kp, vp, table, lens, starts, q, scale, seen):
    """attention() of rows that see the tokens before their sequence's rows and
    the rows seen[z][i] of it."""
    rows, Hq, D = q.shape
    G = Hq // kp.shape[1]
    out, lse = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
    mass, spread = np.zeros((rows, Hq, D)), np.zeros((rows, Hq))
    with np.errstate(invalid="ignore"):
        for z, ln in enumerate(lens):
            n = starts[z + 1] - starts[z]
            if n == 0 or ln == 0:
                continue
            k, v = tokens(kp, vp, table[z][: -(-ln // PAGE)], ln)
            base = ln - n
            for i in range(n):
                at = list(range(max(base, 0))) + [base + j for j in seen[z][i] if base + j >= 0]
                if not at:
                    continue
                r = starts[z] + i
                for h in range(Hq):
                    kk, vv = k[h // G, at], v[h // G, at]
                    s = scale * (kk @ q[r, h])
                    m = s.max()
                    p = np.exp(s - m)
                    lse[r, h] = m + np.log(p.sum())
                    p /= p.sum()
                    out[r, h] = p @ vv
                    mass[r, h] = p @ np.abs(vv)
                    spread[r, h] = (scale * (np.abs(kk) @ np.abs(q[r, h]))).max()
    return out, lse, mass, spread
