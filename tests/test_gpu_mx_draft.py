"""Rotated appends and drafts on the microscaled paged cache, on the GPU
against the plain 64-bit implementation: codes bit for bit, trees and kept
paths exactly, rotated queries and attention within bounds that follow from
their roundings."""
import numpy as np
import pytest
import torch

import mx_ref
from tensor_compression_amd import kvtc
from test_gpu_mx import DT, FORMATS, Case, dev, hard_rows, np64

pytestmark = pytest.mark.gpu

INV = 1 << kvtc.ERR_INVALID_ARG


def freqs_of(rot, theta=1e4):
    return [theta ** (-2.0 * j / rot) for j in range(rot // 2)]


def rope_of(rot, half=True, axis=None, theta=1e4):
    return kvtc.MxRope(dev(freqs_of(rot, theta), torch.float64), kvtc.ROPE_HALF if half else kvtc.ROPE_INTERLEAVED, axis)


def own_positions(c):
    """Each row's position in the cache."""
    return [ln - (c.starts[z + 1] - c.starts[z]) + i for z, ln in enumerate(c.lens)
            for i in range(c.starts[z + 1] - c.starts[z])]


def check_queries(q, got, pos, rot, half, axis, dtype, what, theta=1e4):
    """cos and sin are within 2.3 2^-24, one product is rounded, then the sum:
    at most 4 2^-24 of |a| + |b|, and the fp64 angle's own error
    (2^-53 of it, with a factor of 4); then half a step of the output."""
    want = mx_ref.rotate(np64(q), pos, freqs_of(rot, theta), axis, half)
    x = np.abs(np64(q))
    size = x.copy()
    p = rot // 2
    a, b = (np.arange(p), np.arange(p) + p) if half else (2 * np.arange(p), 2 * np.arange(p) + 1)
    size[..., a] = size[..., b] = x[..., a] + x[..., b]
    far = 4 * np.abs(np.asarray(pos, np.float64)).max() * 2.0 ** -53
    u = 2.0 ** -8 if dtype == kvtc.BF16 else 2.0 ** -24
    tol = (4 * 2.0 ** -24 + far) * size * (1 + u) + u * np.abs(want) + 1e-38
    err = np.abs(np64(got) - want)
    print(what, "worst error / bound %.3f" % float((err / tol).max()), flush=True)
    assert (err <= tol).all()
    assert torch.equal(got[..., rot:], q[..., rot:])


# ---- rotated appends


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
@pytest.mark.parametrize("D,bk,bv", FORMATS)
def test_write_rope_bytes(D, bk, bv, dtype, half):
    """Rows over the whole range of the type, starts anywhere in a page, a
    sequence with more rows than tokens and one without rows, rows of no
    sequence, one layer of two; positions as they stand in the cache."""
    rows, lens = [1, 5, 16, 0, 17, 40, 3], [1, 5, 16, 7, 45, 40, 2]
    total = sum(rows) + 2
    c = Case(D, bk, bv, dtype, 3, rows, lens, layers=2, seed=D + bk, fill=0xA5, total_rows=total)
    k, v = (hard_rows(c.rng, total, 3, D, dtype) for _ in range(2))
    q = c.rand(total, 6, D)
    out = torch.full_like(q, 7.0)
    print("write_rope", D, bk, bv, dtype, half, flush=True)
    c.cache.write_rope(c.batch, k, v, rope_of(D, half), q=q, out=out, layer=1, status=c.status)
    n = c.starts[-1]
    pos, axis = [own_positions(c)], [0] * (D // 2)
    turned = mx_ref.rotate(np64(k)[:n], pos, freqs_of(D), axis, half)
    want = np.full(c.cache.pool.shape[1:], 0xA5, np.uint8)
    mx_ref.write(want, c.table, lens, c.starts, turned, np64(v)[:n], D, bk, bv)
    got = c.cache.pool.cpu().numpy()
    assert np.array_equal(got[1], want)
    assert (got[0] == 0xA5).all()
    assert c.status.item() == 1 << kvtc.ERR_NONFINITE
    assert (out[n:] == 7.0).all()
    check_queries(q[:n], out[:n], pos, D, half, axis, dtype, "queries")


@pytest.mark.parametrize("rot", [16, 32, 48, 64, 96, 112, 128])
@pytest.mark.parametrize("half", [True, False])
def test_rope_of_some_channels(rot, half):
    """Part of the channels, one to four axes in stretches and in turn, given
    positions of either sign and far out, queries in place."""
    for D, dtype in ((64, kvtc.FP32), (128, kvtc.BF16), (128, kvtc.FP32)):
        if rot > D:
            continue
        for axes in (1, 2, 3, 4):
            rows, lens = [9, 1, 30], [40, 1, 33]
            c = Case(D, 8, 4, dtype, 2, rows, lens, seed=rot + axes)
            axis = [j % axes if axes == 3 else j * axes // (rot // 2) for j in range(rot // 2)]
            pos = c.rng.integers(-2 ** 20, 2 ** 24, (axes, c.total))
            pos[:, :4] = [[0], [1], [-1], [99]][0]
            k, v, q = c.rand(c.total, 2, D), c.rand(c.total, 2, D), c.rand(c.total, 6, D)
            rope = rope_of(rot, half, axis)
            assert rope.axes == max(axis) + 1
            pos = pos[:rope.axes]
            was = q.clone()
            print("rope", D, rot, half, dtype, axes, flush=True)
            out = c.cache.write_rope(c.batch, k, v, rope, positions=dev(pos, torch.int32), q=q, out=q, status=c.status)
            assert out is q
            turned = mx_ref.rotate(np64(k), pos, freqs_of(rot), axis, half)
            want = np.full(c.cache.pool.shape[1:], 0xFF, np.uint8)
            mx_ref.write(want, c.table, lens, c.starts, turned, np64(v), D, 8, 4)
            assert np.array_equal(c.cache.pool[0].cpu().numpy(), want)
            check_queries(was, q, pos, rot, half, axis, dtype, "in place")
            assert c.status.item() == 0


def test_rope_far_positions():
    """The ends of int32; values that would show an angle off by 2^-24."""
    D = 128
    pos = np.array([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30, 2 ** 24 + 1, -12345678, 1000003, 7]])
    rows = pos.shape[1]
    c = Case(D, 8, 8, kvtc.FP32, 2, [rows], [rows], seed=3)
    k, v, q = c.rand(rows, 2, D), c.rand(rows, 2, D), c.rand(rows, 4, D)
    for half in (True, False):
        out = c.cache.write_rope(c.batch, k, v, rope_of(D, half, theta=5e5), positions=dev(pos[0], torch.int32), q=q, status=c.status)
        check_queries(q, out, pos, D, half, [0] * 64, kvtc.FP32, "far", theta=5e5)
        turned = mx_ref.rotate(np64(k), pos, freqs_of(D, 5e5), [0] * 64, half)
        want = np.full(c.cache.pool.shape[1:], 0xFF, np.uint8)
        mx_ref.write(want, c.table, c.lens, c.starts, turned, np64(v), D, 8, 8)
        assert np.array_equal(c.cache.pool[0, :, :, :].cpu().numpy(), want)
    assert c.status.item() == 0


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
@pytest.mark.parametrize("bk", [4, 8])
def test_rope_keys_beside_borders(bk, dtype):
    """Keys whose rotation lies 1e-9 and 1e-13 of itself beside a border of the
    elements or of the scale, where fp32 holds the border itself: one channel
    of a pair, turned by the angle whose cosine brings it there; without a turn
    they are the ties.  Each at several powers of two."""
    D = 64
    top, borders = (8.0, [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]) if bk == 4 else \
        (512.0, [272.0, 304.0, 336.0, 368.0, 400.0, 232.0, 432.0, 464.0])
    at = [t * (1 + d) for t in borders for d in (1e-9, -1e-9, 1e-13, -1e-13)]  # the last four decide the scale
    f = [float(x) for x in np.arccos(np.array(at) / top)]
    rows = []
    for power in (-40, -1, 0, 3, 60):
        for last in (None, 28, 29, 30, 31):  # none of the four, or one
            x = np.zeros(D)
            x[:28] = top
            if last is not None:
                x[last] = top
            rows += [(x * 2.0 ** power, 1)]
            y = np.zeros(D)
            y[:28], y[28:32] = np.round(at[:28], 4), 0 if last is None else borders[-1]
            rows += [(y * 2.0 ** power, 0), (-y * 2.0 ** power, 0), (-x * 2.0 ** power, -1)]
    n = len(rows)
    c = Case(D, bk, 8, dtype, 1, [n], [n], seed=1)
    pos = np.array([[p for _, p in rows]])
    rope = kvtc.MxRope(dev(f, torch.float64))
    k = dev(np.stack([x for x, _ in rows])[:, None], torch.float32).to(DT[dtype])
    assert np.array_equal(np64(k)[:, 0], np.stack([x for x, _ in rows]))
    c.cache.write_rope(c.batch, k, k, rope, positions=dev(pos, torch.int32), status=c.status)
    turned = mx_ref.rotate(np64(k), pos, f, [0] * (D // 2), True)
    near = turned.astype(np.float32)[0, 0, :28].astype(np.float64)
    assert np.array_equal(near, np.repeat(borders[:7], 4) * 2.0 ** -40) and (turned[0, 0, :28] != near).all()
    want = np.full(c.cache.pool.shape[1:], 0xFF, np.uint8)
    mx_ref.write(want, c.table, c.lens, c.starts, turned, np64(k), D, bk, 8)
    assert np.array_equal(c.cache.pool[0].cpu().numpy(), want)


def test_rope_past_the_end_of_fp32_saturates():
    """Equal numbers of a pair by an eighth of a turn: the sum passes fp32 and
    saturates; the difference is nothing but the roundings of cos, sin (2^-53
    each), the products (2^-53) and the sum, at most 2^-51 (|a| + |b|), in the
    kernel and in the reference, plus half a step of the element (2^-4)."""
    D = 64
    c = Case(D, 8, 4, kvtc.FP32, 1, [3], [3], seed=2)
    x = torch.full((3, 1, D), 3.3e38, device="cuda")
    x[1] = -x[1]
    pos = dev([1, 1, 0], torch.int32)
    rope = kvtc.MxRope(torch.full((D // 2,), np.pi / 4, dtype=torch.float64, device="cuda"))
    c.cache.write_rope(c.batch, x, x, rope, positions=pos, status=c.status)
    turned = mx_ref.rotate(np64(x), [[1, 1, 0]], [np.pi / 4] * 32, [0] * 32, True)
    assert np.abs(turned).max() > 3.5e38
    want = np.full(c.cache.pool.shape[1:], 0xFF, np.uint8)
    mx_ref.write(want, c.table, c.lens, c.starts, turned, np64(x), D, 8, 4)
    got = c.cache.pool[0].cpu().numpy()
    at, _, so = mx_ref.places(D, 8, 4, 0)
    kp, _ = c.unpacked()
    pg = c.table[0][0]
    noise = np.abs(turned[:2, 0, :32]).max()
    assert noise <= 2.0 ** -51 * 6.6e38 and np.abs(kp[pg, 0, :2, :32]).max() <= 2.0 ** -51 * 6.6e38 * (1 + 2.0 ** -4)
    for x in (got, want):  # the differences' codes and scales
        x[pg, 0, at[:2, :32].ravel()] = 0
        x[pg, 0, so[:2, 0]] = 0
    assert np.array_equal(got, want) and c.status.item() == 0


def test_rope_without_turning_is_write():
    """Frequencies of zero: the bytes of write, the queries as they are; also
    a whole cache [L, H, T, D] through strides out of order."""
    D, L, H, T = 128, 3, 2, 77
    c = Case(D, 4, 8, kvtc.BF16, H, [T], [T], layers=L, seed=5)
    k, v = c.rand(L, T, H, D).transpose(1, 2), c.rand(L, H, T, D)
    c.cache.write(c.batch, k, v)
    want = c.cache.pool.clone()
    c.cache.pool.fill_(0xFF)
    still = kvtc.MxRope(torch.zeros(64, dtype=torch.float64, device="cuda"))
    c.cache.write_rope(c.batch, k, v, still, status=c.status)
    assert torch.equal(c.cache.pool, want)
    q = c.rand(T, 5, D)
    assert torch.equal(c.cache.write_rope(c.batch, k[1].transpose(0, 1), v[1].transpose(0, 1), still, q=q, layer=1), q)
    assert torch.equal(c.cache.pool, want) and c.status.item() == 0
    # every layer at once is each layer for itself
    rope = rope_of(D)
    c.cache.write_rope(c.batch, k, v, rope)
    want = c.cache.pool.clone()
    c.cache.pool.fill_(0xFF)
    for layer in range(L):
        c.cache.write_rope(c.batch, k[layer:layer + 1], v[layer:layer + 1], rope, layer=layer)
    assert torch.equal(c.cache.pool, want)


def test_rope_slices_and_steps():
    """Slices of one projection, queries rotated in place among them; token by
    token is the same as at once."""
    D, H, G = 128, 3, 5
    c = Case(D, 4, 4, kvtc.BF16, H, [37, 20], [37, 20], seed=6, fill=0)
    qkv = c.rand(57, (G + 2) * H, D)
    was = qkv.clone()
    q, k, v = qkv.split([G * H, H, H], 1)
    rope = rope_of(D)
    c.cache.write_rope(c.batch, k, v, rope, q=q, out=q, status=c.status)
    assert torch.equal(qkv[:, G * H:], was[:, G * H:])
    want, wq = c.cache.pool.clone(), q.clone()
    check_queries(was[:, :G * H], wq, [own_positions(c)], D, True, [0] * 64, kvtc.BF16, "slices")
    c.cache.pool.zero_()
    lens, starts = torch.zeros(2, dtype=torch.int32, device="cuda"), dev([0, 1, 2], torch.int32)
    b = c.cache.batch(c.table_dev, lens, starts, total_rows=2, max_rows=1, max_len=37)
    for t in range(37):
        at = [t, 37 + min(t, 19)]
        lens += dev([1, 1 if t < 20 else 0], torch.int32)
        if t >= 20:
            starts.copy_(dev([0, 1, 1], torch.int32))
        x = was[at]
        got = c.cache.write_rope(b, x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:], rope, q=x[:, :G * H])
        rows = 2 if t < 20 else 1
        assert torch.equal(got[:rows], wq[at][:rows])
    assert torch.equal(c.cache.pool, want) and c.status.item() == 0


@pytest.mark.parametrize("H,heads", [(9, 18), (8, 8), (17, 17), (1, 23)])
@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
def test_rope_many_heads(H, heads, dtype):
    """More vectors than a workgroup takes, part of a workgroup's, full pages
    and parts of pages."""
    for D, half in ((64, True), (128, False), (128, True)):
        rows, lens = [45, 16, 1, 7], [50, 32, 33, 20]
        c = Case(D, 4, 8, dtype, H, rows, lens, seed=H + D)
        k, v, q = c.rand(c.total, H, D), c.rand(c.total, H, D), c.rand(c.total, heads, D)
        out = c.cache.write_rope(c.batch, k, v, rope_of(D, half), q=q, status=c.status)
        pos, axis = [own_positions(c)], [0] * (D // 2)
        want = np.full(c.cache.pool.shape[1:], 0xFF, np.uint8)
        mx_ref.write(want, c.table, lens, c.starts, mx_ref.rotate(np64(k), pos, freqs_of(D), axis, half), np64(v), D, 4, 8)
        assert np.array_equal(c.cache.pool[0].cpu().numpy(), want)
        check_queries(q, out, pos, D, half, axis, dtype, f"heads {H} {heads} D{D}")
        assert c.status.item() == 0


def test_rope_reports_and_skips():
    """Pages outside the pool, bad lengths: reported, nothing written there,
    queries of good sequences rotated; NaN and infinite frequencies."""
    D, H = 64, 2
    for page in (-1, 2 ** 31 - 1, 9999):
        c = Case(D, 8, 8, kvtc.BF16, H, [20, 3], [40, 20], seed=8)
        k, v, q = c.rand(23, H, D), c.rand(23, H, D), c.rand(23, H, D)
        want_q = c.cache.write_rope(c.batch, k, v, rope_of(D), q=q)
        good = c.cache.pool.clone()
        c.cache.pool.fill_(0xFF)
        c.table_dev[0, 1] = page
        got = c.cache.write_rope(c.batch, k, v, rope_of(D), q=q, status=c.status)
        assert c.status.item() == INV and torch.equal(got, want_q)
        good[0, c.table[0][1]] = 0xFF
        assert torch.equal(c.cache.pool, good)
    c = Case(D, 8, 8, kvtc.BF16, H, [20, 3], [40, 20], seed=8)
    out = torch.full_like(q, 7.0)
    b = c.cache.batch(c.table_dev, dev([41, 20], torch.int32), dev([0, 20, 23], torch.int32), total_rows=23, max_rows=20, max_len=40)
    c.cache.write_rope(b, k, v, rope_of(D), q=q, out=out, status=c.status)
    assert c.status.item() == INV and (out[:20] == 7.0).all() and torch.equal(out[20:], want_q[20:])
    assert (c.cache.pool[0, c.table[0]] == 0xFF).all()
    c.status.zero_()
    bad = kvtc.MxRope(dev([float("nan")] + [1.0] * 30 + [float("inf")], torch.float64))
    c.cache.write_rope(c.batch, k, v, bad, status=c.status)
    assert c.status.item() == 1 << kvtc.ERR_NONFINITE
    kp, vp = c.unpacked()
    kk, vv = mx_ref.tokens(kp, vp, c.table[0], 40)
    assert np.isnan(kk[:, 21:]).all() and np.isfinite(vv[:, 20:]).all()


# ---- trees


def random_parents(rng, n):
    """Mostly the row before, some further back, some roots."""
    return [int(max(-1, i - 1 - int(rng.random() ** 3 * 12))) if rng.random() > 0.02 else -1 for i in range(n)]


@pytest.mark.parametrize("rows", [[1], [5, 0, 31, 32, 33], [64, 65, 1, 127], [200, 1000], [2300]])
def test_tree(rows):
    rng = np.random.default_rng(sum(rows))
    lens = [n + int(rng.integers(0, 50)) for n in rows]
    lens[0] = max(rows[0] - 1, 0)  # more rows than tokens: positions from -1 on
    total = sum(rows) + 3
    c = Case(64, 8, 8, kvtc.BF16, 1, rows, lens, total_rows=total)
    parents = [random_parents(rng, n) for n in rows]
    parents[-1] = list(range(-1, rows[-1] - 1)) if rows[-1] != 1000 else [-1] * 1000  # a chain; all roots
    flat = dev([p for ps in parents for p in ps] + [-7] * 3, torch.int32)
    for extra in (0, 3):
        words = -(-max(rows) // 32) + extra
        masks = torch.full((total, words), 99, dtype=torch.int32, device="cuda")
        pos = torch.full((total,), 99, dtype=torch.int32, device="cuda")
        c.cache.tree(c.batch, flat, masks=masks, positions=pos, status=c.status)
        seen = [mx_ref.tree(p) for p in parents]
        want = np.concatenate([mx_ref.mask_words(s, words) for s in seen])
        at = np.concatenate([[ln - n + len(r) - 1 for r in s] for n, ln, s in zip(rows, lens, seen)])
        n = c.starts[-1]
        assert np.array_equal(masks[:n].cpu().numpy(), want)
        assert np.array_equal(pos[:n].cpu().numpy(), at)
        assert (masks[n:] == 99).all() and (pos[n:] == 99).all() and c.status.item() == 0
    m, p = c.cache.tree(c.batch, flat)
    assert torch.equal(m[:n], masks[:n, :m.shape[1]]) and torch.equal(p[:n], pos[:n])


def test_tree_of_the_largest_draft():
    n = 4096
    c = Case(64, 8, 8, kvtc.BF16, 1, [n], [n])
    masks, pos = c.cache.tree(c.batch, torch.arange(-1, n - 1, dtype=torch.int32, device="cuda"), status=c.status)
    bits = ((masks[:, :, None] >> torch.arange(32, dtype=torch.int32, device="cuda")) & 1).reshape(n, n)
    assert torch.equal(bits, torch.ones_like(bits).tril()) and torch.equal(pos, torch.arange(n, dtype=torch.int32, device="cuda"))
    assert c.status.item() == 0


def test_tree_reports_bad_parents():
    """A row's own number, a later one, below -1: roots, reported; a sequence
    outside the bounds is left alone."""
    c = Case(64, 8, 8, kvtc.BF16, 1, [4, 70], [10, 90])
    good = [-1, 0, 1, 1] + list(range(-1, 69))
    for at, bad in ((1, 1), (2, 3), (3, -2), (40, 66), (0, 2 ** 31 - 1), (73, -2 ** 31)):
        p = list(good)
        p[at] = bad
        masks, pos = c.cache.tree(c.batch, dev(p, torch.int32), status=c.status)
        assert c.status.item() == INV, (at, bad)
        c.status.zero_()
        p[at] = -1
        seen = [mx_ref.tree(p[:4]), mx_ref.tree(p[4:])]
        assert np.array_equal(masks.cpu().numpy(), np.concatenate([mx_ref.mask_words(s, 3) for s in seen]))
    b = c.cache.batch(c.table_dev, dev([10, 91], torch.int32), c.batch.row_start, total_rows=74, max_rows=70, max_len=90)
    masks = torch.full((74, 3), 99, dtype=torch.int32, device="cuda")
    c.cache.tree(b, dev(good, torch.int32), masks=masks, status=c.status)
    assert c.status.item() == INV and (masks[4:] == 99).all() and not (masks[:4] == 99).any()


# ---- attention over drafts


def random_masks(c, kind, words=None, junk=True):
    """(seen rows of every sequence, device words): trees, or any rows at all
    (itself or not, later ones, none); bits past a sequence's rows are set."""
    rows = [c.starts[z + 1] - c.starts[z] for z in range(len(c.lens))]
    words = words or max(-(-max(rows) // 32), 1)
    seen = []
    for n in rows:
        if kind == "tree":
            seen.append(mx_ref.tree(random_parents(c.rng, n)))
        else:
            seen.append([[j for j in range(n) if c.rng.random() < 0.4] if c.rng.random() > 0.15 else [] for _ in range(n)])
    w = [mx_ref.mask_words(s, words) for s in seen]
    if junk:
        for x, n in zip(w, rows):
            for j in range(n, 32 * words):
                x.view(np.uint32)[:, j // 32] |= np.uint32(1 << (j % 32))
    flat = np.full((c.total, words), -1, np.int32)
    flat[:c.starts[-1]] = np.concatenate(w) if w else flat[:0]
    return seen, dev(flat, torch.int32)


def check_tree_attention(c, q, got, lse, scale, seen, what):
    """The bounds of check_attention in test_gpu_mx."""
    kp, vp = c.unpacked()
    kp, vp = np.nan_to_num(kp), np.nan_to_num(vp)
    want, wlse, mass, spread = mx_ref.attention_seen(kp, vp, c.table, c.lens, c.starts, np64(q), scale, seen)
    n = c.starts[-1]
    o, s = np64(got)[:n], np64(lse)[:n]
    u = 2.0 ** -8 if c.dtype == kvtc.BF16 else 2.0 ** -23
    T = max(c.lens)
    ew = spread * (c.D * 2.0 ** -24 + 4 * 2.0 ** -24) + 2.0 ** -21
    steps = (T / 32 + 64) * 2.0 ** -24
    tol = (u + 2 * ew[..., None] + 2 * steps) * mass + u * np.abs(want) + 1e-30
    worst = float((np.abs(o - want[:n]) / tol[:n]).max())
    print(what, "worst error / bound %.3f" % worst, flush=True)
    assert worst <= 1.0
    empty = np.isneginf(wlse[:n])
    assert np.array_equal(np.isneginf(s), empty) and not o[empty].any()
    ltol = ew[:n] + steps + np.abs(np.where(empty, 0, wlse[:n])) * 2.0 ** -22
    assert (np.abs(np.where(empty, 0, s) - np.where(empty, 0, wlse[:n])) <= ltol).all()


def run_tree(c, G, masks, shared=0, **kw):
    q = c.rand(c.total, c.H * G, c.D, gain=0.2)
    out = torch.full((c.total, c.H * G, c.D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((c.total, c.H * G), 7.0, device="cuda")
    scale = c.D ** -0.5
    c.cache.attention_tree(c.batch, q, masks, shared, scale, out=out, lse=lse, status=c.status, **kw)
    assert c.status.item() == 0
    n = c.starts[-1]
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()
    return q, out, lse, scale


LENS = [1, 15, 16, 17, 31, 32, 33, 0, 5, 130, 257, 700, 3, 40]
ROWS = [1, 4, 2, 1, 3, 9, 5, 1, 7, 8, 0, 6, 5, 40]  # one with no tokens, one with more rows than tokens, one all draft


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
@pytest.mark.parametrize("D,bk,bv", FORMATS)
def test_tree_attention_formats(D, bk, bv, dtype, kind):
    """Ragged lengths in a pool whose unwritten bytes are all NaN."""
    c = Case(D, bk, bv, dtype, 2, ROWS, LENS, seed=D + bk + bv, total_rows=sum(ROWS) + 3)
    c.fill()
    seen, masks = random_masks(c, kind)
    q, out, lse, scale = run_tree(c, 3, masks)
    check_tree_attention(c, q, out, lse, scale, seen, f"D{D} k{bk} v{bv} dtype {dtype} {kind}")


@pytest.mark.parametrize("G", [1, 2, 5, 16, 24])
@pytest.mark.parametrize("most", [1, 4, 16, 33])
def test_tree_attention_groups(G, most):
    """Tiles of 16, 32 and 128 rows, some part full, in both types; masks of
    more words than needed."""
    for dtype in (kvtc.BF16, kvtc.FP32):
        rows = [1, most, max(most // 2, 1), most]
        lens = [40, 129 + most, max(most // 2, 1), 300]
        c = Case(128, 4, 4, dtype, 2, rows, lens, seed=G + most)
        c.fill()
        for kind in ("tree", "any"):
            seen, masks = random_masks(c, kind, words=3)
            q, out, lse, scale = run_tree(c, G, masks)
            check_tree_attention(c, q, out, lse, scale, seen, f"G{G} rows {most} dtype {dtype} {kind}")


@pytest.mark.parametrize("D,bk,bv", [(64, 8, 8), (128, 4, 4), (128, 8, 4)])
@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
def test_tree_attention_large_drafts(D, bk, bv, dtype):
    """Many rows a sequence, masks of many words that straddle pages and tiles."""
    rows, lens = [200, 61, 90, 130], [200, 333, 77, 1000]
    c = Case(D, bk, bv, dtype, 2, rows, lens, seed=bk)
    c.fill()
    for kind in ("tree", "any"):
        seen, masks = random_masks(c, kind)
        q, out, lse, scale = run_tree(c, 2, masks)
        check_tree_attention(c, q, out, lse, scale, seen, f"large D{D} k{bk} v{bv} dtype {dtype} {kind}")


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
def test_tree_attention_long_context(dtype):
    """One sequence over many ranges, drafts at and across their borders."""
    for ln, n in ((2047, 8), (2049, 30), (2176, 40), (20011, 7)):
        c = Case(128, 8, 4, dtype, 2, [n], [ln], seed=ln)
        c.fill()
        for kind in ("tree", "any"):
            seen, masks = random_masks(c, kind)
            q, out, lse, scale = run_tree(c, 4, masks)
            check_tree_attention(c, q, out, lse, scale, seen, f"context {ln} rows {n} dtype {dtype} {kind}")


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
@pytest.mark.parametrize("shared", [1, 3, 40])
def test_tree_attention_shared_prefix(shared, dtype):
    """Drafts past, at the end of, across the end of, and inside the prefix,
    empty sequences, sequences without rows; few rows and many."""
    p = 16 * shared
    lens = [p + 9, p + 40, p, max(p - 5, 0), 0, p + 300, p + 16, min(p, 3), p + 4]
    for rows in ([9, 2, 1, 3, 1, 0, 20, 5, 9], [1, 2, 1, 3, 1, 0, 1, 1, 8]):
        for D, bk, bv, G in ((128, 4, 4, 4), (64, 8, 4, 1)):
            c = Case(D, bk, bv, dtype, 2, rows, lens, seed=shared + D, shared=shared, total_rows=sum(rows) + 1)
            c.fill()
            for kind in ("tree", "any"):
                seen, masks = random_masks(c, kind)
                q, out, lse, scale = run_tree(c, G, masks, shared)
                check_tree_attention(c, q, out, lse, scale, seen, f"shared {shared} D{D} dtype {dtype} {kind}")
            out2 = torch.full_like(out, 7.0)
            c.table_dev[1:, :shared] = -1  # not read
            c.cache.attention_tree(c.batch, q, masks, shared, scale, out=out2, status=c.status)
            assert torch.equal(out, out2) and c.status.item() == 0


@pytest.mark.parametrize("rows,G", [(8, 2), (16, 4), (33, 3), (60, 8)])
@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
def test_tree_attention_nan_tokens(rows, G, dtype):
    """A NaN value of a draft's row, and of one before it: exactly the rows
    that see it, and only in its channel block, get NaN; a NaN key: the rows
    that see it."""
    D, ln = 64, 200 + rows
    c = Case(D, 8, 8, dtype, 1, [rows], [ln], seed=rows)
    c.fill()
    seen, masks = random_masks(c, "any")
    one = c.cache.batch(c.table_dev, c.batch.kv_lens, dev([0, ln], torch.int32), total_rows=ln, max_rows=ln, max_len=ln)
    k, v = (x[0].clone() for x in c.cache.read(one, *(torch.empty(1, 1, ln, D, dtype=DT[dtype], device="cuda") for _ in range(2))))
    q, good, _, _ = run_tree(c, G, masks)
    for j in (0, rows // 2, rows - 1, -30):
        t = 200 + j
        sees = torch.tensor([j < 0 or j in s for s in seen[0]], device="cuda")
        v2 = v.clone()
        v2[0, t, 40] = float("nan")
        c.cache.write(one, k[None], v2[None])
        out = c.cache.attention_tree(c.batch, q, masks)
        nan = torch.isnan(out)
        assert nan[sees][..., 32:].all() and not nan[sees][..., :32].any() and not nan[~sees].any(), j
        assert torch.equal(out[..., :32], good[..., :32]) and torch.equal(out[~sees], good[~sees])
        k2 = k.clone()
        k2[0, t, 3] = float("nan")
        c.cache.write(one, k2[None], v[None])
        out = c.cache.attention_tree(c.batch, q, masks)
        assert torch.isnan(out[sees]).all() and torch.equal(out[~sees], good[~sees]), j
        c.cache.write(one, k[None], v[None])


@pytest.mark.parametrize("G,most", [(4, 16), (8, 7)])
def test_tree_attention_longest_first(G, most):
    """More sequences in two tiles of 32 rows than the card holds at once: they
    are taken by length; some without rows, some without tokens, some equal."""
    n, H, D = 36, 8, 64
    rng = np.random.default_rng(G)
    lens = [int(x) for x in rng.integers(0, 2101, n)]
    rows = [int(x) for x in rng.integers(0, most + 1, n)]
    lens[0], lens[5], lens[6], lens[7], rows[0], rows[7] = 2100, 0, 1, 2100, most, most
    c = Case(D, 8, 4, kvtc.BF16, H, [1], [2100], seed=G)
    c.fill()
    c.table_dev, c.table = c.table_dev.expand(n, -1).contiguous(), c.table * n
    c.lens, c.rows, c.starts, c.total = lens, rows, [0] + [int(x) for x in np.cumsum(rows)], sum(rows) + 1
    c.batch = c.new_batch(rows, lens, max_rows=most)
    seen, masks = random_masks(c, "tree")
    q, out, lse, scale = run_tree(c, G, masks)
    check_tree_attention(c, q, out, lse, scale, seen, f"by length G{G}")


# How attention over drafts is cut up: (kv heads, query heads of each, sequences, most rows of one, longest, bound on
# the lengths, shared pages).  Rows of a sequence and kv head: up to 16 in one tile, up to 64 in tiles of 32, else of
# 128.  Eight waves a workgroup: one tile of 16, at most 256 workgroups, ranges of more than 512 tokens.  Past the
# caches: under these bounds the smallest record (1088 bytes of 16 tokens and a head) passes 256 MB.  By length: more
# than 256 / kv heads sequences and a bound of 2048 or more.
CUTS = {
    "16 rows": (2, 4, 9, 4, 500, 500, 0),
    "16 rows, eight waves": (2, 4, 128, 4, 600, 600, 0),
    "16 rows, eight waves, past the caches": (2, 4, 128, 4, 600, 16384, 0),
    "16 rows, eight waves, ranges": (32, 1, 1, 5, 4500, 4500, 0),
    "16 rows, eight waves, ranges, past the caches": (32, 1, 1, 5, 4500, 131072, 0),
    "16 rows, by length": (2, 4, 136, 4, 2100, 2100, 0),
    "16 rows, by length, past the caches": (2, 4, 136, 4, 700, 16384, 0),
    "16 rows, ranges": (2, 4, 3, 4, 2100, 2100, 0),
    "32 rows": (2, 4, 9, 16, 700, 700, 0),
    "32 rows, ranges": (2, 4, 2, 16, 2100, 2100, 0),
    "128 rows, ranges": (2, 4, 1, 40, 2100, 2100, 0),
    "prefix of 128 rows beside 16": (2, 4, 20, 4, 800, 800, 32),
    "prefix of 128 rows, 16 past the caches": (2, 4, 20, 4, 800, 131072, 32),
    "prefix of 128 rows, then 32": (2, 4, 9, 16, 800, 800, 32),
    "prefix of 128 rows beside 128": (2, 4, 6, 33, 800, 800, 32),
    "prefix of 32 rows, then 16": (2, 4, 4, 4, 800, 800, 32),
    "prefix of 16 rows": (2, 2, 2, 4, 800, 800, 32),
}


@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
@pytest.mark.parametrize("D,bk,bv", FORMATS)
def test_tree_attention_cuts(D, bk, bv, dtype, cut):
    """Every way that a call is cut up, in every format and type.  All
    sequences lie in the same pages; table entries from the longest on are
    outside the pool."""
    H, G, n, most, longest, bound, shared = CUTS[cut]
    rng = np.random.default_rng(n + D + bk)
    least = 16 * shared
    lens = [int(x) for x in rng.integers(least, longest + 1, n)]
    rows = [int(x) for x in rng.integers(0, most + 1, n)]
    lens[0], rows[0] = longest, most
    if n > 1:
        rows[1] = most
    if n > 3:
        lens[2], lens[3], rows[2], rows[3] = max(least - 5, 0), 1, 1, 1
    if n > 6:
        lens[4], rows[4], lens[6] = 0, 2, lens[5]
    c = Case(D, bk, bv, dtype, H, [1], [longest], seed=D + bv)
    c.fill()
    width = -(-bound // 16)
    assert (n * (bound - least) * H * (D * (bk + bv) // 8 + D // 16) > 2 ** 28) == ("past" in cut)
    c.table_dev = torch.cat([c.table_dev[:, :-1], c.table_dev[:, -1:].expand(1, width)], 1)[:, :width].expand(n, -1).contiguous()
    c.table = c.table * n
    c.lens, c.rows, c.starts, c.total = lens, rows, [0] + [int(x) for x in np.cumsum(rows)], sum(rows) + 1
    c.batch = c.new_batch(rows, lens, max_rows=most, max_len=bound)
    seen, masks = random_masks(c, "any" if (bk == 4) == (bv == 4) else "tree")
    print("cut", cut, D, bk, bv, dtype, flush=True)
    q, out, lse, scale = run_tree(c, G, masks, shared)
    check_tree_attention(c, q, out, lse, scale, seen, f"{cut} D{D} k{bk} v{bv} dtype {dtype}")


@pytest.mark.parametrize("rows", [[2, 3, 1], [20, 30, 25]])
def test_tree_attention_nan_in_the_prefix(rows):
    """A NaN value in the shared prefix reaches the rows that are past it, in
    its channels, and a sequence inside the prefix that ends before it not."""
    D, G, shared = 128, 4, 4
    lens = [64 + rows[0] + 5, 30 + rows[1], 64 + rows[2]]
    lens[1] = min(lens[1], 40)
    rows = [rows[0], min(rows[1], 12), rows[2]]
    c = Case(D, 8, 8, kvtc.BF16, 2, rows, lens, seed=4, shared=shared)
    c.fill()
    seen, masks = random_masks(c, "tree")
    q, good, _, _ = run_tree(c, G, masks, shared)
    at, _, so = mx_ref.places(D, 8, 8, 1)
    page, t = c.table[0][3], 10  # token 58
    c.cache.pool[0, page, 1, int(so[t, 2])] = 255  # channels 64 to 95 of kv head 1
    out = c.cache.attention_tree(c.batch, q, masks, shared)
    nan = torch.isnan(out)
    hit = torch.zeros_like(nan)
    for z in (0, 2):
        hit[c.starts[z]:c.starts[z + 1], G:, 64:96] = True
    assert torch.equal(nan, hit) and torch.equal(out[~hit], good[~hit])


def test_tree_attention_of_a_chain_is_causal():
    """A draft without branches, and a full mask, against the attentions that
    the cache had before: the same result within the bounds of both."""
    for rows, G in ((5, 3), (40, 4)):
        c = Case(128, 4, 8, kvtc.FP32, 2, [rows, rows], [rows, 300], seed=9)
        c.fill()
        q = c.rand(c.total, c.H * G, 128)
        chain = dev(list(range(-1, rows - 1)) * 2, torch.int32)
        masks, pos = c.cache.tree(c.batch, chain)
        assert pos.tolist() == list(range(rows)) + list(range(300 - rows, 300))
        a, b = c.cache.attention_tree(c.batch, q, masks), c.cache.attention(c.batch, q)
        assert (a - b).abs().max() <= 1e-5 * b.abs().max()
        a, b = c.cache.attention_tree(c.batch, q, torch.full_like(masks, -1)), c.cache.attention(c.batch, q, causal=False)
        assert (a - b).abs().max() <= 1e-5 * b.abs().max()


def test_tree_attention_bad_metadata():
    """A sequence outside the bounds is skipped, a page outside the pool is
    masked, and either is reported; the others are as without."""
    D, H, G = 128, 2, 2
    rows, lens = [6, 20, 3], [40, 50, 33]
    c = Case(D, 4, 4, kvtc.BF16, H, rows, lens, seed=8)
    c.fill()
    seen, masks = random_masks(c, "tree")
    q, good, _, scale = run_tree(c, G, masks)
    for bad_lens, starts in (([40, 51, 33], [0, 6, 26, 29]), ([40, -1, 33], [0, 6, 26, 29]), ([40, 50, 33], [0, 6, 27, 26])):
        b = c.cache.batch(c.table_dev, dev(bad_lens, torch.int32), dev(starts, torch.int32), total_rows=29, max_rows=20, max_len=50)
        out = torch.full_like(q, 7.0)
        c.cache.attention_tree(b, q, masks, out=out, status=c.status)
        assert c.status.item() == INV and torch.equal(out[:6], good[:6])
        c.status.zero_()
    c.table_dev[1, 2] = c.pages  # the last 18 tokens of sequence 1 lie in pages 2 and 3
    out = c.cache.attention_tree(c.batch, q, masks, status=c.status)
    assert c.status.item() == INV and torch.equal(out[:6], good[:6]) and torch.equal(out[26:], good[26:])
    kp, vp = c.unpacked()
    k, v = mx_ref.tokens(kp, vp, c.table[1], 50)
    for i in range(20):
        at = [t for t in list(range(30)) + [30 + j for j in seen[1][i]] if t // 16 != 2]
        for h in range(H * G):
            s = scale * (k[h // G, at] @ np64(q)[6 + i, h])
            p = np.exp(s - s.max())
            want = p @ v[h // G, at] / p.sum()
            assert np.abs(np64(out)[6 + i, h] - want).max() <= 2.0 ** -7 * np.abs(v[h // G, at]).max()


# ---- keeping


def check_keep(c, seen, nodes, before, lens_out, layers):
    """Kept tokens hold the codes of the rows that were kept; every byte before
    the draft, of other layers and of other pages is as it was."""
    got, lens = c.cache.pool.cpu().numpy(), lens_out.tolist()
    where = [mx_ref.places(c.D, c.bk, c.bv, kv) for kv in (0, 1)]
    free = np.zeros(got.shape, bool)  # bytes that may be anything
    for z, ln in enumerate(c.lens):
        n = c.starts[z + 1] - c.starts[z]
        base = ln - n
        kept = [j for j in (seen[z][nodes[z]] if n and nodes[z] >= 0 else []) if base + j >= 0]
        assert lens[z] == (max(base, 0) + len(kept) if n else ln), z
        for t in range(max(base, 0), ln):
            pg, r = c.table[z][t // 16], t % 16
            for at, _, so in where:
                free[np.ix_(layers, [pg], range(c.H), np.unique(np.concatenate([at[r], so[r]])))] = True
        for i, j in enumerate(kept):
            a, b = base + j, max(base, 0) + i
            for at, _, so in where:
                for idx in (at, so):
                    x = before[layers][:, c.table[z][a // 16]][:, :, idx[a % 16]]
                    assert np.array_equal(got[layers][:, c.table[z][b // 16]][:, :, idx[b % 16]], x), (z, i)
    assert np.array_equal(got[~free], before[~free])


@pytest.mark.parametrize("D,bk,bv", FORMATS)
def test_keep(D, bk, bv):
    """Trees and any rows, in one layer, some and all; nodes first, last, none;
    a sequence with more rows than tokens, without rows, without tokens."""
    rows, lens = [5, 1, 17, 0, 40, 6, 33, 3], [5, 20, 40, 9, 200, 4, 37, 0]
    for kind in ("tree", "any"):
        for layer, layers in ((0, 3), (1, 1), (1, None)):
            c = Case(D, bk, bv, kvtc.BF16, 3, rows, lens, layers=3, seed=D + bk + bv, total_rows=sum(rows) + 2)
            c.cache.pool.copy_(torch.as_tensor(c.rng.integers(0, 256, tuple(c.cache.pool.shape)), dtype=torch.uint8))
            seen, masks = random_masks(c, kind)
            nodes = [int(c.rng.integers(-1, max(n, 1))) for n in rows]
            nodes[4], nodes[6], nodes[1] = 39, 32, -1
            before = c.cache.pool.cpu().numpy()
            print("keep", D, bk, bv, kind, layer, layers, flush=True)
            out = c.cache.keep(c.batch, dev(nodes, torch.int32), masks, layer=layer, layers=layers, status=c.status)
            assert c.status.item() == 0
            check_keep(c, seen, nodes, before, out, list(range(layer, 3 if layers is None else layer + layers)))


def test_keep_many_heads():
    """Enough heads, layers and sequences that a wave takes several (layer,
    head) pairs, the last of them fewer."""
    rows, lens = [5, 1, 17, 0, 40, 6, 33, 3], [5, 20, 40, 9, 60, 4, 37, 0]
    for D, bk, bv in ((64, 8, 4), (128, 4, 4)):
        c = Case(D, bk, bv, kvtc.BF16, 7, rows, lens, layers=43, seed=D)
        assert 43 * 7 * len(rows) > 2048
        c.cache.pool.copy_(torch.as_tensor(c.rng.integers(0, 256, tuple(c.cache.pool.shape)), dtype=torch.uint8))
        for kind in ("tree", "any"):
            seen, masks = random_masks(c, kind)
            nodes = [int(c.rng.integers(-1, max(n, 1))) for n in rows]
            nodes[4], nodes[6] = 39, 32
            before = c.cache.pool.cpu().numpy()
            out = c.cache.keep(c.batch, dev(nodes, torch.int32), masks, status=c.status)
            assert c.status.item() == 0
            check_keep(c, seen, nodes, before, out, list(range(43)))


def test_keep_long_paths():
    """Hundreds of kept rows: most move within and across the chunks that are
    read before they are written; all rows kept moves nothing."""
    for n, drop in ((300, 1), (300, 17), (1000, 3), (4096, 2)):
        c = Case(64, 8, 8, kvtc.FP32, 1, [n], [n + 21], seed=n)
        c.cache.pool.copy_(torch.as_tensor(c.rng.integers(0, 256, tuple(c.cache.pool.shape)), dtype=torch.uint8))
        before = c.cache.pool.cpu().numpy()
        last = [j for j in range(n) if j % (drop + 1) or j == n - 1]
        seen = [[[]] * (n - 2) + [list(range(n)), last]]
        masks = dev(mx_ref.mask_words(seen[0], -(-n // 32)), torch.int32)
        out = c.cache.keep(c.batch, dev([n - 2], torch.int32), masks, status=c.status)
        assert out.tolist() == [n + 21] and np.array_equal(c.cache.pool.cpu().numpy(), before)
        out = c.cache.keep(c.batch, dev([n - 1], torch.int32), masks, status=c.status)
        check_keep(c, seen, [n - 1], before, out, [0])
        assert c.status.item() == 0


def test_keep_reports_and_skips():
    rows, lens = [6, 8, 5], [40, 50, 33]
    c = Case(64, 4, 8, kvtc.BF16, 2, rows, lens, seed=3)
    c.cache.pool.copy_(torch.as_tensor(c.rng.integers(0, 256, tuple(c.cache.pool.shape)), dtype=torch.uint8))
    seen, masks = random_masks(c, "tree")
    before = c.cache.pool.clone()
    for node in (-2, 8, 2 ** 31 - 1, -2 ** 31):
        out = c.cache.keep(c.batch, dev([-1, node, -1], torch.int32), masks, status=c.status)
        assert out.tolist() == [34, 50, 28] and c.status.item() == INV and torch.equal(c.cache.pool, before)
        c.status.zero_()
    b = c.cache.batch(c.table_dev, dev([40, 51, 33], torch.int32), c.batch.row_start, total_rows=19, max_rows=8, max_len=50)
    out = c.cache.keep(b, dev([-1, 7, -1], torch.int32), masks, status=c.status)
    assert out.tolist() == [34, 51, 28] and c.status.item() == INV and torch.equal(c.cache.pool, before)
    c.status.zero_()
    # rows 0, 3, 6, 7 of sequence 1: tokens 42 to 49 in pages 2 and 3; page 3 (tokens 48, 49: rows 6, 7) outside
    words = dev([[0b11001001]], torch.int32).expand(19, 1).contiguous()
    c.table_dev[1, 3] = -5
    out = c.cache.keep(c.batch, dev([-1, 0, -1], torch.int32), words, status=c.status)
    assert out.tolist() == [34, 46, 28] and c.status.item() == INV
    want = before.cpu().numpy().copy()
    rec, (pk, pv) = want[0, c.table[1][2]], (mx_ref.places(64, 4, 8, kv) for kv in (0, 1))
    for at, _, so in (pk, pv):
        for idx in (at, so):
            rec[:, idx[43 % 16]] = before[0, c.table[1][2]].cpu().numpy()[:, idx[45 % 16]]  # row 3 (token 45) moves to 43
    assert np.array_equal(c.cache.pool.cpu().numpy(), want)


def test_keep_reports_pages_of_tokens_that_stay():
    """A path that keeps its place, as a draft accepted whole, or the first
    part of one: a page outside the pool that a kept token stands in is
    reported though nothing moves there; one of dropped rows alone is not."""
    n, ln = 40, 70  # tokens 30 to 69: pages 1 (rows 0, 1) to 4 (rows 34 to 39)
    first = list(range(20))  # rows 0 to 19, tokens 30 to 49: pages 1, 2 and two tokens of page 3
    gap = first + [39]  # row 39 (page 4) moves to token 50, in page 3
    seen = [[list(range(n)), first, gap] + [[i] for i in range(3, n)]]
    for D, bk, bv, H, layers in ((64, 4, 8, 2, 1), (128, 8, 4, 8, 300)):  # one (layer, head) pair a wave, and four
        c = Case(D, bk, bv, kvtc.BF16, H, [n], [ln], layers=layers, seed=D)
        c.cache.pool.fill_(0x11)
        masks = dev(mx_ref.mask_words(seen[0], 2), torch.int32)
        for node, kept, pages in ((0, 40, (1, 2, 3, 4)), (1, 20, (1, 2, 3)), (2, 21, (1, 2, 3, 4))):
            for page in (1, 2, 3, 4):
                table = c.table_dev.clone()
                table[0, page] = -1 if page % 2 else c.pages
                b = c.cache.batch(table, c.batch.kv_lens, c.batch.row_start, total_rows=n, max_rows=n, max_len=ln)
                before = c.cache.pool.clone()
                out = c.cache.keep(b, dev([node], torch.int32), masks, status=c.status)
                assert out.tolist() == [30 + kept] and c.status.item() == (INV if page in pages else 0), (node, page)
                assert torch.equal(c.cache.pool, before)  # all bytes are alike
                c.status.zero_()


# ---- together


def test_offsets_past_32_bits():
    """The same draft in a small pool and in the last pages of one of 4.5 GB:
    the same codes, outputs and kept tokens."""
    H, D, ln, n = 8, 128, 300, 20
    pages, last = -(-ln // 16), 65000
    cfg = dict(layers=2, kv_heads=H, head_dim=D, dtype=kvtc.BF16, bits_k=8, bits_v=8)
    c = Case(D, 8, 8, kvtc.BF16, H, [n], [ln], seed=16)
    k, v, q = c.rand(ln, H, D), c.rand(ln, H, D), c.rand(n, 2 * H, D)
    seen, masks = random_masks(c, "tree")
    got = []
    for size in (pages, last):
        cache = kvtc.MxCache(cfg, size)
        table = dev([list(range(size - 1, size - 1 - pages, -1))], torch.int32)

        def batch(rows, ln=ln):
            return cache.batch(table, dev([ln], torch.int32), dev([0, rows], torch.int32), rows, rows, ln)

        cache.write_rope(batch(ln), k, v, rope_of(D), layer=1, status=c.status)
        outs = [cache.pool[1, table[0, :ln // 16].long()]]
        for shared in (0, 10):
            outs.append(cache.attention_tree(batch(n), q, masks, shared, layer=1, status=c.status))
        new = cache.keep(batch(n), dev([n - 1], torch.int32), masks, layer=1, status=c.status)
        ko, vo = (torch.empty(int(new.item()), H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        outs += [new, *cache.read(batch(len(ko), len(ko)), ko, vo, layer=1, status=c.status)]
        got.append(outs)
    assert c.status.item() == 0
    for small, big in zip(*got):
        assert torch.equal(small, big)


def test_captured_drafts_follow_the_device_arrays():
    """A whole step captured once (tree, rotated append, attention behind a
    prefix and without, keeping) and replayed while lengths, rows, trees and
    nodes change; every replay against the eager calls.  (At most one sequence
    writes into the two shared pages: two would write the same rows.)"""
    D, H, G, n, most = 128, 2, 4, 3, 3000  # ranges, so workspaces
    c = Case(D, 8, 4, kvtc.BF16, H, [8] * n, [most] * n, seed=14, shared=2)
    c.fill()
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, starts = dev([90, 40, 48], torch.int32), dev([0, 8, 12, 20], torch.int32)
    b = c.cache.batch(c.table_dev, lens, starts, total_rows=24, max_rows=12, max_len=most)
    qkv = c.rand(24, (G + 2) * H, D)
    q, k, v = qkv.split([G * H, H, H], 1)
    rope = rope_of(D)
    parents, nodes = torch.zeros(24, **i32), torch.zeros(n, **i32)
    bufs = [dict(masks=torch.zeros(24, 1, **i32), pos=torch.zeros(24, **i32), q=torch.zeros(24, G * H, D, dtype=q.dtype, device="cuda"),
                 o=torch.zeros(24, G * H, D, dtype=q.dtype, device="cuda"), o2=torch.zeros(24, G * H, D, dtype=q.dtype, device="cuda"),
                 lens=torch.zeros(n, **i32)) for _ in range(2)]
    ws = [c.cache.workspace_tree(b, G * H), c.cache.workspace_tree(b, G * H, 2)]
    assert all(w.nbytes > 16 for w in ws)

    def step(x):
        c.cache.tree(b, parents, masks=x["masks"], positions=x["pos"], status=c.status)
        c.cache.write_rope(b, k, v, rope, positions=x["pos"], q=q, out=x["q"], status=c.status)
        c.cache.attention_tree(b, x["q"], x["masks"], out=x["o"], ws=ws[0], status=c.status)
        c.cache.attention_tree(b, x["q"], x["masks"], 2, out=x["o2"], ws=ws[1], status=c.status)
        c.cache.keep(b, nodes, x["masks"], lens_out=x["lens"], status=c.status)

    parents.fill_(-1)
    start = c.cache.pool.clone()
    step(bufs[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(bufs[0])
    for r, (ln, rows) in enumerate([((90, 40, 48), (8, 4, 8)), ((700, 128, 33), (12, 0, 12)), ((129, 640, 44), (3, 12, 9)),
                                    ((5, 52, 0), (8, 12, 2)), ((257, 90, 40), (1, 1, 1))]):
        lens.copy_(dev(list(ln), torch.int32))
        at = [0] + [int(x) for x in np.cumsum(rows)]
        starts.copy_(dev(at, torch.int32))
        p = [x for m in rows for x in random_parents(c.rng, m)]
        parents.copy_(dev(p + [-1] * (24 - len(p)), torch.int32))
        nodes.copy_(dev([int(c.rng.integers(-1, max(m, 1))) for m in rows], torch.int32))
        qkv.copy_(c.rand(24, (G + 2) * H, D))
        got = []
        for x, f in ((bufs[0], g.replay), (bufs[1], lambda: step(bufs[1]))):
            c.cache.pool.copy_(start)
            for y in x.values():
                y.fill_(7)
            f()
            torch.cuda.synchronize()
            got.append((c.cache.pool.clone(), {name: y.clone() for name, y in x.items()}))
        assert torch.equal(got[0][0], got[1][0]), r
        for name in got[0][1]:
            assert torch.equal(got[0][1][name], got[1][1][name]), (r, name)
            if name not in ("lens",):
                assert (got[0][1][name][at[-1]:] == 7).all(), (r, name)
    assert c.status.item() == 0


def test_on_other_streams_at_once():
    rows, lens = [8] * 6, [900, 9, 77, 2000, 512, 8]
    c = Case(128, 4, 8, kvtc.BF16, 2, rows, lens, seed=13)
    c.fill()
    q = c.rand(48, 8, 128)
    seen, masks = random_masks(c, "tree")
    parents = dev([p for _ in rows for p in random_parents(c.rng, 8)], torch.int32)
    good, tree = c.cache.attention_tree(c.batch, q, masks), c.cache.tree(c.batch, parents)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for s in streams:  # both at once, each with a workspace of its own
            outs.append((c.cache.attention_tree(c.batch, q, masks, stream=s), *c.cache.tree(c.batch, parents, stream=s)))
    torch.cuda.synchronize()
    for o, m, p in outs:
        assert torch.equal(o, good) and torch.equal(m, tree[0]) and torch.equal(p, tree[1])


def test_drafted_decoding_is_plain_decoding():
    """A conversation decoded in drafts (tree, rotated append at the nodes'
    positions, attention, a path kept) against one decoded token by token: the
    kept cache is byte for byte the plain one's, and the rows on the path get
    what the plain steps got.  Layers, ragged sequences, a path that ends in
    the middle, drafts of which nothing or everything is right."""
    L, H, G, D, n = 2, 2, 3, 64, 3
    cfg = dict(layers=L, kv_heads=H, head_dim=D, dtype=kvtc.BF16, bits_k=8, bits_v=4)
    rng = np.random.default_rng(77)
    first, total, most = [20, 33, 7], 24, 6
    pages = -(-(max(first) + total + most) // 16)
    table = dev(rng.permutation(n * pages).reshape(n, pages), torch.int32)
    plain, spec = kvtc.MxCache(cfg, n * pages), kvtc.MxCache(cfg, n * pages)
    for x in (plain, spec):
        x.pool.zero_()
    rope = rope_of(D)
    gen = torch.Generator(device="cuda").manual_seed(5)
    rows = sum(first)
    qkv = torch.randn(L, rows, (G + 2) * H, D, generator=gen, device="cuda").to(torch.bfloat16)
    starts = dev([0] + [int(x) for x in np.cumsum(first)], torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for x in (plain, spec):  # the prompts
        b = x.batch(table, dev(first, torch.int32), starts, rows, max(first), pages * 16)
        for l in range(L):
            x.write_rope(b, qkv[l, :, G * H:(G + 1) * H], qkv[l, :, (G + 1) * H:], rope, layer=l, status=status)
    # what a model would give for token t of sequence z, and for a wrong token instead
    right, wrong = (torch.randn(L, n, total, (G + 2) * H, D, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    want = torch.zeros(L, n, total, G * H, D, dtype=torch.bfloat16, device="cuda")
    lens = dev(first, torch.int32)
    one = plain.batch(table, lens, dev(list(range(n + 1)), torch.int32), n, 1, pages * 16)
    for t in range(total):
        lens += 1
        for l in range(L):
            x = right[l, :, t]
            q = plain.write_rope(one, x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:], rope, q=x[:, :G * H], layer=l, status=status)
            want[l, :, t] = plain.attention(one, q, layer=l, status=status)
    at, lens = [0] * n, dev(first, torch.int32)
    while min(at) < total:
        parents, good, nodes, rowstart = [], [], [], [0]
        for z in range(n):
            m = int(rng.integers(0, most + 1)) if at[z] < total else 0
            ps = [int(rng.integers(-1, i)) for i in range(m)]
            # one path through the tree is right: follow children from the root
            path, cur = [], -1
            for i in range(m):
                if ps[i] == cur and len(path) < total - at[z] and rng.random() < 0.8:
                    path.append(i)
                    cur = i
            parents += ps
            good.append(path)
            nodes.append(cur)
            rowstart.append(rowstart[-1] + m)
        r = rowstart[-1]
        if r == 0:
            continue
        grown = dev([int(x) + rowstart[z + 1] - rowstart[z] for z, x in enumerate(lens.tolist())], torch.int32)
        b = spec.batch(table, grown, dev(rowstart, torch.int32), r, most, pages * 16)
        masks, pos = spec.tree(b, dev(parents, torch.int32), status=status)
        for l in range(L):
            x = torch.empty(r, (G + 2) * H, D, dtype=torch.bfloat16, device="cuda")
            for z in range(n):
                for i in range(rowstart[z + 1] - rowstart[z]):
                    ok = i in good[z]
                    x[rowstart[z] + i] = right[l, z, at[z] + good[z].index(i)] if ok else wrong[l, z, (at[z] + i) % total]
            q = spec.write_rope(b, x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:], rope, positions=pos, q=x[:, :G * H], layer=l, status=status)
            out = spec.attention_tree(b, q, masks, layer=l, status=status)
            for z in range(n):
                for d, i in enumerate(good[z]):
                    a, w = out[rowstart[z] + i].float(), want[l, z, at[z] + d].float()
                    # both within 2^-8 of the terms' and of the output's magnitude; at most 64 weights of the values' size
                    assert (a - w).abs().max() <= 4 * 2.0 ** -8 * 8, (l, z, d)
        lens = spec.keep(b, dev(nodes, torch.int32), masks, status=status)
        for z in range(n):
            at[z] += len(good[z])
            assert lens[z].item() == first[z] + at[z]
    assert status.item() == 0
    where = [mx_ref.places(D, 8, 4, kv) for kv in (0, 1)]
    a, b = plain.pool.cpu().numpy(), spec.pool.cpu().numpy()
    for z in range(n):
        for t in range(first[z] + total):
            pg = int(table[z, t // 16])
            for at_, _, so in where:
                for idx in (at_, so):
                    assert np.array_equal(a[:, pg][:, :, idx[t % 16]], b[:, pg][:, :, idx[t % 16]]), (z, t)
