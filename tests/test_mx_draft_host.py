"""Rotated appends and drafts on the microscaled cache, on the CPU: the plain
implementation's own pins, and what the library and the binding refuse before
anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import mx_ref
from tensor_compression_amd import kvtc
from test_mx_host import CAP, INV, P, UNS, batch, cfg, size, strides

CALLS = ("rope", "attn", "keep")


def rope(axis=None, **kw):
    r = dict(style=0, rot_dim=128, axes=1, reserved=0, freqs=P, axis=axis)
    r.update(kw)
    return kvtc.MxRopeStruct(*[r[f] for f, _ in kvtc.MxRopeStruct._fields_])


def call(name, c=None, b=None, r=None, **kw):
    c, b, r = c or cfg(), b or batch(), r or rope()
    a = dict(layer=0, n_layers=1, positions=P, k=P, ks=strides(0, 128, 512), v=P, vs=strides(0, 128, 512), q=P, q_stride=1024,
             q_heads=8, q_out=P + 4096, q_out_stride=1024, pool=P, pool_bytes=1 << 40, status=P, masks=P, words=1, shared=2,
             scale=0.1, out=P, lse=P, ws=P, ws_bytes=1 << 40, nodes=P, lens_out=P + 64, parents=P + 8192, tree_positions=P + 12288)
    a.update(kw)
    L, cr, br = kvtc.lib(), ctypes.byref(c), ctypes.byref(b)
    if name == "rope":
        return L.kvtc_mx_write_rope(cr, br, a["layer"], a["n_layers"], ctypes.byref(r), a["positions"], a["k"], a["ks"],
                                    a["v"], a["vs"], a["q"], a["q_stride"], a["q_heads"], a["q_out"], a["q_out_stride"],
                                    a["pool"], a["pool_bytes"], a["status"], None)
    if name == "tree":
        return L.kvtc_mx_tree(br, a["parents"], a["masks"], a["words"], a["tree_positions"], a["status"], None)
    if name == "keep":
        return L.kvtc_mx_keep(cr, br, a["layer"], a["n_layers"], a["masks"], a["words"], a["nodes"], a["pool"],
                              a["pool_bytes"], a["lens_out"], a["status"], None)
    return L.kvtc_mx_attn_tree(cr, br, a["layer"], a["pool"], a["pool_bytes"], a["shared"], a["masks"], a["words"], a["q"],
                               a["q_stride"], a["q_heads"], a["scale"], a["out"], a["lse"], a["ws"], a["ws_bytes"],
                               a["status"], None)


# ---- the plain implementation


@pytest.mark.parametrize("half", [True, False])
def test_rotation_keeps_lengths_and_adds_up(half):
    """A pair's length stays; turning by t and then u is turning by t + u; the
    product of two rotated vectors depends on the distance alone."""
    rng = np.random.default_rng(0)
    f, axis = [10000.0 ** (-j / 32) for j in range(32)], [j % 2 for j in range(32)]
    x, y = rng.standard_normal((2, 5, 3, 80))
    t, u = rng.integers(-1000, 1000, (2, 2, 5))
    a = mx_ref.rotate(x, t, f, axis, half)
    assert np.allclose(np.square(a).sum(-1), np.square(x).sum(-1), rtol=1e-12) and np.array_equal(a[..., 64:], x[..., 64:])
    assert np.allclose(mx_ref.rotate(a, u, f, axis, half), mx_ref.rotate(x, t + u, f, axis, half), atol=1e-10)
    b = mx_ref.rotate(y, t + 77, f, axis, half)
    want = (x * mx_ref.rotate(y, np.full((2, 5), 77), f, axis, half)).sum(-1)
    assert np.allclose((a * b).sum(-1), want, atol=1e-10)
    # the first pair by a radian
    one = mx_ref.rotate(np.eye(80)[:1, None], np.ones((2, 1), int), f, axis, half)[0, 0]
    assert np.isclose(one[0], np.cos(1)) and np.isclose(one[32 if half else 1], np.sin(1))


def test_tree_and_masks():
    seen = mx_ref.tree([-1, 0, 0, 2, -1, 4, 3])
    assert seen == [[0], [0, 1], [0, 2], [0, 2, 3], [4], [4, 5], [0, 2, 3, 6]]
    assert mx_ref.mask_words(seen, 2).tolist() == [[1, 0], [3, 0], [5, 0], [13, 0], [16, 0], [48, 0], [77, 0]]
    assert mx_ref.mask_words([[31, 32]], 2).tolist() == [[-2 ** 31, 1]]


def test_attention_of_a_chain_is_causal():
    rng = np.random.default_rng(1)
    D, bk, bv = 64, 8, 8
    pool = np.zeros((4, 2, mx_ref.record_bytes(D, bk, bv)), np.uint8)
    lens, starts, table = [20, 33], [0, 20, 25], [[0], [1, 3, 2]]
    table[0] = [0, 0]
    k, v = rng.standard_normal((2, 33, 2, D))
    mx_ref.write(pool, table[1:], [33], [0, 33], k, v, D, bk, bv)
    kp, vp = mx_ref.unpack(pool, D, bk, bv)
    q = rng.standard_normal((25, 4, D))
    seen = [mx_ref.tree(list(range(-1, n - 1))) for n in (20, 5)]
    for a, b in zip(mx_ref.attention_seen(kp, vp, table, lens, starts, q, 0.1, seen),
                    mx_ref.attention(kp, vp, table, lens, starts, q, 0.1, True)):
        # sums of at most 64 terms below 10, whose order may differ: 64 steps of 2^-53 of 640
        assert np.array_equal(np.isinf(a), np.isinf(b)) and np.allclose(a, b, rtol=0, atol=64 * 2.0 ** -53 * 640)


# ---- refusals


@pytest.mark.parametrize("bad,want", [
    (dict(layers=0), INV), (dict(kv_heads=0), INV), (dict(pool_pages=0), INV), (dict(dtype=2), INV),
    (dict(bits_k=5), INV), (dict(bits_v=16), INV), (dict(head_dim=96), UNS), (dict(layers=8193, kv_heads=8), UNS)])
def test_bad_configurations(bad, want):
    for name in CALLS:
        assert call(name, c=cfg(**bad)) == want, name
    n = ctypes.c_size_t(0)
    assert kvtc.lib().kvtc_mx_attn_tree_workspace(ctypes.byref(cfg(**bad)), ctypes.byref(batch()), 8, 0, ctypes.byref(n)) == want


@pytest.mark.parametrize("bad", [
    dict(n_seqs=-1), dict(max_pages=0), dict(total_rows=-1), dict(max_rows=-1), dict(max_len=-1), dict(max_len=97),
    dict(reserved=1), dict(page_table=None), dict(kv_lens=None), dict(row_start=None), dict(page_table=P + 2),
    dict(kv_lens=P + 1), dict(row_start=P + 2)])
def test_bad_batches(bad):
    for name in CALLS + ("tree",):
        assert call(name, b=batch(**bad)) == INV, name
    n = ctypes.c_size_t(0)
    assert kvtc.lib().kvtc_mx_attn_tree_workspace(ctypes.byref(cfg()), ctypes.byref(batch(**bad)), 8, 0, ctypes.byref(n)) == INV


@pytest.mark.parametrize("name", CALLS)
def test_bad_pool_layer_status(name):
    need = size(cfg())[2]
    for bad, want in ((dict(pool=None), INV), (dict(pool=P + 8), INV), (dict(pool_bytes=need - 1), CAP),
                      (dict(layer=-1), INV), (dict(layer=2), INV), (dict(status=P + 2), INV)):
        assert call(name, **bad) == want, bad


@pytest.mark.parametrize("bad,want", [
    (dict(style=2), INV), (dict(rot_dim=0), INV), (dict(rot_dim=144), INV), (dict(rot_dim=-16), INV), (dict(rot_dim=24), UNS),
    (dict(rot_dim=127), UNS), (dict(axes=0), INV), (dict(axes=5), INV), (dict(reserved=1), INV), (dict(freqs=None), INV),
    (dict(freqs=P + 4), INV), (dict(axis=bytes([0] * 63 + [1])), INV), (dict(axes=3, axis=bytes([3] + [0] * 63)), INV)])
def test_bad_rotations(bad, want):
    assert call("rope", r=rope(**bad)) == want
    assert call("rope", r=rope(**bad), q_heads=0, q=None, q_out=None) == want


def test_bad_rotated_rows():
    for bad in (dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 2), dict(ks=None), dict(vs=None),
                dict(ks=strides(0, 128, -512)), dict(vs=strides(0, 124, 512)), dict(ks=strides(0, 128, 2 ** 47)),
                dict(n_layers=0), dict(n_layers=3), dict(layer=1, n_layers=2), dict(positions=P + 2), dict(q=None),
                dict(q_out=None), dict(q=P + 8), dict(q_out=P + 4), dict(q_heads=-1), dict(q_stride=-8), dict(q_stride=12),
                dict(q_out_stride=12), dict(q_out_stride=1016), dict(q_out_stride=2 ** 47), dict(n_layers=2),
                dict(q_out=P, q_stride=2048)):
        assert call("rope", **bad) == INV, bad
    assert call("rope", r=rope(axes=2, axis=bytes([0, 1] * 32)), positions=None) == INV
    assert call("rope", b=batch(n_seqs=2 ** 20, total_rows=2 ** 20, max_rows=2 ** 10)) == UNS
    assert call("rope", c=cfg(layers=16384), n_layers=1, q_heads=2 ** 30 // 128, q_stride=2 ** 30, q_out_stride=2 ** 30) == UNS


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 30, 2 ** 31 - 31])
def test_rotated_rows_past_a_launch(rows):
    """Row bounds at the end of int32: more pages than a launch has workgroups."""
    for heads in (0, 8):
        assert call("rope", b=batch(total_rows=rows, max_rows=rows), q_heads=heads) == UNS


def test_rotated_queries_apart_from_what_is_read():
    """Slices of any strides and heads near each other: refused exactly where
    a written element is one that the call reads, but for queries in place."""
    rng = np.random.default_rng(11)
    D, unit = 64, 8  # elements of 2 bytes, strides in whole 16 bytes

    def taken(at, strides, extent):  # 16-byte units
        i = np.add.outer(np.arange(extent[0]) * strides[0], np.arange(extent[1]) * strides[1])
        return set((at // 16 + np.add.outer(i.ravel() // unit, np.arange(D // unit))).ravel().tolist())

    def some(*choices):
        return int(rng.choice(choices))

    seen = [0, 0, 0]
    for trial in range(3000):
        rows, H, G = some(1, 2, 5), some(1, 2), some(1, 2, 3)
        fused = (G + 2) * H * D
        qw = G * H * D
        qs, os = some(0, qw, fused, fused, qw + 8, 2 * qw), some(qw, fused, fused, 2 * qw, qw + 24)
        ks = [(D, fused), (D, fused), (D, H * D), (rows * D, D), (0, D), (D, 0), (D + 8, 3 * D + 8)][some(*range(7))]
        base = P + 0x100000
        q = base + 16 * some(0, 0, 0, *range(0, 200, 7))
        q_out = q if trial % 3 == 0 else base + 16 * some(*range(-60, 260))
        k = q + 2 * qw if trial % 2 else base + 16 * some(*range(-100, 300))
        v = k + 2 * H * D if trial % 5 else base + 16 * some(*range(2000, 2500))
        out = taken(q_out, (os, D), (rows, G * H))
        b = batch(n_seqs=1, total_rows=rows, max_rows=rows, page_table=P, kv_lens=P + 0x10000, row_start=P + 0x20000)
        bad = q == q_out and qs != os  # in place: the same strides
        bad |= q != q_out and bool(out & taken(q, (qs, D), (rows, G * H)))
        bad |= any(out & taken(x, (ks[1], ks[0]), (rows, H)) for x in (k, v))
        got = call("rope", c=cfg(head_dim=D, kv_heads=H), b=b, r=rope(rot_dim=D, freqs=P + 0x30000), positions=P + 0x40000, k=k, v=v,
                   ks=strides(0, *ks), vs=strides(0, *ks), q=q, q_stride=qs, q_heads=G * H, q_out=q_out, q_out_stride=os,
                   pool=P + 0x8000000)
        assert got == INV if bad else launched(got), (trial, rows, H, G, qs, os, ks, q - base, q_out - base, k - base, v - base)
        seen[2 if bad else q == q_out] += 1
    assert min(seen) > 100, seen  # of each kind


def test_rotated_queries_apart_from_small_inputs_and_the_pool():
    need = size(cfg())[2]
    b = batch(n_seqs=3, total_rows=5, max_rows=5, page_table=P, kv_lens=P + 0x10000, row_start=P + 0x20000)
    for at, n in ((P, 3 * 6 * 4), (P + 0x10000, 3 * 4), (P + 0x20000, 4 * 4), (P + 0x30000, 64 * 8), (P + 0x40000, 2 * 5 * 4),
                  (P + 0x8000000, need)):
        last = at + n - 1 - (at + n - 1) % 16
        for q_out, want in ((at, INV), (last, INV), (at - 5 * 8 * 128 * 2 + 16, INV), (at - 5 * 8 * 128 * 2, None), (last + 16, None)):
            got = call("rope", b=b, r=rope(freqs=P + 0x30000, axes=2, axis=bytes([0, 1] * 32)), positions=P + 0x40000, k=P + 0x1000000,
                       v=P + 0x2000000, q=P + 0x3000000, q_out=q_out, pool=P + 0x8000000, pool_bytes=need)
            assert got == INV if want else launched(got), (hex(at), q_out - at)


@pytest.mark.parametrize("name", ["attn", "keep", "tree"])
def test_bad_masks(name):
    for bad, want in ((dict(masks=None), INV), (dict(masks=P + 2), INV), (dict(words=0), INV), (dict(words=-1), INV),
                      (dict(words=129), UNS)):
        assert call(name, **bad) == want, bad
    assert call(name, b=batch(max_rows=33)) == INV
    assert call(name, b=batch(max_rows=4097, total_rows=4097), words=129) == UNS


def test_bad_trees_and_nodes():
    for bad in (dict(parents=None), dict(parents=P + 2), dict(tree_positions=P + 2), dict(status=P + 1), dict(parents=P + 12288),
                dict(parents=P + 12304), dict(masks=P + 8208), dict(masks=P + 12288 - 4 * 4)):
        assert call("tree", **bad) == INV, bad
    for bad in (dict(nodes=None), dict(nodes=P + 2), dict(lens_out=None), dict(lens_out=P + 2), dict(lens_out=P), dict(lens_out=P + 8), dict(nodes=P + 128, lens_out=P + 120),
                dict(n_layers=0), dict(n_layers=3), dict(layer=1, n_layers=2)):
        assert call("keep", **bad) == INV, bad
    for name in ("tree", "keep"):
        assert call(name, b=batch(n_seqs=2 ** 24)) == UNS


def apart(**kw):
    """The arrays of a batch of 3 sequences, 5 rows and 6 pages each, 64 KB apart."""
    a = dict(page_table=P, kv_lens=P + 0x10000, row_start=P + 0x20000)
    a.update(kw)
    return batch(n_seqs=3, total_rows=5, max_rows=5, max_pages=6, max_len=96, **a)


def launched(status):
    """A call that nothing refused: without a GPU its launch fails."""
    if torch.cuda.is_available():
        pytest.skip("would be launched with these addresses")
    return status == kvtc.ERR_HIP


def test_kept_lengths_apart_from_what_is_read():
    """The lengths after it overlap nothing that other workgroups still read,
    and may lie right beside it."""
    need = size(cfg())[2]
    a = dict(masks=P + 0x30000, words=2, nodes=P + 0x40000, pool=P + 0x50000, pool_bytes=need)
    # start and size of what is read
    for at, n in ((P, 3 * 6 * 4), (P + 0x10000, 3 * 4), (P + 0x20000, 4 * 4), (P + 0x30000, 5 * 2 * 4), (P + 0x40000, 3 * 4),
                  (P + 0x50000, need)):
        for lens_out in (at, at + n - 4, at - 8, at - 4):
            assert call("keep", b=apart(), lens_out=lens_out, **a) == INV, (hex(at), lens_out - at)
    for at, n in ((P, 3 * 6 * 4), (P + 0x10000, 3 * 4), (P + 0x20000, 4 * 4), (P + 0x30000, 5 * 2 * 4), (P + 0x40000, 3 * 4),
                  (P + 0x50000, need)):
        for lens_out in (at - 12, at + n):
            assert launched(call("keep", b=apart(), lens_out=lens_out, **a)), (hex(at), lens_out - at)


def test_masks_and_positions_apart_from_what_is_read():
    """Neither overlaps the parents, lengths or rows of the batch, or each
    other; they may lie right beside them.  The page table is not read."""
    a = dict(parents=P + 0x30000, masks=P + 0x40000, words=2, tree_positions=P + 0x50000)
    read = ((P + 0x10000, 3 * 4), (P + 0x20000, 4 * 4), (P + 0x30000, 5 * 4))  # lengths, rows, parents
    for at, n in read + ((P + 0x40000, 5 * 2 * 4),):
        for positions in (at, at + n - 4, at - 16, at - 4):
            assert call("tree", b=apart(), **{**a, "tree_positions": positions}) == INV, (hex(at), positions - at)
    for at, n in read + ((P + 0x50000, 5 * 4),):
        for masks in (at, at + n - 4, at - 36, at - 4):
            assert call("tree", b=apart(), **{**a, "masks": masks}) == INV, (hex(at), masks - at)
    for at, n in read:
        for positions, masks in ((at - 20, at + n), (at + n, at - 40)):
            assert launched(call("tree", b=apart(), **{**a, "tree_positions": positions, "masks": masks})), hex(at)
    assert launched(call("tree", b=apart(), **{**a, "masks": P})) and launched(call("tree", b=apart(), **{**a, "tree_positions": P}))


def test_bad_tree_attention():
    for bad in (dict(q=None), dict(out=None), dict(q=P + 2), dict(out=P + 8), dict(lse=P + 2), dict(ws=P + 8),
                dict(q_stride=-8), dict(q_stride=12), dict(q_heads=0), dict(q_heads=6), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=2.0 ** 101), dict(shared=-1), dict(shared=7)):
        assert call("attn", **bad) == INV, bad
    assert call("attn", b=batch(total_rows=2 ** 28)) == UNS
    n = ctypes.c_size_t(0)
    assert kvtc.lib().kvtc_mx_attn_tree_workspace(ctypes.byref(cfg()), ctypes.byref(batch()), 8, 2, ctypes.byref(n)) == kvtc.OK
    assert n.value > 0
    assert call("attn", ws_bytes=n.value - 1) == CAP and call("attn", ws=None) == INV
    assert kvtc.lib().kvtc_mx_attn_tree_workspace(ctypes.byref(cfg()), ctypes.byref(batch()), 8, 2, None) == INV


@pytest.mark.parametrize("name", ("rope", "attn", "tree"))
def test_nothing_to_do(name):
    for b in (batch(n_seqs=0, page_table=None, kv_lens=None, row_start=None), batch(total_rows=0), batch(max_rows=0)):
        assert call(name, b=b, k=None, v=None, q=None, q_out=None, out=None, ws=None, ws_bytes=0, masks=None, parents=None) == kvtc.OK
    assert call("keep", b=batch(n_seqs=0, page_table=None, kv_lens=None, row_start=None), masks=None, nodes=None, lens_out=None) == kvtc.OK


def test_rotations_of_the_binding():
    """Frequencies that the kernels could not read, axes past four."""
    f = kvtc.rope_freqs(64, 1e4, device="cpu")
    assert f.dtype == torch.float64 and f[0] == 1 and np.isclose(f[16].item(), 1e-2) and f.numel() == 32
    with pytest.raises(ValueError):
        kvtc.MxRope(f)
    with pytest.raises(ValueError):
        kvtc.MxRope(f.float())
