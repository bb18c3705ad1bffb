"""The microscaled paged cache on the CPU: the plain implementation's own
pins, and what the library refuses before anything is launched."""
import ctypes
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import mx_ref
from tensor_compression_amd import kvtc


@pytest.mark.parametrize("b", [4, 8])
def test_elements_are_the_nearest_and_none_saturates(b):
    rng = np.random.default_rng(b)
    x = rng.standard_normal((400, 32)) * 2.0 ** rng.integers(-30, 30, (400, 1))
    code, s = mx_ref.quantise(x, b)
    y = mx_ref.values(code, s, b)
    g = np.concatenate([-mx_ref.grid(b)[::-1], mx_ref.grid(b)])
    for r in range(0, 400, 7):
        all_values = g * 2.0 ** (int(s[r, 0]) - 127)
        best = np.abs(x[r][:, None] - all_values[None]).min(1)
        assert np.array_equal(np.abs(x[r] - y[r]), best)
        # the scale is the smallest one: half of it would saturate
        assert np.abs(x[r]).max() >= mx_ref.OVER[b] * 2.0 ** (int(s[r, 0]) - 128)


def test_scale_borders_and_clamps():
    for b, over, top in ((4, 1.75, 252), (8, 1.8125, 246)):
        x = np.zeros((7, 32))
        x[0, 3] = over                      # exactly the border: the next scale
        x[1, 3] = over * (1 - 2.0 ** -23)   # just below
        x[3, 0] = 2.0 ** -126               # below the smallest scale's half step: zeros
        x[4, 0] = np.finfo(np.float32).max  # saturates under the largest scale
        x[5, 9] = np.inf
        x[6, 9] = np.nan
        code, s = mx_ref.quantise(x, b)
        base = 127 - (2 if b == 4 else 8)
        assert list(s[:, 0]) == [base + 1, base, 15, 15, top, 255, 255]
        y = mx_ref.values(code, s, b)
        assert not y[2].any() and not y[3].any() and np.isfinite(y[4]).all() and np.isnan(y[5:]).all()
        assert y[4, 0] == mx_ref.TOP[b] * 2.0 ** (top - 127) and y[4, 0] < 3.39e38


@pytest.mark.parametrize("D,bk,bv", [(64, 4, 4), (64, 8, 4), (128, 4, 8), (128, 8, 8)])
def test_record_layout_is_a_bijection(D, bk, bv):
    seen = np.zeros(mx_ref.record_bytes(D, bk, bv) * 2, int)  # nibbles
    for kv, b in ((0, bk), (1, bv)):
        at, sh, so = mx_ref.places(D, bk, bv, kv)
        for half in range(b // 4):
            np.add.at(seen, (at * 2 + sh // 4 + half).ravel(), 1)
        for half in (0, 1):
            np.add.at(seen, (so * 2 + half).ravel(), 1)
    assert (seen == 1).all()


def test_write_then_unpack_is_quantise():
    rng = np.random.default_rng(3)
    D, bk, bv, H = 64, 4, 8, 2
    pool = np.full((5, H, mx_ref.record_bytes(D, bk, bv)), 0xFF, np.uint8)
    k, v = rng.standard_normal((2, 21, H, D))
    mx_ref.write(pool, [[3, 1, 0]], [37], [0, 21], k, v, D, bk, bv)
    kp, vp = mx_ref.unpack(pool, D, bk, bv)
    for x, xp, b in ((k, kp, bk), (v, vp, bv)):
        got = xp[[3, 1, 0]].transpose(1, 0, 2, 3).reshape(H, 48, D)
        assert np.array_equal(got[:, 16:37].transpose(1, 0, 2), mx_ref.values(*mx_ref.quantise(x, b), b))
        assert np.isnan(got[:, :16]).all() and np.isnan(got[:, 37:]).all()


# ---- refusals: every one of them before a launch, so no GPU is needed

P = 0x7F0000000000  # a device address that is never touched


def cfg(**kw):
    c = dict(layers=2, kv_heads=4, head_dim=128, dtype=kvtc.BF16, bits_k=4, bits_v=8, pool_pages=10)
    c.update(kw)
    return kvtc.MxConfig(*[c[f] for f, _ in kvtc.MxConfig._fields_])


def batch(**kw):
    b = dict(n_seqs=3, max_pages=6, total_rows=5, max_rows=4, max_len=96, reserved=0, page_table=P, kv_lens=P,
             row_start=P)
    b.update(kw)
    return kvtc.MxBatchStruct(*[b[f] for f, _ in kvtc.MxBatchStruct._fields_])


def size(c):
    r, t = ctypes.c_size_t(0), ctypes.c_size_t(0)
    st = kvtc.lib().kvtc_mx_pool_size(ctypes.byref(c), ctypes.byref(r), ctypes.byref(t))
    return st, r.value, t.value


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def call(name, c=None, b=None, **kw):
    c, b = c or cfg(), b or batch()
    a = dict(layer=0, n_layers=1, k=P, ks=strides(0, 128, 512), v=P, vs=strides(0, 128, 512), pool=P, pool_bytes=1 << 40,
             out_dtype=kvtc.FP32, status=P, q=P, q_stride=1024, q_heads=8, scale=0.1, causal=1, out=P, lse=P, ws=P,
             ws_bytes=1 << 40, shared=2)
    a.update(kw)
    L, cr, br = kvtc.lib(), ctypes.byref(c), ctypes.byref(b)
    if name == "write":
        return L.kvtc_mx_write(cr, br, a["layer"], a["n_layers"], a["k"], a["ks"], a["v"], a["vs"], a["pool"],
                               a["pool_bytes"], a["status"], None)
    if name == "read":
        return L.kvtc_mx_read(cr, br, a["layer"], a["n_layers"], a["pool"], a["pool_bytes"], a["k"], a["ks"], a["v"],
                              a["vs"], a["out_dtype"], a["status"], None)
    head = (cr, br, a["layer"], a["pool"], a["pool_bytes"])
    tail = (a["q"], a["q_stride"], a["q_heads"], a["scale"], a["causal"], a["out"], a["lse"], a["ws"], a["ws_bytes"],
            a["status"], None)
    if name == "attn":
        return L.kvtc_mx_attn(*head, *tail)
    return L.kvtc_mx_attn_shared(*head, a["shared"], *tail)


CALLS = ("write", "read", "attn", "shared")
INV, UNS, CAP = kvtc.ERR_INVALID_ARG, kvtc.ERR_UNSUPPORTED, kvtc.ERR_CAPACITY


def test_pool_size():
    st, rec, total = size(cfg())
    assert st == kvtc.OK and rec == mx_ref.record_bytes(128, 4, 8) and total == 2 * 10 * 4 * rec
    assert size(cfg(layers=16384, kv_heads=4, pool_pages=2 ** 31 - 1))[2] == 65536 * (2 ** 31 - 1) * rec


@pytest.mark.parametrize("bad,want", [
    (dict(layers=0), INV), (dict(kv_heads=0), INV), (dict(pool_pages=0), INV), (dict(dtype=2), INV),
    (dict(bits_k=5), INV), (dict(bits_v=16), INV), (dict(head_dim=96), UNS), (dict(head_dim=256), UNS),
    (dict(layers=8193, kv_heads=8), UNS)])
def test_bad_configurations(bad, want):
    assert size(cfg(**bad))[0] == want
    for name in CALLS:
        assert call(name, c=cfg(**bad)) == want, name


@pytest.mark.parametrize("bad", [
    dict(n_seqs=-1), dict(max_pages=0), dict(total_rows=-1), dict(max_rows=-1), dict(max_len=-1), dict(max_len=97),
    dict(reserved=1), dict(page_table=None), dict(kv_lens=None), dict(row_start=None), dict(page_table=P + 2),
    dict(kv_lens=P + 1), dict(row_start=P + 2), dict(max_pages=2 ** 27, max_len=2 ** 30 + 1)])
def test_bad_batches(bad):
    for name in CALLS:
        assert call(name, b=batch(**bad)) == INV, name
    n = ctypes.c_size_t(0)
    assert kvtc.lib().kvtc_mx_attn_workspace(ctypes.byref(cfg()), ctypes.byref(batch(**bad)), 8, 0, ctypes.byref(n)) == INV


@pytest.mark.parametrize("name", CALLS)
def test_bad_pool_layer_status(name):
    need = size(cfg())[2]
    for bad, want in ((dict(pool=None), INV), (dict(pool=P + 8), INV), (dict(pool_bytes=need - 1), CAP),
                      (dict(layer=-1), INV), (dict(layer=2), INV), (dict(status=P + 2), INV)):
        assert call(name, **bad) == want, bad


@pytest.mark.parametrize("name", ["write", "read"])
def test_bad_rows(name):
    for bad in (dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 2), dict(ks=None), dict(vs=None),
                dict(ks=strides(0, 128, -512)), dict(vs=strides(0, 124, 512)) if name == "write" else dict(out_dtype=3),
                dict(ks=strides(0, 128, 2 ** 47)), dict(n_layers=0), dict(n_layers=3), dict(layer=1, n_layers=2)):
        assert call(name, **bad) == INV, bad


def test_overlapping_outputs():
    for s in (strides(0, 128, 0), strides(0, 0, 512), strides(0, 128, 384), strides(0, 64, 512)):
        assert call("read", ks=s) == INV
        assert call("read", vs=s) == INV
    # a layer stride of 0 is an overlap only when there are two layers
    assert call("read", n_layers=2, ks=strides(0, 128, 512)) == INV


def test_overlapping_outputs_of_huge_strides():
    """Spans past 64 bits: row 1 of layer 0 and row 0 of layer 1 lie 8 elements apart."""
    b = batch(n_seqs=0, total_rows=2 ** 31 - 1)
    for rows, layers in ((2 ** 34, 2 ** 34 + 8), (2 ** 33, 2 ** 46), (2 ** 46, 2 ** 46)):
        assert call("read", b=b, n_layers=2, ks=strides(layers, 128, rows)) == INV
        assert call("read", b=b, n_layers=2, ks=strides(layers, 128, 512), vs=strides(layers, 128, rows)) == INV
    assert call("read", b=b, n_layers=2, ks=strides(2 ** 45, 128, 512), vs=strides(2 ** 45, 128, 512)) == kvtc.OK


@pytest.mark.parametrize("name", ["attn", "shared"])
def test_bad_attention(name):
    for bad in (dict(q=None), dict(out=None), dict(q=P + 2), dict(out=P + 8), dict(lse=P + 2), dict(ws=P + 8),
                dict(q_stride=-8), dict(q_stride=12), dict(q_heads=0), dict(q_heads=6), dict(q_heads=2),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=2.0 ** 101),
                dict(scale=2.0 ** -127), dict(causal=2)):
        assert call(name, **bad) == INV, bad
    big = batch(total_rows=2 ** 28)
    assert call(name, b=big, q_heads=8) == UNS


def test_bad_prefix_and_workspace():
    assert call("shared", shared=-1) == INV and call("shared", shared=7) == INV
    n = ctypes.c_size_t(0)
    assert kvtc.lib().kvtc_mx_attn_workspace(ctypes.byref(cfg()), ctypes.byref(batch()), 8, 2, ctypes.byref(n)) == kvtc.OK
    assert n.value > 0
    assert call("shared", ws_bytes=n.value - 1) == CAP and call("shared", ws=None) == INV


def test_grids_of_both_passes():
    """Each pass within a launch's workgroups: planned.  The own tokens' past
    them: refused."""
    c, n = cfg(kv_heads=1), ctypes.c_size_t(0)
    for seqs, want in ((2 ** 24 - 1, kvtc.OK), (2 ** 24, UNS)):
        b = batch(n_seqs=seqs, total_rows=4096, max_rows=1)
        for shared in (0, 2):
            assert kvtc.lib().kvtc_mx_attn_workspace(ctypes.byref(c), ctypes.byref(b), 1, shared, ctypes.byref(n)) == want
    assert call("shared", c=c, b=b, q_heads=1) == UNS and call("attn", c=c, b=b, q_heads=1) == UNS


def test_a_pool_in_host_memory_is_refused():
    """The kernels would follow a host pointer."""
    c = dict(layers=1, kv_heads=2, head_dim=64, dtype=kvtc.BF16, bits_k=4, bits_v=4)
    with pytest.raises(ValueError):
        kvtc.MxCache(c, 3, device="cpu")
    with pytest.raises(ValueError):
        kvtc.MxCache(c, 3, pool=torch.empty(1, 3, 2, mx_ref.record_bytes(64, 4, 4), dtype=torch.uint8))


def test_a_stream_of_another_device_is_refused():
    """Before anything is launched on it."""
    cache, ran = object.__new__(kvtc.MxCache), []
    cache._index, cache.device = 0, torch.device("cuda", 0)
    with pytest.raises(ValueError):
        cache._call(lambda *a: ran.append(a), SimpleNamespace(device_index=1, cuda_stream=0))
    assert not ran


@pytest.mark.parametrize("name", CALLS)
def test_nothing_to_do(name):
    """No sequences, no rows: fine, whatever the row pointers are."""
    for b in (batch(n_seqs=0, page_table=None, kv_lens=None, row_start=None), batch(total_rows=0), batch(max_rows=0)):
        assert call(name, b=b, k=None, v=None, q=None, out=None, ws=None, ws_bytes=0) == kvtc.OK
