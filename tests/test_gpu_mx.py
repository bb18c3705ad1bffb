"""The microscaled paged cache on the GPU against the plain 64-bit
implementation: writing and reading bit for bit, attention within bounds that
follow from its roundings."""
import numpy as np
import pytest
import torch

import mx_ref
from tensor_compression_amd import kvtc

pytestmark = pytest.mark.gpu

FORMATS = [(64, 4, 4), (64, 8, 4), (64, 4, 8), (64, 8, 8), (128, 4, 4), (128, 8, 4), (128, 4, 8), (128, 8, 8)]
DT = {kvtc.BF16: torch.bfloat16, kvtc.FP32: torch.float32}


def dev(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype).cuda()


class Case:
    """A cache, a batch of sequences (lens after their rows) in scattered pages."""

    def __init__(self, D, bk, bv, dtype, H, rows, lens, layers=1, seed=0, fill=0xFF, shared=0, total_rows=None):
        self.rng = np.random.default_rng(seed)
        self.D, self.bk, self.bv, self.dtype, self.H, self.layers = D, bk, bv, dtype, H, layers
        self.rows, self.lens = list(rows), list(lens)
        self.starts = [0] + [int(x) for x in np.cumsum(rows)]
        self.total = self.starts[-1] if total_rows is None else total_rows
        need = [max(-(-x // 16), shared) for x in lens]
        self.pages = shared + sum(x - shared for x in need) + 2
        perm = [int(x) for x in self.rng.permutation(self.pages)]
        at, self.table = shared, []
        for x in need:
            self.table.append(perm[:shared] + perm[at:at + x - shared])
            at += x - shared
        width = max(max(need, default=0), 1) + 1
        # entries past a sequence's pages are outside the pool: nothing may follow them
        self.table_dev = dev([t + [2 ** 30 + 5] * (width - len(t)) for t in self.table], torch.int32)
        self.cache = kvtc.MxCache(dict(layers=layers, kv_heads=H, head_dim=D, dtype=dtype, bits_k=bk, bits_v=bv), self.pages)
        self.cache.pool.fill_(fill)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.batch = self.new_batch(rows, lens)

    def new_batch(self, rows, lens, **kw):
        starts = [0] + [int(x) for x in np.cumsum(rows)]
        a = dict(total_rows=self.total, max_rows=max(rows), max_len=max(lens))
        a.update(kw)
        return self.cache.batch(self.table_dev, dev(list(lens), torch.int32), dev(starts, torch.int32), **a)

    def rand(self, *shape, gain=0.6):
        x = self.rng.standard_normal(shape) * np.exp(gain * self.rng.standard_normal(shape[-1]))
        return dev(x, torch.float32).to(DT[self.dtype])

    def fill(self):
        """The whole sequences written by the library; returns the pool's bytes."""
        t = sum(self.lens)
        k, v = self.rand(t, self.H, self.D), self.rand(t, self.H, self.D)
        b = self.cache.batch(self.table_dev, dev(self.lens, torch.int32),
                             dev([0] + [int(x) for x in np.cumsum(self.lens)], torch.int32), total_rows=t,
                             max_rows=max(self.lens), max_len=max(self.lens))
        for layer in range(self.layers):
            self.cache.write(b, k, v, layer=layer, status=self.status)
        return self.cache.pool.cpu().numpy()

    def unpacked(self, layer=0):
        return mx_ref.unpack(self.cache.pool[layer].cpu().numpy(), self.D, self.bk, self.bv)


def np64(x):
    return x.double().cpu().numpy()


# ---- writing and reading


def hard_rows(rng, rows, H, D, dtype):
    """Rows over the whole range of the type: blocks of every size, ties,
    zeros of both signs, subnormals, the largest numbers, NaN and infinity."""
    x = rng.standard_normal((rows, H, D)) * 2.0 ** rng.integers(-120, 120, (rows, H, D // 32, 1)).repeat(32, -1).reshape(rows, H, D)
    flat = x.reshape(-1, 32)
    m = len(flat)
    flat[0 % m] = 0.0
    flat[1 % m] = -0.0
    flat[2 % m] = rng.integers(-14, 15, 32) / 4.0        # ties of both formats
    flat[3 % m] = rng.integers(-1000, 1000, 32) / 2.0
    flat[4 % m] = 2.0 ** -133 * rng.integers(-8, 8, 32)  # subnormals
    flat[5 % m] = 3.38e38 * rng.uniform(-1, 1, 32)
    flat[5 % m, 7] = 3.38e38
    flat[6 % m, 3] = np.inf
    flat[7 % m, 31] = -np.inf
    flat[8 % m, 0] = np.nan
    for i, lead in enumerate((1.75, 1.8125, 1.7421875, 1.8046875)):  # the scale's borders
        flat[(9 + i) % m] = 0.25
        flat[(9 + i) % m, 5] = lead * 2.0 ** (i - 2)
    return dev(flat.reshape(rows, H, D), torch.float32).to(DT[dtype])


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
@pytest.mark.parametrize("D,bk,bv", FORMATS)
def test_write_bytes(D, bk, bv, dtype):
    rows, lens = [1, 5, 16, 0, 17, 40, 3], [1, 5, 16, 7, 45, 40, 2]  # the last has a row before its first token
    c = Case(D, bk, bv, dtype, 3, rows, lens, layers=2, seed=D + bk, fill=0xA5)
    k, v = (hard_rows(c.rng, c.total, 3, D, dtype) for _ in range(2))
    print("write", D, bk, bv, dtype, flush=True)
    c.cache.write(c.batch, k, v, layer=1, status=c.status)
    want = np.full(c.cache.pool.shape[1:], 0xA5, np.uint8)
    mx_ref.write(want, c.table, lens, c.starts, np64(k), np64(v), D, bk, bv)
    got = c.cache.pool.cpu().numpy()
    assert np.array_equal(got[1], want)
    assert (got[0] == 0xA5).all()
    assert c.status.item() == 1 << kvtc.ERR_NONFINITE


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,bk,bv", FORMATS)
def test_read_values(D, bk, bv, out):
    rows, lens = [1, 5, 16, 0, 17, 33, 3], [1, 9, 16, 7, 45, 40, 2]
    total = sum(rows) + 2
    c = Case(D, bk, bv, kvtc.BF16, 3, rows, lens, layers=2, seed=D + bv, total_rows=total)
    c.fill()
    k = torch.full((total, 3, D), 7.0, dtype=out, device="cuda")
    v = torch.full((total, 5, D), 7.0, dtype=out, device="cuda")[:, 1:4]  # a slice: strides of its own
    print("read", D, bk, bv, out, flush=True)
    c.cache.read(c.batch, k, v, layer=1, status=c.status)
    for x, pages in ((k, c.unpacked(1)[0]), (v, c.unpacked(1)[1])):
        want = np.full((total, 3, D), 7.0)
        for z, ln in enumerate(lens):
            for i in range(rows[z]):
                pos = ln - rows[z] + i
                if pos >= 0:
                    want[c.starts[z] + i] = pages[c.table[z][pos // 16], :, pos % 16]
        assert np.array_equal(np64(x), want)
    assert c.status.item() == 0


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
def test_write_and_read_whole_cache(dtype):
    """[L, H, T, D] in and out, through strides, in one call for all layers;
    NaN blocks come back as NaN."""
    D, L, H, T = 128, 3, 2, 77
    c = Case(D, 8, 4, dtype, H, [T], [T], layers=L, seed=5)
    k = c.rand(L, T, H, D).transpose(1, 2)  # layer, head and token strides out of order
    v = c.rand(L, H, T, D)
    v[1, 1, 3, 40] = float("nan")
    c.cache.write(c.batch, k, v, status=c.status)
    ko, vo = (torch.empty(L, H, T, D, dtype=DT[dtype], device="cuda") for _ in range(2))
    c.cache.read(c.batch, ko, vo, status=c.status)
    for x, y, b in ((k, ko, 8), (v, vo, 4)):
        want = mx_ref.values(*mx_ref.quantise(np64(x), b), b)
        assert np.array_equal(np64(y), want, equal_nan=True)
    assert torch.isnan(vo[1, 1, 3, 32:64]).all() and not torch.isnan(vo[1, 1, 3, :32]).any()
    assert c.status.item() == 1 << kvtc.ERR_NONFINITE
    with pytest.raises(kvtc.KvtcError):
        c.cache.read(c.batch, ko[:1].expand(L, H, T, D), vo)
    with pytest.raises(ValueError):
        c.cache.write(c.batch, k[:, :1], v)


def test_appending_token_by_token_is_writing_at_once():
    D, H = 64, 2
    c = Case(D, 4, 8, kvtc.BF16, H, [37, 20], [37, 20], seed=6, fill=0)
    k, v = c.rand(57, H, D), c.rand(57, H, D)
    c.cache.write(c.batch, k, v)
    want = c.cache.pool.clone()
    c.cache.pool.zero_()
    c.total = 2
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    starts = dev([0, 1, 2], torch.int32)
    b = c.cache.batch(c.table_dev, lens, starts, total_rows=2, max_rows=1, max_len=37)
    for t in range(37):
        at = [t, 37 + min(t, 19)]
        lens += dev([1, 1 if t < 20 else 0], torch.int32)
        if t >= 20:
            starts.copy_(dev([0, 1, 1], torch.int32))
        c.cache.write(b, k[at], v[at])
    assert torch.equal(c.cache.pool, want)


# ---- attention


def check_attention(c, q, got, lse, scale, causal, what):
    """Bounds: bf16 weights and outputs are off by at most 2^-8 of themselves
    each (fp32: the three-part weights and the output 2^-23), the scores by
    D 2^-24 of the sum of their terms' magnitudes (exact products, fp32 sums)
    and a few roundings of the exponent, the sums of T weights in 32-token
    steps by T / 32 + 64 roundings of 2^-24."""
    kp, vp = c.unpacked()
    kp, vp = np.nan_to_num(kp), np.nan_to_num(vp)
    want, wlse, mass, spread = mx_ref.attention(kp, vp, c.table, c.lens, c.starts, np64(q), scale, causal)
    n = c.starts[-1]
    o, s = np64(got)[:n], np64(lse)[:n]
    u = 2.0 ** -8 if c.dtype == kvtc.BF16 else 2.0 ** -23
    T = max(c.lens)
    ew = spread * (c.D * 2.0 ** -24 + 4 * 2.0 ** -24) + 2.0 ** -21
    steps = (T / 32 + 64) * 2.0 ** -24
    tol = (u + 2 * ew[..., None] + 2 * steps) * mass + u * np.abs(want) + 1e-30
    err = np.abs(o - want[:n])
    worst = float((err / tol[:n]).max())
    print(what, "worst error / bound %.3f" % worst, flush=True)
    assert worst <= 1.0
    empty = np.isneginf(wlse[:n])
    assert np.array_equal(np.isneginf(s), empty) and not o[empty].any()
    ltol = ew[:n] + steps + np.abs(np.where(empty, 0, wlse[:n])) * 2.0 ** -22
    assert (np.abs(np.where(empty, 0, s) - np.where(empty, 0, wlse[:n])) <= ltol).all()


def run_attention(c, G, causal=True, shared=None, scale=None, **kw):
    q = c.rand(c.total, c.H * G, c.D, gain=0.2)
    out = torch.full((c.total, c.H * G, c.D), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((c.total, c.H * G), 7.0, device="cuda")
    scale = c.D ** -0.5 if scale is None else scale
    if shared is None:
        c.cache.attention(c.batch, q, scale, causal, out=out, lse=lse, status=c.status, **kw)
    else:
        c.cache.attention_shared(c.batch, q, shared, scale, causal, out=out, lse=lse, status=c.status, **kw)
    assert c.status.item() == 0
    n = c.starts[-1]
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()
    return q, out, lse, scale


LENS = [1, 15, 16, 17, 31, 32, 33, 0, 5, 130, 257, 700]


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
@pytest.mark.parametrize("D,bk,bv", FORMATS)
def test_attention_formats(D, bk, bv, dtype):
    """Ragged lengths, sequences with no rows, no tokens, or more rows than
    tokens, in a pool whose unwritten bytes are all NaN."""
    rows = [1, 1, 2, 1, 3, 1, 5, 1, 7, 1, 0, 2]
    c = Case(D, bk, bv, dtype, 2, rows, LENS, seed=D + bk + bv, total_rows=sum(rows) + 3)
    c.fill()
    q, out, lse, scale = run_attention(c, 3)
    check_attention(c, q, out, lse, scale, True, f"D{D} k{bk} v{bv} dtype {dtype}")


@pytest.mark.parametrize("G", [1, 2, 5, 8, 16, 24])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_groups(G, causal):
    """Groups of 1 to 24 heads: tiles of 16, 32 and 64 rows, some part full."""
    for dtype in (kvtc.BF16, kvtc.FP32):
        rows = [1, 4, 2, 1]
        c = Case(128, 4, 4, dtype, 3, rows, [40, 129, 2, 300], seed=G)
        c.fill()
        q, out, lse, scale = run_attention(c, G, causal)
        check_attention(c, q, out, lse, scale, causal, f"G{G} causal {causal} dtype {dtype}")


@pytest.mark.parametrize("D,bk,bv", [(64, 8, 8), (128, 4, 4), (128, 8, 4)])
def test_attention_long_rows(D, bk, bv):
    """Prompts: many rows a sequence, with and without tokens before them."""
    for dtype in (kvtc.BF16, kvtc.FP32):
        rows, lens = [200, 61, 90], [200, 333, 64]
        c = Case(D, bk, bv, dtype, 2, rows, lens, seed=bk)
        c.fill()
        q, out, lse, scale = run_attention(c, 2)
        check_attention(c, q, out, lse, scale, True, f"rows D{D} k{bk} v{bv} dtype {dtype}")


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
def test_attention_long_context(dtype):
    """One sequence over many ranges, lengths around their borders."""
    for ln in (2047, 2049, 20011):
        c = Case(128, 8, 4, dtype, 2, [2], [ln], seed=ln)
        c.fill()
        q, out, lse, scale = run_attention(c, 4)
        check_attention(c, q, out, lse, scale, True, f"context {ln} dtype {dtype}")


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
@pytest.mark.parametrize("shared", [0, 1, 3, 40])
def test_attention_shared_prefix(shared, dtype):
    """Sequences past, at the end of, and inside the prefix, empty ones, and
    sequences without rows; equal to the plain call on the same tables."""
    p = 16 * shared
    lens = [p + 1, p + 40, p, max(p - 5, 0), 0, p + 300, p + 16, min(p, 3)]
    rows = [1, 2, 1, 3, 1, 0, 1, 1]
    for D, bk, bv, G in ((128, 4, 4, 4), (64, 8, 4, 3)):
        c = Case(D, bk, bv, dtype, 2, rows, lens, seed=shared + D, shared=shared, total_rows=sum(rows) + 1)
        c.fill()
        q, out, lse, scale = run_attention(c, G, shared=shared)
        check_attention(c, q, out, lse, scale, True, f"shared {shared} D{D} dtype {dtype}")
        # entries of the other sequences for the prefix are not read
        out2 = torch.full_like(out, 7.0)
        if shared:
            c.table_dev[1:, :shared] = -1
            c.cache.attention_shared(c.batch, q, shared, scale, out=out2, status=c.status)
            assert torch.equal(out, out2) and c.status.item() == 0


def test_attention_with_nothing_but_the_prefix():
    """Every sequence inside the prefix, whose last page is not full; and
    sequences without any token."""
    for G in (2, 40):
        c = Case(128, 8, 4, kvtc.BF16, 2, [1, 2, 1], [37, 20, 0], seed=G, shared=3)
        one = c.cache.batch(c.table_dev[:1], dev([37], torch.int32), dev([0, 37], torch.int32), total_rows=37, max_rows=37,
                            max_len=37)
        c.cache.write(one, c.rand(37, 2, 128), c.rand(37, 2, 128))
        q, out, lse, scale = run_attention(c, G, shared=3)
        check_attention(c, q, out, lse, scale, True, f"only prefix G{G}")
    for shared in (None, 3):
        c.batch = c.new_batch([1, 2, 1], [0, 0, 0])
        c.lens = [0, 0, 0]
        q, out, lse, scale = run_attention(c, 40, shared=shared)
        assert not out.any() and torch.isneginf(lse).all()


def test_attention_shared_prefix_many_rows():
    """Enough rows together for whole 64-row tiles of the prefix pass."""
    lens = [160 + int(x) for x in np.random.default_rng(1).integers(0, 90, 70)]
    c = Case(128, 4, 4, kvtc.BF16, 2, [1 + z % 2 for z in range(70)], lens, seed=2, shared=10)
    c.fill()
    for causal in (True, False):
        q, out, lse, scale = run_attention(c, 4, causal, shared=10)
        check_attention(c, q, out, lse, scale, causal, f"shared rows causal {causal}")


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
def test_attention_long_ranges(dtype):
    """Ranges of more pages than a workgroup knows the numbers of at once: few
    rows (many sequences over the same pages leave no room to split) and many."""
    n, H, ln = 64, 8, 17003
    c = Case(128, 4, 4, dtype, H, [1], [ln], seed=21)
    c.fill()
    q = c.rand(n, H, 128)
    table = c.table_dev.expand(n, -1).contiguous()
    lens = [ln - 37 * z for z in range(n)]
    b = c.cache.batch(table, dev(lens, torch.int32), dev(list(range(n + 1)), torch.int32), total_rows=n, max_rows=1, max_len=ln)
    lse = torch.empty(n, H, device="cuda")
    out, _ = c.cache.attention(b, q, lse=lse, status=c.status)
    for z in (0, 41, 63):
        c.lens = [lens[z]]
        check_attention(c, q[z:z + 1], out[z:z + 1], lse[z:z + 1], 128 ** -0.5, True, f"long range {z} dtype {dtype}")
    c = Case(64, 8, 4, dtype, 8, [300], [5003], seed=22)
    c.fill()
    q, out, lse, scale = run_attention(c, 1)
    check_attention(c, q, out, lse, scale, True, f"long rows dtype {dtype}")
    assert c.status.item() == 0


@pytest.mark.parametrize("D,bk,bv,dtype", [(128, 4, 4, kvtc.BF16), (128, 8, 4, kvtc.FP32), (64, 4, 8, kvtc.BF16),
                                           (64, 8, 8, kvtc.FP32)])
def test_attention_one_workgroup_a_unit(D, bk, bv, dtype):
    """About as many sequences and heads as compute units, each long enough for
    a larger workgroup; under bounds of hundreds of megabytes of codes too."""
    n, H = 30, 8
    lens = [1500 - 29 * z for z in range(n - 6)] + [0, 1, 16, 17, 255, 257]
    c = Case(D, bk, bv, dtype, H, [1], [1500], seed=D + bk)
    c.fill()
    q = c.rand(n + 1, 2 * H, D)
    table = torch.full((n, 640), 2 ** 30, dtype=torch.int32, device="cuda")
    table[:, :94] = c.table_dev[:1, :94]
    kv, starts = dev(lens, torch.int32), dev(list(range(n + 1)), torch.int32)
    for max_len in (1500, 10240):
        b = c.cache.batch(table, kv, starts, total_rows=n + 1, max_rows=1, max_len=max_len)
        lse = torch.full((n + 1, 2 * H), 7.0, device="cuda")
        out = torch.full_like(q, 7.0)
        c.cache.attention(b, q, out=out, lse=lse, status=c.status)
        assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all() and c.status.item() == 0
        for z in (0, 11, 24, 25, 26, 27, 28, 29):
            c.lens = [lens[z]]
            check_attention(c, q[z:z + 1], out[z:z + 1], lse[z:z + 1], D ** -0.5, True, f"sequence {z} bound {max_len}")


@pytest.mark.parametrize("n,H,G", [(33, 8, 1), (64, 8, 5), (65, 5, 1), (150, 2, 1), (256, 2, 1), (257, 1, 1), (300, 1, 20)])
def test_attention_sequences_by_length(n, H, G):
    """More whole sequences than compute units take: every length, equal ones,
    0 and the longest, each computed once; lengths outside the bounds too."""
    D, longest = 64, 2100
    c = Case(D, 4, 8, kvtc.BF16, H, [1], [longest], seed=n)
    c.fill()
    lens = [int(x) for x in c.rng.integers(0, longest + 1, n)]
    lens[3], lens[7], lens[8], lens[9], lens[n - 1] = longest, 0, 900, 900, 901
    q = c.rand(n, H * G, D)
    table = c.table_dev.expand(n, -1).contiguous()
    starts = dev(list(range(n + 1)), torch.int32)

    def run(lens):
        b = c.cache.batch(table, dev(lens, torch.int32), starts, total_rows=n, max_rows=1, max_len=longest)
        out, lse = torch.full_like(q, 7.0), torch.full((n, H * G), 7.0, device="cuda")
        c.cache.attention(b, q, out=out, lse=lse, status=c.status)
        return out, lse

    out, lse = run(lens)
    assert c.status.item() == 0
    c.lens, c.starts, c.table = lens, list(range(n + 1)), c.table * n
    check_attention(c, q, out, lse, D ** -0.5, True, f"{n} sequences")
    bad = {5: -3, 11: longest + 1, 20: -2 ** 31, 21: 2 ** 31 - 1}
    got, _ = run([bad.get(z, x) for z, x in enumerate(lens)])
    assert c.status.item() == 1 << kvtc.ERR_INVALID_ARG
    for z in range(n):
        assert (got[z] == 7.0).all() if z in bad else torch.equal(got[z], out[z]), z


@pytest.mark.parametrize("scale", [1e-3, 1.0, 8.0])
def test_attention_scales(scale):
    """Flat and needle-sharp weights, scores that grow along the sequence."""
    c = Case(64, 8, 8, kvtc.FP32, 1, [3], [500], seed=9)
    c.fill()
    q, out, lse, scale = run_attention(c, 4, scale=scale)
    check_attention(c, q, out, lse, scale, True, f"scale {scale}")
    t = c.lens[0]
    k = torch.ones(t, 1, 64, device="cuda") * torch.linspace(-30, 30, t, device="cuda")[:, None, None]
    b = c.new_batch([t], [t], total_rows=t)
    c.cache.write(b, k, c.rand(t, 1, 64))
    for sign in (1.0, -1.0):
        q = torch.full((3, 4, 64), sign, device="cuda")
        lse = torch.empty(3, 4, device="cuda")
        out, _ = c.cache.attention(c.batch, q, scale, lse=lse)
        check_attention(c, q, out, lse, scale, True, f"ramp {sign} scale {scale}")


@pytest.mark.parametrize("rows", [3, 20, 80])
@pytest.mark.parametrize("D,bv", [(64, 4), (64, 8), (128, 4), (128, 8)])
@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
def test_nan_tokens_reach_only_rows_that_attend_to_them(D, bv, dtype, rows):
    """Few, some and many rows (a kernel each)."""
    ln, H, G = rows + 80, 2, 2
    for kv, back in ((0, 2), (1, 2), (1, 1), (1, rows - 1), (0, 1), (1, rows + 40)):
        pos = ln - back
        c = Case(D, 8, bv, dtype, H, [rows], [ln], seed=pos)
        k, v = c.rand(ln, H, D), c.rand(ln, H, D)
        (k, v)[kv][pos, 1, 33] = float("nan")
        b = c.new_batch([ln], [ln], total_rows=ln)
        c.cache.write(b, k, v)
        q = c.rand(rows, H * G, D)
        out = c.cache.attention(c.batch, q)
        want = torch.zeros(rows, H * G, D, dtype=torch.bool, device="cuda")
        first = max(pos - (ln - rows), 0)
        want[first:, G:, :] = kv == 0
        want[first:, G:, 32:64] = True
        assert torch.equal(torch.isnan(out), want), (kv, pos)
    # as a query: its own row and head only
    q[2, 1, 5] = float("nan")
    want = torch.isnan(out)
    out2 = c.cache.attention(c.batch, q)
    want[2, 1] = True
    assert torch.equal(torch.isnan(out2), want)


@pytest.mark.parametrize("n", [3, 40])
def test_nan_token_in_the_prefix(n):
    """A sequence inside the prefix does not see the NaN that the others see,
    with few rows together and with many."""
    lens = [32 + 7 * (z % 3) if z % 4 else 20 for z in range(n)]
    lens[0] = 32
    c = Case(128, 4, 4, kvtc.BF16, 1, [1] * n, lens, shared=2, seed=n)
    first = c.cache.batch(c.table_dev[:1], dev([32], torch.int32), dev([0, 32], torch.int32), total_rows=32, max_rows=32,
                          max_len=32)
    k, v = c.rand(32, 1, 128), c.rand(32, 1, 128)
    v[25, 0, 100] = float("nan")
    c.cache.write(first, k, v)
    rest = [max(x - 32, 0) for x in lens]
    own = c.cache.batch(c.table_dev, dev(lens, torch.int32), dev([0] + [int(x) for x in np.cumsum(rest)], torch.int32),
                        total_rows=max(sum(rest), 1), max_rows=max(max(rest), 1), max_len=max(lens))
    c.cache.write(own, c.rand(max(sum(rest), 1), 1, 128), c.rand(max(sum(rest), 1), 1, 128), status=c.status)
    q = c.rand(n, 2, 128)
    nan = torch.isnan(c.cache.attention_shared(c.batch, q, 2, status=c.status))
    want = torch.zeros_like(nan)
    want[[z for z in range(n) if lens[z] > 25], :, 96:] = True
    assert torch.equal(nan, want) and c.status.item() == 0


def test_attention_infinite_query():
    """An infinite query spoils its own row and head, nothing else."""
    c = Case(64, 8, 4, kvtc.BF16, 1, [4], [60], seed=12)
    c.fill()
    q = c.rand(4, 2, 64)
    good = c.cache.attention(c.batch, q)
    q[1, 0, 3] = float("inf")
    out = c.cache.attention(c.batch, q)
    keep = torch.ones(4, 2, dtype=torch.bool, device="cuda")
    keep[1, 0] = False
    assert torch.equal(out[keep], good[keep])


# ---- metadata that is wrong, streams, graphs


def test_bad_metadata_is_reported_and_skipped():
    bad_bit = 1 << kvtc.ERR_INVALID_ARG
    H, D = 2, 128

    def fresh():
        c = Case(D, 4, 4, kvtc.BF16, H, [2, 3, 1], [40, 20, 33], seed=8)
        c.fill()
        q = c.rand(6, H * 2, D)
        return c, q, c.cache.attention(c.batch, q)

    # lengths outside the bounds, row ranges outside the tensors or backwards
    for lens, starts in (([40, 41, 33], [0, 2, 5, 6]), ([40, -1, 33], [0, 2, 5, 6]), ([40, 20, 33], [0, 2, 6, 7]),
                         ([40, 20, 33], [0, 5, 2, 3]), ([40, 20, 33], [0, 2, 6, 6])):
        c, q, good = fresh()
        b = c.cache.batch(c.table_dev, dev(lens, torch.int32), dev(starts, torch.int32), total_rows=6, max_rows=3, max_len=40)
        out = torch.full_like(q, 7.0)
        print("bad metadata", lens, starts, flush=True)
        c.cache.attention(b, q, out=out, status=c.status)
        assert c.status.item() == bad_bit
        if starts[1] == 2:
            assert torch.equal(out[:2], good[:2])
        before = c.cache.pool.clone()
        c.status.zero_()
        c.cache.write(b, c.rand(6, H, D), c.rand(6, H, D), status=c.status)
        assert c.status.item() == bad_bit
        for z in range(3):
            n = starts[z + 1] - starts[z]
            if not (0 <= lens[z] <= 40 and 0 <= n <= 3 and starts[z + 1] <= 6 and starts[z] >= 0):
                assert torch.equal(c.cache.pool[0, c.table[z]], before[0, c.table[z]])
        c.status.zero_()
        c.cache.read(b, torch.empty(6, H, D, device="cuda"), torch.empty(6, H, D, device="cuda"), status=c.status)
        assert c.status.item() == bad_bit
    # pages outside the pool: their tokens are masked, everything else as without them
    for page in (-1, 2 ** 31 - 1, "pages"):
        c, q, good = fresh()
        page = c.pages if page == "pages" else page
        c.table_dev[1, 1] = page
        out = torch.full_like(q, 7.0)
        print("bad page", page, flush=True)
        c.cache.attention(c.batch, q, out=out, status=c.status)
        assert c.status.item() == bad_bit and torch.equal(out[:2], good[:2]) and torch.equal(out[5:], good[5:])
        kp, vp = c.unpacked()
        want, _, _, _ = mx_ref.attention(kp, vp, [c.table[1]], [16], [0, 1], np64(q)[4:5], D ** -0.5, True)
        assert np.abs(np64(out[4:5]) - want).max() < 0.05
        before = c.cache.pool.clone()
        c.cache.write(c.batch, c.rand(6, H, D), c.rand(6, H, D), status=c.status)
        assert torch.equal(c.cache.pool[0, c.table[1]], before[0, c.table[1]])
        k = torch.full((6, H, D), 7.0, device="cuda")
        c.cache.read(c.batch, k, k.clone(), status=c.status)
        assert (k[2:5] == 7.0).all() and not (k[:2] == 7.0).any()
    # a call that is fine adds nothing
    c, q, good = fresh()
    c.cache.attention(c.batch, q, status=c.status)
    assert c.status.item() == 0


@pytest.mark.parametrize("rows,page", [(2, 5), (2, 150), (40, 60), (200, 0), (200, 100), (200, 180)])
def test_pages_outside_the_pool_anywhere(rows, page):
    """Near the start and far behind it, for few, some and many rows: exactly
    that page's tokens are missing."""
    H, G, D, ln = 1, 1 if rows > 2 else 2, 64, 3000
    c = Case(D, 8, 8, kvtc.FP32, H, [rows], [ln], seed=rows + page)
    c.fill()
    q = c.rand(rows, H * G, D)
    c.table_dev[0, page] = c.pages + 3
    out = c.cache.attention(c.batch, q, status=c.status)
    assert c.status.item() == 1 << kvtc.ERR_INVALID_ARG
    kp, vp = c.unpacked()
    k, v = mx_ref.tokens(kp, vp, c.table[0], ln)
    keep = np.arange(ln) // 16 != page
    for r in (0, rows // 2, rows - 1):
        lim = ln - rows + r + 1
        m = keep[:lim]
        s = D ** -0.5 * (k[0, :lim][m] @ np64(q)[r].T)
        p = np.exp(s - s.max(0))
        want = (p / p.sum(0)).T @ v[0, :lim][m]
        assert np.abs(np64(out)[r] - want).max() < 1e-5 * np.abs(v[0, :lim][m]).max()


def test_loose_bounds_give_the_same():
    """Bounds far above what the device arrays hold (a captured step's) choose
    other kernels and other splits, not other results."""
    rows, lens = [1, 2, 1, 0, 3], [700, 33, 1, 90, 400]
    for shared in (None, 1):
        c = Case(128, 8, 4, kvtc.FP32, 2, rows, lens, seed=31, shared=shared or 0)
        c.fill()
        q, out, lse, scale = run_attention(c, 4, shared=shared)
        check_attention(c, q, out, lse, scale, True, "tight bounds")
        wide = torch.full((5, 300), -1, dtype=torch.int32, device="cuda")
        wide[:, :c.table_dev.shape[1]] = c.table_dev
        c.table_dev = wide
        for max_rows, max_len in ((8, 4800), (7, 700), (1000, 4800)):
            c.batch = c.new_batch(rows, lens, max_rows=max_rows, max_len=max_len)
            q2, out2, lse2, _ = run_attention(c, 4, shared=shared)
            check_attention(c, q2, out2, lse2, scale, True, f"bounds {max_rows} {max_len}")


def test_pool_offsets_past_32_bits():
    """The same tokens in a small pool and in the last pages of one of 4.5 GB,
    behind a whole layer: the same bytes, values and outputs."""
    H, D, ln = 8, 128, 700
    pages, last = -(-ln // 16), 65000
    cfg = dict(layers=2, kv_heads=H, head_dim=D, dtype=kvtc.BF16, bits_k=8, bits_v=8)
    c = Case(D, 8, 8, kvtc.BF16, H, [1], [ln], seed=16)
    k, v = c.rand(ln, H, D), c.rand(ln, H, D)
    got = []
    for n in (pages, last):
        cache = kvtc.MxCache(cfg, n)
        table = dev([list(range(n - 1, n - 1 - pages, -1))], torch.int32)

        def batch(rows):
            return cache.batch(table, dev([ln], torch.int32), dev([0, rows], torch.int32), rows, rows, ln)

        cache.write(batch(ln), k, v, layer=1, status=c.status)
        ko, vo = torch.empty_like(k), torch.empty_like(v)
        cache.read(batch(ln), ko, vo, layer=1, status=c.status)
        outs = [cache.pool[1, table[0, :ln // 16].long()], ko, vo]  # (the last page is not full: anything behind its tokens)
        for rows in (2, 17, 200):
            q = k[:rows].repeat(1, 2, 1) + v[:rows].repeat(1, 2, 1)
            outs.append(cache.attention(batch(rows), q, layer=1, status=c.status))
            outs.append(cache.attention_shared(batch(rows), q, 20, layer=1, status=c.status))
        got.append(outs)
    assert last * H * cache.record_bytes * 2 > 2 ** 32 and c.status.item() == 0
    for small, big in zip(*got):
        assert torch.equal(small, big) and not torch.isnan(big.float()).any()


def test_repeatable_and_on_other_streams():
    c = Case(128, 4, 8, kvtc.BF16, 2, [1] * 6, [900, 3, 77, 2000, 512, 1], seed=13)
    c.fill()
    q = c.rand(6, 8, 128)
    good = c.cache.attention(c.batch, q)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):
        for s in streams:  # both at once, each with a workspace of its own
            outs.append(c.cache.attention(c.batch, q, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, good) for o in outs)


def test_captured_calls_follow_the_device_arrays():
    """A step (write, attend, shared prefix) captured once and replayed while
    lengths, pages and rows change; every replay against the eager call."""
    D, H, G, n = 128, 2, 4, 3
    c = Case(D, 8, 4, kvtc.BF16, H, [1] * n, [300, 300, 300], seed=14, shared=2)
    c.fill()
    lens, starts = dev([33, 40, 35], torch.int32), dev([0, 1, 2, 3], torch.int32)
    b = c.cache.batch(c.table_dev, lens, starts, total_rows=n, max_rows=1, max_len=300)
    k, v, q = c.rand(n, H, D), c.rand(n, H, D), c.rand(n, H * G, D)
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    ws, ws2 = c.cache.workspace(b, H * G), c.cache.workspace(b, H * G, 2)

    def step(o, o2):
        c.cache.write(b, k, v, status=c.status)
        c.cache.attention(b, q, out=o, ws=ws, status=c.status)
        c.cache.attention_shared(b, q, 2, out=o2, ws=ws2, status=c.status)

    step(out, out2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(out, out2)
    for r in range(6):
        lens.copy_(dev([33 + 40 * r, 40 + 3 * r, 35 + 50 * r], torch.int32))
        q.copy_(c.rand(n, H * G, D))
        k.copy_(c.rand(n, H, D))
        if r == 3:
            c.table_dev[0, 5], c.table_dev[1, 5] = int(c.table[1][5]), int(c.table[0][5])
        g.replay()
        torch.cuda.synchronize()
        pool = c.cache.pool.clone()
        e, e2 = torch.empty_like(q), torch.empty_like(q)
        step(e, e2)
        assert torch.equal(pool, c.cache.pool) and torch.equal(out, e) and torch.equal(out2, e2), r
    assert c.status.item() == 0


def test_decoded_cache_is_served_and_encoded_again():
    """As a serving program uses the two together: a container is decoded, its
    cache goes into pages, a conversation goes on for some steps (fused
    projections, one layer after the other), and the grown cache is read back
    and encoded."""
    L, H, G, D, T = 2, 2, 4, 128, 300
    cfg = dict(layers=L, kv_heads=H, head_dim=D, dtype=kvtc.BF16, transform=kvtc.PCA, sink_tokens=4, recent_tokens=32,
               bits_k=4.0, bits_v=4.0, max_bits=8, rope_keys=0, rope_style=0, rope_theta=10000.0, rans_scale_bits=12,
               rans_lanes=32, chunk_tokens=1024, tile_tokens=128, basis_per_head=0, wht_keys=0)
    basis = torch.eye(D).expand(L, 2, D, D).contiguous()
    plan = kvtc.Plan(cfg, basis, max_tokens=400)
    c = Case(D, 8, 4, kvtc.BF16, H, [T], [T], layers=L, seed=15)
    data, st = plan.encode(c.rand(L, H, T, D), c.rand(L, H, T, D))
    assert st == kvtc.OK
    K, V, st = plan.decode(data, T, kvtc.BF16)
    assert st == kvtc.OK
    total = T + 10
    table = dev([list(range(-(-total // 16)))], torch.int32)
    cache = kvtc.MxCache(dict(layers=L, kv_heads=H, head_dim=D, dtype=kvtc.BF16, bits_k=8, bits_v=4), table.shape[1])
    lens = dev([T], torch.int32)
    cache.write(cache.batch(table, lens, dev([0, T], torch.int32), T, T, total), K, V, status=c.status)
    rows_k, rows_v = [np64(K)], [np64(V)]
    step = cache.batch(table, lens, dev([0, 1], torch.int32), total_rows=1, max_rows=1, max_len=total)
    for t in range(T, total):
        lens += 1
        new = []
        for layer in range(L):
            qkv = c.rand(1, (G + 2) * H, D)
            q, k, v = qkv.split([G * H, H, H], 1)
            cache.write(step, k, v, layer=layer, status=c.status)
            out = cache.attention(step, q, layer=layer, status=c.status)
            new.append((np64(k)[0], np64(v)[0]))
            kp, vp = mx_ref.unpack(cache.pool[layer].cpu().numpy(), D, 8, 4)
            want, _, mass, _ = mx_ref.attention(kp, vp, [list(range(table.shape[1]))], [t + 1], [0, 1], np64(q), D ** -0.5, True)
            assert (np.abs(np64(out) - want) <= 2.0 ** -7 * mass + 2.0 ** -8 * np.abs(want)).all()
        rows_k.append(np.stack([x[0] for x in new])[:, :, None])
        rows_v.append(np.stack([x[1] for x in new])[:, :, None])
    ko, vo = (torch.empty(L, H, total, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.read(cache.batch(table, lens, dev([0, total], torch.int32), total, total, total), ko, vo, status=c.status)
    for got, rows, b in ((ko, rows_k, 8), (vo, rows_v, 4)):
        want = mx_ref.values(*mx_ref.quantise(np.concatenate(rows, 2), b), b)
        assert np.array_equal(np64(got), want)
    data, st = plan.encode(ko, vo)
    assert st == kvtc.OK and c.status.item() == 0
    k2, v2, st = plan.decode(data, total, kvtc.BF16)
    assert st == kvtc.OK and torch.equal(k2[:, :, -32:], ko[:, :, -32:])


# ---- every kernel in every format, batches of unlike sequences, captured ranges


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
@pytest.mark.parametrize("D,bk,bv", FORMATS)
def test_attention_many_rows_formats(D, bk, bv, dtype):
    """The kernel for many rows in every format: prompts with and without
    tokens before them, a lone row and a sequence without rows among them."""
    rows, lens = [150, 1, 0, 70, 129], [150, 260, 40, 70, 300]
    for G, causal in ((2, True), (3, False)):
        c = Case(D, bk, bv, dtype, 2, rows, lens, seed=D + 2 * bk + bv, total_rows=sum(rows) + 2)
        c.fill()
        q, out, lse, scale = run_attention(c, G, causal)
        check_attention(c, q, out, lse, scale, causal, f"many rows D{D} k{bk} v{bv} dtype {dtype} causal {causal}")


@pytest.mark.parametrize("most", [2, 7, 40])
@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
@pytest.mark.parametrize("D,bk,bv", FORMATS)
def test_attention_behind_a_prefix_formats(D, bk, bv, dtype, most):
    """More than 64 rows together behind a prefix, in every format: a few own
    rows a sequence (both passes in one launch), some, and many."""
    rng = np.random.default_rng(D + bk + bv + most)
    n = 30 if most < 40 else 4
    lens = [160 + int(x) for x in rng.integers(0, 150, n)]
    lens[0], lens[1], lens[n - 1] = 160, 90, 161
    rows = [1 + int(x) for x in rng.integers(0, most, n)]
    rows[2], rows[3] = most, 0
    c = Case(D, bk, bv, dtype, 2, rows, lens, seed=most, shared=10, total_rows=sum(rows) + 1)
    c.fill()
    for causal in (True, False):
        q, out, lse, scale = run_attention(c, 3, causal, shared=10)
        check_attention(c, q, out, lse, scale, causal, f"behind D{D} k{bk} v{bv} dtype {dtype} rows {most} causal {causal}")


@pytest.mark.parametrize("D,bk,bv,dtype,H,shared", [(64, 4, 4, kvtc.BF16, 8, 1100), (64, 8, 4, kvtc.FP32, 8, 1100),
                                                    (128, 4, 4, kvtc.BF16, 4, 2200)])
def test_attention_few_rows_behind_a_long_prefix(D, bk, bv, dtype, H, shared):
    """At most 16 rows together: ranges of the prefix long enough for the
    larger workgroups, a sequence inside the prefix, one at its end."""
    p = 16 * shared
    lens = [p + 5, p, p + 300, p - 7000, 40]
    c = Case(D, bk, bv, dtype, H, [1, 1, 2, 1, 1], lens, seed=D + bk, shared=shared, total_rows=8)
    c.fill()
    q, out, lse, scale = run_attention(c, 2, shared=shared)
    check_attention(c, q, out, lse, scale, True, f"long prefix D{D} k{bk} v{bv} dtype {dtype}")


@pytest.mark.parametrize("rows,G", [(1, 20), (5, 4), (1, 32)])
def test_attention_sequences_by_length_of_some_rows(rows, G):
    """More whole sequences than compute units take, in tiles of 32 rows, in
    part and all full."""
    n, H, D = 36, 8, 64
    lens = [int(x) for x in np.random.default_rng(G).integers(0, 2101, n)]
    lens[0], lens[5], lens[6], lens[7] = 2100, 0, 1, 2100
    c = Case(D, 8, 4, kvtc.BF16, H, [1], [2100], seed=G)
    c.fill()
    c.table_dev, c.table = c.table_dev.expand(n, -1).contiguous(), c.table * n
    take = [rows if z % 3 else max(rows - 1, 0) for z in range(n)]
    c.lens, c.rows, c.starts, c.total = lens, take, [0] + [int(x) for x in np.cumsum(take)], sum(take) + 1
    c.batch = c.new_batch(take, lens, max_rows=rows)
    q, out, lse, scale = run_attention(c, G)
    check_attention(c, q, out, lse, scale, True, f"by length {rows} rows of {G}")


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_prompts_beside_single_rows(dtype, causal):
    """One call for a prompt's chunk and the decode steps of the others: some
    long, some empty, some with more rows than tokens (which see no token when
    causal, and all of them when not)."""
    lens = [400, 1, 0, 17, 900, 2, 33, 64, 5, 1500] + [100 + 13 * z for z in range(12)]
    rows = [130, 1, 1, 1, 1, 5, 1, 0, 9, 2] + [1] * 12
    for D, bk, bv in ((128, 4, 4), (64, 8, 8)):
        c = Case(D, bk, bv, dtype, 2, rows, lens, seed=D, total_rows=sum(rows) + 4)
        c.fill()
        q, out, lse, scale = run_attention(c, 4, causal)
        check_attention(c, q, out, lse, scale, causal, f"mixed D{D} dtype {dtype} causal {causal}")


@pytest.mark.parametrize("rows", [2, 20, 80])
@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
def test_attention_scores_up_to_their_bound(dtype, rows):
    """Scores of up to 2^25 of either sign and values of 2^64.  Keys of one
    channel and a query of one power of two: products and scores are exact and
    at least 2^16 apart, so a row is the mean of the tokens with its largest score, and
    its log-sum-exp that score and the logarithm of their number."""
    D, ln = 64, 300
    u = 2.0 ** -8 if dtype == kvtc.BF16 else 2.0 ** -23
    for sign in (1.0, -1.0):
        for order in ("up", "down", "mixed"):
            c = Case(D, 8, 8, dtype, 1, [rows], [ln], seed=rows)
            t = {"up": np.arange(ln), "down": np.arange(ln)[::-1].copy(), "mixed": c.rng.permutation(ln)}[order] // 7
            lead = (8 + t % 8) * 2.0 ** (t // 8)  # 42 values with four significant bits, 8 to 320
            k, v = torch.zeros(ln, 1, D, dtype=DT[dtype], device="cuda"), c.rand(ln, 1, D) * 2.0 ** 60
            v = v.clamp(-2.0 ** 64, 2.0 ** 64)
            k[:, 0, 0] = dev(lead, torch.float32).to(DT[dtype])
            b = c.new_batch([ln], [ln], total_rows=ln)
            c.cache.write(b, k, v, status=c.status)
            q = torch.zeros(rows, 2, D, dtype=DT[dtype], device="cuda")
            q[:, :, 0] = sign * 2.0 ** 10
            lse = torch.empty(rows, 2, device="cuda")
            out, _ = c.cache.attention(c.batch, q, 2.0 ** 6, lse=lse, status=c.status)
            score = sign * 2.0 ** 16 * lead
            assert np.abs(score).max() < 2.0 ** 25
            vp = mx_ref.tokens(*c.unpacked(), c.table[0], ln)[1][0]
            for i in range(rows):
                lim = ln - rows + i + 1
                top = score[:lim] == score[:lim].max()
                want = vp[:lim][top].mean(0)
                # weights and output are rounded once each, the sum of the few weights by as many steps of 2^-24
                tol = 2 * u * np.abs(vp[:lim][top]).mean(0) + 64 * 2.0 ** -24 * np.abs(vp[:lim][top]).max()
                assert (np.abs(np64(out)[i] - want) <= tol).all(), (sign, order, i)
                wl = score[:lim].max() + np.log(top.sum())
                # roundings of scale log2(e), of the sum, of ln 2, of their product and of the join
                assert (np.abs(np64(lse)[i] - wl) <= 5 * 2.0 ** -24 * abs(wl)).all(), (sign, order, i)
    assert c.status.item() == 0


@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
def test_captured_ranges_follow_lengths_and_rows(dtype):
    """A call captured under bounds that split the tokens into ranges, replayed
    while lengths cross the ranges' borders, rows move between the sequences
    and one of them has none; every replay against the plain implementation
    and against the eager call, rows of no sequence left alone."""
    D, H, G, n, most = 64, 2, 2, 4, 3000
    c = Case(D, 8, 4, dtype, H, [1] * n, [most] * n, seed=44, shared=8, total_rows=9)
    c.fill()
    lens, starts = dev([1] * n, torch.int32), dev([0] * (n + 1), torch.int32)
    b = c.cache.batch(c.table_dev, lens, starts, total_rows=9, max_rows=4, max_len=most)
    q = c.rand(9, H * G, D)
    outs = [torch.empty_like(q) for _ in range(2)]
    lses = [torch.empty(9, H * G, device="cuda") for _ in range(2)]
    ws = [c.cache.workspace(b, H * G), c.cache.workspace(b, H * G, 8)]
    assert all(w.nbytes > 16 for w in ws)

    def step(o, s):
        c.cache.attention(b, q, out=o[0], lse=s[0], ws=ws[0], status=c.status)
        c.cache.attention_shared(b, q, 8, out=o[1], lse=s[1], ws=ws[1], status=c.status)

    step(outs, lses)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(outs, lses)
    for r, (ln, rows) in enumerate([((128, 129, 127, 1), (1, 1, 1, 1)), ((3000, 256, 2999, 130), (4, 0, 2, 1)),
                                    ((0, 5, 128, 2177), (1, 3, 0, 4)), ((64, 1000, 2048, 257), (0, 0, 4, 0)),
                                    ((2945, 2944, 2943, 40), (2, 2, 2, 3)), ((128, 129, 127, 1), (1, 1, 1, 1))]):
        c.lens, c.starts = list(ln), [0] + [int(x) for x in np.cumsum(rows)]
        lens.copy_(dev(c.lens, torch.int32))
        starts.copy_(dev(c.starts, torch.int32))
        q.copy_(c.rand(9, H * G, D))
        for x in (*outs, *lses):
            x.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        e, es = [torch.full_like(x, 7.0) for x in outs], [torch.full_like(x, 7.0) for x in lses]
        step(e, es)
        for o, s, o2, s2 in zip(outs, lses, e, es):
            assert torch.equal(o, o2) and torch.equal(s, s2), r
            assert (o[c.starts[-1]:] == 7.0).all() and (s[c.starts[-1]:] == 7.0).all(), r
            check_attention(c, q, o, s, D ** -0.5, True, f"replay {r} dtype {dtype}")
    assert c.status.item() == 0


@pytest.mark.parametrize("D,bk,bv,dtype", [(128, 4, 4, kvtc.BF16), (64, 8, 8, kvtc.FP32)])
def test_attention_one_workgroup_a_unit_behind_a_prefix(D, bk, bv, dtype):
    """Own tokens for the larger workgroups in a launch after the prefix's: the
    rows together fit one of its tiles or many, under bounds of hundreds of
    megabytes of codes too."""
    H, ln = 8, 1500
    lens = [1500 - 29 * z for z in range(24)] + [0, 48, 49, 20, 303, 304]
    n = len(lens)
    for G, bounds in ((2, (1500, 12800)), (4, (1500, 12800))):
        c = Case(D, bk, bv, dtype, H, [1], [ln], seed=D + G)
        c.fill()
        c.table_dev = torch.cat([c.table_dev.expand(n, -1), torch.full((n, 720), 2 ** 30, dtype=torch.int32, device="cuda")], 1)
        c.table, c.rows, c.lens, c.starts, c.total = c.table * n, [1] * n, lens, list(range(n + 1)), n + 1
        for bound in bounds:
            c.batch = c.new_batch(c.rows, lens, max_len=bound)
            q, out, lse, scale = run_attention(c, G, shared=3)
            check_attention(c, q, out, lse, scale, True, f"D{D} G{G} bound {bound}")


@pytest.mark.parametrize("rows", [2, 20, 80])
@pytest.mark.parametrize("dtype", [kvtc.BF16, kvtc.FP32])
def test_attention_products_near_the_end_of_fp32(dtype, rows):
    """Products of -3.2e38, -2.8e38 and -1.6e38 under a scale that makes them
    ordinary scores, the least ones alone, first, last and in between."""
    D, ln = 64, 150
    for order in (np.full(ln, 120.0), np.where(np.arange(ln) < 70, 120.0, 104.0), np.where(np.arange(ln) < 50, 60.0, 120.0),
                  np.tile([120.0, 104.0, 120.0, 120.0, 60.0], 30)):
        c = Case(D, 8, 8, dtype, 1, [rows], [ln], seed=rows)
        k, v = torch.zeros(ln, 1, D, dtype=DT[dtype], device="cuda"), c.rand(ln, 1, D)
        k[:, 0, 5] = dev(order * 2.0 ** 58, torch.float32).to(DT[dtype])
        c.cache.write(c.new_batch([ln], [ln], total_rows=ln), k, v, status=c.status)
        q = torch.zeros(rows, 2, D, dtype=DT[dtype], device="cuda")
        q[:, :, 5] = -2.0 ** 63
        lse = torch.empty(rows, 2, device="cuda")
        for scale in (2.0 ** -124, 2.0 ** -126):
            out, _ = c.cache.attention(c.batch, q, scale, lse=lse, status=c.status)
            check_attention(c, q, out, lse, scale, True, f"products {order[:3]} scale {scale}")
    assert c.status.item() == 0
