"""A decoder's self attention against plain 64-bit implementations: rotary positions, appending to a paged cache,
attention over it behind a shared prefix, and a run of them together.

Tolerances, from the arithmetic (u = 2^-24, one fp32 rounding):
  results         half a step: bf16 2^-8 |y|, fp32 2^-24 |y|
  rotation        sine and cosine of the reduced angle are off by pi u for its rounding and, fp32, two units in the last place
                  (2^-22 at most together); bf16, 2^-21.19 of the hardware's and pi u: 16 u covers either. The
                  factor, two products and an addition: 4 u more. All of it times |u| + |v| and the factor.
                  fp64: the angle p f is off by 2^-51 of itself and by p 2^-63, here and in the reference
  attention       a score is off by 2 u (dh + 4) scale sum|q||k|, and its weight by twice that, relatively; bf16 weights
                  by 2^-8 more; sums of n fp32 terms by 2 u (n + 8); the exponential of a rounded argument by 2^-20;
                  the joining factors of parts by 2^-20 again
"""
import math

import pytest
import torch

from vision_transformer_encoder_gb300 import api

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = {BF: 2.0 ** -8, F32: U, F64: 2.0 ** -53}
DEV = "cuda:0"
LAYOUTS = [api.ROTARY_HALF, api.ROTARY_INTERLEAVED]


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert api.device_error() == 0


def rand(*shape, seed=0, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed * 7919 + sum(shape))
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def close(got, ref, tol):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    bad = ~((got - ref).abs() <= tol) & ~torch.isnan(ref) & ~(got == ref)
    if bad.any():
        i = int(torch.argmax(((got - ref).abs() / tol.clamp_min(1e-300)).nan_to_num(0).reshape(-1)))
        raise AssertionError("%d of %d outside: worst got %g ref %g tol %g" % (
            int(bad.sum()), bad.numel(), got.reshape(-1)[i], ref.reshape(-1)[i], tol.expand_as(ref).reshape(-1)[i]))


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# --------------------------------------------------------------------------------- rotary
def rotary_ref(x, f, pos, layout, scale=1.0):
    """(rotated x, what its errors go by) in 64 bits."""
    x, n = x.double(), f.numel()
    a = pos.double()[:, :, None, None] * f.double()
    c, s = torch.cos(a) * scale, torch.sin(a) * scale
    i = torch.arange(n, device=x.device)
    i, j = (i, i + n) if layout == api.ROTARY_HALF else (2 * i, 2 * i + 1)
    y, w = x.clone(), torch.zeros_like(x)
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    w[..., i] = w[..., j] = (x[..., i].abs() + x[..., j].abs()) * abs(scale)
    return y, w


def rotary_tol(y, w, dt, f, pos):
    if dt == F64:
        a = pos.double().abs()[:, :, None, None] * f.abs().max()
        return w * (a * 2.0 ** -50 + pos.double().abs()[:, :, None, None] * 2.0 ** -60 + 2.0 ** -49) + HALF[dt] * y.abs()
    return w * 20 * U + HALF[dt] * y.abs() * 1.01


def check_rotary(x, f, pos=None, layout=api.ROTARY_HALF, scale=1.0, **kw):
    got = api.rotary(x, f, positions=pos, layout=layout, scale=scale, **kw)
    if pos is None:
        pos = torch.arange(x.shape[1], device=DEV).expand(x.shape[0], -1)
    y, w = rotary_ref(x, f, pos, layout, scale)
    close(got, y, rotary_tol(y, w, x.dtype, f, pos))
    return got


ROTARY_SHAPES = [(1, 1, 1, 2, 2), (1, 1, 1, 64, 64), (3, 5, 3, 64, 32), (2, 7, 4, 80, 80), (1, 300, 16, 128, 128), (2, 33, 5, 96, 6),
                 (5, 1, 12, 64, 64), (1, 3, 2, 17, 10), (2, 2, 3, 512, 512), (1, 2, 7, 40, 8), (700, 1, 20, 64, 48),
                 (1, 2600, 12, 64, 16), (1, 2, 256, 80, 80), (1, 9, 103, 80, 64), (1, 300, 70, 512, 512), (1, 3, 700, 64, 64)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", [BF, F32, F64], ids=str)
@pytest.mark.parametrize("shape", ROTARY_SHAPES, ids=str)
def test_rotary(shape, dt, layout):
    B, T, H, dh, width = shape
    x = rand(B, T, H, dh, seed=1, dtype=dt)
    f = api.rotary_frequencies(width, device=DEV)
    check_rotary(x, f, layout=layout)
    pos = torch.randint(-1000, 5000, (B, T), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(DEV)
    check_rotary(x, f, pos, layout, 1.25)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
def test_rotary_at_far_positions(dt, layout):
    x = rand(1, 6, 3, 64, seed=2, dtype=dt)
    for f in (api.rotary_frequencies(64, device=DEV), api.rotary_frequencies(64, 500000.0, factor=8, trained=8192, device=DEV),
              torch.tensor([7.0, -3.0, 6.283185307179586, 0.0, 1e3, -1e-3], dtype=F64, device=DEV)):
        pos = ints([[0, -1, 1 << 20, -(1 << 24) + 1, (1 << 31) - 1, -(1 << 31)]])
        # the reference's own angle: p f 2^-53, and as much for f / 2 pi
        y, w = rotary_ref(x, f, pos, layout)
        a = pos.double().abs()[:, :, None, None] * f.abs().max() * 2.0 ** -51
        close(api.rotary(x, f, positions=pos, layout=layout), y, rotary_tol(y, w, dt, f, pos) + w * a)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", [BF, F32, F64], ids=str)
def test_rotary_layouts_in_place_and_unaligned(dt, layout):
    B, T, H, dh = 3, 10, 4, 64
    f = api.rotary_frequencies(48, device=DEV)
    qkv = rand(B, T, H + 4, dh, seed=4, dtype=dt)
    for x in (qkv[:, :, 1:1 + H], rand(B, H, T, dh, seed=5, dtype=dt).transpose(1, 2), qkv[:, :, :1].expand(-1, -1, H, -1),
              rand(T, B, H, dh, seed=6, dtype=dt).transpose(0, 1), rand(B * T * H * dh + 1, seed=7, dtype=dt)[1:].view(B, T, H, dh),
              rand(B, T, H, dh + 3, seed=8, dtype=dt)[..., :dh]):
        got = check_rotary(x, f, layout=layout)
        assert got.is_contiguous()
        shifted = torch.empty(x.numel() + 1, dtype=dt, device=DEV)[1:].view(x.shape)
        assert same(check_rotary(x, f, layout=layout, out=shifted), got) and same(shifted, got)
    ref = check_rotary(qkv[:, :, 1:1 + H], f, layout=layout)
    whole = qkv.clone()
    view = qkv[:, :, 1:1 + H]
    assert api.rotary(view, f, layout=layout, out=view) is view
    assert same(view, ref) and same(qkv[:, :, 0], whole[:, :, 0]) and same(qkv[:, :, 1 + H:], whole[:, :, 1 + H:])


def test_rotary_frequencies():
    """By parts: pairs that turn often within the trained length keep their frequency, slow ones are stretched."""
    f = api.rotary_frequencies(64)
    assert f.dtype == F64 and f.shape == (32,) and f[0] == 1
    assert torch.allclose(f, torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=F64), rtol=1e-14)
    assert torch.allclose(api.rotary_frequencies(64, factor=4), f / 4, rtol=1e-14)
    g = api.rotary_frequencies(64, factor=4, trained=4096)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32]) and torch.allclose(g[turns < 1], f[turns < 1] / 4, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((g[mid] < f[mid]) & (g[mid] > f[mid] / 4)).all()
    for bad in (dict(width=0), dict(width=3), dict(width=8, factor=0), dict(width=8, slow=2, fast=1)):
        with pytest.raises(ValueError):
            api.rotary_frequencies(**bad)


# ------------------------------------------------------------------------------ the cache
def pool(pages, page, Hkv, dh, dt, fill=math.nan):
    """(keys, values), contiguous pools with `fill` everywhere."""
    return [torch.full((pages, page, Hkv, dh), fill, dtype=dt, device=DEV) for _ in range(2)]


def tables(held, page, spare=1, seed=0, width=None):
    """A page table for sequences with `held` keys each, pages in no order; entries behind them are rubbish. And the pages
    that the pool needs."""
    need = [-(-n // page) for n in held]
    total = sum(need) + spare
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    width = max(max(need), 1) + 1 if width is None else width
    t = torch.full((len(held), width), 1 << 30, dtype=torch.int32)
    t[:, 1::2] = -5
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return t.to(DEV), total


def slots(table, b, u, page):
    return int(table[b, u // page]), u % page


def append_ref(k, v, kp, vp, table, starts, lens, f, pos, layout, scale):
    """(keys, values) pools in 64 bits, and what the keys' errors go by."""
    k64, w = (k.double(), torch.zeros_like(k, dtype=F64)) if f is None else rotary_ref(k, f, pos, layout, scale)
    kp, vp, wp = kp.double(), vp.double(), torch.zeros_like(kp, dtype=F64)
    P, page = kp.shape[:2]
    t = table.cpu()
    for b in range(k.shape[0]):
        for i in range(k.shape[1] if lens is None else max(0, min(int(lens[b]), k.shape[1]))):
            u = int(starts[b]) + i
            if u < 0 or u >= t.shape[1] * page:
                continue
            pg, s = slots(t, b, u, page)
            if 0 <= pg < P:
                kp[pg, s], vp[pg, s], wp[pg, s] = k64[b, i], v[b, i].double(), w[b, i]
    return kp, vp, wp


def check_append(k, v, q, page, starts, lens=None, f=None, pos=None, layout=0, scale=1.0, table=None, pages=None, pools=None, **kw):
    B, T, Hkv, dh = k.shape
    dt = k.dtype
    if table is None:
        table, pages = tables([s + T for s in starts], page)
    kp, vp = pools or pool(pages, page, Hkv, dh, dt)
    starts = ints(starts)
    p = starts.long()[:, None] + torch.arange(T, device=DEV) if pos is None else pos   # past 32 bits too
    rk, rv, w = append_ref(k, v, kp, vp, table, starts, lens, f, p, layout, scale)
    got = api.cache_append(k, v, kp, vp, table, starts, lens=lens, q=q, frequencies=f, positions=pos, layout=layout, scale=scale, **kw)
    pp = torch.zeros((1, 1), dtype=torch.int32, device=DEV) if f is None else p.abs().max()[None, None]
    close(kp, rk, rotary_tol(rk, w, dt, f if f is not None else torch.zeros(1, dtype=F64, device=DEV), pp))
    assert torch.equal(vp.double().nan_to_num(7.0), rv.nan_to_num(7.0))
    if q is None:
        assert got is None
    elif f is None:
        assert same(got, q)
    else:
        y, w = rotary_ref(q, f, p, layout, scale)
        close(got, y, rotary_tol(y, w, dt, f, p))
    return got, kp, vp


APPEND_SHAPES = [(1, 1, 1, 1, 2, 2, 1), (3, 1, 16, 16, 64, 64, 16), (2, 5, 16, 2, 128, 128, 64), (2, 37, 12, 4, 80, 40, 16),
                 (4, 3, 6, 3, 17, 10, 5), (1, 300, 4, 4, 64, 64, 32), (64, 1, 12, 3, 96, 96, 128), (2, 9, 0, 2, 64, 32, 7),
                 (2, 40, 200, 28, 80, 80, 16), (1, 5, 0, 300, 64, 64, 16)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", [BF, F32, F64], ids=str)
@pytest.mark.parametrize("shape", APPEND_SHAPES, ids=str)
def test_cache_append(shape, dt, layout):
    B, T, H, Hkv, dh, width, page = shape
    k, v = rand(B, T, Hkv, dh, seed=1, dtype=dt), rand(B, T, Hkv, dh, seed=2, dtype=dt)
    q = rand(B, T, H, dh, seed=3, dtype=dt) if H else None
    f = api.rotary_frequencies(width, device=DEV)
    starts = [(7 * b) % 40 for b in range(B)]
    check_append(k, v, q, page, starts, f=f, layout=layout)
    lens = ints([(T * (b + 1)) // B - (b == 1) for b in range(B)])
    pos = torch.randint(0, 900, (B, T), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(DEV)
    check_append(k, v, q, page, starts, lens=lens, f=f, pos=pos, layout=layout, scale=0.9)
    check_append(k, v, q, page, starts)   # nothing turned


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
def test_cache_append_keeps_to_its_slots(dt):
    """Absent pages, slots outside the table, lengths outside [0, T]: nothing of those is written."""
    B, T, Hkv, dh, page = 6, 9, 2, 64, 4
    k, v, q = (rand(B, T, h, dh, seed=i, dtype=dt) for i, h in ((1, Hkv), (2, Hkv), (3, 4)))
    f = api.rotary_frequencies(64, device=DEV)
    table, pages = tables([24] * B, page, spare=3, width=6)
    table[0, 1], table[0, 2], table[1, 0], table[2, 5] = -1, pages, -(1 << 31), (1 << 31) - 1
    lens = ints([9, 9, 20, -3, 0, 9])
    check_append(k, v, q, page, [2, 0, 18, 3, 1, 22], lens=lens, f=f, table=table, pages=pages)
    check_append(k, v, q, page, [-4, 23, 24, 1 << 30, (1 << 31) - 1, -(1 << 31)], f=f, table=table, pages=pages)


@pytest.mark.parametrize("dt", [BF, F32, F64], ids=str)
def test_cache_append_layouts(dt):
    """A fused projection's parts, pools side by side in a page and heads before tokens, queries turned where they lie."""
    B, T, H, Hkv, dh, page = 2, 11, 4, 2, 64, 16
    qkv = rand(B, T, H + 2 * Hkv, dh, seed=1, dtype=dt)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    f = api.rotary_frequencies(64, device=DEV)
    table, pages = tables([30, 30], page)
    ref, kp, vp = check_append(k, v, q, page, [19, 3], f=f, table=table, pages=pages)
    side = torch.full((pages, 2, page, Hkv, dh), math.nan, dtype=dt, device=DEV)
    heads = torch.full((2, pages, Hkv, page, dh), math.nan, dtype=dt, device=DEV).transpose(2, 3)
    odd = torch.full((2, pages, page, Hkv, dh + 1), math.nan, dtype=dt, device=DEV)[..., :dh]
    for pools in ((side[:, 0], side[:, 1]), (heads[0], heads[1]), (odd[0], odd[1])):
        got, a, b = check_append(k, v, q, page, [19, 3], f=f, table=table, pages=pages, pools=pools)
        assert same(got, ref) and same(a, kp) and same(b, vp)
    keep = qkv.clone()
    pools = pool(pages, page, Hkv, dh, dt)
    assert api.cache_append(k, v, *pools, table, ints([19, 3]), q=q, frequencies=f, q_out=q) is q
    assert same(q, ref) and same(pools[0], kp) and same(qkv[:, :, H:], keep[:, :, H:])
    api.cache_append(k[:, :, :1], v[:, :, :1], kp[:, :, :1], vp[:, :, :1], table, ints([19, 3]), frequencies=f)
    assert same(kp, pools[0])


# --------------------------------------------------------------------------- paged attention
class Held:
    """Sequences in a paged cache: own[b] keys each (the new ones last), behind prefix[g] keys of their group. Pools hold NaN
    wherever there is no key."""

    def __init__(self, Tq, H, Hkv, dh, page, own, prefix=(), dt=BF, seed=0, q_lens=None):
        self.B, self.page, self.own, self.prefix, self.dt = len(own), page, list(own), list(prefix), dt
        self.q = rand(self.B, Tq, H, dh, seed=seed + 1, dtype=dt)
        held = self.own + self.prefix
        table, pages = tables(held, page, seed=seed)
        self.kp, self.vp = pool(pages, page, Hkv, dh, dt)
        kv = rand(sum(held) + 1, 2, Hkv, dh, seed=seed + 2, dtype=dt)
        at, where = 0, []
        for b, n in enumerate(held):
            for u in range(0, n, page):
                m = min(page, n - u)
                pg = int(table[b, u // page])
                self.kp[pg, :m], self.vp[pg, :m] = kv[at + u:at + u + m, 0], kv[at + u:at + u + m, 1]
            where.append((at, n))
            at += n
        self.k, self.v, self.where = kv[:, 0], kv[:, 1], where
        self.table = table[:self.B].contiguous()
        self.prefix_table = table[self.B:].contiguous() if prefix else None
        self.kv_lens, self.prefix_lens = ints(self.own), ints(self.prefix) if prefix else None
        self.q_lens = None if q_lens is None else ints(q_lens)

    def keys(self, b):
        """Rows of k and v that sequence b holds: (prefix, own)."""
        g = b // (self.B // len(self.prefix)) if self.prefix else None
        r = [torch.arange(a, a + n) for a, n in ([self.where[self.B + g]] if self.prefix else [(0, 0)]) + [self.where[b]]]
        return r

    def ref(self, scale, gone=()):
        """(o, sums of w |v|, largest sum |q||k| times |scale|, keys seen) in 64 bits; gone: (sequence, first, last) of own
        keys that are absent."""
        B, Tq, H, dh = self.q.shape
        Hkv = self.k.shape[1]
        G = H // Hkv
        out = [torch.zeros(B, Tq, H, n, dtype=F64, device=DEV) for n in (dh, dh, 1, 1)]
        for b in range(B):
            pre, mine = self.keys(b)
            idx = torch.cat([pre, mine]).to(DEV)
            new = Tq if self.q_lens is None else max(0, min(Tq, int(self.q_lens[b])))
            if not new or not len(idx):
                continue
            k, v = self.k[idx].double(), self.v[idx].double()
            u = torch.arange(len(idx), device=DEV) - len(pre)
            see = u < (self.own[b] - new + 1 + torch.arange(new, device=DEV))[:, None]
            see = see | (u < 0)
            for s, a, e in gone:
                if s == b:
                    see &= ~((u >= a) & (u < e))
            q = self.q[b, :new].double().reshape(new, Hkv, G, dh)
            x = torch.einsum("thgd,khd->thgk", q, k) * scale
            live = see[:, None, None, :]
            p = torch.softmax(x.masked_fill(~live, -math.inf), 3).masked_fill(~live.any(3, keepdim=True), 0.0)
            mag = (torch.einsum("thgd,khd->thgk", q.abs(), k.abs()) * abs(scale)).masked_fill(~live, 0).amax(3)
            out[0][b, :new] = torch.einsum("thgk,khd->thgd", p, v).reshape(new, H, dh)
            out[1][b, :new] = torch.einsum("thgk,khd->thgd", p, v.abs()).reshape(new, H, dh)
            out[2][b, :new] = mag.reshape(new, H, 1)
            out[3][b, :new] = live.sum(3).expand(-1, Hkv, G).reshape(new, H, 1).double()
        return out

    def call(self, scale=None, **kw):
        a = dict(q=self.q, k_pages=self.kp, v_pages=self.vp, page_table=self.table, kv_lens=self.kv_lens, q_lens=self.q_lens,
                 prefix_table=self.prefix_table, prefix_lens=self.prefix_lens, scale=scale)
        return api.paged_attention(**(a | kw))


def paged_tol(h, o, w, mag, n, dh):
    dt = h.dt
    u = 2.0 ** -53 if dt == F64 else U
    es = 2 * u * (dh + 4) * mag
    tol = (2 * es + 2 * u * (n + 8) + (0 if dt == F64 else 2.0 ** -19)) * w + HALF[dt] * o.abs() * 1.01
    return tol + 2.0 ** -8 * w if dt == BF else tol


def check_paged(h, scale=None, gone=(), **kw):
    dh = h.q.shape[3]
    o, w, mag, n = h.ref(dh ** -0.5 if scale is None else scale, gone)
    got = h.call(scale, **kw)
    close(got, o, paged_tol(h, o, w, mag, n, dh))
    return got


# Tq, H, Hkv, dh, page, own, prefix
PAGED_SHAPES = [
    (1, 1, 1, 64, 16, [1], []), (1, 3, 3, 64, 16, [5, 17], []), (1, 4, 2, 64, 32, [127, 1, 300], []),
    (1, 16, 16, 64, 16, [128, 577, 3, 290], []), (1, 16, 2, 128, 64, [1000, 63], []), (1, 2, 1, 96, 128, [4000], []),
    (3, 6, 3, 64, 16, [63, 3, 100], []), (2, 8, 4, 72, 16, [200, 2], []), (4, 12, 3, 80, 64, [300, 64], []),
    (17, 4, 1, 64, 16, [17, 90], []), (33, 3, 3, 64, 32, [577, 33], []), (100, 15, 5, 96, 16, [100, 140], []),
    (128, 4, 4, 128, 64, [128, 500], []), (129, 8, 2, 64, 128, [385, 129], []), (300, 4, 4, 80, 16, [300], []),
    (260, 2, 1, 128, 256, [1025, 260], []), (513, 6, 2, 96, 32, [700], []), (150, 6, 2, 64, 48, [3000], []),
    (1, 4, 4, 64, 16, [1, 9, 30, 17], [100]), (1, 16, 2, 128, 64, [70, 1, 33, 5, 129, 64], [257, 1000]),
    (1, 16, 16, 64, 16, [20] * 32, [1025]), (3, 16, 2, 128, 64, [30, 3, 577, 70], [700, 200]),
    (2, 12, 4, 80, 32, [5, 2, 60], [33, 1, 500]), (5, 8, 2, 64, 16, [5] * 16, [2000]), (40, 3, 3, 64, 16, [40, 77, 41], [130]),
    (16, 4, 2, 96, 16, [16] * 9, [385]), (150, 4, 4, 80, 32, [150, 200], [600]), (260, 6, 2, 128, 64, [260, 300], [1000, 64]),
    (1, 6, 2, 64, 16, [0, 4, 0], [50]), (3, 5, 5, 64, 16, [3, 3], [1]),
    # what the fast forms do not take: pages, widths
    (1, 4, 2, 64, 1, [5, 30], [7]), (2, 4, 2, 64, 20, [45, 2], [30]), (9, 4, 4, 40, 16, [40, 9], [20]), (3, 2, 1, 33, 8, [50], []),
    (2, 4, 1, 160, 16, [40, 2], [50]), (2, 2, 2, 300, 16, [40, 2], []), (20, 2, 1, 512, 16, [70], [33]),
]


@pytest.mark.parametrize("dt", [BF, F32, F64], ids=str)
@pytest.mark.parametrize("shape", PAGED_SHAPES, ids=str)
def test_paged_attention(shape, dt):
    Tq, H, Hkv, dh, page, own, prefix = shape
    h = Held(Tq, H, Hkv, dh, page, own, prefix, dt=dt)
    got = check_paged(h)
    assert same(h.call(), got)


@pytest.mark.parametrize("prefix", [[], [90], [90, 5], [600], [1300, 64]])
@pytest.mark.parametrize("Tq,H,Hkv,dh", [(3, 4, 2, 64), (4, 16, 4, 128), (40, 4, 4, 64), (70, 6, 2, 80), (300, 2, 1, 64)])
def test_paged_attention_of_ragged_queries(Tq, H, Hkv, dh, prefix):
    """Lengths of zero and one, more new tokens than keys, lengths outside their range; rows behind are zeros."""
    own = [Tq, 1, 0, 400, Tq + 1, 2, 77, 130]
    lens = [Tq, 1, 0, Tq // 2, 1, min(Tq, 3), Tq // 3, 0]
    for dt in (BF, F32):
        h = Held(Tq, H, Hkv, dh, 16, own, prefix, dt=dt, q_lens=lens)
        got = check_paged(h)
        for b, n in enumerate(lens):
            assert (got[b, n:] == 0).all()
        more = ints([n + 9 if n == Tq else n or -4 for n in lens])
        assert same(h.call(q_lens=more), got)
        many = h.kv_lens.clone()
        many[2] = -7
        assert same(h.call(kv_lens=many), got)


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("Tq,H,Hkv,dh,page", [(1, 4, 2, 64, 16), (2, 8, 2, 128, 64), (40, 4, 4, 64, 16), (200, 4, 2, 80, 32), (3, 2, 2, 64, 12)])
def test_paged_attention_lengths_past_the_table(Tq, H, Hkv, dh, page, dt):
    own = [page * 9, page * 9]
    h = Held(Tq, H, Hkv, dh, page, own, [page * 5], dt=dt)
    h.table, h.prefix_table = h.table[:, :9].contiguous(), h.prefix_table[:, :5].contiguous()
    got = check_paged(h)
    assert same(h.call(kv_lens=ints([1 << 30, (1 << 31) - 1]), prefix_lens=ints([page * 5 + 1])), got)


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("Tq,H,Hkv,dh,page", [(1, 4, 2, 64, 16), (2, 8, 2, 128, 64), (4, 16, 4, 96, 32), (40, 4, 4, 64, 16),
                                              (200, 4, 2, 80, 32), (130, 2, 2, 128, 128), (300, 2, 2, 64, 16), (3, 2, 2, 64, 12)])
def test_paged_attention_does_not_see_absent_pages(Tq, H, Hkv, dh, page, dt):
    """Pages dropped from the front, the middle and the whole of a sequence, and all of a prefix."""
    own = [800, 500, 300]
    for prefix in ([], [400]):
        h = Held(Tq, H, Hkv, dh, page, own, prefix, dt=dt)
        P = h.kp.shape[0]
        last = 300 // page   # pages of the last sequence, all of them
        h.table[0, 0], h.table[0, 3], h.table[0, 4] = -1, P, -(1 << 31)
        h.table[1, 500 // page - 1] = (1 << 31) - 1
        h.table[2, :last + 1] = -1
        gone = [(0, 0, page), (0, 3 * page, 5 * page), (1, (500 // page - 1) * page, 500 // page * page), (2, 0, 300)]
        check_paged(h, gone=gone)
        if prefix:
            h.prefix_table[:] = -1
            h.prefix = []
            o, w, mag, n = h.ref(dh ** -0.5, gone)
            got = h.call()
            close(got, o, paged_tol(h, o, w, mag, n, dh))
            assert (got[2] == 0).all()


@pytest.mark.parametrize("dt", [BF, F32, F64], ids=str)
@pytest.mark.parametrize("Tq,H,Hkv,dh,page", [(1, 4, 2, 64, 16), (3, 8, 2, 128, 64), (40, 4, 4, 64, 16), (200, 4, 2, 80, 32)])
def test_paged_attention_layouts(Tq, H, Hkv, dh, page, dt):
    """Queries in a fused projection, tokens or heads first; pools side by side in a page, heads before tokens, unaligned."""
    B = 4
    h = Held(Tq, H, Hkv, dh, page, [Tq + 70 * b for b in range(B)], [300, 33], dt=dt)
    check_paged(h)
    P = h.kp.shape[0]
    wide = torch.full((B, Tq, H + 3, dh), math.nan, dtype=dt, device=DEV)
    wide[:, :, 1:1 + H] = h.q
    early = torch.empty(Tq, B, H, dh, dtype=dt, device=DEV).transpose(0, 1).copy_(h.q)
    heads = torch.empty(B, H, Tq, dh, dtype=dt, device=DEV).transpose(1, 2).copy_(h.q)
    off = torch.empty(h.q.numel() + 1, dtype=dt, device=DEV)[1:].view(h.q.shape).copy_(h.q)
    # other layouts may take another kernel, whose weights are rounded elsewhere: each is held to the reference
    o, w, mag, n = h.ref(dh ** -0.5)
    tol = paged_tol(h, o, w, mag, n, dh)
    for q in (wide[:, :, 1:1 + H], early, heads, off):
        close(h.call(q=q), o, tol)
    side = torch.empty(P, 2, page, Hkv, dh, dtype=dt, device=DEV)
    inner = torch.empty(2, P, Hkv, page, dh, dtype=dt, device=DEV).transpose(2, 3)
    odd = torch.empty(2, P, page, Hkv, dh + 1, dtype=dt, device=DEV)[..., :dh]
    for kp, vp in ((side[:, 0], side[:, 1]), (inner[0], inner[1]), (odd[0], odd[1])):
        kp.copy_(h.kp)
        vp.copy_(h.vp)
        close(h.call(k_pages=kp, v_pages=vp), o, tol)
    out = torch.full((h.q.numel() + 1,), math.nan, dtype=dt, device=DEV)[1:].view(h.q.shape)
    assert h.call(out=out) is out
    close(out, o, tol)


SPECIAL = [(1, 4, 2, 64, [300, 70], []), (3, 8, 2, 128, [400, 9], [500]), (1, 16, 16, 64, [30] * 20, [700]), (40, 4, 4, 64, [300, 70], [200]),
           (200, 4, 2, 80, [400, 250], []), (200, 2, 2, 128, [250, 200], [400])]


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("Tq,H,Hkv,dh,own,prefix", SPECIAL)
def test_paged_attention_special_scores(Tq, H, Hkv, dh, own, prefix, dt):
    h = Held(Tq, H, Hkv, dh, 16, own, prefix, dt=dt)
    check_paged(h, scale=0.0)
    check_paged(h, scale=-0.3)
    check_paged(h, scale=3.0)
    # one key's scores of minus infinity carry no weight
    pg, s = slots(h.table, 0, 2, 16)
    h.q = h.q.abs() + 0.01
    keep = h.kp.clone()
    h.kp[pg, s] = -math.inf
    o, w, mag, n = h.ref(dh ** -0.5, [(0, 2, 3)])
    close(h.call(), o, (2.0 ** -7 if dt == BF else 2.0 ** -16) * w)
    # nothing else: zeros
    if not prefix:
        h.kp.copy_(torch.where(torch.isnan(keep), keep, -math.inf))
        assert (h.call() == 0).all()
    # a key that is not a number spoils the rows of its sequence and head that see it, no others
    h.kp.copy_(keep)
    ref = h.call()
    h.kp[pg, s, 0] = math.nan
    got = h.call()
    G = H // Hkv
    sees = torch.arange(Tq, device=DEV) + own[0] - Tq >= 2
    assert torch.isnan(got[0, sees, :G]).all() and same(got[1:], ref[1:]) and same(got[0, :, G:], ref[0, :, G:])
    assert same(got[0, ~sees], ref[0, ~sees])


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("Tq,H,Hkv,dh,own,prefix", [(4, 4, 2, 64, [90, 4], []), (3, 8, 2, 128, [400, 9], [500]), (40, 4, 4, 64, [300, 40], [200]),
                                                    (200, 4, 2, 80, [400, 250], []), (200, 2, 2, 128, [250, 200], [400])])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_paged_attention_later_tokens_do_not_reach_earlier_ones(Tq, H, Hkv, dh, own, prefix, dt, value):
    """The key and value of a sequence's newest token are seen by its last query alone, whatever they hold. (Rows on
    tensor cores that meet such a value are made again with weights that are not rounded: held to the reference, not to the bits.)"""
    h = Held(Tq, H, Hkv, dh, 16, own, prefix, dt=dt)
    o, w, mag, n = h.ref(dh ** -0.5)
    tol = paged_tol(h, o, w, mag, n, dh)
    for b, n in enumerate(own):
        pg, s = slots(h.table, b, n - 1, 16)
        h.vp[pg, s] = value
    got = h.call()
    close(got[:, :-1], o[:, :-1], tol[:, :-1])
    assert not torch.isfinite(got[:, -1]).any()
    for b, n in enumerate(own):
        pg, s = slots(h.table, b, n - 1, 16)
        h.kp[pg, s] = value
    got = h.call()
    close(got[:, :-1], o[:, :-1], tol[:, :-1])
    assert not torch.isfinite(got[:, -1]).any()


@pytest.mark.parametrize("scale", [1e9, 7e17, 1e30])
@pytest.mark.parametrize("dt", [BF, F32, F64], ids=str)
@pytest.mark.parametrize("Tq,H,Hkv,dh,own,prefix", SPECIAL)
def test_paged_attention_of_large_scores(Tq, H, Hkv, dh, own, prefix, dt, scale):
    """Queries and keys of small whole numbers have exact scores, and differences of 1 leave no weight: the mean of the
    values under the largest score, the weights all exactly 1."""
    h = Held(Tq, H, Hkv, dh, 16, own, prefix, dt=dt)
    whole = [t.float().round().clamp(-2, 2).to(dt) for t in (h.q, h.kp, h.k)]
    h.q, h.kp, h.k = whole
    for sc in (scale, -scale):
        o, w, _, n = h.ref(sc)
        tol = (2 * U * (n + 8) + (2.0 ** -20 if dt == F32 else 0)) * w + HALF[dt] * o.abs() * 1.01
        close(h.call(sc), o, tol)


def inside(shape, dt, lead, fn):
    """fn(out) with out a contiguous tensor between two margins; nothing outside it changes."""
    n = math.prod(shape) * torch.empty(0, dtype=dt).element_size()
    buf = torch.full((lead + n + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    fn(buf[lead:lead + n].view(dt).view(shape))
    assert (buf[:lead] == 0x5A).all() and (buf[lead + n:] == 0x5A).all()


@pytest.mark.parametrize("lead", [4096, 4104])
def test_nothing_outside_the_outputs_is_written(lead):
    for dt in (BF, F32):
        x, f = rand(3, 7, 5, 80, dtype=dt), api.rotary_frequencies(64, device=DEV)
        inside(tuple(x.shape), dt, lead, lambda t: api.rotary(x, f, out=t))
        for Tq, H, Hkv, dh, own, prefix in SPECIAL + [(131, 6, 2, 64, [140, 131], []), (37, 5, 1, 128, [37, 90], [64]), (7, 3, 3, 40, [9], [])]:
            h = Held(Tq, H, Hkv, dh, 16, own, prefix, dt=dt)
            inside(tuple(h.q.shape), dt, lead, lambda t: h.call(out=t))


@pytest.mark.parametrize("dt,Tq,dh", [(BF, 1, 64), (BF, 150, 128), (F32, 1, 64), (BF, 4, 64), (BF, 20, 72)], ids=str)
def test_pools_past_32_bit_offsets(dt, Tq, dh):
    """Pages, or tokens, that lie more than 2^32 elements apart: appended to, and read."""
    Hkv, page = 2, 16
    for strides in (((1 << 32) + 64, Hkv * dh, dh), (Hkv * dh, 1 << 29, dh)):
        span = 2 * strides[0] + 15 * strides[1] + Hkv * dh
        buf = torch.empty(span, dtype=dt, device=DEV)
        far = buf.as_strided((3, page, Hkv, dh), strides + (1,))
        far.fill_(math.nan)
        h = Held(Tq, 4, Hkv, dh, page, [40], dt=dt) if Tq < 40 else Held(Tq, 4, Hkv, dh, page, [160], dt=dt)
        P = h.kp.shape[0]
        near = [pool(3, page, Hkv, dh, dt)[0] for _ in range(2)]
        k, v = rand(1, 40, Hkv, dh, seed=1, dtype=dt), rand(1, 40, Hkv, dh, seed=2, dtype=dt)
        f, table = api.rotary_frequencies(dh, device=DEV), ints([[2, 0, 1]])
        q = rand(1, min(Tq, 40), 4, dh, seed=3, dtype=dt)
        for i in range(2):   # the far pool as keys, as values
            far.fill_(math.nan)
            other = near[1].clone()
            a = (far, other) if i == 0 else (other, far)
            b = (near[0].clone(), near[1].clone())
            for pools in (a, b):
                api.cache_append(k, v, *pools, table, ints([0]), frequencies=f)
            assert same(a[0], b[0]) and same(a[1], b[1])
            got = [api.paged_attention(q, *pools, table, ints([40])) for pools in (a, b)]
            assert same(*got) and torch.isfinite(got[0]).all()
        del buf, far


def test_outputs_past_32_bit_offsets():
    T, n = 1 << 20, 4096
    x = torch.empty(1, T + 600, 16, 256, dtype=BF, device=DEV).normal_()
    f = api.rotary_frequencies(256, device=DEV)
    pos = torch.arange(T + 600, dtype=torch.int32, device=DEV)[None]
    got = api.rotary(x, f)
    assert same(got[:, -n:], api.rotary(x[:, -n:], f, positions=pos[:, -n:].contiguous()))
    del got
    x = x.view(1, -1, 32, 128)[:, :T + 600]
    # rows that see 600 keys at most; the last ones alone, with the same keys, see the same
    h = Held(1, 32, 2, 128, 64, [600])
    got = h.call(q=x)
    assert same(got[:, -600:], h.call(q=x[:, -600:])) and (got[:, :-600] == 0).all()


@pytest.mark.parametrize("B", [37, 200])
def test_paged_attention_of_many_ragged_sequences(B):
    """More work than one round of CTAs, sequences in any order of length, empty ones among them."""
    g = torch.Generator().manual_seed(B)
    own = torch.randint(0, 400, (B,), generator=g).tolist()
    for Tq, prefix in ((1, []), (140, []), (140, [200]), (20, [300]), (2, [300])):
        lens = [min(n, Tq, 1 + i % Tq) for i, n in enumerate(own)]
        check_paged(Held(Tq, 6, 3, 64, 16, own, prefix, q_lens=lens))


@pytest.mark.parametrize("dh", [40, 64, 96, 128])
@pytest.mark.parametrize("Tq,H,Hkv", [(1, 12, 12), (1, 16, 8), (4, 24, 8), (8, 16, 8)])
@pytest.mark.parametrize("most,prefix", [(1, []), (33, [70]), (64, []), (64, [300]), (65, [40]), (96, []), (97, []), (330, [])])
def test_paged_attention_of_few_queries_and_many_heads(Tq, H, Hkv, dh, most, prefix):
    """More key heads than half the SMs: short sequences, whose warps have a tile at most, some empty; absent values and
    later tokens that are no numbers; any number of CTAs to a head."""
    own = [Tq + (most - 1) * i // 12 for i in range(13)]
    h = Held(Tq, H, Hkv, dh, 16, own, prefix, q_lens=[min(Tq, n) if i != 3 else 0 for i, n in enumerate(own)])
    check_paged(h)
    o, w, mag, n = h.ref(dh ** -0.5)
    pg, s = slots(h.table, 12, own[12] - 1, 16)
    h.vp[pg, s] = math.nan
    got = h.call()
    assert torch.isnan(got[12, Tq - 1]).all()
    got[12, Tq - 1] = o[12, Tq - 1].to(got.dtype)
    close(got, o, paged_tol(h, o, w, mag, n, dh))


@pytest.mark.parametrize("dh", [64, 80, 128])
@pytest.mark.parametrize("B", [1, 7, 9, 12, 14, 17, 36])
def test_paged_attention_of_few_queries_in_any_cluster(B, dh):
    """One to eight CTAs to a key head, as many as run at once."""
    for n in (150, 190, 400, 770, 1000, 1200, 1500, 3000):
        check_paged(Held(1 + n % 2, 8, 2, dh, 32, [n - n * b // (3 * B) for b in range(B)]))


@pytest.mark.parametrize("Tq,H,Hkv,dh", [(1, 4, 2, 64), (2, 16, 2, 128), (100, 4, 2, 64), (260, 2, 2, 96)])
def test_paged_attention_where_keys_are_dealt_out(Tq, H, Hkv, dh):
    """Few rows over many keys: parts go to different CTAs, some of them, or all but one key, without any."""
    for own, prefix in (([5000], []), ([Tq, 4000], []), ([Tq, Tq, Tq], [6000]), ([300, Tq, 2000], [1, 129, 3000])):
        h = Held(Tq, H, Hkv, dh, 64, own, prefix)
        got = check_paged(h)
        for _ in range(3):
            assert same(h.call(), got)


@pytest.mark.parametrize("Tq,H,Hkv,dh,own,prefix", SPECIAL + [(40, 4, 4, 96, [300] * 3, [500])])
def test_paged_attention_of_broadcast_queries(Tq, H, Hkv, dh, own, prefix):
    """One set of queries for all sequences, one token's for all tokens, one head's for all heads (strides of zero)."""
    h = Held(Tq, H, Hkv, dh, 16, own, prefix)
    q = h.q
    for wide in (q[:1].expand(q.shape), q[:, :1].expand(q.shape), q[:, :, :1].expand(q.shape)):
        h.q = wide.contiguous()
        o, w, mag, n = h.ref(dh ** -0.5)
        close(h.call(q=wide), o, paged_tol(h, o, w, mag, n, dh))


@pytest.mark.parametrize("Tq,H,Hkv,dh,own,prefix", SPECIAL + [(300, 4, 4, 64, [1500, 600], []), (130, 4, 2, 96, [800, 500], [700])])
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
def test_paged_attention_of_values_that_are_no_numbers(Tq, H, Hkv, dh, own, prefix, dt):
    """All values NaN, or one early one infinite: rows that see them are not finite, and the call ends in its time."""
    h = Held(Tq, H, Hkv, dh, 16, own, prefix, dt=dt)
    keep = h.vp.clone()
    h.vp[:] = math.nan
    assert torch.isnan(h.call()).all()
    h.vp.copy_(keep)
    ref = h.call()
    pg, s = slots(h.table, 0, 0, 16)
    h.vp[pg, s, 0] = math.inf
    got, G = h.call(), H // Hkv
    assert not torch.isfinite(got[0, :, :G]).any() and same(got[1:], ref[1:]) and same(got[0, :, G:], ref[0, :, G:])


@pytest.mark.parametrize("Tq,H,Hkv,dh,own,prefix", [(40, 4, 4, 64, [300, 140], [200]), (200, 4, 2, 80, [400, 250], []), (24, 4, 4, 96, [2900], []),
                                                    (200, 6, 2, 128, [250, 3000], [400]), (3, 8, 2, 128, [400, 90], [])])
def test_paged_attention_later_tokens_behind_absent_pages(Tq, H, Hkv, dh, own, prefix):
    """Rows that are made again see what they see: not the pages that are absent, the prefix, parts of the keys."""
    h = Held(Tq, H, Hkv, dh, 16, own, prefix)
    pg, s = slots(h.table, 0, own[0] - 1, 16)
    h.vp[pg, s, :, 1::2] = math.nan
    gone = []
    for b, page in ((0, 1), (len(own) - 1, 4)):
        h.table[b, page] = -7 if b else 1 << 20
        gone.append((b, 16 * page, 16 * page + 16))
    o, w, mag, n = h.ref(dh ** -0.5, gone)
    tol = paged_tol(h, o, w, mag, n, dh)
    got = h.call()
    last = torch.isnan(got[0, -1])
    assert last[:, 1::2].all() and not last[:, 0::2].any()
    got[0, -1] = o[0, -1].to(got.dtype)
    close(got, o, tol)
    assert same(h.call()[:, :-1], got[:, :-1])


@pytest.mark.parametrize("n", [(1 << 17) + 1, (1 << 17) + (1 << 16) + 5])
def test_paged_attention_of_keys_past_one_part(n):
    """Enough sequences to fill the GPU, each longer than one part may be. Scores of zero and whole values: exact sums, one
    division, one rounding. The pages are the same few in turn."""
    B, Tq, page, P = 80, 20, 64, 8
    kp, vp = rand(P, page, 1, 64, dtype=BF), rand(P, page, 1, 64, seed=1).round().to(BF)
    table = (torch.arange((n + page - 1) // page) % P).int().to(DEV).repeat(B, 1)
    got = api.paged_attention(torch.zeros(B, Tq, 1, 64, dtype=BF, device=DEV), kp, vp, table, ints([n] * B))
    at = torch.cat([torch.zeros(1, 64, dtype=F64, device=DEV), vp.double().reshape(P * page, 64).cumsum(0)])
    sees = torch.arange(n - Tq + 1, n + 1, device=DEV)
    o = (at[-1] * (sees // (P * page))[:, None] + at[sees % (P * page)]) / sees[:, None]
    close(got[:, :, 0], o.expand(B, Tq, 64), (HALF[BF] * 1.01 + 4 * U) * o.abs().expand(B, Tq, 64))


@pytest.mark.parametrize("scale", [1.0, 1e5, 1e8, -1e7])
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("Tq,H,Hkv,dh,own,prefix", SPECIAL + [(40, 4, 2, 128, [900, 41], []), (300, 2, 1, 64, [1100], [300])])
def test_paged_attention_weights_sum_to_one_behind_later_tokens(Tq, H, Hkv, dh, own, prefix, dt, scale):
    """Values of 1 come out as 1, however far the scores are from zero (where the rounding of a score is a factor in its weight),
    also where the newest token's value is not a number: a weight is off by its rounding to bf16, the sums by that of
    each of their terms and of a rescale, the result by its own rounding."""
    h = Held(Tq, H, Hkv, dh, 16, own, prefix, dt=dt)
    h.vp.copy_(torch.where(torch.isnan(h.vp), h.vp, 1.0))
    for b, n in enumerate(own):
        pg, s = slots(h.table, b, n - 1, 16)
        h.vp[pg, s] = math.nan
    got, one = h.call(scale=scale), torch.ones((), dtype=F64, device=DEV)
    terms = 4 * U * (max(own) + (max(prefix) if prefix else 0) + 64)
    close(got[:, :-1], one.expand_as(got[:, :-1]), one * (terms + HALF[dt] * (2 if dt == BF else 1)) * 1.01)
    assert torch.isnan(got[:, -1]).all()


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dt", [BF, F32, F64], ids=str)
@pytest.mark.parametrize("Tq,H,Hkv,dh,own,prefix", SPECIAL + [(1, 1, 1, 64, [300], []), (2, 2, 2, 128, [90], [70]), (5, 3, 1, 72, [90], []), (20, 2, 1, 40, [90], [70])])
def test_paged_attention_of_seen_keys_without_weight(Tq, H, Hkv, dh, own, prefix, dt, value):
    """A key that a row sees, so far below the others that its weight is zero: its value still counts as 0 times it."""
    h = Held(Tq, H, Hkv, dh, 16, own, prefix, dt=dt)
    h.q = h.q.abs() + 0.5
    pg, s = slots(h.table, 0, 0, 16)
    h.kp[pg, s], h.vp[pg, s] = -1e4, value
    got = h.call()
    assert torch.isnan(got[0]).all() and torch.isfinite(got[1:]).all()
    if prefix:   # of the prefix: all sequences of the group
        h = Held(Tq, H, Hkv, dh, 16, own, prefix, dt=dt)
        h.q = h.q.abs() + 0.5
        pg, s = slots(h.prefix_table, 0, 0, 16)
        h.kp[pg, s], h.vp[pg, s] = -1e4, value
        assert torch.isnan(h.call()).all()


@pytest.mark.parametrize("page", [8, 16, 48, 80, 96, 112, 144, 160, 384])
@pytest.mark.parametrize("Tq,H,Hkv,dh,dt", [(1, 4, 2, 64, BF), (3, 8, 2, 128, BF), (50, 4, 4, 80, BF), (200, 2, 2, 64, BF), (2, 4, 2, 80, F32)], ids=str)
def test_paged_attention_page_sizes(Tq, H, Hkv, dh, dt, page):
    """Pages that tiles straddle, and that end inside a tile."""
    h = Held(Tq, H, Hkv, dh, page, [Tq, 3 * page + Tq, 500 + Tq], [2 * page + 5], dt=dt)
    check_paged(h)
    check_paged(Held(Tq, H, Hkv, dh, page, [Tq + page - 1, 1000 + Tq], [], dt=dt))


# ------------------------------------------------------------------------------- together
def step(p, x, kp, vp, table, starts, kv_lens, f, H, Hkv, lens=None, positions=None, before=None, out=None):
    """The self attention of a decoder's layer on new tokens x (B, T, D): projection, rotation and append, attention."""
    B, T, D = x.shape
    dh = D // H
    q8, qs = api.rmsnorm(x, 1e-6, gamma=p["g"], out_dtype=torch.float8_e4m3fn)
    qkv = api.linear_fp8(q8, qs, *p["wqkv"]).view(B, T, H + 2 * Hkv, dh)
    q = api.cache_append(qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:], kp, vp, table, starts, lens=lens, q=qkv[:, :, :H],
                         frequencies=f, positions=positions)
    table_, lens_ = before if before else (None, None)
    return api.paged_attention(q, kp, vp, table, kv_lens, q_lens=lens, prefix_table=table_, prefix_lens=lens_, out=out)


def make_step(D, H, Hkv, seed=0):
    dh = D // H
    w = rand(D, (H + 2 * Hkv) * dh, seed=seed + 1, std=D ** -0.5, dtype=BF)
    return dict(g=1 + rand(D, seed=seed, std=0.1), wqkv=api.quantize_weight(w))


@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2)])
def test_tokens_one_by_one_and_in_parts_see_what_the_whole_text_sees(H, Hkv):
    """A text of 150 tokens at once, in parts of 64, token by token from the 140th, and behind a shared prefix of its
    first 100 tokens that another page table holds: the same rows, up to what rounding weights and joining parts differ by."""
    D, page, n = 64 * H, 16, 150
    p, f, x = make_step(D, H, Hkv), api.rotary_frequencies(64, device=DEV), rand(2, n, D, seed=9, dtype=BF)
    table, pages = tables([n, n], page)

    def fresh():
        return pool(pages, page, Hkv, 64, BF)

    kp, vp = fresh()
    whole = step(p, x, kp, vp, table, ints([0, 0]), ints([n, n]), f, H, Hkv)
    kp2, vp2 = fresh()
    got = []
    for a, b in [(0, 64), (64, 128), (128, 140)] + [(i, i + 1) for i in range(140, n)]:
        got.append(step(p, x[:, a:b].contiguous(), kp2, vp2, table, ints([a, a]), ints([b, b]), f, H, Hkv))
    # the same products in another kernel's order of additions can round a key to its neighbour in bf16
    tol = 2.0 ** -6 * (whole.double().abs() + 0.25)
    close(torch.cat(got, 1), whole.double(), tol)
    # one text as a prefix for three continuations
    kp3, vp3 = fresh()
    t1 = table[:1].contiguous()
    step(p, x[:1, :100].contiguous(), kp3, vp3, t1, ints([0]), ints([100]), f, H, Hkv)
    own, more = tables([50] * 3, page, seed=4)
    kp3, vp3 = (torch.cat([t, torch.full((more,) + t.shape[1:], math.nan, dtype=BF, device=DEV)]) for t in (kp3, vp3))
    own = torch.where(own < more, own + pages, own)
    tail = x[:1, 100:].expand(3, -1, -1).contiguous()
    pos = torch.arange(100, n, dtype=torch.int32, device=DEV).expand(3, -1).contiguous()
    got = step(p, tail, kp3, vp3, own, ints([0] * 3), ints([50] * 3), f, H, Hkv, positions=pos, before=(t1, ints([100])))
    close(got, whole[:1, 100:].double().expand(3, -1, -1, -1), tol[:1, 100:])
    assert same(got[0], got[1]) and same(got[0], got[2])


@pytest.mark.parametrize("T", [1, 3, 40])
def test_a_captured_step_replays_on_new_inputs_and_streams_agree(T):
    """Two graphs of a step behind a shared prefix, each with a cache of its own, replayed at once."""
    B, H, Hkv, D, page = 6, 8, 2, 512, 16
    p, f = make_step(D, H, Hkv), api.rotary_frequencies(64, device=DEV)
    h = Held(T, H, Hkv, 64, page, [40, T, 47, 90, T + 1, 64], [300, 700])
    x = rand(B, T, D, seed=30, dtype=BF)
    starts, lens = h.kv_lens - T, h.kv_lens.clone()
    pos = (starts[:, None] + 700 + torch.arange(T, device=DEV)).int().contiguous()
    args = lambda kp, vp: (p, x, kp, vp, h.table, starts, lens, f, H, Hkv, None, pos, (h.prefix_table, h.prefix_lens))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*args(h.kp.clone(), h.vp.clone()))
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        kp, vp = h.kp.clone(), h.vp.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = step(*args(kp, vp))
        graphs.append((g, y, kp, vp))
    for seed in (40, 41):
        x.copy_(rand(B, T, D, seed=seed, dtype=BF))
        kp, vp = graphs[0][2].clone(), graphs[0][3].clone()
        eager = step(*args(kp, vp))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for _ in range(3):
            for (g, *_), st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for _, y, a, b in graphs:
            assert same(y, eager) and same(a, kp) and same(b, vp)


def test_calls_on_explicit_streams_and_at_once():
    """Calls that need scratch memory, on three streams in turn without waiting."""
    hs = [Held(t, 16, 2, 128, 64, [70 + t] * 4, [900], seed=t) for t in (1, 2, 30)]
    ref = [h.call() for h in hs]
    x, f = rand(3, 5, 4, 64, dtype=BF), api.rotary_frequencies(64, device=DEV)
    r = api.rotary(x, f)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in hs]
    for _ in range(5):
        got = [h.call(stream=s) for h, s in zip(hs, streams)]
        z = api.rotary(x, f, stream=streams[0].cuda_stream)
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, ref)) and same(z, r)
    kp, vp = hs[0].kp.clone(), hs[0].vp.clone()
    k = rand(4, 1, 2, 128, dtype=BF)
    api.cache_append(k, k, kp, vp, hs[0].table, ints([3] * 4), stream=streams[1])
    streams[1].synchronize()
    api.cache_append(k, k, hs[0].kp, hs[0].vp, hs[0].table, ints([3] * 4))
    assert same(kp, hs[0].kp) and same(vp, hs[0].vp)


def test_the_binding_refuses_what_does_not_fit():
    h = Held(2, 4, 2, 64, 16, [5, 7], [20])
    x, f = h.q, api.rotary_frequencies(64, device=DEV)
    k = rand(2, 3, 2, 64, dtype=BF)
    s, P = ints([0, 0]), h.kp
    append = lambda **kw: api.cache_append(**(dict(k=k, v=k, k_pages=P, v_pages=h.vp, page_table=h.table, starts=s) | kw))
    bad = [
        lambda: api.rotary(x[0], f), lambda: api.rotary(x.half(), f), lambda: api.rotary(x, f.float()), lambda: api.rotary(x, f.cpu()),
        lambda: api.rotary(x, f, positions=s), lambda: api.rotary(x, f, layout=2), lambda: api.rotary(x, f[:0]), lambda: api.rotary(x, None),
        lambda: api.rotary(x.transpose(2, 3), f), lambda: api.rotary(x[:0], f), lambda: api.rotary(x, f, out=x[:, :, :2]),
        lambda: api.rotary(x, f, positions=s[:, None].expand(2, 2)), lambda: api.rotary(x, f[None]),
        lambda: append(k=k.float()), lambda: append(v=k[:, :2]), lambda: append(k=k[..., :32]), lambda: append(page_table=h.table[:1]),
        lambda: append(starts=None), lambda: append(starts=s.long()), lambda: append(lens=s[:1]), lambda: append(q_out=x),
        lambda: append(q=x), lambda: append(v_pages=P[:1]), lambda: append(page_table=h.table.t()), lambda: append(frequencies=f.float()),
        lambda: append(positions=s), lambda: append(k_pages=P[0]),
        lambda: h.call(q=x.float()), lambda: h.call(q=x[..., :32]), lambda: h.call(kv_lens=None), lambda: h.call(kv_lens=s.long()),
        lambda: h.call(prefix_lens=None), lambda: h.call(prefix_table=None), lambda: h.call(prefix_table=h.table.repeat(2, 1)[:3], prefix_lens=ints([1] * 3)),
        lambda: h.call(q_lens=s[:1]), lambda: h.call(page_table=h.table[0]), lambda: h.call(out=x.float()), lambda: h.call(v_pages=h.vp.float()),
        lambda: h.call(q=x.cpu()), lambda: h.call(page_table=h.table[:, ::2]),
    ]
    for i, fn in enumerate(bad):
        with pytest.raises(ValueError):
            fn()
            raise AssertionError("call %d was taken" % i)
    for fn in (lambda: api.rotary(x, api.rotary_frequencies(128, device=DEV)),          # wider than the heads
               lambda: api.rotary(x[:, :, :1].expand(-1, -1, 4, -1), f, out=x[:, :, :1].expand(-1, -1, 4, -1)),   # rows upon each other
               lambda: api.rotary(x, f, scale=math.nan), lambda: append(v_pages=P),     # one pool for both
               lambda: append(k=P[:1, :3].expand(2, -1, -1, -1)),                       # out of the pool
               lambda: append(k_pages=P[:1].expand(P.shape)), lambda: h.call(scale=math.inf), lambda: h.call(out=x),
               lambda: h.call(q=rand(2, 2, 3, 64, dtype=BF))):                          # 3 heads on 2
        with pytest.raises(api.VitError):
            fn()


@pytest.mark.parametrize("dt", [BF, F32, F64], ids=str)
def test_an_output_at_the_inputs_address_is_the_input_or_is_refused(dt):
    """Rows of a wider buffer, and an output that starts where they do but steps otherwise: refused, and nothing is written.
    Dimensions of one have no stride to compare."""
    B, T, H, dh, page = 2, 5, 4, 64, 16
    buf, f = rand(B, T, H + 2, dh, seed=1, dtype=dt), api.rotary_frequencies(48, device=DEV)
    k = rand(B, T, 2, dh, seed=2, dtype=dt)
    table, pages = tables([T] * B, page)
    pools = pool(pages, page, 2, dh, dt, fill=0.0)
    keep = buf.clone()
    x, packed = buf[:, :, :H], buf.view(-1)[:B * T * H * dh].view(B, T, H, dh)
    for a, b in ((x, packed), (packed, x), (x, buf.as_strided(x.shape, (T * H * dh, dh, T * dh, 1)))):
        with pytest.raises(ValueError):
            api.rotary(a, f, out=b)
        with pytest.raises(ValueError):
            api.cache_append(k, k, *pools, table, ints([0] * B), q=a, frequencies=f, q_out=b)
        assert same(buf, keep) and all((p == 0).all() for p in pools)
    # one sequence of one token: whatever those strides say, it is x
    for shape, at in (((1, 1, H, dh), (3, 7, dh, 1)), ((1, T, H, dh), (1, (H + 2) * dh, dh, 1)), ((B, 1, 1, dh), (T * (H + 2) * dh, 5, 11, 1))):
        buf.copy_(keep)
        x = buf[:shape[0], :shape[1], :shape[2]]
        ref = api.rotary(x, f)
        out = buf.as_strided(shape, at)
        assert api.rotary(x, f, out=out) is out and same(x, ref)
        buf.copy_(keep)
        kk = k[:shape[0], :shape[1]].contiguous()
        assert api.cache_append(kk, kk, *pools, table[:shape[0]].contiguous(), ints([0] * shape[0]), q=x, frequencies=f, q_out=out) is out and same(x, ref)


def pi_floor(bits):
    """floor(2^bits pi), by 16 atan(1/5) - 4 atan(1/239)."""
    def atan_of(n):   # 2^(bits + 32) atan(1/n), each term off by less than 1
        term = total = (1 << (bits + 32)) // n
        i = 1
        while term:
            term //= n * n
            i += 2
            total += term // i if i % 4 == 1 else -(term // i)
        return total
    return (16 * atan_of(5) - 4 * atan_of(239)) >> 32


def cos_sin_exactly(pos, f):
    """Cosines and sines (B, T, 1, n) in 64 bits of the angles positions * frequencies, reduced in whole numbers of 2^-256 turns."""
    K = 256
    pi = pi_floor(K)
    c, s = [], []
    for p in pos.reshape(-1).tolist():
        for x in f.tolist():
            num, den = float(x).as_integer_ratio()
            r = ((p * num << 2 * K) // (2 * den * pi)) % (1 << K)
            r -= (1 << K) if r >> (K - 1) else 0
            a = (2 * r * pi) / (1 << 2 * K)   # rounded once
            c.append(math.cos(a))
            s.append(math.sin(a))
    shape = tuple(pos.shape) + (1, f.numel())
    return [torch.tensor(v, dtype=F64).view(shape).to(DEV) for v in (c, s)]


@pytest.mark.parametrize("layout", LAYOUTS)
def test_rotary_in_64_bits_at_any_position(layout):
    """Angles from a reduction in whole numbers. Off by, in units of 2^-53 of |u| + |v|: the half turn in [-1, 1) by 1 (its
    conversion and one sum), so the angle by pi; sincospi by 2 last places, 2; the factor 1; a product 1 and the rounding of the
    result, counted apart. The reference: its angle's rounding 2, cos and sin 1, two products and a sum 3. 14 in all."""
    assert abs(pi_floor(60) / (1 << 60) - math.pi) < 2.0 ** -51
    x = rand(2, 8, 3, 64, seed=2, dtype=F64)
    pos = ints([[0, 1, -1, 300, 4097, 99991, 1000000, -123456], [(1 << 31) - 1, -(1 << 31), 1 << 24, -(1 << 30) + 1, 7, 1 << 20, 2, 31]])
    for f in (api.rotary_frequencies(64, device=DEV), api.rotary_frequencies(48, 500000.0, factor=8, trained=8192, device=DEV),
              -api.rotary_frequencies(64, device=DEV),
              torch.tensor([7.0, -3.0, 6.283185307179586, 0.0, 1e3, -1e-3, 1e-9, -1e-12, 1e-25, -3e-40], dtype=F64, device=DEV)):
        n = f.numel()
        c, s = cos_sin_exactly(pos, f)
        i = torch.arange(n, device=DEV)
        i, j = (i, i + n) if layout == api.ROTARY_HALF else (2 * i, 2 * i + 1)
        y, w = x.clone(), torch.zeros_like(x)
        y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
        w[..., i] = w[..., j] = x[..., i].abs() + x[..., j].abs()
        close(api.rotary(x, f, positions=pos, layout=layout), y, w * 14 * 2.0 ** -53 * 1.01 + HALF[F64] * y.abs() * 1.01)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", [BF, F32, F64], ids=str)
def test_rotary_by_a_negative_frequency_is_rotary_at_a_negative_position(dt, layout):
    """The same angle, to the bit: a frequency's sign costs nothing of its turn's bits."""
    x = rand(1, 6, 3, 64, seed=2, dtype=dt)
    pos = ints([[0, 5, 1 << 20, -(1 << 24) + 1, (1 << 31) - 1, -(1 << 30)]])
    f = torch.cat([api.rotary_frequencies(40), torch.tensor([1e-9, 3e-13, 0.7, 2.5], dtype=F64)]).to(DEV)
    assert same(api.rotary(x, -f, positions=pos, layout=layout), api.rotary(x, f, positions=-pos, layout=layout))


# --------------------------------------------------------------------- which kernel works a call off
G_, R_, T_, F_ = api.PAGED_GENERIC, api.PAGED_ROWS, api.PAGED_TC, api.PAGED_F32


def check_form(h, kernel, prefix_kernel=-1, scale=None, **kw):
    """The call has this kernel, launches what its plan says, and is right."""
    a = dict(q=h.q, k_pages=h.kp, v_pages=h.vp, page_table=h.table, kv_lens=h.kv_lens, q_lens=h.q_lens, prefix_table=h.prefix_table,
             prefix_lens=h.prefix_lens, scale=scale) | kw
    before = api.launch_count()
    p = api.paged_attention_plan(**a)
    assert api.launch_count() == before
    assert (p["kernel"], p["prefix_kernel"]) == (kernel, prefix_kernel), p
    check_paged(h, scale, **kw)
    assert api.launch_count() - before == p["launches"]
    assert (p["scratch"] > 0) == (p["launches"] > 1)
    return p


@pytest.mark.parametrize("dh", [8, 16, 24, 56, 64, 72, 80, 88, 96, 104, 120, 128, 136])
@pytest.mark.parametrize("Tq,H,Hkv", [(1, 4, 4), (16, 2, 2), (2, 16, 2), (17, 2, 2), (3, 12, 2)])
def test_which_kernel_bf16_has(Tq, H, Hkv, dh):
    """At most 16 query rows per key head and widths of a multiple of 8 up to 128: the kernel of few queries. Prefixes, and more rows,
    of widths 64, 80, 96 and 128: tensor cores. Just outside either: the generic one."""
    few, wide, tc = Tq * H // Hkv <= 16, dh > 128, dh in (64, 80, 96, 128)
    own = G_ if wide else R_ if few else T_ if tc else G_
    check_form(Held(Tq, H, Hkv, dh, 16, [Tq, 40 + Tq, 100], []), own)
    p = check_form(Held(Tq, H, Hkv, dh, 16, [Tq, 40 + Tq, 100, 30], [70, 200]), own, T_ if tc else G_)
    assert p["own_rows"] == (min(Tq * H // Hkv, 4 if Tq * H // Hkv <= 4 else 16) if own == G_ else Tq * H // Hkv)


@pytest.mark.parametrize("Tq,dh", [(1, 64), (5, 80), (40, 64), (40, 80), (40, 128)])
def test_which_kernel_bf16_has_by_pages_scales_and_layouts(Tq, dh):
    fast, H, Hkv = R_ if Tq <= 16 else T_, 2, 2
    for page, kernel in ((16, fast), (48, fast), (8, G_), (24, G_), (1, G_)):
        h = Held(Tq, H, Hkv, dh, page, [Tq, Tq + 90, 100], [50])
        check_form(h, kernel, G_ if kernel == G_ else T_)
    h = Held(Tq, H, Hkv, dh, 16, [Tq, Tq + 90], [50])
    neg = G_ if fast == T_ else R_
    check_form(h, neg, G_, scale=-0.1)
    check_form(h, neg, G_, scale=0.0)
    off = torch.empty(h.q.numel() + 1, dtype=BF, device=DEV)[1:].view(h.q.shape).copy_(h.q)
    check_form(h, G_, G_, q=off)
    odd = torch.empty(2, *h.kp.shape[:3], dh + 1, dtype=BF, device=DEV)[..., :dh]
    odd[0].copy_(h.kp)
    odd[1].copy_(h.vp)
    check_form(h, G_, G_, k_pages=odd[0], v_pages=odd[1])
    # tokens before sequences: a group's queries are no single run of rows
    early = torch.empty(Tq, 2, H, dh, dtype=BF, device=DEV).transpose(0, 1).copy_(h.q)
    p = check_form(h, fast, G_ if 1 < Tq <= 16 else T_, q=early)
    if fast == T_:
        assert p["prefix_parts"] == 0
    wide = torch.empty(2, Tq, H + 2, dh, dtype=BF, device=DEV)[:, :, :H].copy_(h.q)
    check_form(h, fast, T_, q=wide)


@pytest.mark.parametrize("dh,page,kernel", [(4, 16, F_), (60, 8, F_), (64, 16, F_), (68, 24, F_), (128, 16, F_), (132, 16, G_), (66, 16, G_), (63, 16, G_),
                                            (64, 12, G_), (64, 20, G_)])
@pytest.mark.parametrize("Tq,H,Hkv", [(1, 3, 3), (1, 4, 2), (3, 4, 2), (30, 4, 2)])
def test_which_kernel_fp32_has(Tq, H, Hkv, dh, page, kernel):
    p = check_form(Held(Tq, H, Hkv, dh, page, [Tq, 70 + Tq], [], dt=F32), kernel)
    R = Tq * H // Hkv
    assert p["own_rows"] == min(R, 4 if kernel == F_ else 16)
    check_form(Held(Tq, H, Hkv, dh, page, [Tq, 70 + Tq], [90], dt=F32), kernel, kernel)
    h = Held(Tq, H, Hkv, dh, page, [Tq, 70 + Tq], [90], dt=F64)
    check_form(h, G_, G_)
    h = Held(Tq, H, Hkv, dh, page, [Tq, 70 + Tq], [90], dt=F32)
    off = torch.empty(h.q.numel() + 1, dtype=F32, device=DEV)[1:].view(h.q.shape).copy_(h.q)
    check_form(h, G_, G_, q=off)


def test_which_work_is_cut_along_the_keys():
    """Few rows over many keys are cut into parts, by the room in the tables; many are not."""
    for Tq, dt, kernel in ((40, BF, T_), (1, F32, F_), (1, F64, G_)):
        p = check_form(Held(Tq, 2, 2, 64, 64, [4000], [], dt=dt), kernel)
        assert p["own_parts"] > 1 and p["launches"] == 2
        h = Held(Tq, 2, 2, 64, 64, [Tq + 20], [], dt=dt)
        p = check_form(h, kernel)
        assert p["own_parts"] == 1 and p["launches"] == 1 and p["scratch"] == 0
    p = check_form(Held(1, 2, 2, 64, 64, [4000], []), R_)
    assert p["launches"] == 1 and p["scratch"] == 0
    p = check_form(Held(1, 16, 16, 64, 16, [20] * 32, [1025]), R_, T_)   # rows of all sequences behind their prefix at once
    assert p["prefix_rows"] == 32 and p["prefix_parts"] > 1
    p = check_form(Held(300, 2, 2, 64, 16, [300, 310], [1000]), T_, T_)   # in front of the own keys
    assert p["prefix_parts"] == 0 and p["prefix_rows"] == 256


@pytest.mark.parametrize("dh", [60, 64, 96, 128])
@pytest.mark.parametrize("S,Tq,G,own_rows,prefix_rows", [(1, 1, 1, 1, 1), (2, 1, 1, 1, 2), (3, 1, 1, 1, 2), (8, 1, 1, 1, 2), (9, 1, 1, 1, 4), (33, 1, 1, 1, 4),
                                                         (1, 2, 1, 2, 2), (3, 1, 2, 2, 4), (1, 1, 3, 3, 3), (5, 1, 3, 3, 4), (2, 3, 2, 4, 4)])
def test_an_fp32_prefix_is_read_for_several_sequences_at_once(S, Tq, G, own_rows, prefix_rows, dh):
    """Rows of different sequences in one warp: empty ones among them, pages that are absent, and a prefix cut along its keys."""
    for prefix in ([77], [700, 33]):
        n = S * len(prefix)
        own = [(Tq + 40 * b) % 130 + (Tq if b % 4 != 2 else 0) for b in range(n)]
        lens = [min(Tq, own[b]) if b % 4 != 3 else 0 for b in range(n)]
        for q_lens in (None, lens):
            h = Held(Tq, 2 * G, 2, dh, 16, own, prefix, dt=F32, q_lens=q_lens)
            p = check_form(h, F_, F_)
            assert (p["own_rows"], p["prefix_rows"]) == (own_rows, prefix_rows)
            assert same(h.call(), h.call())
        h = Held(Tq, 2 * G, 2, dh, 16, own, prefix, dt=F32)
        ref = h.call()
        pg, s = slots(h.prefix_table, len(prefix) - 1, 5, 16)
        h.vp[pg, s, 0] = math.nan   # one key head of the last group's prefix: its sequences' rows, no others
        got = h.call()
        assert torch.isnan(got[n - S:, :, :G]).all() and same(got[:n - S], ref[:n - S]) and same(got[n - S:, :, G:], ref[n - S:, :, G:])
        h.prefix_table[len(prefix) - 1, 0] = -1   # with the page that holds it absent, the value is not there
        assert torch.isfinite(h.call()).all()


def test_a_generic_prefix_is_read_for_several_rows_at_once():
    for Tq, G, rows in ((1, 1, 4), (2, 2, 4), (1, 5, 16), (9, 2, 16)):
        p = check_form(Held(Tq, 2 * G, 2, 40, 20, [Tq + 3 * b for b in range(6)], [77], dt=F32), G_, G_)
        assert p["prefix_rows"] == rows


# ------------------------------------------------------------------- tables as a server keeps them
FORMS = [(1, 4, 2, 64, 16, BF), (3, 8, 2, 128, 64, BF), (2, 4, 2, 72, 16, BF), (40, 4, 4, 64, 16, BF), (200, 4, 2, 80, 32, BF), (140, 2, 2, 128, 128, BF),
         (20, 4, 2, 72, 16, BF), (1, 4, 4, 64, 16, F32), (2, 4, 2, 128, 8, F32), (30, 4, 2, 64, 16, F32), (1, 4, 2, 64, 12, F32), (2, 2, 1, 64, 16, F64)]


def widened(table, by, pages, seed):
    """A table with room for `by` times as many pages: entries behind the held ones are any numbers, pages of the pool among them."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(-3, pages + 3, (table.shape[0], table.shape[1] * by), generator=g, dtype=torch.int32)
    t[:, 3::7] = torch.randint(-(1 << 31), (1 << 31) - 1, t[:, 3::7].shape, generator=g).int()
    t[:, :table.shape[1]] = table.cpu()
    return t.to(DEV)


@pytest.mark.parametrize("by", [16, 128, 3000])
@pytest.mark.parametrize("Tq,H,Hkv,dh,page,dt", FORMS, ids=str)
def test_paged_attention_of_tables_much_wider_than_what_is_held(Tq, H, Hkv, dh, page, dt, by):
    """Room for long texts, and short ones in it: the same results, whatever stands behind the held pages."""
    for prefix in ([], [130, 33]):
        h = Held(Tq, H, Hkv, dh, page, [Tq, Tq + 90, 2 * Tq, 100 + Tq], prefix, dt=dt)
        P = h.kp.shape[0]
        # rubbish stands in the spare entry behind the last page too
        h.table = widened(h.table, by, P, by)
        if prefix:
            h.prefix_table = widened(h.prefix_table, by, P, by + 1)
        got = check_paged(h)
        assert same(h.call(), got)


@pytest.mark.parametrize("Tq,H,Hkv,dh,page,dt", FORMS, ids=str)
def test_paged_attention_reads_a_page_as_often_as_tables_name_it(Tq, H, Hkv, dh, page, dt):
    """The same page twice in a sequence, in several sequences and in a prefix."""
    n = 5 * page + 3
    n = max(n, Tq)
    need = -(-n // page)
    P = 3
    kp, vp = rand(P, page, Hkv, dh, seed=1, dtype=dt), rand(P, page, Hkv, dh, seed=2, dtype=dt)
    order = [[(i * i + b) % P for i in range(need)] for b in range(2)]
    table, pre = ints(order), ints([[1, 1, 0, 1]])
    q = rand(2, Tq, H, dh, seed=3, dtype=dt)
    got = api.paged_attention(q, kp, vp, table, ints([n, n]), prefix_table=pre, prefix_lens=ints([3 * page + 1]))
    # the same keys, each in a page of its own
    rows = order + [[1, 1, 0, 1]]
    own = [torch.cat([p[i] for r in rows for i in r]).view(-1, page, Hkv, dh) for p in (kp, vp)]
    t2 = torch.arange(2 * need, dtype=torch.int32, device=DEV).view(2, need)
    p2 = torch.arange(2 * need, 2 * need + 4, dtype=torch.int32, device=DEV).view(1, 4)
    assert same(got, api.paged_attention(q, own[0], own[1], t2, ints([n, n]), prefix_table=p2, prefix_lens=ints([3 * page + 1])))
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("Tq,H,Hkv,dh,page,dt", FORMS, ids=str)
def test_paged_attention_of_nothing_and_of_padding_that_is_no_number(Tq, H, Hkv, dh, page, dt):
    """Lengths of zero throughout; a prefix of nothing; and queries behind a sequence's new tokens that are NaN."""
    B = 4
    h = Held(Tq, H, Hkv, dh, page, [Tq + 50 * b for b in range(B)], [90, 40], dt=dt)
    zero, none = ints([0] * B), ints([0, -5])
    assert (h.call(kv_lens=zero, prefix_lens=none) == 0).all()
    assert (h.call(q_lens=zero) == 0).all() and (h.call(q_lens=zero, kv_lens=zero, prefix_lens=none) == 0).all()
    alone = h.call(prefix_table=None, prefix_lens=None)
    h.prefix, h.prefix_lens = [0, 0], none   # the same rows without one
    keep, h.where = h.where, h.where[:B] + [(0, 0), (0, 0)]
    o, w, mag, n = h.ref(dh ** -0.5)
    close(h.call(), o, paged_tol(h, o, w, mag, n, dh))
    close(alone, o, paged_tol(h, o, w, mag, n, dh))
    h.where, h.prefix, h.prefix_lens = keep, [90, 40], ints([90, 40])
    lens = [Tq, max(1, Tq // 2), 0, max(1, Tq - 1)]
    h.q_lens = ints(lens)
    ref = check_paged(h)
    for b, m in enumerate(lens):
        h.q[b, m:] = math.nan
    assert same(h.call(), ref)


@pytest.mark.parametrize("B,Tq,H,Hkv,dh,dt", [(2500, 1, 4, 4, 64, BF), (1200, 2, 4, 2, 128, BF), (500, 20, 2, 2, 64, BF), (1200, 1, 4, 2, 64, F32), (400, 1, 2, 2, 40, F64)], ids=str)
def test_paged_attention_of_thousands_of_sequences(B, Tq, H, Hkv, dh, dt):
    g = torch.Generator().manual_seed(B)
    own = (torch.randint(0, 70, (B,), generator=g)).tolist()
    for prefix, groups in ((0, 0), (50, 1), (20, B // 4)):
        h = Held(Tq, H, Hkv, dh, 16, own, [prefix] * groups, dt=dt)
        got = h.call()
        some = list(range(0, B, 97)) + [B - 1]
        small = Held.__new__(Held)
        small.__dict__.update(h.__dict__)
        S = B // groups if groups else 0
        small.B, small.own, small.q, small.q_lens = len(some), [own[b] for b in some], h.q[some], None
        small.where = [h.where[b] for b in some] + ([h.where[B + b // S] for b in some] if groups else [])
        small.prefix = [prefix] * len(some) if groups else []
        o, w, mag, n = small.ref(dh ** -0.5)
        close(got[some], o, paged_tol(small, o, w, mag, n, dh))


@pytest.mark.parametrize("H,Hkv,dh,dt", [(8, 2, 64, BF), (4, 4, 72, BF), (4, 4, 64, F32)], ids=str)
@pytest.mark.parametrize("T", [1, 2, 24])
def test_a_text_grows_without_waiting_as_it_grows_with_waiting(T, H, Hkv, dh, dt):
    """Append and attention in turn, each launched while the one before still runs, against the same with a wait behind each
    call: tokens, lengths, starts and page tables are all made on the stream."""
    B, page, steps = 6, 16, 12
    h = Held(T, H, Hkv, dh, page, [30 + 9 * b for b in range(B)], [300, 77, 500], dt=dt)
    f = api.rotary_frequencies(dh if dh != 72 else 64, device=DEV)
    x = rand(steps, B, T, H + 2 * Hkv, dh, seed=5, dtype=dt)
    width = -(-(80 + steps * T + page) // page)
    P0 = h.kp.shape[0]

    def run(wait):
        kp, vp = (torch.cat([p, torch.full((B * width,) + p.shape[1:], math.nan, dtype=dt, device=DEV)]) for p in (h.kp, h.vp))
        table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        held = h.table[:, :6]   # of at most 75 keys; what is behind a sequence's own is rubbish
        table[:, :6] = torch.where((held < P0) & (page * torch.arange(6, device=DEV) < h.kv_lens[:, None]), held, -1)
        lens, q, outs = h.kv_lens.clone(), torch.empty(B, T, H, dh, dtype=dt, device=DEV), []
        torch.cuda.synchronize()
        for i in range(steps):
            sync = torch.cuda.synchronize if wait else (lambda: None)
            starts = lens.clone()
            lens += T
            for j in range(width):   # a page for each slot that starts to be used
                table[:, j] = torch.where((table[:, j] < 0) & (lens > j * page), P0 + j + width * torch.arange(B, device=DEV), table[:, j]).int()
            sync()
            a = x[i]
            api.cache_append(a[:, :, H:H + Hkv], a[:, :, H + Hkv:], kp, vp, table, starts, q=a[:, :, :H], frequencies=f, q_out=q)
            sync()
            o = api.paged_attention(q, kp, vp, table, lens, prefix_table=h.prefix_table, prefix_lens=h.prefix_lens)
            sync()
            x2 = o + 0   # an ordinary kernel between
            outs.append(api.paged_attention(x2, kp, vp, table, lens, prefix_table=h.prefix_table, prefix_lens=h.prefix_lens, out=o))
            sync()
        torch.cuda.synchronize()
        return outs, kp, vp

    ref, rk, rv = run(True)
    assert all(torch.isfinite(o).all() for o in ref)
    for _ in range(3):
        got, gk, gv = run(False)
        assert all(same(a, b) for a, b in zip(got, ref)) and same(gk, rk) and same(gv, rv)
