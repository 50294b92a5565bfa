"""The serving stages against plain 64-bit implementations: root-mean-square norm, 8-bit
quantisation, the 8-bit product, cross attention, and a run of them together.

Tolerances, from the arithmetic (u = 2^-24, one fp32 rounding):
  bf16 result     half a step, 2^-8 |y|;   fp32 result 2^-24 |y|
  e4m3 result     q * scale: half a step, 2^-4 |y|, or 2^-10 scale below the normal range
  norm            sum of squares: a chain of at most ceil(D / 256) + 8 additions in one thread and
                  10 in the tree; square root, division and two products: 8 more
  scales          the error of the largest value of the block, and one division
  product         a block of 128 products and the blocks in turn, each addition off by at most
                  2 u of the sum of magnitudes (tensor cores may truncate): 2 u (128 + blocks + 8)
  GELU            slope at most 1.13; its own arithmetic 2^-19 |z|
  attention       a score is off by 2 u (dh + 2) scale sum|q||k|, and its weight by twice that,
                  relatively; bf16 weights by 2^-8 more; sums of Tk fp32 terms by 2 u (Tk + 8)
"""
import math

import pytest
import torch

from vision_transformer_encoder_gb300 import api

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F8 = torch.float8_e4m3fn
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = {BF: 2.0 ** -8, F32: U, F64: 2.0 ** -53}
DEV = "cuda:0"
TINY = 2.0 ** -126


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    assert api.device_error() == 0


def rand(*shape, seed=0, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed * 7919 + sum(shape))
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def unaligned(t):
    """t's values at an address that is a multiple of its element size only."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    buf[1:].copy_(t.reshape(-1))
    return buf[1:].view(t.shape)


def close(got, ref, tol):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    bad = ~((got - ref).abs() <= tol) & ~torch.isnan(ref) & ~(got == ref)
    if bad.any():
        i = int(torch.argmax(((got - ref).abs() / tol.clamp_min(1e-300)).nan_to_num(0).reshape(-1)))
        raise AssertionError("%d of %d outside: worst got %g ref %g tol %g" % (
            int(bad.sum()), bad.numel(), got.reshape(-1)[i], ref.reshape(-1)[i], tol.expand_as(ref).reshape(-1)[i]))


def spread(scales, n, rows=None):
    s = scales.double().repeat_interleave(128, 1)[:, :n]
    return s if rows is None else s.repeat_interleave(128, 0)[:rows]


def block_max(y):
    pad = torch.nn.functional.pad(y.abs(), (0, -y.shape[1] % 128))
    return pad.view(y.shape[0], -1, 128).amax(2)


def close8(q, scales, y, err):
    """q * scales against y (rows, n), itself known to within err (rows, n)."""
    top, n = block_max(y), y.shape[1]
    serr = block_max(err) / 448 + 2 * U * scales.double() + TINY * 2.0 ** -20
    assert ((scales.double() - (top / 448).clamp_min(TINY)).abs() <= serr).all()
    sc = spread(scales, n)
    # a scale that is off moves the grid, not the values; the codes saturate at 448
    close(q.double() * sc, y, (2.0 ** -4 + 2.0 ** -20) * (y.abs() + err) + 2.0 ** -10 * sc + err + 448 * spread(serr, n))


# ----------------------------------------------------------------------------------- norm
def norm_ref(x, residual, gamma, eps):
    s = x.double() + (residual.double() if residual is not None else 0)
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return s, y * gamma.double() if gamma is not None else y


NORM_TYPES = [(BF, BF, BF), (BF, F32, BF), (BF, None, F8), (BF, BF, F8), (BF, F32, F8), (F32, F32, F32),
              (F32, None, BF), (F32, F32, F8), (BF, None, F32), (F64, F64, F64)]


@pytest.mark.parametrize("types", NORM_TYPES, ids=str)
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 5), (7, 127), (2, 128), (5, 129), (64, 192), (33, 1280), (9, 1000),
                                    (3, 4096), (2, 8192), (3, 8200), (1, 40001), (1100, 264), (2500, 1024)])
def test_rmsnorm(rows, D, types):
    xt, rt, ot = types
    x = rand(rows, D, seed=1, dtype=xt)
    residual = rand(rows, D, seed=2, std=3.0, dtype=rt) if rt is not None else None
    gamma = (1 + rand(D, seed=3, std=0.2)).to(F64 if xt == F64 else BF if D % 2 else F32)
    check_norm(x, residual, gamma, ot)


def check_norm(x, residual, gamma, ot, **kw):
    rows, D = x.shape
    eps = 1e-6
    s, y = norm_ref(x, residual, gamma, eps)
    got = api.rmsnorm(x, eps, gamma=gamma, residual=residual, out_dtype=ot, **kw)
    got = list(got) if isinstance(got, tuple) else [got]
    if residual is not None:
        close(got[-1], s, HALF[residual.dtype] * s.abs() * (1 + 2.0 ** -10) + (0 if ot == F64 else U) * s.abs())
    chain = math.ceil(D / 256) + 26
    err = chain * (2.0 ** -53 if ot == F64 else U) * y.abs()
    if ot == F8:
        close8(got[0], got[1], y, err)
    else:
        close(got[0], y, HALF[ot] * y.abs() * (1 + 2.0 ** -10) + err)
    return got


@pytest.mark.parametrize("ot", [BF, F8])
@pytest.mark.parametrize("D", [136, 1024])
def test_rmsnorm_in_place_and_unaligned(D, ot):
    x, r, g = rand(17, D, seed=1, dtype=BF), rand(17, D, seed=2, dtype=BF), rand(D, seed=3, dtype=BF)
    ref = [t.clone() for t in check_norm(x, r, g, ot)]
    for which in ("residual", "x"):
        x2, r2 = x.clone(), r.clone()
        t = r2 if which == "residual" else x2
        got = api.rmsnorm(x2, 1e-6, gamma=g, residual=r2, out_dtype=ot, sum_out=t)
        assert got[-1] is t
        for a, b in zip(got, ref):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    check_norm(unaligned(x), unaligned(r), unaligned(g), ot)
    check_norm(x, r, g, ot, out=unaligned(ref[0].view(torch.uint8)).view(ot) if ot == F8 else unaligned(ref[0]))


def test_rmsnorm_special_rows():
    x = rand(6, 512, seed=4, dtype=BF)
    x[0] = 0
    x[1, 7] = math.nan
    x[2, 300] = math.inf
    x[3] = 1e-30
    x[4] = 2.0 ** 60
    out = api.rmsnorm(x, 1e-6)
    q, s = api.rmsnorm(x, 1e-6, out_dtype=F8)
    assert (out[0] == 0).all() and (q[0].float() == 0).all() and (s[0] == TINY).all()
    assert torch.isnan(out[1]).all() and torch.isnan(q[1].float() * s[1].repeat_interleave(128)).all()
    ref = norm_ref(x, None, None, 1e-6)[1]
    assert torch.equal(torch.isnan(out[2]), torch.isnan(ref[2])) and (out[2, :300] == 0).all()
    close(out[3:], ref[3:], 2.0 ** -7 * ref[3:].abs())


@pytest.mark.parametrize("rows,D", [(3, 8), (1500, 264), (2, 5)])   # registers, many rows, generic
def test_rmsnorm_large_rows_and_eps(rows, D):
    """Squares past the fp32 range beside an eps of their size: mean square 1e38, eps 1e38."""
    x = torch.full((rows, D), 1e19, device=DEV)
    x[:, ::2] *= -1
    for eps in (1e38, 1e-6):
        y = norm_ref(x, None, None, eps)[1]
        close(api.rmsnorm(x, eps), y, 2.0 ** -19 * y.abs())


@pytest.mark.parametrize("eps", [1e-6, 1e300])
@pytest.mark.parametrize("value", [1e19, 1e150, 1e200, 1e300])
@pytest.mark.parametrize("D", [5, 264, 3000])
def test_rmsnorm_large_rows_in_fp64(D, value, eps):
    """fp64 rows have fp64's range: squares past it are summed from scaled values, eps beside them."""
    x = rand(3, D, seed=2, dtype=F64) * value
    x[1] = 1.7e308
    s, y = norm_ref(x * 2.0 ** -520, None, None, eps * 2.0 ** -1040)
    # y of the scaled rows; a chain of ceil(D / 256) + 8 additions per thread, 10 in the tree, 8 more operations
    close(api.rmsnorm(x, eps), y, 2 * (math.ceil(D / 256) + 26) * 2.0 ** -53 * y.abs())
    r = rand(3, D, seed=3, dtype=F64) * value
    r[1] = -1e308
    out, total = api.rmsnorm(x, eps, residual=r)
    s, y = norm_ref((x + r) * 2.0 ** -520, None, None, eps * 2.0 ** -1040)
    assert torch.equal(total, x + r)
    close(out, y, 2 * (math.ceil(D / 256) + 26) * 2.0 ** -53 * y.abs())


@pytest.mark.parametrize("types", [(BF, BF, F8), (BF, F32, BF), (F32, F32, F32)], ids=str)
@pytest.mark.parametrize("rows,D", [(2500, 1024), (1501, 5120), (700, 10240), (5, 8200), (3, 1001)])   # rows to a warp, to 2 to 8 warps, few, generic
def test_rmsnorm_in_place_in_every_form(rows, D, types):
    xt, rt, ot = types
    x, r, g = rand(rows, D, seed=1, dtype=xt), rand(rows, D, seed=2, dtype=rt), rand(D, seed=3)
    ref = check_norm(x, r, g, ot)
    for over in (["residual", "x"] if xt == rt else ["residual"]):
        x2, r2 = x.clone(), r.clone()
        got = api.rmsnorm(x2, 1e-6, gamma=g, residual=r2, out_dtype=ot, sum_out=r2 if over == "residual" else x2)
        for a, b in zip(got, ref):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(r2 if over == "x" else x2, r if over == "x" else x)
    # x as its own residual: a sum of 2 x
    got = api.rmsnorm(x, 1e-6, gamma=g, residual=x)
    assert torch.equal(got[1], (x.double() * 2).to(xt))


@pytest.mark.parametrize("rows,D", [(2500, 1024), (1501, 5120), (6, 1001)])
def test_rmsnorm_special_rows_in_every_form(rows, D):
    x = rand(rows, D, seed=4, dtype=BF)
    plain, (pq, ps) = api.rmsnorm(x, 1e-6), api.rmsnorm(x, 1e-6, out_dtype=F8)
    x[0], x[1, 7], x[2, 300], x[4] = 0, math.nan, math.inf, 2.0 ** 60
    out, (q, s) = api.rmsnorm(x, 1e-6), api.rmsnorm(x, 1e-6, out_dtype=F8)
    v = q.float() * spread(s, D).float()
    assert (out[0] == 0).all() and (v[0] == 0).all() and (s[0] == TINY).all()
    assert torch.isnan(out[1]).all() and torch.isnan(v[1]).all()
    for t in (out, v):
        assert torch.isnan(t[2, 300]) and (t[2, :300] == 0).all() and (t[2, 301:] == 0).all()
    y = norm_ref(x[4:5], None, None, 1e-6)[1]
    close(out[4:5], y, 2.0 ** -7 * y.abs())
    keep = torch.tensor([i for i in range(rows) if i not in (0, 1, 2, 4)], device=DEV)
    assert torch.equal(out[keep], plain[keep]) and torch.equal(s[keep], ps[keep])
    assert torch.equal(q.view(torch.uint8)[keep], pq.view(torch.uint8)[keep])


def test_rmsnorm_leading_dimensions_and_no_gain():
    x = rand(2, 3, 5, 64, seed=5, dtype=BF)
    out = api.rmsnorm(x, 1e-5)
    assert out.shape == x.shape and out.dtype == BF
    y = norm_ref(x.view(-1, 64), None, None, 1e-5)[1]
    close(out.view(-1, 64), y, 2.0 ** -7 * y.abs())


# ------------------------------------------------------------------------------- quantise
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 127), (2, 128), (5, 129), (7, 264), (300, 1024), (4, 1000), (1, 20000),
                                    (20011, 136)])
def test_quantize(rows, K, dt):
    x = rand(rows, K, seed=6, dtype=dt)
    x[0, : min(K, 130)] = 0
    for t in (x, unaligned(x)):
        q, s = api.quantize(t)
        close8(q, s, x.double(), torch.zeros_like(x, dtype=F64))


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("K,N", [(1, 1), (127, 130), (128, 128), (200, 72), (264, 520), (1024, 384), (16, 1000)])
def test_quantize_weight(K, N, dt):
    w = rand(K, N, seed=7, dtype=dt)
    for t in (w, unaligned(w)):
        q, s = api.quantize_weight(t)
        assert q.shape == (N, K) and s.shape == ((N + 127) // 128, (K + 127) // 128)
        wt = w.double().t().contiguous()
        for nb in range(s.shape[0]):
            rows = wt[nb * 128:(nb + 1) * 128]
            sc = (block_max(rows).amax(0) / 448).clamp_min(TINY)
            assert ((s[nb].double() - sc).abs() <= 2 * U * sc).all()
        sc = spread(s, K, N)
        close(q.double() * sc, wt, (2.0 ** -4 + 2.0 ** -20) * wt.abs() + 2.0 ** -10 * sc)


def test_quantize_special_values():
    x = torch.zeros(3, 256, device=DEV)
    x[0, 3], x[1, 200] = math.nan, -math.inf
    x[1, 201] = 1.0
    x[2] = 1e-42            # below the floor of the scale: codes of zero or the smallest step
    q, s = api.quantize(x)
    v = q.float() * s.repeat_interleave(128, 1)
    assert torch.isnan(v[0, 3]) and (v[0, 4:] == 0).all()
    assert torch.isnan(v[1, 128:]).all() and (v[1, :128] == 0).all()
    assert (s[2] == TINY).all() and (v[2].abs() <= 2.0 ** -135).all()


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("K,N", [(256, 264), (255, 131)])   # by 8, generic
def test_quantize_special_values_in_every_form(K, N, dt):
    x = rand(K, N, seed=6, dtype=dt)
    q0, s0 = api.quantize(x)
    w0, t0 = api.quantize_weight(x)
    x[1, 3], x[2, 130], x[3, 130] = math.nan, math.inf, -math.inf
    q, s = api.quantize(x)
    v = q.double() * spread(s, N)
    # a NaN is one; the block of an infinity is NaN throughout; the rest is as before
    assert torch.isnan(v[1, 3]) and not torch.isnan(v[1, 4:]).any() and not torch.isnan(v[2:4, :128]).any()
    assert torch.isnan(v[2:4, 128:256]).all() and not torch.isnan(v[2:4, 256:]).any() and torch.isinf(s[2:4, 1]).all()
    assert torch.equal(q.view(torch.uint8)[4:], q0.view(torch.uint8)[4:]) and torch.equal(s[4:], s0[4:])
    w, t = api.quantize_weight(x)   # the infinities are in the block of rows 128.. of the transpose, columns ..127
    v = w.double() * spread(t, K, N)
    assert torch.isnan(v[128:256, :128]).all() and torch.isinf(t[1, 0]) and torch.isnan(v[3, 1])
    assert torch.isnan(v).sum() == 1 + (min(N, 256) - 128) * 128 and torch.equal(t[:, 1], t0[:, 1])
    assert torch.equal(w.view(torch.uint8)[:, 128:], w0.view(torch.uint8)[:, 128:])


# -------------------------------------------------------------------------------- product
def linear_ref(a, sa, w, sw):
    """z and the sum of magnitudes of its terms."""
    av, wv = a.double() * spread(sa, a.shape[1]), w.double() * spread(sw, w.shape[1], w.shape[0])
    return av @ wv.t(), av.abs() @ wv.abs().t()


def gelu64(z):
    return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def make_product(M, K, N, seed=0):
    a, sa = api.quantize(rand(M, K, seed=seed + 1) * torch.exp(rand(K, seed=seed + 2, std=0.7)))
    w, sw = api.quantize_weight(rand(K, N, seed=seed + 3, std=K ** -0.5))
    return a, sa, w, sw


def check_linear(ops, epi=api.EPI_STORE, bias=None, residual=None, ot=BF, **kw):
    a, sa, w, sw = ops
    z, mag = linear_ref(*ops)
    err = 2 * U * (128 + sa.shape[1] + 8) * mag
    if bias is not None:
        z = z + bias.double()
        err = err + 2 * U * z.abs()
    if epi == api.EPI_GELU:
        err, z = 1.13 * err + 2.0 ** -19 * z.abs(), gelu64(z)
    elif epi == api.EPI_RESIDUAL:
        z = z + residual.double()
        err = err + 2 * U * z.abs()
    got = api.linear_fp8(a, sa, w, sw, bias=bias, residual=residual, epilogue=epi, out_dtype=ot, **kw)
    if ot == F8:
        close8(got[0], got[1], z, err)
    else:
        # the bf16 GELU may use the hardware tangent, 2^-11 of the half that it scales
        more = 2.0 ** -11 * z.abs() + 2.0 ** -12 * linear_ref(*ops)[0].abs() if epi == api.EPI_GELU and ot == BF else 0
        close(got, z, HALF[ot] * z.abs() * (1 + 2.0 ** -8) + err + more)
    return got


LINEAR_SHAPES = [(1, 1, 1), (3, 130, 5), (1, 128, 128), (2, 16, 8), (7, 144, 200), (16, 1024, 384), (17, 272, 136),
                 (33, 512, 1000), (64, 80, 64), (65, 640, 257), (128, 1280, 256), (130, 128, 520), (200, 1264, 1286),
                 (257, 384, 640), (300, 192, 129), (513, 2048, 256), (1000, 256, 2048), (1731, 1280, 1280),
                 (1300, 272, 4104), (1290, 144, 4112)]


@pytest.mark.parametrize("M,K,N", LINEAR_SHAPES)
@pytest.mark.parametrize("form", ["store bf16", "store f32", "store e4m3", "gelu e4m3", "gelu bf16 bias", "gelu f32",
                                  "residual bf16", "residual f32 bias", "residual f32 to bf16", "residual e4m3"])
def test_linear_fp8(M, K, N, form):
    ops = make_product(M, K, N, seed=M % 5)
    words = form.split()
    epi = {"store": api.EPI_STORE, "gelu": api.EPI_GELU, "residual": api.EPI_RESIDUAL}[words[0]]
    ot = F8 if words[-1] == "e4m3" else BF if words[-1] == "bf16" or "bf16" in words[1:2] else F32
    bias = rand(N, seed=8, std=0.5, dtype=F32 if M % 2 else BF) if "bias" in words or ot == F8 else None
    residual = None
    if words[0] == "residual":
        residual = rand(M, N, seed=9, dtype=F32 if "f32" in words else BF)
    check_linear(ops, epi, bias, residual, ot)


@pytest.mark.parametrize("M", [3, 300])
def test_linear_fp8_unaligned_and_in_place(M):
    a, sa, w, sw = make_product(M, 256, 264)
    u8 = lambda t: unaligned(t.view(torch.uint8)).view(F8)  # noqa: E731
    bias = rand(264, seed=1, dtype=BF)
    for ops in ((u8(a), sa, w, sw), (a, sa, u8(w), sw), (a, unaligned(sa), w, unaligned(sw))):
        check_linear(ops, bias=unaligned(bias))
    check_linear((a, sa, w, sw), ot=BF, out=unaligned(torch.empty(M, 264, dtype=BF, device=DEV)))
    for dt in (BF, F32):
        r = rand(M, 264, seed=2, dtype=dt)
        ref = api.linear_fp8(a, sa, w, sw, residual=r, epilogue=api.EPI_RESIDUAL, out_dtype=dt)
        got = api.linear_fp8(a, sa, w, sw, residual=r, epilogue=api.EPI_RESIDUAL, out=r)
        assert got is r and torch.equal(got, ref)
        r = unaligned(rand(M, 264, seed=2, dtype=dt))
        assert torch.equal(api.linear_fp8(a, sa, w, sw, residual=r, epilogue=api.EPI_RESIDUAL, out_dtype=dt), ref)


@pytest.mark.parametrize("M", [2, 40, 600])
def test_linear_fp8_special_values(M):
    """NaN and infinite operands reach the rows and columns that they belong to, and no others."""
    a, sa, w, sw = make_product(M, 384, 256)
    ref = api.linear_fp8(a, sa, w, sw)
    a2, sa2 = a.clone(), sa.clone()
    a2.view(torch.uint8)[1, 200] = 0x7F          # NaN
    got = api.linear_fp8(a2, sa, w, sw)
    assert torch.isnan(got[1]).all() and torch.equal(got[0], ref[0]) and torch.equal(got[2:], ref[2:])
    sa2[0, 1] = math.inf
    got = api.linear_fp8(a, sa2, w, sw)
    assert not torch.isfinite(got[0]).any() and torch.equal(got[1:], ref[1:])
    zero = api.linear_fp8(torch.zeros_like(a.view(torch.uint8)).view(F8), sa, w, sw, out_dtype=F8)
    assert (zero[0].float() == 0).all() and (zero[1] == TINY).all()


@pytest.mark.parametrize("ot", [BF, F32, F8], ids=str)
@pytest.mark.parametrize("M,K", [(4, 256), (40, 256), (600, 256), (4, 255)])   # rows, pairs, generic
def test_linear_fp8_gelu_of_large_values(M, K, ot):
    """GELU of -1e25 is zero and of 1e25 is itself, beside rows of ordinary size."""
    a, sa, w, sw = make_product(M, K, 256)
    sa = sa.clone()
    sa[1::2] *= 1e25
    z = linear_ref(a, sa, w, sw)[0]
    got = api.linear_fp8(a, sa, w, sw, epilogue=api.EPI_GELU, out_dtype=ot)
    v = got[0].double() * spread(got[1], 256) if ot == F8 else got.double()
    below, above = z < -1e23, z > 1e23
    assert below.any() and above.any() and (v[below] == 0).all()
    # e4m3: half a step of the block's scale, at most 448 of which are the largest value
    tol = (2.0 ** -4 if ot == F8 else 2.0 ** -7) * z[above].abs() + (2.0 ** -17 * z.abs().max() if ot == F8 else 0)
    close(v[above], z[above], tol)


# 16 and 32 rows to a tile, CTA pairs with tiles of 128 and of 256 columns, CUDA cores (on 152 SMs: 32-row tiles up to
# one wave of CTAs, then pairs)
GEMM_FORMS = [(4, 256, 384), (600, 256, 384), (2400, 256, 384), (2400, 256, 4096), (4, 255, 384)]
PAIR_SHAPES = [(2405, 272, 392), (2405, 272, 4104), (2405, 272, 389)]


@pytest.mark.parametrize("M,K,N", GEMM_FORMS)
def test_linear_fp8_gelu_to_bf16_is_rounded_once(M, K, N):
    """No more than the fp32 GELU's own error beside the output's half step: no 8-bit kernel takes the hardware tangent."""
    ops = make_product(M, K, N)
    z, mag = linear_ref(*ops)
    err = 1.13 * 2 * U * (128 + ops[1].shape[1] + 8) * mag + 2.0 ** -19 * z.abs()
    y = gelu64(z)
    close(api.linear_fp8(*ops, epilogue=api.EPI_GELU, out_dtype=BF), y, HALF[BF] * y.abs() * (1 + 2.0 ** -8) + err)


@pytest.mark.parametrize("ot", [BF, F32, F8], ids=str)
@pytest.mark.parametrize("M,K,N", GEMM_FORMS)
def test_linear_fp8_values_of_any_size(M, K, N, ot):
    """GELU of -1e25 is zero and of 1e25 itself; NaN and infinities stay in their rows."""
    a, sa, w, sw = make_product(M, K, N)
    sa = sa.clone()
    sa[1::2] *= 1e25
    z = linear_ref(a, sa, w, sw)[0]
    got = api.linear_fp8(a, sa, w, sw, epilogue=api.EPI_GELU, out_dtype=ot)
    v = got[0].double() * spread(got[1], N) if ot == F8 else got.double()
    below, above = z < -1e23, z > 1e23
    assert below.any() and above.any() and (v[below] == 0).all()
    # e4m3: half a step of the block's scale, at most 448 of which are the largest value
    tol = (2.0 ** -4 if ot == F8 else 2.0 ** -7) * z[above].abs() + (2.0 ** -17 * z.abs().max() if ot == F8 else 0)
    close(v[above], z[above], tol)
    a, sa, w, sw = make_product(M, K, N)
    ref = api.linear_fp8(a, sa, w, sw, out_dtype=ot)
    a.view(torch.uint8)[M - 2, 200] = 0x7F          # NaN
    sa[0, 1] = math.inf
    got = api.linear_fp8(a, sa, w, sw, out_dtype=ot)
    if ot == F8:
        assert torch.equal(got[1][1:M - 2], ref[1][1:M - 2]) and torch.equal(got[1][M - 1], ref[1][M - 1])
        got, ref = got[0], ref[0]
    assert torch.isnan(got[M - 2].float()).all() and not torch.isfinite(got[0].float()).any()
    same = got.view(torch.uint8) == ref.view(torch.uint8)
    assert same[1:M - 2].all() and same[M - 1].all()


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("M,K,N", PAIR_SHAPES)
def test_linear_fp8_of_pairs_in_place_and_unaligned(M, K, N, dt):
    ops = make_product(M, K, N)
    r = rand(M, N, seed=2, dtype=dt)
    ref = check_linear(ops, api.EPI_RESIDUAL, residual=r, ot=dt)
    apart = unaligned(r)
    assert torch.equal(api.linear_fp8(*ops, residual=apart, epilogue=api.EPI_RESIDUAL, out_dtype=dt), ref)
    assert torch.equal(api.linear_fp8(*ops, residual=apart, epilogue=api.EPI_RESIDUAL, out=apart), ref)
    got = api.linear_fp8(*ops, residual=r, epilogue=api.EPI_RESIDUAL, out=r)
    assert got is r and torch.equal(got, ref)


@pytest.mark.parametrize("lead", [4096, 4104])
@pytest.mark.parametrize("M,K,N", PAIR_SHAPES)
def test_nothing_outside_the_outputs_of_pairs_is_written(M, K, N, lead):
    ops = make_product(M, K, N)
    for dt in (BF, F32, F8):
        inside((M, N), dt, lead, lambda t: api.linear_fp8(*ops, out=t))
    inside((M, (N + 127) // 128), F32, lead, lambda t: api.linear_fp8(*ops, out_dtype=F8, out_scales=t))


# -------------------------------------------------------------------------- cross attention
def cross_ref(q, k, v, lens, scale):
    """o, the sum of weights times |v|, and the largest sum of magnitudes in a row's scores."""
    B, Tq, H, dh = q.shape
    Tk, G = k.shape[1], H // k.shape[2]
    qd = q.double().permute(0, 2, 1, 3)
    kd, vd = (t.double().repeat_interleave(G, 2).permute(0, 2, 1, 3) for t in (k, v))
    live = torch.arange(Tk, device=q.device)[None] < (lens[:, None] if lens is not None else Tk)
    kd, vd = (torch.where(live[:, None, :, None], t, 0.0) for t in (kd, vd))
    x = torch.where(live[:, None, None], scale * (qd @ kd.transpose(2, 3)), -math.inf)
    p = torch.where(live[:, None, None].any(3, keepdim=True), torch.softmax(x, 3), 0.0)
    mag = abs(scale) * (qd.abs() @ kd.abs().transpose(2, 3)).amax(3, keepdim=True)
    return [t.permute(0, 2, 1, 3) for t in (p @ vd, p @ vd.abs(), mag)]


def check_cross(q, k, v, lens=None, scale=None, **kw):
    dh, Tk, dt = q.shape[3], k.shape[1], q.dtype
    sc = dh ** -0.5 if scale is None else scale
    o, w, mag = cross_ref(q, k, v, lens, sc)
    got = api.cross_attention(q, k, v, kv_lens=lens, scale=scale, **kw)
    u = 2.0 ** -53 if dt == F64 else U
    es = 2 * u * (dh + 4) * mag
    # 2^-20: the exponential of a rounded argument, up to 16 units of the scores' base
    tol = (2 * es + 2 * u * (Tk + 8) + (0 if dt == F64 else 2.0 ** -20)) * w + HALF[dt] * o.abs() * 1.01
    if dt == BF:
        tol = tol + 2.0 ** -8 * w
    close(got, o, tol)
    return got


def make_cross(B, Tq, Tk, H, Hkv, dh, dt=BF, seed=0):
    q = rand(B, Tq, H, dh, seed=seed + 1, dtype=dt)
    kv = rand(B, Tk, 2, Hkv, dh, seed=seed + 2, dtype=dt)
    return q, kv[:, :, 0], kv[:, :, 1]


def lens_of(B, Tk, seed=0):
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, Tk + 1, (B,), generator=g, dtype=torch.int32)
    if B > 1:
        lens[0] = 0
    if B > 2:
        lens[1], lens[2] = Tk, 1
    return lens.to(DEV)


CROSS_SHAPES = [(1, 1, 1, 1, 1, 64), (2, 1, 2, 3, 3, 64), (3, 1, 127, 4, 2, 64), (2, 1, 128, 8, 1, 80),
                (4, 1, 129, 16, 16, 64), (2, 1, 1000, 16, 2, 128), (1, 1, 5001, 2, 1, 96), (5, 2, 63, 6, 3, 64),
                (2, 5, 300, 12, 4, 80), (1, 16, 257, 4, 4, 128), (3, 17, 64, 4, 1, 64), (2, 33, 577, 3, 3, 64),
                (2, 100, 40, 15, 5, 96), (2, 128, 128, 4, 4, 128), (3, 129, 385, 8, 2, 64), (1, 300, 130, 4, 4, 80),
                (2, 260, 1025, 2, 1, 128), (1, 513, 700, 6, 2, 96), (3, 257, 3, 3, 1, 64), (1, 90, 3000, 16, 2, 64)]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("shape", CROSS_SHAPES, ids=str)
def test_cross_attention(shape, dt, ragged):
    q, k, v = make_cross(*shape, dt=dt)
    check_cross(q, k, v, lens_of(shape[0], shape[2]) if ragged else None)


@pytest.mark.parametrize("Tq", [1, 3, 20, 130, 260])
@pytest.mark.parametrize("dh", [64, 80, 96, 128])
def test_cross_attention_of_few_queries_over_many_keys(dh, Tq):
    """Parts of the keys go to different CTAs: lengths that leave some of them, or all but one key, without."""
    B, Tk, H, Hkv = 3, 2500, 6, 2
    q, k, v = make_cross(B, Tq, Tk, H, Hkv, dh)
    for lens in ([2500, 1, 0], [1300, 129, 2177]):
        check_cross(q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV))
    check_cross(q[:1], k[:1], v[:1])
    got = check_cross(q, k, v)
    for _ in range(3):
        assert torch.equal(api.cross_attention(q, k, v), got)


@pytest.mark.parametrize("dt", [BF, F32], ids=str)
@pytest.mark.parametrize("B", [2, 37, 128, 130])
def test_cross_attention_of_many_ragged_sequences(B, dt):
    """More work than one round of CTAs, sequences in any order of length, equal and empty ones among them."""
    Tq, H, Tk = (1300, 16, 200) if B == 2 else (140, 6, 200)
    q, k, v = make_cross(B, Tq, Tk, H, H, 64, dt=dt)
    lens = torch.randint(0, Tk + 1, (B,), generator=torch.Generator().manual_seed(B)).to(torch.int32).to(DEV)
    lens[B // 3] = 0
    lens[1::5] = 77
    for t in (Tq, Tq - 30, 30):
        check_cross(q[:, :t], k, v, lens)


@pytest.mark.parametrize("dh", [1, 8, 17, 32, 48, 72, 160, 256, 512])
@pytest.mark.parametrize("dt", [BF, F32, F64], ids=str)
def test_cross_attention_other_head_widths(dh, dt):
    q, k, v = make_cross(2, 5, 70, 4, 2, dh, dt=dt)
    check_cross(q, k, v, torch.tensor([70, 33], dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("Tq", [1, 200])
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
def test_cross_attention_layouts(Tq, dt):
    """Heads before tokens, batch-broadcast states, unaligned and padded views, one key head."""
    B, Tk, H, Hkv, dh = 3, 150, 4, 2, 64
    lens = torch.tensor([150, 1, 77], dtype=torch.int32, device=DEV)
    q, k, v = make_cross(B, Tq, Tk, H, Hkv, dh, dt=dt)
    ref = check_cross(q, k, v, lens)
    heads_first = [t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (q, k, v)]
    assert torch.equal(check_cross(*heads_first, lens), ref)
    assert torch.equal(check_cross(q, k.contiguous(), v.contiguous(), lens), ref)
    check_cross(unaligned(q), k, v, lens)
    check_cross(q, unaligned(k.contiguous()), unaligned(v.contiguous()), lens)
    check_cross(q, k, v, lens, out=unaligned(torch.empty_like(q)))
    wide = torch.nn.functional.pad(k, (0, 3))[..., :dh]           # token rows of no even number of bytes
    check_cross(q, wide, v, lens)
    check_cross(q, k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1), lens)
    check_cross(q, k[:, :, :1].expand(-1, -1, 2, -1), v[:, :, :1].expand(-1, -1, 2, -1), lens)


@pytest.mark.parametrize("Tq,Tk", [(1, 300), (3, 100), (40, 300), (200, 300)])
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
def test_cross_attention_ignores_what_lies_past_the_length(Tq, Tk, dt):
    q, k, v = make_cross(4, Tq, Tk, 4, 2, 64, dt=dt)
    lens = torch.tensor([Tk - 1, 0, 1, 65], dtype=torch.int32, device=DEV)
    ref = check_cross(q, k, v, lens)
    k, v = k.clone(), v.clone()
    for b, n in enumerate(lens.tolist()):
        k[b, n:], v[b, n:] = math.nan, math.nan
        k[b, n + 1:], v[b, n + 1:] = math.inf, -math.inf
    assert torch.equal(api.cross_attention(q, k, v, kv_lens=lens), ref)
    out_of_range = torch.tensor([Tk + 1000, -5, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    q, k, v = make_cross(4, Tq, Tk, 4, 2, 64, dt=dt)
    clamped = torch.tensor([Tk, 0, Tk, 0], dtype=torch.int32, device=DEV)
    assert torch.equal(api.cross_attention(q, k, v, kv_lens=out_of_range),
                       api.cross_attention(q, k, v, kv_lens=clamped))


@pytest.mark.parametrize("Tq", [1, 150])
@pytest.mark.parametrize("dt", [BF, F32], ids=str)
def test_cross_attention_special_scores(Tq, dt):
    q, k, v = make_cross(2, Tq, 400, 2, 2, 64, dt=dt)
    # growing scores make the running maximum climb through every tile; large ones leave one key
    grow = torch.linspace(0, 6, 400, device=DEV)[None, :, None, None]
    check_cross(q, (q[:, :1].float().expand(-1, 400, -1, -1) * grow).to(dt), v, scale=0.125)
    check_cross(q, k, v, scale=0.0)
    check_cross(q, k, v, scale=-0.3)
    # one key's scores of minus infinity carry no weight; a row of nothing else is not a number
    q2, k2 = q.abs() + 0.01, k.clone()
    k2[:, 3] = -math.inf
    got = api.cross_attention(q2, k2, v)
    rest = torch.cat([k2[:, :3], k2[:, 4:]], 1), torch.cat([v[:, :3], v[:, 4:]], 1)
    o, w, mag = cross_ref(q2, *rest, None, 0.125)
    close(got, o, (2.0 ** -7 if dt == BF else 2.0 ** -16) * w)
    k2[:] = -math.inf
    assert torch.isnan(api.cross_attention(q2, k2, v)).all()
    k2 = k.clone()
    k2[0, 399, 1] = math.nan
    got = api.cross_attention(q, k2, v)
    assert torch.isnan(got[0, :, 1]).all()
    keep = api.cross_attention(q, k, v)
    assert torch.equal(got[1], keep[1]) and torch.equal(got[0, :, 0], keep[0, :, 0])


# Scores of 2^31 and more are farther apart in fp32 than the exponential's range is wide, so the largest
# one has to come out as exactly zero behind the maximum. Forms: split and whole tensor-core items, few
# queries on one CTA and on a cluster, fp32 with and without shared rows, CUDA cores.
LARGE_SCORES = [(BF, 2, 150, 400, 4, 2, 64), (BF, 1, 64, 2500, 2, 2, 128), (BF, 40, 1, 300, 16, 16, 64),
                (BF, 1, 2, 3000, 4, 2, 80), (F32, 2, 150, 400, 4, 2, 64), (F32, 2, 3, 400, 4, 2, 80),
                (F32, 2, 20, 70, 4, 2, 128), (BF, 2, 40, 70, 4, 2, 72), (F64, 2, 3, 70, 4, 2, 64)]


@pytest.mark.parametrize("scale", [1e9, 7e17, 1e30])
@pytest.mark.parametrize("form", LARGE_SCORES, ids=str)
def test_cross_attention_of_large_scores(form, scale):
    """Queries and keys of small whole numbers have exact scores, and differences of 1 leave no weight: the mean
    of the values under the largest score, the weights all exactly 1. Then numbers without structure, whose
    scores are too coarse for more than this: every output lies between the values."""
    dt, B, Tq, Tk, H, Hkv, dh = form
    q, k, v = make_cross(B, Tq, Tk, H, Hkv, dh, dt=dt)
    lens = torch.full((B,), Tk, dtype=torch.int32, device=DEV)
    lens[0] = Tk - 45
    qi, ki = (t.float().round().clamp(-2, 2).to(dt) for t in (q, k))
    # the kernels that take the maximum of scaled scores also have negative scales
    for sc in (scale, -scale):
        o, w, _ = cross_ref(qi, ki, v, lens, sc)
        got = api.cross_attention(qi, ki, v, kv_lens=lens, scale=sc)
        # sums of up to Tk values and a division, the low parts of a 3xTF32 product, half a step
        tol = (2 * U * (Tk + 8) + (2.0 ** -20 if dt == F32 else 0)) * w + HALF[dt] * o.abs() * 1.01
        close(got, o, tol)
        got = api.cross_attention(q, k, v, kv_lens=lens, scale=sc).double()
        vd = v.double().repeat_interleave(H // Hkv, 2)
        lo, hi = vd.amin(1, keepdim=True), vd.amax(1, keepdim=True)
        room = 2.0 ** -7 * torch.maximum(lo.abs(), hi.abs())
        assert ((got >= lo - room) & (got <= hi + room)).all()


@pytest.mark.parametrize("dh,Hkv", [(64, 2), (128, 2), (80, 1), (72, 2)])
@pytest.mark.parametrize("Tq", [1, 3, 20, 130])
def test_cross_attention_special_values_where_keys_are_dealt_out(Tq, dh, Hkv):
    """Parts of a long sequence on different CTAs: what lies past the length, keys and whole parts without weight, NaN."""
    B, Tk = 2, 2500
    q, k, v = make_cross(B, Tq, Tk, 2 * Hkv, Hkv, dh)
    lens = torch.tensor([1290, 129], dtype=torch.int32, device=DEV)
    ref = check_cross(q, k, v, lens)
    k2, v2 = k.clone(), v.clone()
    for b, n in enumerate(lens.tolist()):
        k2[b, n:], v2[b, n:] = math.nan, math.nan
        k2[b, n + 1:], v2[b, n + 1:] = math.inf, -math.inf
    assert torch.equal(api.cross_attention(q, k2, v2, kv_lens=lens), ref)
    # scores of minus infinity for all keys but the last ones, or but the first
    q2 = q.abs() + 0.01
    for live in (slice(2300, 2500), slice(0, 100), slice(1200, 1201)):
        k2 = torch.full_like(k, -math.inf)
        k2[:, live] = k[:, live]
        o, w, _ = cross_ref(q2, k[:, live], v[:, live], None, dh ** -0.5)
        close(api.cross_attention(q2, k2, v), o, 2.0 ** -7 * w)
    k2 = torch.full_like(k, -math.inf)
    assert torch.isnan(api.cross_attention(q2, k2, v)).all()
    k2 = k.clone()
    k2[0, 1700, 0] = math.nan
    got, keep = api.cross_attention(q, k2, v), api.cross_attention(q, k, v)
    assert torch.isnan(got[0, :, :2]).all() and torch.equal(got[1], keep[1]) and torch.equal(got[0, :, 2:], keep[0, :, 2:])
    # scores that grow through the parts
    grow = torch.linspace(0, 6, Tk, device=DEV)[None, :, None, None]
    check_cross(q, (k[:, :1].float().expand(-1, Tk, -1, -1) * grow).to(BF), v)


# ----------------------------------------------------------------------- limits of outputs, offsets
def inside(shape, dt, lead, fn):
    """fn(out) with out a contiguous tensor between two margins (the first of `lead` bytes); nothing outside it changes."""
    n = math.prod(shape) * torch.empty(0, dtype=dt).element_size()
    buf = torch.full((lead + n + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    fn(buf[lead:lead + n].view(dt).view(shape))
    assert (buf[:lead] == 0x5A).all() and (buf[lead + n:] == 0x5A).all()


@pytest.mark.parametrize("lead", [4096, 4104])
def test_nothing_outside_the_outputs_is_written(lead):
    for rows, D in ((3, 264), (5, 129), (1501, 1032)):
        x = rand(rows, D, dtype=BF)
        blocks = (rows, (D + 127) // 128)
        inside((rows, D), BF, lead, lambda t: api.rmsnorm(x, 1e-6, out=t))
        inside((rows, D), F8, lead, lambda t: api.rmsnorm(x, 1e-6, out=t))
        inside(blocks, F32, lead, lambda t: api.rmsnorm(x, 1e-6, out_dtype=F8, scales=t))
        inside((rows, D), F32, lead, lambda t: api.rmsnorm(x, 1e-6, residual=x.float(), sum_out=t))
        inside((rows, D), F8, lead, lambda t: api.quantize(x, out=t))
        inside(blocks, F32, lead, lambda t: api.quantize(x, scales=t))
        inside((D, rows), F8, lead, lambda t: api.quantize_weight(x, out=t))
    for M in (3, 29, 45, 333):
        for N in (136, 400, 1032, 5):
            ops = make_product(M, 272, N)
            for dt in (BF, F32, F8):
                inside((M, N), dt, lead, lambda t: api.linear_fp8(*ops, out=t))
            inside((M, (N + 127) // 128), F32, lead, lambda t: api.linear_fp8(*ops, out_dtype=F8, out_scales=t))
    for dt in (BF, F32):
        for Tq, H, Hkv, dh in ((1, 4, 2, 64), (3, 6, 2, 80), (131, 6, 2, 64), (150, 2, 2, 96), (37, 5, 1, 128), (7, 3, 3, 40)):
            q, k, v = make_cross(2, Tq, 333, H, Hkv, dh, dt=dt)
            inside(tuple(q.shape), dt, lead, lambda t: api.cross_attention(q, k, v, out=t))


def big(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(sum(shape)))


def test_rows_past_32_bit_offsets():
    """More than 2^32 elements: the last rows and blocks come out as they do alone."""
    x = big((1 << 21) + 3, 2056)
    q, s = api.quantize(x)
    qe, se = api.quantize(x[-3:])
    assert torch.equal(q[-3:].view(torch.uint8), qe.view(torch.uint8)) and torch.equal(s[-3:], se)
    q, s = api.rmsnorm(x, 1e-6, out=q, scales=s)
    for part in (slice(0, 3), slice(-3, None)):
        y = norm_ref(x[part], None, None, 1e-6)[1]
        close8(q[part], s[part], y, (math.ceil(2056 / 256) + 26) * U * y.abs())
    del x, q, s
    w = big(65544, 65544)
    q, s = api.quantize_weight(w)
    qe, se = api.quantize_weight(w[65408:, 65408:].contiguous())
    assert torch.equal(q[65408:, 65408:].contiguous().view(torch.uint8), qe.view(torch.uint8))
    assert torch.equal(s[511:, 511:], se)


@pytest.mark.parametrize("ot", [BF, F8], ids=str)
def test_product_past_32_bit_offsets(ot):
    a, sa, w, sw = make_product((1 << 17) + 5, 128, 32784)
    got = api.linear_fp8(a, sa, w, sw, out_dtype=ot)
    ref = api.linear_fp8(a[-261:], sa[-261:], w, sw, out_dtype=ot)   # the last whole tile and what is behind it
    for g, r in zip(got, ref) if ot == F8 else ((got, ref),):
        assert torch.equal(g[-261:].view(torch.uint8), r.view(torch.uint8))
    del got, ref
    # a weight of more than 2^32 elements under few rows
    n0, N, K = 1 << 20, (1 << 20) + 72, 4096
    a, sa = api.quantize(rand(3, K))
    w = torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    w[n0:] = api.quantize(rand(72, K, seed=1))[0].view(torch.uint8)
    w, sw = w.view(F8), torch.rand(N // 128 + 1, K // 128, device=DEV) * 1e-3
    got = api.linear_fp8(a, sa, w, sw, out_dtype=F32)
    z, mag = linear_ref(a, sa, w[n0:].contiguous(), sw[n0 // 128:])
    close(got[:, n0:], z, 2 * U * (128 + 32 + 8) * mag)
    assert (got[:, :n0] == 0).all()


@pytest.mark.parametrize("dt,Tq,dh", [(BF, 1, 64), (BF, 150, 128), (F32, 1, 64), (F32, 40, 64), (BF, 20, 72), (F64, 2, 64)], ids=str)
def test_cross_attention_past_32_bit_offsets(dt, Tq, dh):
    """A cache whose sequences, or tokens, lie more than 2^32 elements apart."""
    q, k, v = make_cross(2, Tq, 300, 4, 2, dh, dt=dt)
    lens = torch.tensor([300, 211], dtype=torch.int32, device=DEV)
    for b, t in (((1 << 32) + 64, 2 * dh), (2 * dh, 1 << 24)):
        buf = torch.empty(b + 299 * t + 2 * dh, dtype=dt, device=DEV)
        far = buf.as_strided((2, 300, 2, dh), (b, t, dh, 1))
        far.copy_(k)
        assert torch.equal(api.cross_attention(q, far, v, kv_lens=lens), api.cross_attention(q, k, v, kv_lens=lens))
        far.copy_(v)
        assert torch.equal(api.cross_attention(q, k, far, kv_lens=lens), api.cross_attention(q, k, v, kv_lens=lens))
        del buf, far


@pytest.mark.parametrize("dt,Tq", [(BF, 1 << 21), (F32, 1 << 20)], ids=str)
def test_cross_attention_outputs_past_32_bit_offsets(dt, Tq):
    q = big(1, Tq + 8, 16, 128, dtype=dt)
    _, k, v = make_cross(1, 1, 40, 16, 1, 128, dt=dt)
    got = api.cross_attention(q, k, v)
    assert torch.equal(got[:, -520:], api.cross_attention(q[:, -520:], k, v))


# ------------------------------------------------------------------------------- together
def decoder_layer(p, x, states_kv, lens, H, out=None):
    """One reading layer of a text decoder: x + cross attention over the encoder's states, then the
    feed-forward block, every product in 8 bits and the residual stream in fp32."""
    B, T, D = x.shape
    k, v = states_kv
    q8, qs = api.rmsnorm(x, 1e-6, gamma=p["g1"], out_dtype=F8)
    q = api.linear_fp8(q8, qs, *p["wq"], bias=p["bq"])
    o = api.cross_attention(q.view(B, T, H, D // H), k, v, kv_lens=lens)
    o8, os_ = api.quantize(o.view(B, T, D))
    y = api.linear_fp8(o8, os_, *p["wo"], out_dtype=BF)
    h8, hs, stream = api.rmsnorm(y, 1e-6, gamma=p["g2"], residual=x, out_dtype=F8)
    u8, us = api.linear_fp8(h8, hs, *p["w1"], epilogue=api.EPI_GELU, out_dtype=F8)
    return api.linear_fp8(u8, us, *p["w2"], residual=stream, epilogue=api.EPI_RESIDUAL, out_dtype=F32, out=out)


def make_layer(D, F, Hkv, dh, seed=0):
    def w(k, n, s):
        return api.quantize_weight(rand(k, n, seed=seed + s, std=k ** -0.5, dtype=BF))
    return dict(g1=1 + rand(D, seed=seed + 1, std=0.1), g2=1 + rand(D, seed=seed + 2, std=0.1), wq=w(D, D, 3),
                bq=rand(D, seed=seed + 4, std=0.1, dtype=BF), wo=w(D, D, 5), w1=w(D, F, 6), w2=w(F, D, 7),
                wkv=w(D, 2 * Hkv * dh, 8))


def project_states(p, states, Hkv, dh):
    B, T, D = states.shape
    s8, ss = api.quantize(states)
    kv = api.linear_fp8(s8, ss, *p["wkv"]).view(B, T, 2, Hkv, dh)
    return kv[:, :, 0], kv[:, :, 1]


def layer_ref(p, x, states, lens, H, Hkv, dh):
    """The same from the values that the 8-bit weights stand for, in 64 bits, nothing rounded on the way."""
    val = {n: p[n][0].double() * spread(p[n][1], p[n][0].shape[1], p[n][0].shape[0]) for n in ("wq", "wo", "w1", "w2", "wkv")}
    B, T, D = x.shape
    kv = (states.double() @ val["wkv"].t()).view(B, -1, 2, Hkv, dh)
    s, y = norm_ref(x.view(-1, D), None, p["g1"], 1e-6)
    q = (y @ val["wq"].t() + p["bq"].double()).view(B, T, H, dh)
    o = cross_ref(q, kv[:, :, 0], kv[:, :, 1], lens, dh ** -0.5)[0].reshape(-1, D)
    s, y = norm_ref(o @ val["wo"].t(), x.view(-1, D), p["g2"], 1e-6)
    return (s + gelu64(y @ val["w1"].t()) @ val["w2"].t()).view(B, T, D)


@pytest.mark.parametrize("T", [1, 37])
def test_a_decoder_layer_over_encoder_states(T):
    """Each of the five 8-bit inputs is off by 2^-4 of a value at most, about 2^-5.5 in the mean square; four of them in a
    row, their products averaging independent errors, leave a relative error of about 2 * 2^-5.5, taken as 2^-3 here."""
    B, D, F, H, Hkv, S = 3, 256, 512, 4, 2, 197
    p = make_layer(D, F, Hkv, D // H)
    x, states = rand(B, T, D, seed=20), rand(B, S, D, seed=21, dtype=BF)
    lens = torch.tensor([197, 50, 0], dtype=torch.int32, device=DEV)
    got = decoder_layer(p, x, project_states(p, states, Hkv, D // H), lens, H)
    ref = layer_ref(p, x, states, lens, H, Hkv, D // H)
    assert float((got.double() - ref).norm() / (ref - x.double()).norm()) < 2.0 ** -3


def test_a_captured_layer_replays_on_new_inputs_and_streams_agree():
    B, T, D, F, H, Hkv, S = 2, 1, 256, 512, 4, 2, 577
    p = make_layer(D, F, Hkv, D // H)
    x, states = rand(B, T, D, seed=30), rand(B, S, D, seed=31, dtype=BF)
    lens = torch.tensor([577, 200], dtype=torch.int32, device=DEV)
    kv = project_states(p, states, Hkv, D // H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decoder_layer(p, x, kv, lens, H)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):   # two graphs of the same work, replayed in turn and at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = decoder_layer(p, x, kv, lens, H)
        graphs.append((g, y))
    for seed in (40, 41):
        x.copy_(rand(B, T, D, seed=seed))
        lens.copy_(torch.tensor([577 - seed, seed], dtype=torch.int32))
        eager = decoder_layer(p, x, kv, lens, H)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for _ in range(3):
            for (g, _), st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for _, y in graphs:
            assert torch.equal(y, eager)


def test_calls_on_an_explicit_stream():
    st = torch.cuda.Stream()
    x = rand(50, 256, seed=50, dtype=BF)
    w, sw = api.quantize_weight(rand(256, 384, seed=51, dtype=BF))
    q, k, v = make_cross(2, 20, 90, 4, 2, 64)
    torch.cuda.synchronize()
    q8, s = api.rmsnorm(x, 1e-6, out_dtype=F8, stream=st)
    z = api.linear_fp8(q8, s, w, sw, stream=st.cuda_stream)
    o = api.cross_attention(q, k, v, stream=st)
    st.synchronize()
    q8b, sb = api.rmsnorm(x, 1e-6, out_dtype=F8)
    assert torch.equal(z, api.linear_fp8(q8b, sb, w, sw)) and torch.equal(o, api.cross_attention(q, k, v))


def test_the_binding_refuses_what_does_not_fit():
    x, r = rand(4, 256, dtype=BF), rand(4, 256)
    q8, s = api.quantize(x)
    w, sw = api.quantize_weight(rand(256, 128, dtype=BF))
    q, k, v = make_cross(2, 3, 10, 4, 2, 64)
    bad = [
        lambda: api.rmsnorm(x.t(), 1e-6), lambda: api.rmsnorm(x, 1e-6, gamma=r), lambda: api.rmsnorm(x, 1e-6, sum_out=x),
        lambda: api.rmsnorm(x, 1e-6, residual=r[:2]), lambda: api.rmsnorm(x, 1e-6, scales=s),
        lambda: api.rmsnorm(x.half(), 1e-6), lambda: api.rmsnorm(x, 1e-6, gamma=torch.ones(256)),
        lambda: api.rmsnorm(x[:0], 1e-6), lambda: api.quantize(x.half()), lambda: api.quantize(x[:, ::2]),
        lambda: api.quantize_weight(x[0]), lambda: api.quantize_weight(x.t()), lambda: api.quantize(x, out=x),
        lambda: api.linear_fp8(x, s, w, sw), lambda: api.linear_fp8(q8, s[:2], w, sw),
        lambda: api.linear_fp8(q8, s, w[:, :128], sw), lambda: api.linear_fp8(q8, s, w, sw.t()),
        lambda: api.linear_fp8(q8, s, w, sw, bias=r[0]), lambda: api.linear_fp8(q8, s, w, sw, out_dtype=torch.float16),
        lambda: api.linear_fp8(q8, s, w, sw, out_scales=s), lambda: api.cross_attention(q, k[:1], v),
        lambda: api.cross_attention(q, k, v[:, :5]), lambda: api.cross_attention(q, k.float(), v),
        lambda: api.cross_attention(q, k, v, kv_lens=torch.tensor([1, 2], device=DEV)),
        lambda: api.cross_attention(q, k, v, kv_lens=torch.tensor([1, 2], dtype=torch.int32)),
        lambda: api.cross_attention(q.half(), k.half(), v.half()), lambda: api.cross_attention(q[..., ::2], k, v),
        lambda: api.cross_attention(q, k.transpose(2, 3), v), lambda: api.cross_attention(q[0], k, v),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError("call %d was taken" % i)
    with pytest.raises(api.VitError):
        api.rmsnorm(x, 1e-6, out=x)                                   # over an input
    with pytest.raises(api.VitError):
        api.linear_fp8(q8, s, w, sw, epilogue=api.EPI_RESIDUAL)        # no residual
    with pytest.raises(api.VitError):
        api.cross_attention(q, k, v, out=q)
