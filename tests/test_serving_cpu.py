"""Refusals of the serving stages (rms norm, 8-bit quantisation and product, cross attention),
on the CPU: the C entry points answer before any CUDA call, the binding before any C call."""
import ctypes

import pytest
import torch

from vision_transformer_encoder_gb300 import api, build

ARG, DTYPE, UNSUPPORTED = -1, -2, -6
F32, BF16, F64, E4M3 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def at(i, offset=0):
    """A made-up device address, far from the others; validation fails before it is used."""
    return 0x100000000 * (i + 1) + offset


def norm(lib, x=at(0), xd=BF16, res=at(1), rd=BF16, rows=4, D=256, gamma=at(2), gd=BF16, sum_=at(3), out=at(4),
         od=E4M3, scales=at(5)):
    return lib.vit_rmsnorm(x, xd, res, rd, rows, D, 1e-6, gamma, gd, sum_, out, od, scales, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(out=None), ARG), (dict(rows=0), ARG), (dict(D=-1), ARG),
    (dict(rows=1 << 40, D=1 << 20), ARG),
    (dict(res=None), ARG),                                       # a sum without a residual
    (dict(scales=None), ARG), (dict(od=BF16), ARG),              # scales belong to e4m3 alone
    (dict(xd=7), DTYPE), (dict(xd=E4M3), DTYPE), (dict(od=F64), DTYPE), (dict(rd=F64), DTYPE),
    (dict(xd=F32), DTYPE),                                       # bf16 residual of an fp32 x
    (dict(gd=F64), DTYPE), (dict(gd=E4M3), DTYPE),
    (dict(xd=F64, rd=F64, gd=F64), DTYPE),                       # fp64 goes to fp64 alone
    (dict(out=at(0)), ARG), (dict(out=at(1, 64)), ARG), (dict(out=at(3)), ARG), (dict(scales=at(4, 8)), ARG),
    (dict(sum_=at(1, 2)), ARG), (dict(sum_=at(0, 2)), ARG), (dict(sum_=at(2)), ARG),   # shifted, or over gamma
    (dict(sum_=at(0), rd=F32), ARG),                             # over an x of another type
    (dict(x=at(0, 1)), ARG), (dict(scales=at(5, 2)), ARG), (dict(rd=F32, res=at(1, 2)), ARG),
])
def test_rmsnorm_refuses(lib, kw, code):
    assert norm(lib, **kw) == code


@pytest.mark.parametrize("eps,types", [(float("nan"), (BF16, BF16)), (float("inf"), (F32, F32)), (1e39, (BF16, F32)),
                                       (1e-50, (BF16, BF16)), (-1e300, (F32, F32)), (float("inf"), (F64, F64))])
def test_rmsnorm_refuses_eps_that_its_arithmetic_does_not_hold(lib, eps, types):
    xd, rd = types
    od = F64 if xd == F64 else F32
    assert lib.vit_rmsnorm(at(0), xd, at(1), rd, 4, 256, eps, None, xd, None, at(4), od, None, None) == ARG


@pytest.mark.parametrize("eps,xd", [(0.0, BF16), (1e-44, F32), (3e38, BF16), (1e300, F64), (1e-300, F64), (-1e-6, F32)])
def test_rmsnorm_takes_every_other_eps(lib, eps, xd):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: a CUDA device is present")
    assert lib.vit_rmsnorm(at(0), xd, None, xd, 4, 256, eps, None, xd, None, at(4), xd, None, None) == -3


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(q=None), ARG), (dict(s=None), ARG), (dict(rows=0), ARG), (dict(K=0), ARG),
    (dict(d=F64), DTYPE), (dict(d=E4M3), DTYPE), (dict(q=at(0)), ARG), (dict(s=at(1)), ARG), (dict(x=at(0, 1)), ARG),
    (dict(s=at(2, 1)), ARG), (dict(rows=1 << 45, K=1 << 10), ARG),
])
def test_quantize_refuses(lib, kw, code):
    a = dict(x=at(0), d=BF16, rows=4, K=256, q=at(1), s=at(2)) | kw
    assert lib.vit_quantize(a["x"], a["d"], a["rows"], a["K"], a["q"], a["s"], None) == code
    assert lib.vit_quantize_weight(a["x"], a["d"], a["rows"], a["K"], a["q"], a["s"], None) == code


def linear(lib, a=at(0), sa=at(1), w=at(2), sw=at(3), bias=at(4), bd=BF16, res=None, rd=BF16, M=4, K=256, N=256, epi=0,
           out=at(6), od=BF16, so=None):
    return lib.vit_linear_fp8(a, sa, w, sw, bias, bd, res, rd, M, K, N, epi, out, od, so, None)


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), ARG), (dict(sa=None), ARG), (dict(w=None), ARG), (dict(sw=None), ARG), (dict(out=None), ARG),
    (dict(M=0), ARG), (dict(K=0), ARG), (dict(N=-3), ARG), (dict(M=1 << 40, K=1 << 10), ARG),
    (dict(epi=3), ARG), (dict(epi=-1), ARG), (dict(epi=2), ARG), (dict(res=at(5)), ARG),   # residual and its epilogue
    (dict(od=F64), DTYPE), (dict(bd=F64), DTYPE), (dict(epi=2, res=at(5), rd=F64), DTYPE),
    (dict(od=E4M3), ARG), (dict(so=at(7)), ARG),                                         # scales with e4m3 alone
    (dict(out=at(0)), ARG), (dict(out=at(2, 16)), ARG), (dict(out=at(4)), ARG), (dict(out=at(1)), ARG),
    (dict(od=E4M3, so=at(6)), ARG), (dict(od=E4M3, so=at(3)), ARG),
    (dict(epi=2, res=at(6, 2)), ARG), (dict(epi=2, res=at(6), rd=F32), ARG),             # shifted, or of another type
    (dict(sa=at(1, 1)), ARG), (dict(out=at(6, 1)), ARG), (dict(bias=at(4, 1)), ARG),
])
def test_linear_fp8_refuses(lib, kw, code):
    assert linear(lib, **kw) == code


def cross(lib, q=at(0), qs=None, k=at(1), ks=None, v=at(2), vs=None, lens=at(3), B=2, Tq=3, Tk=5, H=4, Hkv=2, dh=64,
          scale=0.125, d=BF16, o=at(4)):
    st = [None if s is None else (ctypes.c_int64 * 3)(*s) for s in (qs, ks, vs)]
    return lib.vit_cross_attention(q, st[0], k, st[1], v, st[2], lens, B, Tq, Tk, H, Hkv, dh, scale, d, o, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(o=None), ARG),
    (dict(B=0), ARG), (dict(Tq=0), ARG), (dict(Tk=0), ARG), (dict(H=0), ARG), (dict(Hkv=0), ARG), (dict(dh=0), ARG),
    (dict(Hkv=3), ARG),                                          # does not divide H
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(d=E4M3), DTYPE), (dict(d=9), DTYPE), (dict(dh=513), UNSUPPORTED),
    (dict(o=at(0)), ARG), (dict(o=at(1, 128)), ARG), (dict(o=at(3)), ARG),
    (dict(ks=(-640, 128, 64)), ARG), (dict(ks=(1 << 60, 128, 64)), ARG),
    (dict(ks=(1 << 20, 128, 64), o=at(1, (1 << 21) + 64)), ARG),  # between the strided rows of k
    (dict(q=at(0, 1)), ARG), (dict(lens=at(3, 2)), ARG), (dict(Tk=1 << 45), ARG), (dict(B=1 << 40), ARG),
])
def test_cross_attention_refuses(lib, kw, code):
    assert cross(lib, **kw) == code


@pytest.mark.parametrize("d", [BF16, F32])
@pytest.mark.parametrize("scale", [1e300, -1e39, 3e38])
def test_cross_attention_refuses_scales_past_fp32(lib, d, scale):
    assert cross(lib, scale=scale, d=d) == ARG


def test_without_a_device_the_stages_report_a_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    assert norm(lib) == -3 and linear(lib) == -3 and cross(lib) == -3
    assert lib.vit_quantize(at(0), BF16, 4, 256, at(1), at(2), None) == -3


def test_the_binding_refuses_host_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q = torch.zeros(4, 256, dtype=torch.float8_e4m3fn)
    s = torch.zeros(4, 2)
    with pytest.raises(ValueError):
        api.rmsnorm(x, 1e-6)
    with pytest.raises(ValueError):
        api.quantize(x)
    with pytest.raises(ValueError):
        api.quantize_weight(x)
    with pytest.raises(ValueError):
        api.linear_fp8(q, s, q, s)
    with pytest.raises(ValueError):
        api.cross_attention(x.view(1, 4, 4, 64), x.view(1, 4, 4, 64), x.view(1, 4, 4, 64))


@pytest.mark.parametrize("epilogue", [1 << 32, (1 << 32) + 1, -(1 << 32)])
def test_the_binding_refuses_epilogues_past_32_bits(epilogue):
    q = torch.empty(4, 256, dtype=torch.float8_e4m3fn, device="meta")
    with pytest.raises(ValueError, match="epilogue"):
        api.linear_fp8(q, q, q, q, epilogue=epilogue)
