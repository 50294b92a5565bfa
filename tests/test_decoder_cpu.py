"""Refusals of the rotary positions, the paged cache and the attention over it, on the CPU: the C entry points answer before
any CUDA call, the binding before any C call."""
import ctypes

import pytest
import torch

from vision_transformer_encoder_gb300 import api, build

ARG, DTYPE, CUDA, UNSUPPORTED = -1, -2, -3, -6
F32, BF16, F64, E4M3 = 0, 1, 2, 3
VP, I64 = ctypes.c_void_p, ctypes.c_int64


class Rope(ctypes.Structure):
    _fields_ = [("frequencies", VP), ("n", I64), ("layout", ctypes.c_int), ("scale", ctypes.c_double)]


class Cache(ctypes.Structure):
    _fields_ = [("k", VP), ("v", VP), ("k_strides", I64 * 3), ("v_strides", I64 * 3), ("pages", I64), ("page", I64),
                ("heads", I64), ("dh", I64), ("dtype", ctypes.c_int)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def at(i, offset=0):
    """A made-up device address, far from the others; validation fails before it is used."""
    return 0x1000000000 * (i + 1) + offset


def strides(s):
    return None if s is None else (I64 * 3)(*s)


def rope(f=at(9), n=32, layout=0, scale=1.0):
    return ctypes.byref(Rope(f, n, layout, scale))


def rotary(lib, x=at(0), xs=None, pos=at(1), r="own", B=2, T=3, H=4, dh=64, d=BF16, out=at(2), **kw):
    r = rope(**kw) if r == "own" else r
    return lib.vit_rotary(x, strides(xs), pos, r, B, T, H, dh, d, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ARG), (dict(out=None), ARG), (dict(r=None), ARG), (dict(B=0), ARG), (dict(T=-1), ARG), (dict(H=0), ARG),
    (dict(dh=0), ARG), (dict(H=65537), ARG), (dict(dh=513), UNSUPPORTED), (dict(d=E4M3), DTYPE), (dict(d=7), DTYPE),
    (dict(f=None), ARG), (dict(n=0), ARG), (dict(n=33), ARG), (dict(layout=2), ARG), (dict(layout=-1), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(scale=1e31), ARG), (dict(f=at(9, 4)), ARG),
    (dict(B=1 << 45), ARG), (dict(xs=(-192, 64, 64)), ARG), (dict(xs=(1 << 60, 256, 64)), ARG), (dict(x=at(0, 1)), ARG),
    (dict(out=at(0, 2)), ARG), (dict(out=at(0, 128)), ARG), (dict(out=at(1)), ARG), (dict(out=at(9)), ARG), (dict(pos=at(1, 2)), ARG),
    (dict(out=at(0), xs=(768, 256, 0)), ARG), (dict(out=at(0), xs=(512, 256, 64)), ARG),   # in place, rows upon each other
])
def test_rotary_refuses(lib, kw, code):
    assert rotary(lib, **kw) == code


def cache(k=at(10), v=at(11), ks=None, vs=None, pages=50, page=16, heads=2, dh=64, d=BF16):
    own = (page * heads * dh, heads * dh, dh)
    return Cache(k, v, strides(ks or own), strides(vs or own), pages, page, heads, dh, d)


CACHES = [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(pages=0), ARG), (dict(page=0), ARG), (dict(heads=0), ARG), (dict(dh=0), ARG),
    (dict(pages=1 << 31), ARG), (dict(page=1 << 31), ARG), (dict(heads=65537), ARG), (dict(dh=513), UNSUPPORTED), (dict(d=E4M3), DTYPE), (dict(d=-1), DTYPE),
    (dict(ks=(0, 128, 64)), ARG), (dict(vs=(2048, -128, 64)), ARG), (dict(vs=(2048, 128, 0)), ARG), (dict(ks=(1 << 50, 128, 64)), ARG),
    (dict(k=at(10, 1)), ARG), (dict(v=at(11, 1)), ARG), (dict(pages=1 << 30, page=1 << 20), ARG),
]
POOLS = [   # refused where the pools are written
    (dict(v=at(10)), ARG), (dict(v=at(10, 2 * 2048)), ARG), (dict(v=at(10, 2 * 63)), ARG),         # upon each other
    (dict(ks=(1024, 128, 64)), ARG), (dict(vs=(2048, 128, 32)), ARG),                               # a pool upon itself
    (dict(v=at(10, 4096), ks=(4096, 128, 64), vs=(4096, 64, 1024)), ARG),                           # different strides in one buffer
    (dict(v=at(10, 4096 - 2), ks=(4096, 128, 64), vs=(4096, 128, 64)), ARG),
]


def append(lib, k=at(0), ks=None, v=at(1), vs=None, q=at(2), qs=None, c=None, table=at(3), tp=8, starts=at(4), lens=at(5), r="own",
           pos=at(6), B=2, T=3, H=4, qo=at(7)):
    r = rope() if r == "own" else r
    c = cache() if c is None else c
    return lib.vit_cache_append(k, strides(ks), v, strides(vs), q, strides(qs), ctypes.byref(c) if c else None, table, tp, starts, lens, r, pos, B, T, H, qo, None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(c=0), ARG), (dict(table=None), ARG), (dict(starts=None), ARG), (dict(B=0), ARG),
    (dict(T=0), ARG), (dict(tp=0), ARG), (dict(q=None), ARG), (dict(qo=None), ARG), (dict(H=0), ARG), (dict(H=1 << 20), ARG),
    (dict(r=rope(n=40)), ARG), (dict(r=rope(f=None)), ARG), (dict(r=rope(layout=3)), ARG), (dict(r=rope(scale=float("inf"))), ARG),
    (dict(ks=(-1, 128, 64)), ARG), (dict(vs=(1 << 60, 128, 64)), ARG), (dict(k=at(0, 1)), ARG), (dict(v=at(1, 1)), ARG), (dict(q=at(2, 1)), ARG),
    (dict(table=at(3, 1)), ARG), (dict(starts=at(4, 2)), ARG), (dict(lens=at(5, 2)), ARG), (dict(pos=at(6, 1)), ARG),
    (dict(k=at(10)), ARG), (dict(v=at(11, 128)), ARG), (dict(q=at(10, 256)), ARG), (dict(qo=at(11)), ARG), (dict(table=at(10)), ARG),
    (dict(starts=at(11)), ARG), (dict(qo=at(0)), ARG), (dict(qo=at(1, 64)), ARG), (dict(qo=at(2, 64)), ARG), (dict(qo=at(4)), ARG),
    (dict(qo=at(6)), ARG), (dict(qo=at(9)), ARG), (dict(B=1 << 44), ARG), (dict(tp=1 << 46), ARG),
    (dict(qo=at(2), qs=(768, 256, 0)), ARG), (dict(qo=at(2), k=at(2, 2 * 255), qs=(2048, 512, 64), ks=(2048, 512, 64)), ARG),   # in place, upon k
])
def test_cache_append_refuses(lib, kw, code):
    assert append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", CACHES + POOLS)
def test_cache_append_refuses_pools(lib, kw, code):
    assert append(lib, c=cache(**kw)) == code


def test_cache_append_takes_pools_and_projections_side_by_side(lib):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: a CUDA device is present")
    for kw in (dict(), dict(v=at(10, 4096), ks=(4096, 128, 64), vs=(4096, 128, 64)),         # in a page
               dict(v=at(10, 256), ks=(4096, 256, 64), vs=(4096, 256, 64)),                  # in a token
               dict(v=at(10, 128), ks=(4096, 256, 128), vs=(4096, 256, 128)),                # in a head
               dict(ks=(2048, 64, 1024), vs=(2048, 64, 1024))):                              # heads before tokens
        assert append(lib, c=cache(**kw)) == CUDA
    st = (3 * 512, 512, 64)   # queries (four heads), keys and values (two) of one projection, turned in place
    assert append(lib, q=at(0), qo=at(0), k=at(0, 512), v=at(0, 768), qs=st, ks=st, vs=st) == CUDA
    assert append(lib, q=at(0), qo=at(0), k=at(0, 510), v=at(0, 768), qs=st, ks=st, vs=st) == ARG


def paged(lib, q=at(0), qs=None, c=None, table=at(1), tp=8, kv=at(2), ql=at(3), pt=at(4), pp=5, pl=at(5), groups=2, B=4, Tq=3, H=4,
          scale=0.125, o=at(6)):
    c = cache() if c is None else c
    return lib.vit_paged_attention(q, strides(qs), ctypes.byref(c) if c else None, table, tp, kv, ql, pt, pp, pl, groups, B, Tq, H, scale, o, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(c=0), ARG), (dict(table=None), ARG), (dict(kv=None), ARG), (dict(o=None), ARG), (dict(B=0), ARG),
    (dict(Tq=0), ARG), (dict(H=0), ARG), (dict(H=3), ARG), (dict(tp=0), ARG), (dict(pt=None), ARG), (dict(pl=None), ARG), (dict(pp=0), ARG),
    (dict(pt=None, pl=None), ARG), (dict(pt=None, pl=None, pp=0), ARG), (dict(groups=0), ARG), (dict(groups=3), ARG), (dict(groups=-2), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=-float("inf")), ARG), (dict(scale=1e31), ARG), (dict(tp=1 << 27), ARG), (dict(pp=1 << 27), ARG),
    (dict(qs=(-1, 256, 64)), ARG), (dict(q=at(0, 1)), ARG), (dict(table=at(1, 2)), ARG), (dict(kv=at(2, 1)), ARG), (dict(ql=at(3, 1)), ARG),
    (dict(pt=at(4, 1)), ARG), (dict(pl=at(5, 1)), ARG), (dict(o=at(6, 1)), ARG),
    (dict(o=at(0)), ARG), (dict(o=at(10, 512)), ARG), (dict(o=at(11)), ARG), (dict(o=at(1)), ARG), (dict(o=at(2)), ARG), (dict(o=at(3)), ARG),
    (dict(o=at(4)), ARG), (dict(o=at(5)), ARG), (dict(B=1 << 44), ARG), (dict(Tq=1 << 45), ARG), (dict(H=1 << 20), ARG),
])
def test_paged_attention_refuses(lib, kw, code):
    assert paged(lib, **kw) == code


@pytest.mark.parametrize("kw,code", CACHES)
def test_paged_attention_refuses_pools(lib, kw, code):
    assert paged(lib, c=cache(**kw)) == code


def test_without_a_device_the_calls_report_a_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    assert rotary(lib) == CUDA and rotary(lib, pos=None) == CUDA and rotary(lib, out=at(0)) == CUDA
    assert append(lib) == CUDA and append(lib, q=None, qo=None, H=0, r=None, pos=None, lens=None) == CUDA
    assert append(lib, q=at(2), qo=at(2)) == CUDA
    assert paged(lib) == CUDA and paged(lib, pt=None, pl=None, pp=0, groups=1, ql=None) == CUDA
    assert paged(lib, c=cache(v=at(10, 4096), ks=(4096, 128, 64), vs=(4096, 128, 64))) == CUDA   # pools side by side are read


def test_the_binding_refuses_host_tensors():
    x, s = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    f, t = api.rotary_frequencies(64), torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: api.rotary(x, f), lambda: api.cache_append(x, x, x, x, t, s), lambda: api.paged_attention(x, x, x, t, s),
                 lambda: api.rotary(x, f, stream=1)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("layout", [1 << 32, -(1 << 32), 2])
def test_the_binding_refuses_layouts_past_32_bits(layout):
    x = torch.empty(2, 3, 4, 64, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError):
        api.rotary(x, x, layout=layout)


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("kernel", "prefix_kernel", "own_parts", "prefix_parts", "own_rows", "prefix_rows", "launches")]
    _fields_ += [("scratch", I64)]


def plan(lib, p="own", q=at(0), qs=None, c=None, table=at(1), tp=8, kv=at(2), ql=at(3), pt=at(4), pp=5, pl=at(5), groups=2, B=4, Tq=3, H=4,
         scale=0.125, o=at(6)):
    c = cache() if c is None else c
    p = ctypes.byref(Plan()) if p == "own" else p
    return lib.vit_paged_attention_plan(q, strides(qs), ctypes.byref(c) if c else None, table, tp, kv, ql, pt, pp, pl, groups, B, Tq, H, scale, o, p)


@pytest.mark.parametrize("kw", [
    dict(p=None), dict(q=None), dict(c=0), dict(table=None), dict(kv=None), dict(o=None), dict(B=0), dict(Tq=0), dict(H=3), dict(tp=0),
    dict(pl=None), dict(pp=0), dict(groups=3), dict(scale=float("nan")), dict(tp=1 << 27), dict(qs=(-1, 256, 64)), dict(q=at(0, 1)),
    dict(o=at(10, 512)), dict(B=1 << 44), dict(c=cache(page=0)), dict(c=cache(k=at(10, 1)))], ids=str)
def test_the_plan_of_paged_attention_refuses_what_the_call_refuses(lib, kw):
    assert plan(lib, **kw) == ARG


def test_the_plan_of_paged_attention_needs_a_device(lib):
    assert plan(lib, c=cache(dh=513)) == UNSUPPORTED and plan(lib, c=cache(d=E4M3)) == DTYPE
    if not torch.cuda.is_available():
        assert plan(lib) == CUDA and plan(lib, pt=None, pl=None, pp=0, groups=1, ql=None) == CUDA
    x, s = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.paged_attention_plan(x, x, x, torch.zeros(2, 1, dtype=torch.int32), s)


@pytest.mark.parametrize("kw", [
    dict(base=float("nan")), dict(base=0.0), dict(base=-2.0), dict(factor=float("nan")), dict(factor=-1.0), dict(trained=float("nan")),
    dict(trained=4096, slow=float("-inf")), dict(trained=4096, slow=float("nan")), dict(trained=4096, slow=32.0),
    dict(base=1e-300, width=512, factor=1e-30)], ids=str)
def test_rotary_frequencies_are_finite_or_refused(kw):
    """The kernels take finite frequencies only, and cannot look at them before they run."""
    kw = dict(dict(width=64, factor=8.0), **kw)
    with pytest.raises(ValueError):
        api.rotary_frequencies(**kw)


def test_rotary_frequencies_that_are_taken():
    for kw in (dict(), dict(factor=0.25), dict(factor=8, trained=1), dict(factor=8, trained=4096.0, slow=-1, fast=0.5), dict(factor=float("inf")), dict(trained=float("inf")), dict(base=0.5), dict(width=2, base=1e300)):
        f = api.rotary_frequencies(**dict(dict(width=64), **kw))
        assert f.dtype == torch.float64 and torch.isfinite(f).all()
