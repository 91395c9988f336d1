"""Host-side refusals of the latent attention and verification entry points: every bad call returns
before a GPU is touched (the pointers here are never followed)."""
import ctypes

import pytest
import torch

from kimi_delta_attention_06_gb300 import build as kbuild
from kimi_delta_attention_06_gb300 import kda

BAD, UNSUP, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def _arr(*v):
    a = (ctypes.c_int32 * len(v))(*v)
    return a, ctypes.cast(a, ctypes.c_void_p)


def _call(lib, name, order, base, **over):
    a = dict(base)
    a.update(over)
    return getattr(lib, name)(*(a[k] for k in order))


def test_row_bytes(lib):
    assert kda.kda_latent_row_bytes(kda.KDA_CACHE_BF16) == 1152
    assert kda.kda_latent_row_bytes(kda.KDA_CACHE_E4M3) == 656
    with pytest.raises(kda.KdaError):
        kda.kda_latent_row_bytes(2)


def test_append_refusals(lib):
    order = ["c", "ldc", "r", "ldr", "cache", "dt", "pages", "page", "slots", "T", "st"]
    base = dict(c=0x1000, ldc=576, r=0x2000, ldr=576, cache=0x3000, dt=1, pages=4, page=64, slots=0x4000, T=3, st=None)
    f = lambda **o: _call(lib, "kda_latent_append", order, base, **o)
    for o in (dict(dt=2), dict(pages=-1), dict(page=0), dict(T=-1), dict(ldc=504), dict(ldc=577), dict(ldr=56),
              dict(c=None), dict(r=None), dict(slots=None), dict(cache=None), dict(c=0x1008), dict(r=0x2004),
              dict(cache=0x3008), dict(slots=0x4002), dict(pages=1 << 26)):
        assert f(**o) == BAD, o
    assert f(page=24) == UNSUP and f(page=2048) == UNSUP
    assert f(T=0, c=None, r=None, slots=None) == OK


def test_gather_refusals(lib):
    keep, cu = _arr(0, 5, 9)
    order = ["cache", "dt", "pages", "page", "table", "mp", "start", "cu", "cuh", "N", "T", "c", "ldc", "r", "ldr", "st"]
    base = dict(cache=0x1000, dt=0, pages=4, page=16, table=0x2000, mp=2, start=None, cu=0x3000, cuh=cu, N=2, T=9,
                c=0x4000, ldc=512, r=0x5000, ldr=64, st=None)
    f = lambda **o: _call(lib, "kda_latent_gather", order, base, **o)
    k2, dec = _arr(0, 9, 5)
    k3, off = _arr(1, 5, 9)
    for o in (dict(dt=-1), dict(T=8), dict(N=-1), dict(mp=-1), dict(cu=None), dict(cuh=None), dict(cuh=dec, T=5),
              dict(cuh=off), dict(c=None), dict(r=None), dict(table=None), dict(ldc=511), dict(ldr=63), dict(c=0x4002),
              dict(start=0x6002), dict(table=0x2002), dict(cu=0x3001)):
        assert f(**o) == BAD, o
    assert f(page=8) == UNSUP
    k4, zero = _arr(0, 0, 0)
    assert f(cuh=zero, T=0) == OK and f(N=0, T=0, cu=None, cuh=None) == OK


def test_decode_refusals(lib):
    order = ["q", "cache", "dt", "pages", "page", "table", "mp", "lens", "N", "K", "H", "scale", "out", "lse", "st"]
    base = dict(q=0x1000, cache=0x2000, dt=0, pages=4, page=16, table=0x3000, mp=2, lens=0x4000, N=2, K=1, H=32,
                scale=0.07, out=0x5000, lse=None, st=None)
    f = lambda **o: _call(lib, "kda_latent_decode", order, base, **o)
    for o in (dict(dt=3), dict(N=-1), dict(K=-1), dict(H=0), dict(mp=-1), dict(scale=float("nan")),
              dict(scale=float("inf")), dict(q=None), dict(lens=None), dict(out=None), dict(table=None), dict(q=0x1008),
              dict(out=0x5008), dict(lens=0x4001), dict(lse=0x6002), dict(cache=0x2004), dict(mp=1 << 28),
              dict(N=1 << 30, K=2)):
        assert f(**o) == BAD, o
    assert f(K=17) == UNSUP and f(H=513) == UNSUP and f(page=40) == UNSUP
    assert f(N=0) == OK and f(K=0) == OK


def test_prefill_refusals(lib):
    kq, cq = _arr(0, 5, 9)
    kk, ck = _arr(0, 8, 20)
    order = ["q", "k", "ldk", "hdk", "v", "ldv", "hdv", "r", "ldr", "cq", "cqh", "ck", "ckh", "N", "Tq", "Tk", "H",
             "causal", "scale", "out", "lse", "st"]
    base = dict(q=0x1000, k=0x2000, ldk=512, hdk=256, v=0x3000, ldv=512, hdv=256, r=0x4000, ldr=64, cq=0x5000, cqh=cq,
                ck=0x6000, ckh=ck, N=2, Tq=9, Tk=20, H=2, causal=1, scale=0.07, out=0x7000, lse=None, st=None)
    f = lambda **o: _call(lib, "kda_latent_prefill", order, base, **o)
    for o in (dict(N=-1), dict(Tq=8), dict(Tk=21), dict(H=0), dict(causal=2), dict(scale=float("nan")), dict(q=None),
              dict(k=None), dict(v=None), dict(r=None), dict(out=None), dict(cq=None), dict(ckh=None), dict(q=0x1002),
              dict(k=0x2008), dict(v=0x3004), dict(r=0x4008), dict(out=0x7004), dict(lse=0x8001), dict(ldk=120),
              dict(hdk=100), dict(ldv=516), dict(hdv=0), dict(ldr=60)):
        assert f(**o) == BAD, o
    kz, cz = _arr(0, 0, 0)
    assert f(cqh=cz, Tq=0) == OK and f(N=0, Tq=0, Tk=0, cq=None, cqh=None, ck=None, ckh=None) == OK


def test_verify_refusals(lib):
    order = ["p", "ldp", "q", "ldq", "x", "nd", "u", "us", "N", "K", "V", "t", "m", "st"]
    base = dict(p=0x1000, ldp=100, q=0x2000, ldq=100, x=0x3000, nd=None, u=0x4000, us=0x5000, N=2, K=3, V=100, t=0x6000,
                m=0x7000, st=None)
    f = lambda **o: _call(lib, "kda_verify_draft", order, base, **o)
    for o in (dict(N=-1), dict(K=-1), dict(V=0), dict(ldp=99), dict(ldq=99), dict(p=None), dict(x=None), dict(u=None),
              dict(us=None), dict(t=None), dict(m=None), dict(p=0x1002), dict(nd=0x8001)):
        assert f(**o) == BAD, o
    assert f(K=kda.KDA_VERIFY_MAX_DRAFT + 1) == UNSUP
    assert f(N=0) == OK


def test_python_binding_checks_types_and_layouts(lib):
    c = torch.zeros(4, 512, dtype=torch.bfloat16)
    r = torch.zeros(4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 16, 656, dtype=torch.uint8)
    slots = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):                            # rows of the other format
        kda.kda_latent_append(c, r, cache, kda.KDA_CACHE_BF16, slots, 4, stream=0)
    with pytest.raises(TypeError):
        kda.kda_latent_append(c, r, cache, kda.KDA_CACHE_E4M3, slots.long(), 4, stream=0)
    with pytest.raises(TypeError):
        kda.kda_latent_append(c.float(), r, cache, kda.KDA_CACHE_E4M3, slots, 4, stream=0)
    with pytest.raises(ValueError):                            # columns must be contiguous
        kda.kda_latent_append(torch.zeros(512, 4, dtype=torch.bfloat16).t(), r, cache, kda.KDA_CACHE_E4M3, slots, 4, stream=0)
    p = torch.zeros(4, 3, 8)[::2]                              # rows of consecutive sequences unevenly spaced
    with pytest.raises(ValueError):
        kda.kda_verify_draft(p, None, slots, None, p, p, 2, 2, 8, slots, slots, stream=0)
    p = torch.zeros(1, 3, 8).expand(2, 3, 8)                    # one sequence's rows for all
    with pytest.raises(ValueError):
        kda.kda_verify_draft(p, None, slots, None, p, p, 2, 2, 8, slots, slots, stream=0)
    with pytest.raises(TypeError):
        kda.kda_verify_draft(p.double(), None, slots, None, p, p, 2, 2, 8, slots, slots, stream=0)
