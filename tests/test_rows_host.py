"""Refusals of the entry points around a cached latent row, before any launch (no GPU):
pointers are fake, aligned addresses that are never dereferenced.  The 64-bit forms the
GPU tests compare with are checked here against automatic differentiation and numerical
differences."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import rows_util as ru

A = 0x10000000


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_13_gb300 import _build, kda
    _build.build_library()
    return kda.library()


def _p(x):
    return ctypes.c_void_p(x)


ROPE = dict(x=A, xts=4 * 192, xhs=192, out=2 * A, ots=4 * 64, ohs=64, k=3 * A, kts=576, ko=4 * A,
            kots=64, pos=5 * A, freq=6 * A, n=10, H=4, dr=64, inter=1, scale=1.0, tr=0, dtype=1)


def _rope(lib, **over):
    x = dict(ROPE, **over)
    return lib.kda_rope(_p(x["x"]), x["xts"], x["xhs"], _p(x["out"]), x["ots"], x["ohs"],
                        _p(x["k"]), x["kts"], _p(x["ko"]), x["kots"], _p(x["pos"]), _p(x["freq"]),
                        x["n"], x["H"], x["dr"], x["inter"], x["scale"], x["tr"], x["dtype"], None)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(pos=None), 1), (dict(freq=None), 1),
    (dict(k=None), 1), (dict(ko=None), 1), (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(H=0), 1),
    (dict(H=65536), 1), (dict(dr=0), 1), (dict(dr=63), 1), (dict(dr=514), 2), (dict(dtype=2), 2),
    (dict(x=A + 1), 1), (dict(ko=4 * A + 1), 1), (dict(pos=5 * A + 2), 1), (dict(freq=6 * A + 4), 1),
    (dict(xts=-1), 1), (dict(ohs=-64), 1), (dict(ohs=32), 1), (dict(ots=64), 1), (dict(kots=32), 1),
    (dict(ots=0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(out=A), 1),                              # in place, but rows elsewhere
    (dict(out=A + 2, ots=768, ohs=192), 1),        # one channel further: rows meet
    (dict(out=A + 64, ots=768, ohs=192), 1),       # half a row further
    (dict(ko=3 * A + 64, kots=576), 1),
    (dict(ko=2 * A), 1), (dict(out=3 * A), 1),     # on the other output, on the other input
    (dict(ko=A + 64, kots=768), 1),                # on rows of x
    (dict(out=5 * A), 1), (dict(out=6 * A - 64), 1)])
def test_rope_refuses(lib, over, code):
    assert _rope(lib, **over) == code


def test_rope_of_no_tokens_launches_nothing(lib):
    assert _rope(lib, n=0) == 0


NORM = dict(x=A, xrs=576, w=2 * A, b=3 * A, n=10, W=512, dtype=1, center=1, eps=1e-5, out=4 * A,
            ors=512, mean=5 * A, rstd=6 * A)


def _norm(lib, **over):
    x = dict(NORM, **over)
    return lib.kda_norm_fwd(_p(x["x"]), x["xrs"], _p(x["w"]), _p(x["b"]), x["n"], x["W"], x["dtype"],
                            x["center"], x["eps"], _p(x["out"]), x["ors"], _p(x["mean"]),
                            _p(x["rstd"]), None)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(W=0), 1),
    (dict(W=16385), 2), (dict(dtype=7), 2), (dict(center=0), 1), (dict(eps=0.0), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(x=A + 1), 1), (dict(w=2 * A + 2), 1), (dict(mean=5 * A + 2), 1), (dict(xrs=-8), 1),
    (dict(ors=511), 1), (dict(ors=0), 1), (dict(out=A), 1), (dict(out=A + 512, ors=576), 1),
    (dict(out=2 * A), 1), (dict(mean=6 * A), 1), (dict(rstd=A + 16), 1), (dict(rstd=4 * A), 1),
    (dict(mean=2 * A), 1)])
def test_norm_refuses(lib, over, code):
    assert _norm(lib, **over) == code


def test_norm_of_no_rows_launches_nothing(lib):
    assert _norm(lib, n=0) == 0


NGRAD = dict(g=A, grs=512, x=2 * A, xrs=576, w=3 * A, mean=4 * A, rstd=5 * A, n=10, W=512, dtype=1,
             dx=6 * A, dxrs=576, dw=7 * A, db=8 * A, ws=9 * A, wsb=1 << 30)


def _ngrad(lib, **over):
    x = dict(NGRAD, **over)
    return lib.kda_norm_bwd(_p(x["g"]), x["grs"], _p(x["x"]), x["xrs"], _p(x["w"]), _p(x["mean"]),
                            _p(x["rstd"]), x["n"], x["W"], x["dtype"], _p(x["dx"]), x["dxrs"],
                            _p(x["dw"]), _p(x["db"]), _p(x["ws"]), x["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(g=None), 1), (dict(x=None), 1), (dict(rstd=None), 1), (dict(dx=None), 1),
    (dict(n=-1), 1), (dict(W=0), 1), (dict(W=20000), 2), (dict(dtype=3), 2), (dict(g=A + 1), 1),
    (dict(rstd=5 * A + 1), 1), (dict(dw=7 * A + 2), 1), (dict(grs=-1), 1), (dict(dxrs=500), 1),
    (dict(dx=A), 1), (dict(dx=2 * A + 512), 1), (dict(dw=8 * A), 1), (dict(dw=3 * A), 1),
    (dict(db=A), 1), (dict(dx=5 * A), 1), (dict(ws=None), 3), (dict(ws=9 * A + 8), 3),
    (dict(wsb=100), 3)])
def test_norm_gradient_refuses(lib, over, code):
    assert _ngrad(lib, **over) == code


def test_norm_gradient_workspace(lib):
    n = ctypes.c_size_t(0)
    assert lib.kda_norm_bwd_workspace_size(100, 512, 1, ctypes.byref(n)) == 0
    assert 0 < n.value <= 100 * 8 * 512
    assert lib.kda_norm_bwd_workspace_size(0, 512, 1, ctypes.byref(n)) == 0 and n.value == 0
    for args, code in (((-1, 512, 1), 1), ((1, 0, 1), 1), ((1, 16385, 1), 2), ((1, 8, 9), 2)):
        assert lib.kda_norm_bwd_workspace_size(*args, ctypes.byref(n)) == code
    assert lib.kda_norm_bwd_workspace_size(1, 8, 1, None) == 1


WEI = dict(q=A, cache=2 * A, table=3 * A, lens=4 * A, mask=5 * A, lse=6 * A, B=3, T=4, H=8, dc=512,
           dr=64, n_pages=100, page=64, max_pages=20, dtype=1, scale=0.1, decay=1.0, w=7 * A,
           ws=8 * A, wsb=1 << 30)


def _wei(lib, **over):
    x = dict(WEI, **over)
    return lib.kda_latent_weights(_p(x["q"]), _p(x["cache"]), _p(x["table"]), _p(x["lens"]),
                                  _p(x["mask"]), _p(x["lse"]), x["B"], x["T"], x["H"], x["dc"],
                                  x["dr"], x["n_pages"], x["page"], x["max_pages"], x["dtype"],
                                  x["scale"], x["decay"], _p(x["w"]), _p(x["ws"]), x["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(cache=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(lse=None), 1), (dict(w=None), 1), (dict(B=-1), 1), (dict(B=65536), 1), (dict(T=0), 1),
    (dict(T=65), 1), (dict(H=0), 1), (dict(H=1 << 24), 1), (dict(dc=256), 2), (dict(dr=32), 2),
    (dict(dtype=0), 2), (dict(n_pages=0), 1), (dict(page=24), 1), (dict(max_pages=0), 1),
    (dict(max_pages=1 << 25), 1), (dict(q=A + 8), 1), (dict(cache=2 * A + 4), 1),
    (dict(mask=5 * A + 4), 1), (dict(w=7 * A + 2), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(decay=-0.5), 1), (dict(decay=float("inf")), 1),
    (dict(decay=float("nan")), 1), (dict(w=6 * A), 1), (dict(w=2 * A + 64), 1), (dict(ws=None), 3),
    (dict(ws=8 * A + 8), 3), (dict(wsb=64), 3)])
def test_weights_refuse(lib, over, code):
    assert _wei(lib, **over) == code


EV = dict(cache=A, table=2 * A, lens=3 * A, w=4 * A, wo=5 * A, L=2, n_pages=100, page=64, rb=1152,
          B=3, max_pages=20, budget=100, first=4, recent=16, nl=6 * A, orig=7 * A, ws=8 * A,
          wsb=1 << 30, st=9 * A)


def _ev(lib, **over):
    x = dict(EV, **over)
    return lib.kda_cache_evict(_p(x["cache"]), _p(x["table"]), _p(x["lens"]), _p(x["w"]),
                               _p(x["wo"]), x["L"], x["n_pages"], x["page"], x["rb"], x["B"],
                               x["max_pages"], x["budget"], x["first"], x["recent"], _p(x["nl"]),
                               _p(x["orig"]), _p(x["ws"]), x["wsb"], _p(x["st"]), None)


@pytest.mark.parametrize("over,code", [
    (dict(cache=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(w=None), 1),
    (dict(wo=None), 1), (dict(nl=None), 1), (dict(orig=None), 1), (dict(L=0), 1), (dict(B=-1), 1),
    (dict(n_pages=0), 1), (dict(page=0), 1), (dict(rb=8), 1), (dict(rb=0), 1),
    (dict(max_pages=0), 1), (dict(max_pages=1 << 25), 1), (dict(n_pages=1 << 25), 1), (dict(budget=0), 1),
    (dict(budget=(1 << 30) + 1), 1), (dict(first=-1), 1), (dict(recent=-1), 1),
    (dict(first=90, recent=11), 1), (dict(cache=A + 8), 1), (dict(w=4 * A + 2), 1),
    (dict(st=9 * A + 2), 1), (dict(wo=4 * A + 64), 1), (dict(wo=A), 1), (dict(nl=3 * A), 1),
    (dict(orig=6 * A), 1), (dict(orig=4 * A), 1), (dict(ws=None), 3), (dict(ws=8 * A + 4), 3),
    (dict(wsb=100), 3)])
def test_evict_refuses(lib, over, code):
    assert _ev(lib, **over) == code


FAR = (1 << 31) - 1                          # rows


@pytest.mark.parametrize("over", [dict(xts=1 << 39), dict(ots=1 << 39), dict(kts=1 << 39), dict(kots=1 << 39),
                                  dict(xts=1 << 32), dict(n=2, xts=1 << 62), dict(n=1, H=4, xhs=1 << 61)])
def test_rope_refuses_views_past_64_bits(lib, over):
    """Spans of more than 2^63 bytes, which come round to some that meet nothing."""
    near = dict(n=FAR, xts=192 * 4, ots=64 * 4, kts=64, kots=64)
    apart = dict(x=1 << 44, out=2 << 44, k=3 << 44, ko=4 << 44, pos=5 << 44, freq=6 << 44)
    assert _rope(lib, **dict(near, **apart, **over)) == 1


@pytest.mark.parametrize("over", [dict(xrs=1 << 39), dict(ors=1 << 39), dict(xrs=1 << 32)])
def test_norm_refuses_views_past_64_bits(lib, over):
    apart = dict(n=FAR, x=1 << 44, out=2 << 44, mean=3 << 44, rstd=4 << 44)
    assert _norm(lib, **dict(apart, **over)) == 1


@pytest.mark.parametrize("over", [dict(grs=1 << 39), dict(xrs=1 << 39), dict(dxrs=1 << 39)])
def test_norm_gradient_refuses_views_past_64_bits(lib, over):
    apart = dict(n=FAR, g=1 << 44, x=2 << 44, dx=3 << 44, mean=4 << 44, rstd=5 << 44, dw=6 << 44, db=7 << 44)
    assert _ngrad(lib, **dict(apart, **over)) == 1


@pytest.mark.parametrize("over", [
    dict(L=FAR, B=1, budget=1 << 30, cache=1 << 57, orig=1 << 61),          # the workspace
    dict(L=1 << 8, n_pages=1 << 20, rb=1 << 30)])                           # the cache
def test_evict_refuses_tensors_past_64_bits(lib, over):
    """2^64 bytes are counted as none."""
    apart = dict(w=1 << 44, wo=2 << 44, wsb=(1 << 64) - 1)
    assert _ev(lib, **dict(apart, **over)) == 1


def test_evict_workspace_past_64_bits(lib):
    n = ctypes.c_size_t(0)
    assert lib.kda_cache_evict_workspace_size(24, 16, 2048, ctypes.byref(n)) == 0
    assert 24 * 16 * 2048 * 12 <= n.value <= 24 * 16 * (2048 * 12 + 64)
    assert lib.kda_cache_evict_workspace_size(FAR, 1, 1 << 30, ctypes.byref(n)) == 1
    assert lib.kda_cache_evict_workspace_size(1 << 15, 1 << 15, 1 << 30, ctypes.byref(n)) == 1


def test_evict_of_no_sequences_launches_nothing(lib):
    assert _ev(lib, B=0) == 0


def test_rows_of_a_view_are_evenly_spaced():
    from gated_delta_rule_13_gb300 import rows
    step = lambda t, lead: rows._step("x", t.shape, t.stride(), lead)  # noqa: E731
    x = torch.zeros(4, 6, 3, 64)
    assert step(x, 2) == 192
    assert step(x[:, :, :, 8:40], 2) == 192
    assert step(x[:, 2:3], 2) == 6 * 192
    assert step(x[1:2, 2:3], 2) == 192
    assert step(x[:, ::2], 2) == 384
    assert step(x[0, :, 0].expand(6, 64), 1) == 192
    assert step(x[0, 0, 0].expand(5, 64), 1) == 0
    assert step(x[:0], 2) == step(x[:, :0], 2) == 64
    assert step(x[0, 0, 0], 0) == 64
    with pytest.raises(ValueError, match="evenly"):
        step(x[:, :5], 2)
    with pytest.raises(ValueError, match="evenly"):
        step(x.transpose(0, 1), 2)
    with pytest.raises(ValueError, match="contiguous"):
        step(x[..., ::2], 2)


def test_inv_freq():
    from gated_delta_rule_13_gb300 import kda_rope_inv_freq as f
    plain = f(64)
    assert plain.dtype is torch.float64 and plain.shape == (32,)
    assert plain[0] == 1 and abs(plain[16].item() - 0.01) < 1e-15
    assert torch.equal(f(64, scaling="linear", factor=4.0), plain / 4)
    base = f(64, scaling="base", factor=8.0)
    assert base[0] == 1 and abs(base[-1] / plain[-1] * 8 - 1) < 1e-12
    ramp = f(64, scaling="ramp", factor=8.0, original=4096)
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(ramp[turns > 40], plain[turns > 40])
    assert torch.allclose(ramp[turns < 0.8] * 8, plain[turns < 0.8], rtol=1e-14)
    assert (ramp[1:] < ramp[:-1]).all()
    for bad in (dict(dim=7), dict(dim=0), dict(dim=64, base=1.0), dict(dim=64, factor=0.5),
                dict(dim=64, scaling="x"), dict(dim=64, scaling="ramp"),
                dict(dim=64, scaling="ramp", original=100, beta_fast=1.0)):
        with pytest.raises(ValueError):
            f(**bad)


@pytest.mark.parametrize("center", [False, True])
def test_reference_gradient_of_the_norm(center):
    """The formula against automatic differentiation, and that against differences."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(3, 9, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(9, generator=g, dtype=torch.float64, requires_grad=True)
    b = torch.randn(9, generator=g, dtype=torch.float64, requires_grad=True)
    d = torch.randn(3, 9, generator=g, dtype=torch.float64)
    assert torch.autograd.gradcheck(lambda *a: ru.norm_ref(*a, center, 1e-5)[0], (x, w, b))
    y, m, r = ru.norm_ref(x, w, b, center, 1e-5)
    want = torch.autograd.grad(y, (x, w, b), d)
    got = ru.norm_grad_ref(d, x.detach(), w.detach(), m.detach() if center else None, r.detach())
    for u, v in zip(got, want):
        assert torch.allclose(u, v, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_gradient_of_the_rotation(interleaved):
    g = torch.Generator().manual_seed(4)
    x = torch.randn(3, 2, 10, generator=g, dtype=torch.float64, requires_grad=True)
    pos, freq = torch.tensor([0, 7, -3]), torch.rand(5, generator=g, dtype=torch.float64)
    d = torch.randn(3, 2, 10, generator=g, dtype=torch.float64)
    f = lambda t: ru.rope_ref(t, pos, freq, interleaved, 1.3, False)  # noqa: E731
    assert torch.autograd.gradcheck(f, (x,))
    want, = torch.autograd.grad(f(x), x, d)
    assert torch.allclose(ru.rope_ref(d, pos, freq, interleaved, 1.3, True), want, atol=1e-12)


def test_reference_of_the_eviction():
    w = [5.0, 1.0, 7.0, 7.0, 0.0, 9.0, 2.0, 7.0, 3.0, 4.0]
    assert ru.evict_ref(w, 10, 10, 2, 2) == list(range(10))
    # first 1, last 2; of 1 .. 7 stay 5 (9.0), 2 and 3 (7.0, the earlier two)
    assert ru.evict_ref(w, 10, 6, 1, 2) == [0, 5, 2, 3, 8, 9]
    assert ru.evict_ref(w, 10, 1, 0, 0) == [5]
    assert ru.evict_ref(w, 10, 3, 1, 2) == [0, 8, 9]
    assert ru.evict_ref([math.nan, -math.inf, -1.0], 3, 2, 0, 0) == [2, 1]
