"""Refusals of the latent-attention and cache entry points, before any launch
(no GPU): pointers are fake, aligned addresses that are never dereferenced."""
from __future__ import annotations

import ctypes

import pytest
import torch

A = 0x10000000


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_13_gb300 import _build, kda
    _build.build_library()
    return kda.library()


def _p(x):
    return ctypes.c_void_p(x)


EXP = dict(q=A, k=2 * A, v=3 * A, r=4 * A, kts=512, khs=128, vts=512, vhs=128, cuq=5 * A,
           cuk=5 * A + 64, n_seqs=2, nq=100, nk=120, H=4, dk=128, dr=64, dv=128, dtype=1,
           scale=0.1, causal=1, out=6 * A, lse=7 * A, ws=8 * A, wsb=1 << 30)


def _head(x):
    return (_p(x["q"]), _p(x["k"]), _p(x["v"]), _p(x["r"]), x["kts"], x["khs"], x["vts"], x["vhs"],
            _p(x["cuq"]), _p(x["cuk"]), x["n_seqs"], x["nq"], x["nk"], x["H"], x["dk"], x["dr"],
            x["dv"], x["dtype"], x["scale"], x["causal"])


def _fwd(lib, **over):
    x = dict(EXP, **over)
    return lib.kda_latent_fwd(*_head(x), _p(x["out"]), _p(x["lse"]), _p(x["ws"]), x["wsb"], None)


def _bwd(lib, **over):
    x = dict(EXP, do=9 * A, dq=10 * A, gk=11 * A, gv=12 * A, gr=13 * A, gkts=512, gkhs=128,
             gvts=512, gvhs=128)
    x.update(over)
    return lib.kda_latent_bwd(*_head(x), _p(x["out"]), _p(x["lse"]), _p(x["do"]), _p(x["dq"]),
                              _p(x["gk"]), _p(x["gv"]), _p(x["gr"]), x["gkts"], x["gkhs"],
                              x["gvts"], x["gvhs"], _p(x["ws"]), x["wsb"], None)


SHARED = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(r=None), 1),
    (dict(dr=0), 1), (dict(cuq=None), 1), (dict(cuk=None), 1), (dict(out=None), 1),
    (dict(lse=None), 1), (dict(n_seqs=0), 1), (dict(nq=-1), 1), (dict(nk=-1), 1),
    (dict(nq=1 << 31), 1), (dict(H=0), 1), (dict(H=70000), 1), (dict(dk=0), 1),
    (dict(dk=64), 2), (dict(dv=256), 2), (dict(dr=32), 2), (dict(dtype=0), 2), (dict(dtype=5), 2),
    (dict(q=A + 8), 1), (dict(k=2 * A + 2), 1), (dict(out=6 * A + 4), 1), (dict(lse=7 * A + 2), 1),
    (dict(kts=0), 1), (dict(kts=508), 1), (dict(khs=132), 1), (dict(khs=64), 1),
    (dict(vts=-512), 1), (dict(vts=256), 1),          # rows of a token would overlap the next's
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1),
    (dict(ws=None), 3), (dict(ws=8 * A + 8), 3), (dict(wsb=100), 3),
]


@pytest.mark.parametrize("over,code", SHARED + [
    (dict(out=A + 1024), 1), (dict(lse=3 * A), 1), (dict(lse=6 * A + 512), 1)])
def test_fwd_refuses(lib, over, code):
    assert _fwd(lib, **over) == code


@pytest.mark.parametrize("over,code", SHARED + [
    (dict(do=None), 1), (dict(dq=None), 1), (dict(gk=None), 1), (dict(gv=None), 1),
    (dict(gr=None), 1), (dict(do=9 * A + 8), 1), (dict(dq=A), 1), (dict(gk=2 * A), 1),
    (dict(gv=11 * A), 1), (dict(gr=10 * A), 1), (dict(gkts=8), 1), (dict(gvhs=4), 1)])
def test_bwd_refuses(lib, over, code):
    assert _bwd(lib, **over) == code


DEC = dict(q=A, cache=2 * A, table=3 * A, lens=4 * A, mask=5 * A, B=3, T=4, H=8, dc=512, dr=64,
           n_pages=100, page=64, max_pages=20, dtype=1, scale=0.1, out=6 * A, lse=7 * A, ws=8 * A,
           wsb=1 << 31)


def _dec(lib, **over):
    x = dict(DEC, **over)
    return lib.kda_latent_decode(_p(x["q"]), _p(x["cache"]), _p(x["table"]), _p(x["lens"]),
                                 _p(x["mask"]), x["B"], x["T"], x["H"], x["dc"], x["dr"],
                                 x["n_pages"], x["page"], x["max_pages"], x["dtype"], x["scale"],
                                 _p(x["out"]), _p(x["lse"]), _p(x["ws"]), x["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(cache=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(out=None), 1), (dict(B=-1), 1), (dict(T=0), 1), (dict(H=0), 1), (dict(dc=0), 1),
    (dict(dc=256), 2), (dict(dr=16), 2), (dict(dtype=0), 2), (dict(n_pages=0), 1),
    (dict(page=0), 1), (dict(page=24), 1), (dict(max_pages=0), 1), (dict(T=65), 1),
    (dict(n_pages=1 << 27), 1), (dict(T=1 << 16, H=1 << 10, mask=None), 1),
    (dict(q=A + 8), 1), (dict(cache=2 * A + 2), 1), (dict(mask=5 * A + 4), 1),
    (dict(out=A), 1), (dict(lse=6 * A), 1), (dict(out=2 * A + 4096), 1),
    (dict(scale=0.0), 1), (dict(scale=float("inf")), 1),
    (dict(ws=None), 3), (dict(ws=8 * A + 4), 3), (dict(wsb=0), 3)])
def test_decode_refuses(lib, over, code):
    assert _dec(lib, **over) == code


WR = dict(cache=A, rows=10 * A, ls=4 * 1152, bs=2 * 1152, ts=1152, table=20 * A, start=21 * A,
          path=22 * A, n=23 * A, L=2, n_pages=10, page=16, row=1152, B=2, T=2, max_pages=4,
          status=24 * A)


def _wr(lib, **over):
    x = dict(WR, **over)
    return lib.kda_cache_write(_p(x["cache"]), _p(x["rows"]), x["ls"], x["bs"], x["ts"],
                               _p(x["table"]), _p(x["start"]), _p(x["path"]), _p(x["n"]), x["L"],
                               x["n_pages"], x["page"], x["row"], x["B"], x["T"], x["max_pages"],
                               _p(x["status"]), None)


@pytest.mark.parametrize("over", [
    dict(cache=None), dict(table=None), dict(start=None), dict(rows=None, path=None),
    dict(L=-1), dict(B=-1), dict(T=0), dict(T=1025), dict(n_pages=0), dict(page=0),
    dict(max_pages=0), dict(row=0), dict(row=1160), dict(cache=A + 8), dict(rows=10 * A + 8),
    dict(ts=1160), dict(bs=-16), dict(start=21 * A + 2), dict(status=24 * A + 1),
    dict(rows=A + 1152)])
def test_cache_write_refuses(lib, over):
    assert _wr(lib, **over) == 1


@pytest.mark.parametrize("args", [
    (None, 2 * A, 3 * A, 1, 1, 4, 64, None), (A, None, 3 * A, 1, 1, 4, 64, None),
    (A, 2 * A, None, 1, 1, 4, 64, None), (A, 2 * A, 3 * A, -1, 1, 4, 64, None),
    (A, 2 * A, 3 * A, 1, -1, 4, 64, None), (A, 2 * A, 3 * A, 1, 1, 0, 64, None),
    (A, 2 * A, 3 * A, 1, 1, 4, 0, None), (A, 2 * A, 3 * A, 1, 1, 4, 72, None),
    (A + 4, 2 * A, 3 * A, 1, 1, 4, 64, None), (A, 2 * A + 1, 3 * A, 1, 1, 4, 64, None),
    (A, 2 * A, 3 * A, 1, 1, 4, 64, 5 * A + 2)])
def test_copy_pages_refuses(lib, args):
    c, s, d, n, L, n_pages, nbytes, st = args
    assert lib.kda_cache_copy_pages(_p(c), _p(s), _p(d), n, L, n_pages, nbytes, _p(st), None) == 1


def test_workspace_sizes(lib):
    import gated_delta_rule_13_gb300 as pkg
    assert pkg.kda_latent_fwd_workspace_size(1, 100, 100, 4) >= 256
    small = pkg.kda_latent_bwd_workspace_size(1, 100, 100, 4, dr=64)
    assert small <= pkg.kda_latent_bwd_workspace_size(1, 10000, 10000, 4, dr=64)
    assert pkg.kda_latent_decode_workspace_size(1, 1, 96) >= 256
    for bad, code in ((dict(dk=64), 2), (dict(dr=1), 2), (dict(dtype=0), 2)):
        with pytest.raises(pkg.KDAError) as e:
            pkg.kda_latent_fwd_workspace_size(1, 1, 1, 1, **bad)
        assert e.value.code == code
    with pytest.raises(pkg.KDAError):
        pkg.kda_latent_decode_workspace_size(1, 0, 1)


def test_binding_wants_cuda_tensors():
    import gated_delta_rule_13_gb300 as pkg
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        pkg.kda_latent_fwd(q, q, q)
    with pytest.raises(TypeError):
        pkg.kda_latent_decode(torch.zeros(1, 1, 2, 512, dtype=torch.bfloat16), q, q, q)
    with pytest.raises(TypeError):
        pkg.kda_cache_write(q, None, q, q)
    with pytest.raises(TypeError):
        pkg.kda_cache_copy_pages(q, q, q)
