"""The bounded waits of latent attention run out without faulting or hanging anything: a
block's loader withholds a tile, the waits for it give up after two milliseconds, the
status says which block, the kernels end, and the next call with the same workspace is as
ever."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_13_gb300 as pkg
from gated_delta_rule_13_gb300 import kda, latent
from test_gpu_latent import DEV, _bwd, _decode_problem, _fwd, _problem, _randn

pytestmark = pytest.mark.gpu
WAIT_US = 2000


def _status(ws):
    torch.cuda.synchronize()
    return kda.kda_read_device_status_detail(ws)


def _same(want, got):
    assert all(torch.equal(a, b) for a, b in zip(want, got, strict=True))


def _gave_up(run, ws, want, block, tile, chains):
    """The armed call reports one of these blocks; the next call gives what it should."""
    for _ in range(3):      # (a block that another took over before it started meets nothing)
        latent.kda_latent_test_timeout(ws, block, tile, WAIT_US)
        got = run()
        code, where, chain, _ = _status(ws)
        if code != kda.KDA_OK:
            break
    assert code == kda.KDA_ERR_TIMEOUT and chain in chains, (code, where, chain)
    got = [t.clone() for t in got]
    again = run()
    assert _status(ws)[0] == kda.KDA_OK
    _same(want, again)
    return got


# blocks 0 and 1: 144 queries over 400 keys, in two tiles; 2 and 3: 44 over 300, in one
@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("block,tile", [(0, 0), (1, 1), (2, 0), (3, 2)])
def test_forward(block, tile, dr):
    x = _problem([400, 300], [400, 300], H=2, dr=dr)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    want = _fwd(x, workspace=ws)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])

    def run():
        out.fill_(3.0)
        lse.fill_(3.0)
        return _fwd(x, out=out, lse=lse, workspace=ws)

    got = _gave_up(run, ws, want, block, tile, [block])
    # the block's rows are not written, all others as ever
    left = (got[1] == 3.0) & (want[1] != 3.0)
    assert 0 < int(left.sum()) <= 256
    assert torch.equal(got[1][~left], want[1][~left])
    assert torch.equal(got[0][~left], want[0][~left]) and bool((got[0][left] == 3.0).all())


@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("block,tile", [(0, 0), (3, 2), (13, 0), (20, 0)])
def test_gradient(block, tile, dr):
    """Keys of 400 and 300 tokens make 14 blocks of the keys pass, then come the queries'."""
    x = _problem([400, 300], [400, 300], H=2, dr=dr)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    out, lse = _fwd(x)
    d_out = _randn(700, 2, 128, seed=9)
    d_kv = torch.empty(2, 700, 2, 128, dtype=torch.bfloat16, device=DEV)

    def run():
        d_kv.fill_(3.0)
        return [t for t in _bwd(x, out, lse, d_out, d_k=d_kv[0], d_v=d_kv[1], workspace=ws)
                if t is not None]

    want = [t.clone() for t in run()]
    got = _gave_up(run, ws, want, block, tile, [block])
    for a, b in zip(want[1:3], got[1:3]):
        left = (a != b).any(-1)
        assert int(left.sum()) <= (128 if block < 14 else 0)
        assert bool((b[left] == 3.0).all())


@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("block,tile", [(0, 0), (1, 0), (4, 1), (5, 1)])
def test_decode(block, tile, dr):
    """Two CTAs exchange scores: when one gives up, so does the other."""
    x = _decode_problem([3000, 5000, 1200, 7000], 2, 16, dr, 64)
    ws = torch.empty(pkg.kda_latent_decode_workspace_size(4, 2, 16, dr=dr), dtype=torch.uint8,
                     device=DEV)

    def run():
        return [pkg.kda_latent_decode(x["q"], x["cache"], x["table"], x["lens"], workspace=ws)]

    want = [t.clone() for t in run()]
    _gave_up(run, ws, want, block, tile, [block & ~1, block | 1])


@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("block", [0, 1])
def test_decode_gives_up_in_time(block, dr):
    """What is in flight is waited for, and nothing else: only one CTA of a pair, and only
    with a rotary part, copies queries.  (The limit of those waits is two seconds.)"""
    x = _decode_problem([3000, 5000], 1, 16, dr, 64)
    ws = torch.empty(pkg.kda_latent_decode_workspace_size(2, 1, 16, dr=dr), dtype=torch.uint8,
                     device=DEV)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    latent.kda_latent_test_timeout(ws, block, 0, WAIT_US)
    begin.record()
    pkg.kda_latent_decode(x["q"], x["cache"], x["table"], x["lens"], workspace=ws)
    end.record()
    assert _status(ws)[0] == kda.KDA_ERR_TIMEOUT
    assert begin.elapsed_time(end) < 1000


def test_a_control_that_meets_nothing():
    x = _problem([100], [100], H=1, dr=0)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    other = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    want = _fwd(x)
    for arm in (lambda: latent.kda_latent_test_timeout(ws, 50, 0, 100000),
                lambda: latent.kda_latent_test_timeout(other, 0),
                lambda: (latent.kda_latent_test_timeout(ws, 0),
                         latent.kda_latent_test_timeout(ws, -1))):
        arm()
        _same(want, _fwd(x, workspace=ws))
        assert _status(ws)[0] == kda.KDA_OK
    latent.kda_latent_test_timeout(ws, -1)
    for bad in ((0, -1, 100), (0, 0, 0), (0, 0, 3000000)):
        with pytest.raises(pkg.KDAError):
            latent.kda_latent_test_timeout(ws, *bad)
