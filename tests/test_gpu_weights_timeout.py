"""The bounded waits of kda_latent_weights run out without faulting or hanging anything, as
those of latent attention do: a block's loaders withhold a tile, the status says which
block, the kernel ends, and the next call with the same workspace is as ever."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_13_gb300 as pkg
from gated_delta_rule_13_gb300 import kda, latent
from test_gpu_latent_timeout import _gave_up, _status, WAIT_US
from test_gpu_weights import DEV, _data

pytestmark = pytest.mark.gpu


def _runner(d, ws):
    lse = torch.full(d["q"].shape[:3], 7.0, device=DEV)
    return lambda: [pkg.kda_latent_weights(d["q"], d["cache"], d["table"], d["seq_lens"], lse,
                                           d["old"].clone(), workspace=ws)]


def _case(pair, dr):
    """One CTA for the keys, with two tiles or more each; pairs, with two or more each."""
    d = _data([20000, 31000], 1, 16, dr, 64) if not pair else _data([60000, 45000], 4, 48, dr, 64)
    T, H = d["q"].shape[1:3]
    ws = torch.empty(pkg.kda_latent_weights_workspace_size(2, T, H, dr=dr), dtype=torch.uint8,
                     device=DEV)
    return d, ws


@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("block,tile", [(0, 0), (3, 1), (151, 0)])
def test_one_cta(block, tile, dr):
    d, ws = _case(False, dr)
    run = _runner(d, ws)
    want = [t.clone() for t in run()]
    got = _gave_up(run, ws, want, block, tile, [block])
    # the block's tiles from this one on are not written
    assert 0 < int((got[0] != want[0]).sum()) <= 128 * 3


@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("block,tile", [(0, 0), (1, 0), (4, 1), (5, 1)])
def test_pair(block, tile, dr):
    """When one CTA of a pair gives up, so does the other."""
    d, ws = _case(True, dr)
    run = _runner(d, ws)
    want = [t.clone() for t in run()]
    _gave_up(run, ws, want, block, tile, [block & ~1, block | 1])


@pytest.mark.parametrize("pair", [False, True])
def test_gives_up_in_time(pair):
    d, ws = _case(pair, 64)
    run = _runner(d, ws)
    run()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    latent.kda_latent_test_timeout(ws, 0, 0, WAIT_US)
    begin.record()
    run()
    end.record()
    assert _status(ws)[0] == kda.KDA_ERR_TIMEOUT
    assert begin.elapsed_time(end) < 1000
