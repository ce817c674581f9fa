"""Latent attention called many times over one problem: every call reports success and
gives the same bits, whichever warp, CTA or kernel happens to run ahead."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_13_gb300 as pkg
from gated_delta_rule_13_gb300 import kda
from test_gpu_latent import (DEV, _bwd, _decode_problem, _fwd, _problem, _randn, check_both,
                             check_decode)

pytestmark = pytest.mark.gpu
REPEATS = 100


def _same(run, ws):
    first = None
    for _ in range(REPEATS):
        got = run()
        assert kda.kda_read_device_status(ws) == kda.KDA_OK
        got = [t for t in got if t is not None]
        if first is None:
            first = [t.clone() for t in got]
            assert all(bool(torch.isfinite(t).all()) for t in first)
        for s, t in zip(first, got):
            assert torch.equal(s, t)


@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("lens,H", [([2000, 1, 900], 16), ([130] * 40, 3), ([6000], 2)])
def test_both_directions(lens, H, dr):
    x = _problem(lens, lens, H, dr)
    ws = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    _same(lambda: _fwd(x, workspace=ws), ws)
    out, lse = _fwd(x)
    d_out = _randn(*out.shape, seed=9)
    _same(lambda: _bwd(x, out, lse, d_out, workspace=ws), ws)


@pytest.mark.parametrize("lens,T,H", [([900, 33, 4000, 1], 1, 128), ([3000] * 24, 8, 16),
                                      ([20000], 1, 16)])
def test_decode(lens, T, H):
    x = _decode_problem(lens, T, H, 64, 64)
    ws = torch.empty(pkg.kda_latent_decode_workspace_size(len(lens), T, H, dr=64),
                     dtype=torch.uint8, device=DEV)
    _same(lambda: [pkg.kda_latent_decode(x["q"], x["cache"], x["table"], x["lens"],
                                         workspace=ws)], ws)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("lens_q,lens_k,H", [
    ([0, 300, 0, 1, 700, 0], [900, 300, 128, 3000, 700, 64], 24),   # keys nobody queries
    ([1] * 40 + [129], [1] * 20 + [0] * 20 + [129], 40),            # items of one tile, rows without keys
    ([513], [513], 96),
])
def test_many_items_a_block(lens_q, lens_k, H, dr, causal):
    """A block works through many items of different lengths, some of them empty."""
    check_both(_problem(lens_q, lens_k, H, dr), causal=causal)


@pytest.mark.parametrize("B", [1, 2, 9, 10, 11, 12, 40])
def test_joined_sequences(B):
    """Few sequences have many parts to join, many sequences have few."""
    check_decode(_decode_problem([1500 + 7 * b for b in range(B)], 1, 40, 64, 64))
