"""Latent attention where its work is laid out in ways that smaller problems do not reach,
against the definition in 64 bits: whole rounds of items and shared-out keys in one call of
the forward, and decode with many tiles of query rows, down to one pair of CTAs a tile."""
from __future__ import annotations

import math

import pytest
import torch

import latent_util as lu
from test_gpu_latent import DEV, _decode_problem, _fwd, _problem, check_decode

pytestmark = pytest.mark.gpu


def _heads(tiles, rest):
    """Heads for which `tiles` of 256 queries fill the SMs once or more and leave at least
    ``rest`` items, at most half an SM's round: their keys are shared out."""
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    for H in range(sms // tiles + 1, 4 * sms):
        if rest <= tiles * H % sms <= sms // 2:
            return H
    raise AssertionError("no such number of heads")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("lens_q,lens_k,rest", [
    ([1280], [2000], 1), ([1280], [2000], 20),                 # many parts, few parts
    ([700, 580], [1500, 2100], 3),
    ([5] * 40 + [600], [5] * 40 + [3001], 2),                  # found through the table
])
def test_whole_rounds_and_shared_out_keys(lens_q, lens_k, rest, dr, causal):
    H = _heads(sum((n + 255) // 256 for n in lens_q), rest)
    x = _problem(lens_q, lens_k, H, dr)
    out, lse = _fwd(x, causal=causal)
    r_out, r_lse, t_out, t_lse = lu.fwd_ref(**x, causal=causal, scale=1 / math.sqrt(128 + dr))
    lu.check("out", out, r_out, t_out)
    lu.check("lse", lse, r_lse, t_lse)


@pytest.mark.parametrize("T,H,tree", [(3, 128, False), (13, 97, True), (20, 128, True),
                                      (39, 128, False), (64, 80, True), (77, 128, False)])
@pytest.mark.parametrize("dr", [0, 64])
def test_many_query_rows(T, H, tree, dr):
    """3, 10, 20, 39, 40 and 77 tiles of 128 rows; from 39 on one pair has all keys of a
    tile, and 77 are more pairs than run at once."""
    check_decode(_decode_problem([200, 77, 1000, 0, 333], T, H, dr, 64, tree=tree))
