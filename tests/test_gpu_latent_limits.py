"""Decode at the lengths the table can address: tile numbers and positions stay in range up
to 2^31 - 1, and a list of more tiles than that is refused on the device."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_13_gb300 as pkg
from gated_delta_rule_13_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE, PAGES = 8176, 262657           # together 2^31 - 16 positions
LAST = PAGE * PAGES


def _problem(lens, H=3):
    """Every page of every sequence is the same one, and all its rows are the same."""
    g = torch.Generator(device=DEV).manual_seed(3)
    row = torch.tensor([-1.0, -0.5, 0.5, 1.0, 2.0], device=DEV)[
        torch.randint(0, 5, (512,), generator=g, device=DEV)].bfloat16()
    q = torch.randint(-1, 2, (len(lens), 1, H, 512), generator=g, device=DEV).bfloat16()
    table = torch.zeros(len(lens), PAGES, dtype=torch.int32, device=DEV)
    return row, q, row.expand(1, PAGE, 512).contiguous(), table, torch.tensor(
        lens, dtype=torch.int32, device=DEV)


def test_the_longest_sequence():
    lens = [70, LAST]
    row, q, cache, table, at = _problem(lens)
    lse = torch.zeros(2, 1, 3, device=DEV)
    out = torch.full((2, 1, 3, 512), 7.0, device=DEV).bfloat16()
    ws = torch.empty(pkg.kda_latent_decode_workspace_size(2, 1, 3), dtype=torch.uint8, device=DEV)
    pkg.kda_latent_decode(q, cache, table, at, scale=0.0625, out=out, lse=lse, workspace=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_OK
    # equal scores: the mean of equal rows, which are exact in bf16
    assert torch.equal(out, row.expand_as(out))
    want = (q.double() @ row.double()) * 0.0625 + torch.tensor(
        [math.log(n) for n in lens], dtype=torch.float64, device=DEV).view(2, 1, 1)
    # a reference and a logarithm of at most 2^6 in base 2, and three fp32 roundings
    assert bool(((lse - want).abs() <= 4 * 2.0 ** (6 - 24)).all())


def test_more_tiles_than_can_be_counted():
    lens = [0] + [LAST] * 64         # 64 * 2^25 tiles
    _, q, cache, table, at = _problem(lens, H=1)
    out = torch.full((65, 1, 1, 512), 7.0, device=DEV).bfloat16()
    ws = torch.empty(pkg.kda_latent_decode_workspace_size(65, 1, 1), dtype=torch.uint8, device=DEV)
    pkg.kda_latent_decode(q, cache, table, at, out=out, workspace=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_ERR_INVALID_ARG
    assert bool((out[0] == 0).all()) and bool((out[1:] == 7).all())
    at[1:] = 5
    pkg.kda_latent_decode(q, cache, table, at, out=out, workspace=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_OK
