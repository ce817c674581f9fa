"""The entry points around a cached row run on the device their tensors are on, like those
of latent attention: with another current device, or a stream of another one, they refuse
before anything is allocated or launched."""
from __future__ import annotations

import types

import pytest
import torch

from gated_delta_rule_13_gb300 import kda_rope_inv_freq, rows
from test_latent_device import current  # noqa: F401

DEV = torch.device("cuda:0")


@pytest.mark.gpu
def test_every_entry_point_refuses(current):  # noqa: F811
    bf = dict(dtype=torch.bfloat16, device=DEV)
    x, one = torch.zeros(4, 2, 64, **bf), torch.ones(1, dtype=torch.int32, device=DEV)
    pos, freq = torch.arange(4, dtype=torch.int32, device=DEV), kda_rope_inv_freq(64, device=DEV)
    q, cache = torch.zeros(1, 1, 2, 512, **bf), torch.zeros(2, 16, 512, **bf)
    weights, lse = torch.zeros(1, 16, device=DEV), torch.zeros(1, 1, 2, device=DEV)
    _, mean, rstd = rows.kda_norm_fwd(x)
    calls = [lambda s: rows.kda_rope(x, pos, freq, stream=s),
             lambda s: rows.kda_norm_fwd(x, stream=s),
             lambda s: rows.kda_norm_bwd(x, x, None, mean, rstd, bias=True, stream=s),
             lambda s: rows.kda_latent_weights(q, cache, one.view(1, 1), one, lse, weights, stream=s),
             lambda s: rows.kda_cache_evict(cache, one.view(1, 1), one, weights, 4, stream=s)]
    for call in calls:
        call(None)
        call(torch.cuda.current_stream())
    torch.cuda.synchronize()
    current(1)
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call(None)
    current(0)
    other = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    for call in calls:
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call(other)


def test_tensors_of_the_host_are_refused():
    t = torch.zeros(4, 2, 64)
    for call in (lambda: rows.kda_rope(t, t, t), lambda: rows.kda_norm_fwd(t),
                 lambda: rows.kda_norm_bwd(t, t, None, None, t),
                 lambda: rows.kda_latent_weights(t, t, t, t, t, t),
                 lambda: rows.kda_cache_evict(t, t, t, t, 4)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
