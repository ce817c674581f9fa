"""A host cu_seqlens belongs to the caller again when the call returns: what is written
there later, while the call waits its turn on the stream or before a captured call is
replayed, changes nothing."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_13_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FEW, FEW_LATER = [0, 100, 400], [0, 300, 400]
# more sequences than one launch carries
MANY, MANY_LATER = [0, 150] + [400] * 9000, [0, 250] + [400] * 9000


def _randn(*shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).bfloat16()


def _problem():
    return dict(q=_randn(400, 2, 192, seed=1), k=_randn(400, 2, 128, seed=2),
                v=_randn(400, 2, 128, seed=3), k_rope=_randn(400, 64, seed=4))


def _calls(x, d_out, cu_q, cu_k):
    out, lse = pkg.kda_latent_fwd(**x, cu_seqlens_q=cu_q, cu_seqlens_k=cu_k)
    return (out, lse, *pkg.kda_latent_bwd(**x, out=out, lse=lse, d_out=d_out, cu_seqlens_q=cu_q,
                                          cu_seqlens_k=cu_k))


def _host(values, pinned):
    t = torch.tensor(values, dtype=torch.int32)
    return t.pin_memory() if pinned else t


@pytest.mark.parametrize("now,later", [(FEW, FEW_LATER), (MANY, MANY_LATER)])
@pytest.mark.parametrize("pinned", [True, False])
def test_written_while_the_call_waits(pinned, now, later):
    x, d_out = _problem(), _randn(400, 2, 128, seed=5)
    want = _calls(x, d_out, *[torch.tensor(now, dtype=torch.int32, device=DEV)] * 2)
    cu_q, cu_k = _host(now, pinned), _host(now, pinned)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)               # about a tenth of a second
    got = _calls(x, d_out, cu_q, cu_k)
    cu_q.copy_(torch.tensor(later, dtype=torch.int32))
    cu_k.copy_(cu_q)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("pinned", [True, False])
def test_written_before_a_captured_call_is_replayed(pinned):
    x, d_out = _problem(), _randn(400, 2, 128, seed=5)
    want = _calls(x, d_out, *[torch.tensor(FEW, dtype=torch.int32, device=DEV)] * 2)
    cu_q, cu_k = _host(FEW, pinned), _host(FEW, pinned)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _calls(x, d_out, cu_q, cu_k)
    cu_q.copy_(torch.tensor(FEW_LATER, dtype=torch.int32))
    cu_k.copy_(cu_q)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
