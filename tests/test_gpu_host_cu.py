"""A host cu_seqlens of the recurrence's entry points belongs to the caller again when the
call returns: what is written there while the call waits its turn on the stream, or before
a captured call is replayed, changes nothing."""
from __future__ import annotations

import pytest
import torch

from gated_delta_rule_13_gb300 import inputs, kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NOW, LATER = [0, 100, 400], [0, 300, 400]


def _problem():
    x = inputs.prefill_inputs([100, 300], H=2, init_state=True, device=DEV, seed=5)
    return [x[n] for n in ("q", "k", "v", "log_alpha", "beta")], x["init_state"]


def _call(entry, cu):
    x, state = _problem()
    if entry == "transitions":
        return lambda: kda.kda_chunk_fwd_transitions(*x, cu)
    if entry == "bwd":
        return lambda: kda.kda_chunk_bwd(*x, state, cu, x[2])
    return lambda: getattr(kda, entry)(*x, state, cu)


ENTRIES = ["kda_chunk_fwd", "kda_chunk_fwd_noalloc", "transitions", "bwd"]


def _host(values, pinned):
    t = torch.tensor(values, dtype=torch.int32)
    return t.pin_memory() if pinned else t


def _same(want, got):
    assert all(torch.equal(a, b) for a, b in zip(want, got, strict=True))


@pytest.mark.parametrize("pinned", [True, False])
@pytest.mark.parametrize("entry", ENTRIES)
def test_written_while_the_call_waits(entry, pinned):
    want = _call(entry, torch.tensor(NOW, dtype=torch.int32, device=DEV))()
    cu = _host(NOW, pinned)
    call = _call(entry, cu)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)               # about a tenth of a second
    got = call()
    cu.copy_(torch.tensor(LATER, dtype=torch.int32))
    torch.cuda.synchronize()
    _same(want, got)


@pytest.mark.parametrize("entry", ENTRIES)
def test_written_before_a_captured_call_is_replayed(entry):
    want = _call(entry, torch.tensor(NOW, dtype=torch.int32, device=DEV))()
    cu = _host(NOW, False)
    call = _call(entry, cu)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    cu.copy_(torch.tensor(LATER, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    _same(want, got)
