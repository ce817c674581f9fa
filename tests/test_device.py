"""The recurrence's entry points refuse tensors and streams of another device than the
current one, on which their kernels would run.  Device numbers are stand-ins."""
from __future__ import annotations

import types

import pytest
import torch

from gated_delta_rule_13_gb300 import inputs, kda

DEV = torch.device("cuda:0")


def _current(monkeypatch, index):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: index, raising=False)


def test_a_stream_of_another_device(monkeypatch):
    stream = types.SimpleNamespace(device=DEV, cuda_stream=7)
    _current(monkeypatch, 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        kda._stream_handle(stream)
    _current(monkeypatch, 0)
    assert kda._stream_handle(stream).value == 7


@pytest.mark.gpu
def test_every_entry_point_refuses(monkeypatch):
    x = inputs.prefill_inputs([40, 30], H=2, init_state=True, device=DEV, seed=1)
    args, state, cu = [x[n] for n in ("q", "k", "v", "log_alpha", "beta")], x["init_state"], \
        x["cu_seqlens"]
    b, m = kda.kda_chunk_fwd_transitions(*args, cu)
    one = [t[:2].contiguous() for t in args]
    drafts = [t[:4].reshape(2, 2, *t.shape[1:]).contiguous() for t in args]
    count = torch.ones(2, dtype=torch.int32, device=DEV)
    ws = torch.zeros(kda.kda_chunk_fwd_workspace_size(2, 70, 2), dtype=torch.uint8, device=DEV)
    gamma = torch.ones(128, device=DEV)
    calls = [lambda **s: kda.kda_chunk_fwd(*args, state, cu, **s),
             lambda **s: kda.kda_chunk_fwd_noalloc(*args, state, cu, **s),
             lambda **s: kda.kda_chunk_fwd_transitions(*args, cu, **s),
             lambda **s: kda.kda_chunk_bwd(*args, state, cu, x["v"], **s),
             lambda **s: kda.kda_state_combine(b, m, 1, state, **s),
             lambda **s: kda.kda_decode_step(state.clone(), *one, **s),
             lambda **s: kda.kda_decode_replay(state.clone(), *drafts, count, **s),
             lambda **s: kda.kda_post_fwd(x["v"], x["v"], gamma, **s),
             lambda **s: kda.kda_read_device_status(ws, **s)]
    for call in calls:
        call()
        call(stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream()
    with monkeypatch.context() as other:
        _current(other, 1)
        for call in calls:
            for kw in ({}, dict(stream=stream)):
                with pytest.raises(ValueError, match="current device is cuda:1"):
                    call(**kw)
    away = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    for call in calls:
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call(stream=away)
