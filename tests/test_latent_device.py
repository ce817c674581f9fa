"""A call runs on the device its tensors are on: with another current device, or a stream
of another one, it is refused before anything is allocated or launched.  Device numbers
are stand-ins; nothing runs on a second device."""
from __future__ import annotations

import types

import pytest
import torch

from gated_delta_rule_13_gb300 import latent

DEV = torch.device("cuda:0")


@pytest.fixture
def current(monkeypatch):
    """Sets what the binding takes for the current device."""
    def set_to(index):
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: index, raising=False)
        monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    return set_to


def test_another_current_device_is_refused(current, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    current(1)
    with pytest.raises(ValueError, match="current device"):
        latent._stream(None, DEV)
    with pytest.raises(ValueError, match="current device"):
        latent._stream(types.SimpleNamespace(device=DEV, cuda_stream=7), DEV)
    current(0)
    assert latent._stream(None, DEV) == 100


def test_a_stream_of_another_device_is_refused(current):
    current(0)
    other = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=7)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        latent._stream(other, DEV)
    assert latent._stream(types.SimpleNamespace(device=DEV, cuda_stream=7), DEV) == 7


def test_workspace_sizes_are_kept_by_device(current, monkeypatch):
    """The size follows from the SM count, which need not be the same on two devices."""
    asked = []

    class Library:
        def __getattr__(self, name):
            def size(*args):
                asked.append(torch._C._cuda_getDevice())
                args[-1]._obj.value = 1000 * (1 + torch._C._cuda_getDevice())
                return 0
            return size

    monkeypatch.setattr(latent, "library", Library)
    latent._size.cache_clear()
    for size in (lambda: latent.kda_latent_fwd_workspace_size(1, 7, 7, 3),
                 lambda: latent.kda_latent_bwd_workspace_size(1, 7, 7, 3),
                 lambda: latent.kda_latent_decode_workspace_size(2, 1, 3)):
        asked.clear()
        for device in (0, 1, 0, 1):
            current(device)
            assert size() == 1000 * (1 + device)
        assert asked == [0, 1]
    latent._size.cache_clear()


@pytest.mark.gpu
def test_every_entry_point_refuses(current):
    bf = dict(dtype=torch.bfloat16, device=DEV)
    q, rows = torch.zeros(4, 2, 128, **bf), torch.zeros(1, 1, 2, 512, **bf)
    cache = torch.zeros(2, 16, 512, **bf)
    one = torch.ones(1, dtype=torch.int32, device=DEV)
    out, lse = latent.kda_latent_fwd(q, q, q)
    calls = [lambda s: latent.kda_latent_fwd(q, q, q, stream=s),
             lambda s: latent.kda_latent_bwd(q, q, q, None, out, lse, q, stream=s),
             lambda s: latent.kda_latent_decode(rows, cache, one.view(1, 1), one, stream=s),
             lambda s: latent.kda_cache_write(cache, rows[0, :, :1], one.view(1, 1), one, stream=s),
             lambda s: latent.kda_cache_copy_pages(cache[None], one, one - 1, stream=s)]
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
