"""The gradient's d_k and d_v may be two views of one tensor, but no row of one may meet a
row of the other (no GPU: pointers are fake; a call that is not refused for its views is
refused for its missing workspace)."""
from __future__ import annotations

import random

import pytest

from test_latent_host import A, _bwd, _fwd, lib  # noqa: F401

REFUSED, TAKEN = 1, 3


def _views(lib, offset, ts, hs, n, H, ts2=None, hs2=None):  # noqa: F811
    """offset: of d_v from d_k, in elements."""
    q_strides = dict(kts=H * 128, khs=128, vts=H * 128, vhs=128)
    return _bwd(lib, gk=11 * A, gv=11 * A + 2 * offset, gkts=ts, gkhs=hs, gvts=ts2 or ts,
                gvhs=hs2 or hs, nk=n, H=H, ws=None, **q_strides)


@pytest.mark.parametrize("offset,want", [
    (128, TAKEN), (-128, TAKEN), (64, REFUSED), (-64, REFUSED), (120, REFUSED), (136, REFUSED),
    (1024, REFUSED), (3 * 1024 + 128, TAKEN), (3 * 1024 + 256, REFUSED), (-5 * 1024 - 256, REFUSED),
    (120 * 1024, TAKEN), (119 * 1024, REFUSED), (119 * 1024 + 768 + 128, TAKEN),
    (119 * 1024 + 768 + 120, REFUSED), (3 * 256 + 128, TAKEN), (-3 * 256 - 128, TAKEN)])
def test_interleaved_heads(lib, offset, want):  # noqa: F811
    assert _views(lib, offset, 1024, 256, 120, 4) == want


@pytest.mark.parametrize("offset,want", [
    (120 * 128, TAKEN), (119 * 128, REFUSED), (120 * 128 + 8, REFUSED), (-120 * 128, TAKEN),
    (7 * 240 * 128, TAKEN), (3 * 240 * 128, REFUSED)])
def test_head_major(lib, offset, want):  # noqa: F811
    assert _views(lib, offset, 128, 240 * 128, 120, 4) == want


def test_strides_of_a_single_row_do_not_matter(lib):  # noqa: F811
    assert _views(lib, 128, 8, 8, 1, 1) == TAKEN
    assert _views(lib, 120, 8, 8, 1, 1) == REFUSED
    assert _views(lib, 120, 8, 256, 1, 4, ts2=16) == REFUSED
    assert _views(lib, 128, 8, 256, 1, 4, ts2=16) == TAKEN
    assert _views(lib, 120, 256, 8, 9, 1, hs2=16) == REFUSED
    assert _views(lib, 128, 256, 8, 9, 1, hs2=16) == TAKEN


def test_against_every_pair_of_rows(lib):  # noqa: F811
    rng = random.Random(1)
    seen = {REFUSED: 0, TAKEN: 0}
    for _ in range(400):
        n, H = rng.randint(1, 5), rng.randint(1, 5)
        small = 128 + 8 * rng.randint(0, 40)
        if rng.random() < 0.5:
            hs, ts = small, (H - 1) * small + 128 + 8 * rng.randint(0, 80)
        else:
            ts, hs = small, (n - 1) * small + 128 + 8 * rng.randint(0, 80)
        offset = 8 * rng.randint(-300, 300)
        rows = [i * ts + h * hs for i in range(n) for h in range(H)]
        meet = any(abs(offset + b - a) < 128 for a in rows for b in rows)
        want = REFUSED if meet else TAKEN
        seen[want] += 1
        assert _views(lib, offset, ts, hs, n, H) == want, (offset, ts, hs, n, H)
    assert min(seen.values()) > 50


# Spans of 2^64 bytes and more, which come round to some that meet nothing; ws=None: a call
# that is not refused for its views is refused for its missing workspace.
FAR = dict(nk=(1 << 31) - 256, H=1, ws=None, k=1 << 44, v=2 << 44, r=3 << 44, gk=5 << 44, gv=6 << 44,
           gr=7 << 44)


@pytest.mark.parametrize("over", [dict(kts=1 << 38), dict(vts=1 << 38), dict(vts=1 << 33)])
def test_views_past_64_bits(lib, over):  # noqa: F811
    assert _fwd(lib, **dict(FAR, **over)) == REFUSED
    assert _bwd(lib, **dict(FAR, **over)) == REFUSED


@pytest.mark.parametrize("over", [dict(gkts=1 << 38), dict(gvts=1 << 38), dict(gkts=1 << 38, gvts=1 << 38)])
def test_gradient_views_past_64_bits(lib, over):  # noqa: F811
    assert _bwd(lib, **dict(FAR, **over)) == REFUSED
