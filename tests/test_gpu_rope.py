"""Rotary positions against their 64-bit form, over layouts, views and positions."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_13_gb300 as kda
import rows_util as ru

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def _in(shape, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def _pos(n, far, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-far, far, n, generator=g, device=DEV).to(torch.int32)


def _freq(dr):
    return kda.kda_rope_inv_freq(dr, device=DEV)


def _check(got, x, pos, freq, interleaved, scale, transpose):
    want = ru.rope_ref(x, pos, freq, interleaved, scale, transpose)
    tol = ru.rope_bound(x, interleaved, scale, x.dtype, want)
    # the 64-bit form's own angle: a position times 2^-53 of a turn or so, far below
    err = (got.double() - want).abs()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.3g} of the bound"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,H,dr", [(1, 1, 2), (1, 96, 64), (3, 3, 6), (64, 96, 64), (300, 16, 64),
                                    (5, 128, 128), (700, 1, 64), (33, 7, 512), (40, 5, 74),
                                    (2000, 40, 16), (9, 300, 8)])
def test_against_64_bits(dtype, interleaved, n, H, dr):
    x, pos, freq = _in((n, H, dr), dtype), _pos((n,), 1 << 20), _freq(dr)
    k = _in((n, dr), dtype, 5)
    before = x.clone()
    got = kda.kda_rope(x, pos, freq, interleaved=interleaved)
    _check(got, x, pos, freq, interleaved, 1.0, False)
    back, k_back = kda.kda_rope(x, pos, freq, k=k, interleaved=interleaved, scale=1.35,
                                transpose=True)
    _check(back, x, pos, freq, interleaved, 1.35, True)
    _check(k_back, k, pos, freq, interleaved, 1.35, True)
    assert torch.equal(x, before)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("n,H,dr,off", [(2500, 33, 68, 0), (3000, 40, 20, 0), (700, 16, 126, 0), (40, 3, 510, 2),
                                        (2000, 96, 72, 4), (1, 200, 12, 0), (900, 17, 64, 2), (20000, 1, 2, 0),
                                        (5, 7, 200, 1)])
def test_pieces_of_any_width(dtype, interleaved, n, H, dr, off):
    """Rows that start on 8, 4 or 2 bytes, and of any number of pieces."""
    buf, pos, freq = _in((n, H, dr + 2 * off), dtype), _pos((n,), 1 << 20), _freq(dr)
    before, x = buf.clone(), buf[..., off:off + dr]
    k = _in((n, dr), dtype, 5)
    out, k_out = kda.kda_rope(x, pos, freq, k=k, interleaved=interleaved)
    _check(out, x, pos, freq, interleaved, 1.0, False)
    _check(k_out, k, pos, freq, interleaved, 1.0, False)
    kda.kda_rope(x, pos, freq, interleaved=interleaved, out=x)          # in place
    assert torch.equal(x, out)
    x.copy_(before[..., off:off + dr])
    assert torch.equal(buf, before)                                     # nothing around it


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_views_in_place_and_between_buffers(dtype, off):
    """The rotary channels of wider heads and of cached rows, both parts of one
    projection: nothing around them changes."""
    n, H, dr = 37, 6, 64
    base = _in((n, off + H * 192 + 576), dtype)
    pos, freq = _pos((n,), 5000), _freq(dr)
    q = base[:, off:off + H * 192].unflatten(1, (H, 192))[..., 128:]
    k = base[:, off + H * 192:][:, 512:]
    want_q, want_k, before = q.clone(), k.clone(), base.clone()
    to = _in((n, H, 576), dtype, 9)
    to_before = to.clone()
    got = kda.kda_rope(q, pos, freq, out=to[..., 512:])
    assert got.data_ptr() == to[..., 512:].data_ptr()
    _check(got, want_q, pos, freq, True, 1.0, False)
    assert torch.equal(to[..., :512], to_before[..., :512]) and torch.equal(base, before)
    a, b = kda.kda_rope(q, pos, freq, k=k, out=q, k_out=k, interleaved=False)
    assert a is q and b is k
    _check(q, want_q, pos, freq, False, 1.0, False)
    _check(k, want_k, pos, freq, False, 1.0, False)
    rest = torch.ones(base.shape[1], dtype=torch.bool, device=DEV)
    rest[off:off + H * 192].view(H, 192)[:, 128:] = False
    rest[off + H * 192 + 512:] = False
    assert torch.equal(base[:, rest], before[:, rest])


def test_batches_of_tokens_and_no_heads():
    B, T, H, dr = 3, 5, 4, 64
    rows = _in((B, T, 576), BF)
    pos, freq = _pos((B, T), 100000), _freq(dr)
    got = kda.kda_rope(rows[..., 512:], pos, freq)
    assert got.shape == (B, T, dr)
    _check(got, rows[..., 512:], pos, freq, True, 1.0, False)
    q = _in((B, T, H, 192), BF)[..., 128:]
    _check(kda.kda_rope(q, pos, freq), q, pos, freq, True, 1.0, False)
    one = _in((1, dr), BF)                       # the same row for all heads and tokens
    x = one[:, None].expand(7, 3, dr)
    p = _pos((7,), 1000)
    _check(kda.kda_rope(x, p, freq), x, p, freq, True, 1.0, False)
    here = torch.tensor(77, dtype=torch.int32, device=DEV)   # one token, by itself
    _check(kda.kda_rope(q[0, 0], here, freq), q[0, 0], here, freq, True, 1.0, False)
    empty = kda.kda_rope(q[:0], pos[:0], freq)
    assert empty.shape == (0, T, H, dr)


def test_the_farthest_positions():
    """Positions at the ends of 32 bits: the angle is a fraction of a turn all the same.
    The 64-bit form is taken from the frequency's exact fraction."""
    from fractions import Fraction
    dr = 64
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 1 << 30, 12345678], dtype=torch.int32, device=DEV)
    freq = _freq(dr)
    x = _in((5, 2, dr), F32)
    # 1 / (2 pi) to 120 bits
    inv = Fraction(211553206025302378997855913028439351, 2 ** 120)
    turns = torch.tensor([[float((Fraction(f) * inv * p) % 1) for f in freq.tolist()]
                          for p in pos.tolist()], dtype=torch.float64, device=DEV)
    c, s = torch.cos(2 * torch.pi * turns)[:, None], torch.sin(2 * torch.pi * turns)[:, None]
    a, b = x[..., 0::2].double(), x[..., 1::2].double()
    want = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    got = kda.kda_rope(x, pos, freq)
    assert ((got.double() - want).abs() <= ru.rope_bound(x, True, 1.0, F32, want)).all()


def _turned_exactly(x, pos, freq):
    """x [n, 2 m] of neighbouring pairs, by fractions of a turn of integers."""
    from fractions import Fraction
    inv = Fraction(0x28be60db9391054a7f09d5f47d4d377036d8a5664f10e4107f9458eaf7ae, 2 ** 240)    # 1 / (2 pi)
    turns = torch.tensor([[float(Fraction(f) * inv * p % 1) for f in freq.tolist()] for p in pos.tolist()],
                         dtype=torch.float64, device=DEV)
    c, s = torch.cos(2 * torch.pi * turns), torch.sin(2 * torch.pi * turns)
    a, b = x[..., 0::2].double(), x[..., 1::2].double()
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_frequencies_that_have_no_angle(dtype, interleaved):
    """No number, infinite or of 2^64 and more: no number in their pairs, others as without."""
    freq = _freq(64)
    bad = freq.clone()
    none = {0: float("nan"), 3: float("inf"), 8: float("-inf"), 13: 2.0 ** 64, 14: -2.0 ** 118, 31: 1.5e308}
    for i, f in none.items():
        bad[i] = f
    x, pos = _in((7, 3, 64), dtype), _pos((7,), 1000)
    pos[2] = 0
    want, got = (kda.kda_rope(x, pos, f, interleaved=interleaved) for f in (freq, bad))
    for i in range(32):
        for ch in ((2 * i, 2 * i + 1) if interleaved else (i, i + 32)):
            if i in none:
                assert got[..., ch].isnan().all(), i
            else:
                assert torch.equal(got[..., ch], want[..., ch]), i


def test_frequencies_of_any_magnitude():
    """Up to 2^64 radians a position the angle is right, whatever the position."""
    freq = torch.tensor([2.0 ** -1070, 1e-300, 3e-20, 2.0 ** -40, 0.7, -0.7, 123.456, 1e6 / 3, 2.0 ** 40 + 0.25,
                         -1.7e15, 1.9 * 2.0 ** 62, -1.99999 * 2.0 ** 63], dtype=torch.float64, device=DEV)
    pos = torch.tensor([0, 1, -1, 77, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32, device=DEV)
    x = _in((7, 24), F32)
    want = _turned_exactly(x, pos, freq)
    got = kda.kda_rope(x, pos, freq)
    assert ((got.double() - want).abs() <= ru.rope_bound(x, True, 1.0, F32, want)).all()


@pytest.mark.parametrize("interleaved", [True, False])
def test_tokens_past_two_to_the_31_elements(interleaved):
    far, n, H, dr = (1 << 31) + 64, 3, 5, 64
    buf = torch.zeros(2 * far + H * dr, dtype=BF, device=DEV)
    x = buf.as_strided((n, H, dr), (far, dr, 1))
    x.copy_(_in((n, H, dr), BF, 3))
    pos, freq = _pos((n,), 1 << 20), _freq(dr)
    _check(kda.kda_rope(x, pos, freq, interleaved=interleaved), x, pos, freq, interleaved, 1.0, False)
    want = kda.kda_rope(x, pos, freq, interleaved=interleaved)
    kda.kda_rope(x, pos, freq, interleaved=interleaved, out=x)
    assert torch.equal(x, want)


def test_turning_back_is_the_gradient():
    """<g, rope(x)> = <rope^T(g), x>, and its difference along any direction."""
    x, g = _in((50, 8, 64), F32), _in((50, 8, 64), F32, 3)
    v = _in((50, 8, 64), F32, 4)
    pos, freq = _pos((50,), 3000), _freq(64)
    f = lambda t: (g.double() * kda.kda_rope(t, pos, freq, scale=1.2).double()).sum()  # noqa: E731
    grad = kda.kda_rope(g, pos, freq, scale=1.2, transpose=True).double()
    # every value is off by at most 10 u of its pair's length; the map is linear, so that
    # the difference has no other error: |g| |x| 10 u scale sqrt 2 each side, and x + v's
    # own rounding, u |x + v|
    off = 20 * ru.U * 1.2 * g.double().norm() * (x.double().norm() + v.double().norm()) * 2
    assert abs((f(x + v) - f(x - v)) / 2 - (grad * v.double()).sum()) <= off
    assert abs(f(x) - (grad * x.double()).sum()) <= off


def test_not_a_number_stays_in_its_pair():
    x = _in((4, 2, 64), BF)
    x[1, 1, 10] = float("nan")
    pos, freq = _pos((4,), 100), _freq(64)
    got = kda.kda_rope(x, pos, freq)
    bad = torch.isnan(got).nonzero().tolist()
    assert bad == [[1, 1, 10], [1, 1, 11]]


def test_streams_and_graphs():
    x, pos, freq = _in((64, 96, 64), BF), _pos((64,), 4096), _freq(64)
    want = kda.kda_rope(x, pos, freq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.kda_rope(x, pos, freq, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_rope(x, pos, freq, out=out)
    pos.add_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, kda.kda_rope(x, pos, freq))


def test_refusals():
    x, pos, freq = _in((8, 4, 64), BF), _pos((8,), 100), _freq(64)
    k = _in((8, 64), BF)
    for bad in (dict(x=x.half()), dict(x=x.cpu()), dict(positions=pos.long()), dict(positions=pos[:4]),
                dict(inv_freq=freq.float()), dict(inv_freq=freq[:16]), dict(k=k.float()),
                dict(k=k[:4]), dict(k_out=k), dict(out=x[:, :2]), dict(out=x.float()),
                dict(scale=float("nan")), dict(x=x[..., ::2], inv_freq=freq[:16]),
                dict(x=x.transpose(0, 1).contiguous().transpose(0, 1)[..., :63], inv_freq=freq)):
        args = dict(x=x, positions=pos, inv_freq=freq)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            kda.kda_rope(args.pop("x"), args.pop("positions"), args.pop("inv_freq"), **args)
    wide = _in((8, 4, 100), BF)
    for bad in (wide[..., 1:65], wide[..., 30:94]):     # meets x's rows
        with pytest.raises(kda.KDAError):
            kda.kda_rope(wide[..., :64], pos, freq, out=bad)
    with pytest.raises(kda.KDAError):
        kda.kda_rope(x, pos, freq, out=x[:1, :1].expand(8, 4, 64))


def test_small_sines_keep_their_digits():
    """Positions that come to within 2^-10 of half a turn and of whole ones: an angle in fp32
    would be off by 2^-25 of half a turn there, 9e-8.  Of 32 bits and the ones below it is off
    by at most 2^-32 of a turn, and the frequency's share; a small sine rounds by little: four
    times by half a step, and CUDA's own 2 steps, 8 u of itself."""
    pos = torch.arange(-(1 << 20), 1 << 20, dtype=torch.int32, device=DEV)
    sine = torch.sin(pos.double())
    pos = pos[sine.abs() < 2.0 ** -10]
    assert len(pos) > 1000
    sine, x = torch.sin(pos.double()), torch.zeros(len(pos), 2, device=DEV)
    x[:, 0] = 1.0
    freq = torch.ones(1, dtype=torch.float64, device=DEV)
    tol = 2 * torch.pi * 2.0 ** -31 + 8 * ru.U * sine.abs()
    for transpose in (False, True):
        got = kda.kda_rope(x, pos, freq, transpose=transpose)
        err = (got[:, 1].double() - (-sine if transpose else sine)).abs()
        assert (err <= tol).all(), f"worst {(err / tol).max().item():.3g} of the bound"
