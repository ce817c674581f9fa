"""The norm over a row's channels and its gradient against their 64-bit forms."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_13_gb300 as kda
import rows_util as ru

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
WIDTHS = [1, 2, 7, 64, 100, 512, 513, 1024, 1025, 2047, 3584, 4100, 7168, 8192, 9001, 16384]


def _in(shape, dtype, seed=0, std=1.0, mean=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dtype)


def _vec(W, seed, mean=0.0):
    return _in((W,), F32, seed, 0.3, mean)


def _within(got, want, tol, what):
    err = (got.double() - want).abs()
    assert (err <= tol).all(), f"{what}: worst {(err / tol).max().item():.3g} of the bound"


def _check_fwd(got, x, w, b, center, eps):
    y, mean, rstd = got
    want = ru.norm_ref(x, w, b, center, eps)
    tol = ru.norm_bounds(x, w, b, center, eps, x.dtype)
    _within(y, want[0], tol[0], "out")
    assert (mean is None) == (not center)
    if center:
        _within(mean, want[1], tol[1], "mean")
    _within(rstd, want[2], tol[2], "rstd")


def _check_bwd(got, g, x, w, mean, rstd):
    want = ru.norm_grad_ref(g, x, w, mean, rstd)
    tol = ru.norm_grad_bounds(g, x, w, mean, rstd, x.dtype)
    for name, a, b, t in zip(("d_x", "d_weight", "d_bias"), got, want, tol):
        if a is not None:
            _within(a, b, t, name)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("W", WIDTHS)
def test_against_64_bits(dtype, center, W):
    for n, affine in ((1, True), (5, False), (260, True)):
        x, g = _in((n, W), dtype, 1, 1.5, 0.3), _in((n, W), dtype, 2)
        w, b = (_vec(W, 3, 1.0), _vec(W, 4)) if affine else (None, None)
        got = kda.kda_norm_fwd(x, w, b, center=center)
        _check_fwd(got, x, w, b, center, 1e-5)
        _, mean, rstd = got
        back = kda.kda_norm_bwd(g, x, w, mean, rstd, bias=affine)
        assert (back[1] is None) == (back[2] is None) == (not affine)
        _check_bwd(back, g, x, w, mean, rstd)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off,stride", [(0, 576), (1, 577), (3, 600), (64, 576)])
def test_views(dtype, off, stride):
    """Channels of wider rows, starting on 16 bytes and not; in place; nothing around
    them changes."""
    n, W = 70, 512
    base, gbase = _in((n, stride), dtype, 1), _in((n, stride), dtype, 2)
    x, g = base[:, off:off + W], gbase[:, off:off + W]
    w = _vec(W, 3, 1.0)
    got = kda.kda_norm_fwd(x, w, None, center=False)
    _check_fwd(got, x, w, None, False, 1e-5)
    to = _in((n, stride), dtype, 5)
    around = to.clone()
    kda.kda_norm_fwd(x, w, None, center=False, out=to[:, off:off + W])
    assert torch.equal(to[:, off:off + W], got[0])
    to[:, off:off + W] = around[:, off:off + W]
    assert torch.equal(to, around)
    back = kda.kda_norm_bwd(g, x, w, None, got[2], d_x=to[:, off:off + W])
    _check_bwd(back, g, x, w, None, got[2])
    want = [t.clone() for t in back[:2]]
    into = gbase.clone()
    same = kda.kda_norm_bwd(into[:, off:off + W], x, w, None, got[2], d_x=into[:, off:off + W])
    assert torch.equal(same[0], want[0]) and torch.equal(same[1], want[1])
    copy = base.clone()
    kda.kda_norm_fwd(copy[:, off:off + W], w, None, center=False, out=copy[:, off:off + W])
    assert torch.equal(copy[:, off:off + W], got[0])
    assert torch.equal(copy[:, :off], base[:, :off])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,W,stride", [(7, 513, 520), (5000, 513, 520), (900, 7170, 7176), (3, 30, 32),
                                        (30000, 30, 32)])
def test_rows_that_end_inside_16_bytes(n, W, stride, dtype):
    x, g = _in((n, stride), dtype, 1)[:, :W], _in((n, stride), dtype, 2)[:, :W]
    w = _vec(W, 3, 1.0)
    to = _in((n, stride), dtype, 5)
    around = to[:, W:].clone()
    got = kda.kda_norm_fwd(x, w, w, out=to[:, :W])
    _check_fwd(got, x, w, w, True, 1e-5)
    assert torch.equal(to[:, W:], around)
    _check_bwd(kda.kda_norm_bwd(g, x, w, got[1], got[2], bias=True, d_x=to[:, :W]), g, x, w, *got[1:])
    assert torch.equal(to[:, W:], around)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,W", [(40000, 1), (40000, 25), (20000, 33), (20000, 60), (9000, 100), (5000, 201),
                                 (5000, 300), (5000, 513), (5000, 999), (1300, 1025), (1300, 2047),
                                 (1300, 4095), (700, 7169), (700, 8191), (650, 9001), (650, 16383)])
def test_many_rows_that_start_anywhere(n, W, dtype):
    """Input, output and gradients each at an address and a distance of their own; between the
    rows nothing is written."""
    def view(seed, off, gap):
        buf = _in((off + n * (W + gap),), dtype, seed)
        return buf, buf[off:].view(n, W + gap)[:, :W]

    (_, x), (xo, o) = view(1, 1, 1), view(2, 3, 2)
    (_, g), (xd, d) = view(3, 2, 0), view(4, 0, 5)
    w, b = _vec(W + 1, 5, 1.0)[1:], _vec(W, 6)
    x[5, W // 2] = float("nan")                     # stays in its row
    g[5] = 0.0
    beside, beside_d = xo.clone(), xd.clone()
    got = kda.kda_norm_fwd(x, w, b, out=o)
    keep = torch.arange(n, device=DEV) != 5
    _check_fwd((o[keep], got[1][keep], got[2][keep]), x[keep], w, b, True, 1e-5)
    assert o[5].isnan().all()
    bits = o.clone()
    o.copy_(beside[3:].view(n, W + 2)[:, :W])
    assert torch.equal(xo, beside)                  # all but the rows
    x[5], got[1][5], got[2][5] = 0.0, 0.0, 1.0
    back = kda.kda_norm_bwd(g, x, w, got[1], got[2], bias=True, d_x=d)
    _check_bwd(back, g, x, w, got[1], got[2])
    want = d.clone()
    again = kda.kda_norm_bwd(g, x, w, got[1], got[2], bias=True)
    assert all(torch.equal(u, v) for u, v in zip(back, again))
    d.copy_(beside_d.view(n, W + 5)[:, :W])
    assert torch.equal(xd, beside_d)
    kda.kda_norm_bwd(g, x, w, got[1], got[2], bias=True, d_x=g)     # in place
    assert torch.equal(g, want)
    kda.kda_norm_fwd(x, w, b, out=x)
    assert torch.equal(x[keep], bits[keep])


def test_one_row_and_vectors_anywhere():
    x, w = _in((300,), BF, 1), _vec(301, 3, 1.0)[1:]          # a weight that starts on 4 bytes
    got = kda.kda_norm_fwd(x, w)
    assert got[0].shape == (300,) and got[1].shape == ()
    _check_fwd(got, x, w, None, True, 1e-5)
    rows = x.expand(9, 300)                                   # the same row, nine times
    got = kda.kda_norm_fwd(rows, w)
    _check_fwd(got, rows, w, None, True, 1e-5)
    _check_bwd(kda.kda_norm_bwd(rows, rows, w, *got[1:], bias=True), rows, rows, w, *got[1:])


@pytest.mark.parametrize("n,W,stride", [(3, 512, (1 << 31) + 64), (3, 100, (1 << 31) + 1),
                                        (4_300_000, 512, 512)])
def test_rows_past_two_to_the_31_elements(n, W, stride):
    x = torch.zeros((n - 1) * stride + W, dtype=BF, device=DEV).as_strided((n, W), (stride, 1))
    few = min(n, 300)
    x[-few:] = _in((few, W), BF, 1)
    g, w = x.flip(1) if n == few else x, _vec(W, 3, 1.0)
    out, mean, rstd = kda.kda_norm_fwd(x, w, w)
    _check_fwd((out[-few:], mean[-few:], rstd[-few:]), x[-few:], w, w, True, 1e-5)
    d_x, d_w, d_b = kda.kda_norm_bwd(g, x, w, mean, rstd, bias=True)
    # the other rows' gradients are zeros: they give the sums nothing
    _check_bwd((d_x[-few:], d_w, d_b), g[-few:], x[-few:], w, mean[-few:], rstd[-few:])
    if n == few:
        kda.kda_norm_fwd(x, w, w, out=x)
        assert torch.equal(x, out)


def test_a_mean_far_from_zero():
    x = _in((40, 7168), F32, 1, 1.0, 300.0)
    _check_fwd(kda.kda_norm_fwd(x, None, None), x, None, None, True, 1e-5)


def test_constant_and_zero_rows():
    x = torch.full((3, 200), 2.5, dtype=F32, device=DEV)
    x[1] = 0
    y, mean, rstd = kda.kda_norm_fwd(x, None, None)
    assert torch.equal(y, torch.zeros_like(y))
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
    y, _, rstd = kda.kda_norm_fwd(x, None, None, center=False)
    assert torch.equal(y[1], torch.zeros_like(y[1]))


def test_rows_of_more_dimensions_and_none():
    x = _in((4, 6, 5, 64), BF)[:, :, :3]
    with pytest.raises(ValueError, match="evenly"):
        kda.kda_norm_fwd(x)
    x = _in((4, 6, 64), BF)
    y, mean, rstd = kda.kda_norm_fwd(x)
    assert y.shape == x.shape and mean.shape == rstd.shape == (4, 6)
    _check_fwd((y, mean, rstd), x, None, None, True, 1e-5)
    w = _vec(64, 1)
    y, mean, rstd = kda.kda_norm_fwd(x[:0], w)
    d = kda.kda_norm_bwd(x[:0], x[:0], w, mean, rstd, bias=True)
    assert d[0].shape == (0, 6, 64)
    assert torch.equal(d[1], torch.zeros_like(w)) and torch.equal(d[2], torch.zeros_like(w))
    y, mean, rstd = kda.kda_norm_fwd(x, w, stats=False)
    assert mean is None and rstd is None


def test_not_a_number_stays_in_its_row():
    x, g = _in((20, 700), BF, 1), _in((20, 700), BF, 2)
    x[3, 5] = float("nan")
    x[7, 1] = float("inf")
    y, mean, rstd = kda.kda_norm_fwd(x, None, None)
    good = [i for i in range(20) if i not in (3, 7)]
    assert torch.isfinite(y[good]).all() and torch.isnan(y[3]).all()
    d = kda.kda_norm_bwd(g, x, None, mean, rstd)[0]
    assert torch.isfinite(d[good]).all()


@pytest.mark.parametrize("n,W,dtype", [
    (5000, 512, F32), (3001, 7168, BF), (40001, 40, BF), (40001, 128, BF), (40001, 96, F32), (20001, 256, F32), (20001, 128, BF),
    (20001, 1024, BF), (10001, 500, F32), (5001, 4096, BF), (5001, 2048, F32), (2501, 4096, F32),
    (1301, 16384, BF), (1301, 8192, F32), (1301, 16384, F32), (20001, 25, BF), (5001, 513, BF),
    (3001, 4001, F32), (2001, 7169, BF), (1301, 16383, F32), (1301, 16383, BF)])
def test_many_rows_and_the_same_bits(n, W, dtype):
    x, g = _in((n, W), dtype, 1, 1.2, 0.1), _in((n, W), dtype, 2)
    w = _vec(W, 3, 1.0)
    got = kda.kda_norm_fwd(x, w, None)
    _check_fwd(got, x, w, None, True, 1e-5)
    back = kda.kda_norm_bwd(g, x, w, got[1], got[2], bias=True)
    _check_bwd(back, g, x, w, got[1], got[2])
    got = kda.kda_norm_fwd(x, w, w, center=False)
    _check_fwd(got, x, w, w, False, 1e-5)
    _check_bwd(kda.kda_norm_bwd(g, x, w, None, got[2]), g, x, w, None, got[2])
    got = kda.kda_norm_fwd(x, w, None)
    again = kda.kda_norm_bwd(g, x, w, got[1], got[2], bias=True)
    for a, b in zip(back, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W,gap", [(8, 0), (16, 0), (32, 0), (40, 0), (48, 0), (64, 0), (25, 0), (31, 1), (55, 2)])
def test_short_rows_many_for_each_group(dtype, W, gap):
    """Four or eight threads a row, every group with more rows than it copies ahead (four): on
    16 bytes and anywhere."""
    group = 4 if W <= 32 else 8
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # of the forward 1024 threads an SM, of the gradient 4 blocks of 512
    n = 6 * sms * (4 * 512 // group) + 1
    x, g = _in((n, W + gap), dtype, 1, 1.2, 0.1)[:, :W], _in((n, W + gap), dtype, 2)[:, :W]
    w, b = _vec(W, 3, 1.0), _vec(W, 4)
    got = kda.kda_norm_fwd(x, w, b)
    _check_fwd(got, x, w, b, True, 1e-5)
    back = kda.kda_norm_bwd(g, x, w, got[1], got[2], bias=True)
    _check_bwd(back, g, x, w, got[1], got[2])
    again = kda.kda_norm_bwd(g, x, w, got[1], got[2], bias=True)
    assert all(torch.equal(u, v) for u, v in zip(back, again))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("n,W", [(1, 8), (400001, 8), (500003, 32), (500003, 27), (300007, 64), (300007, 61), (160001, 128),
                                 (160001, 100), (100003, 256), (50001, 512), (40001, 1000), (20001, 1025),
                                 (9001, 4096), (4001, 7169), (3001, 16384)])
def test_sums_over_rows_lose_no_row(n, W, center, dtype):
    """Rows of whole numbers a whole mean apart, of deviation 1: z is -1 or 1 and the gradient
    a small whole number, so that every partial sum, below 3 n < 2^24, is exact in fp32 and a
    row left out or taken twice shows."""
    gen = torch.Generator(device=DEV).manual_seed(7)
    z = torch.randint(0, 2, (n, W), generator=gen, device=DEV, dtype=torch.int32) * 2 - 1
    g = torch.randint(-3, 4, (n, W), generator=gen, device=DEV, dtype=torch.int32)
    m = torch.randint(-9, 10, (n, 1), generator=gen, device=DEV, dtype=torch.int32) if center else 0
    mean = m[:, 0].to(F32) if center else None
    one = torch.ones(n, dtype=F32, device=DEV)
    _, d_w, d_b = kda.kda_norm_bwd(g.to(dtype), (z + m).to(dtype), _vec(W, 3, 1.0), mean, one, bias=True)
    assert torch.equal(d_w, (g * z).sum(0).to(F32))
    assert torch.equal(d_b, g.sum(0).to(F32))


def test_gradient_against_differences():
    """f = <g, y>: f(x + h v) - f(x - h v) is the gradient along the step, but for the
    bounds of the values, those of the gradient, and what a central difference leaves, which
    is taken from the 64-bit form."""
    x, g, v = _in((4, 64), F32, 1), _in((4, 64), F32, 2), _in((4, 64), F32, 3)
    w, b = _vec(64, 4, 1.0), _vec(64, 5)
    h = 2.0 ** -6
    for center in (True, False):
        f = lambda t: (g.double() * kda.kda_norm_fwd(t, w, b, center=center)[0].double()).sum()  # noqa: E731
        f64 = lambda t: (g.double() * ru.norm_ref(t, w, b, center, 1e-5)[0]).sum()  # noqa: E731
        xp, xm = x + h * v, x - h * v                    # as the kernel gets them
        tol = sum((g.double().abs() * ru.norm_bounds(t, w, b, center, 1e-5, F32)[0]).sum()
                  for t in (xp, xm))
        step = (xp.double() - xm.double())
        _, mean, rstd = kda.kda_norm_fwd(x, w, b, center=center)
        d = kda.kda_norm_bwd(g, x, w, mean, rstd)[0].double()
        exact_grad = ru.norm_grad_ref(g, x, w, *(t if t is None else t.double() for t in
                                                 (mean, rstd)))[0]
        curve = abs(f64(xp.double()) - f64(xm.double()) - (exact_grad * step).sum())
        slack = (ru.norm_grad_bounds(g, x, w, mean, rstd, F32)[0] * step.abs()).sum()
        assert abs(f(xp) - f(xm) - (d * step).sum()) <= tol + slack + curve
        assert curve < 0.05 * abs((exact_grad * step).sum()) + 0.02


def test_streams_and_graphs():
    x, g, w = _in((300, 512), BF, 1), _in((300, 512), BF, 2), _vec(512, 3, 1.0)
    want = kda.kda_norm_fwd(x, w, w)
    grad = kda.kda_norm_bwd(g, x, w, want[1], want[2], bias=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.kda_norm_fwd(x, w, w, stream=s)
    back = kda.kda_norm_bwd(g, x, w, got[1], got[2], bias=True, stream=s)
    s.synchronize()
    for a, b in zip((*got, *back), (*want, *grad)):
        assert torch.equal(a, b)
    ws = torch.empty(kda.kda_norm_bwd_workspace_size(300, 512), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, mean, rstd = kda.kda_norm_fwd(x, w, w)
        d = kda.kda_norm_bwd(g, x, w, mean, rstd, bias=True, workspace=ws)
    x.mul_(0.5)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    _check_fwd((y, mean, rstd), x, w, w, True, 1e-5)
    _check_bwd(d, g, x, w, mean, rstd)


def test_refusals():
    x, w = _in((8, 64), BF), _vec(64, 1)
    _, mean, rstd = kda.kda_norm_fwd(x, w)
    for call in (lambda: kda.kda_norm_fwd(x.half()), lambda: kda.kda_norm_fwd(x.cpu()),
                 lambda: kda.kda_norm_fwd(x, w.bfloat16()), lambda: kda.kda_norm_fwd(x, w[:32]),
                 lambda: kda.kda_norm_fwd(x, eps=0.0), lambda: kda.kda_norm_fwd(x[:, ::2]),
                 lambda: kda.kda_norm_fwd(x, out=x.float()), lambda: kda.kda_norm_fwd(x, out=x[:4]),
                 lambda: kda.kda_norm_bwd(x[:4], x, w, mean, rstd),
                 lambda: kda.kda_norm_bwd(x, x, w, mean[:4], rstd),
                 lambda: kda.kda_norm_bwd(x, x, w, mean, rstd.double()),
                 lambda: kda.kda_norm_bwd(x.float(), x, w, mean, rstd)):
        with pytest.raises((TypeError, ValueError)):
            call()
    wide = _in((8, 100), BF)
    with pytest.raises(kda.KDAError):
        kda.kda_norm_fwd(wide[:, :64], out=wide[:, 1:65])
    with pytest.raises(kda.KDAError):
        kda.kda_norm_fwd(_in((2, 16385), BF))
    with pytest.raises(kda.KDAError):
        kda.kda_norm_bwd(x, x, w, mean, rstd, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
