"""Latent attention on the GPU against its definition in 64 bits, element by
element within the bounds derived in latent_util."""
from __future__ import annotations

import math

import pytest
import torch

import gated_delta_rule_13_gb300 as pkg
import latent_util as lu

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _cu(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)


def _randn(*shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).bfloat16()


def _problem(lens_q, lens_k, H, dr, layout="kv", seed=0):
    nq, nk = sum(lens_q), sum(lens_k)
    if layout == "kv":          # two views of one projection
        kv = _randn(nk, H, 256, seed=seed)
        k, v = kv[..., :128], kv[..., 128:]
    elif layout == "heads":     # head-major
        k = _randn(H, nk, 128, seed=seed).transpose(0, 1)
        v = _randn(H, nk, 136, seed=seed + 1).transpose(0, 1)[..., 8:]
    else:
        k, v = _randn(nk, H, 128, seed=seed), _randn(nk, H, 128, seed=seed + 1)
    return dict(q=_randn(nq, H, 128 + dr, seed=seed + 2), k=k, v=v,
                k_rope=_randn(nk, dr, seed=seed + 3) if dr else None,
                cu_q=_cu(lens_q), cu_k=_cu(lens_k))


def _fwd(x, **kw):
    return pkg.kda_latent_fwd(x["q"], x["k"], x["v"], x["k_rope"], x["cu_q"], x["cu_k"], **kw)


def _bwd(x, out, lse, d_out, **kw):
    return pkg.kda_latent_bwd(x["q"], x["k"], x["v"], x["k_rope"], out, lse, d_out, x["cu_q"],
                              x["cu_k"], **kw)


def check_both(x, causal=True, scale=None, seed=50):
    sc = scale or 1 / math.sqrt(x["q"].shape[2])
    out, lse = _fwd(x, causal=causal, scale=scale)
    r_out, r_lse, t_out, t_lse = lu.fwd_ref(**x, causal=causal, scale=sc)
    lu.check("out", out, r_out, t_out)
    lu.check("lse", lse, r_lse, t_lse)
    d_out = _randn(*out.shape, seed=seed)
    got = _bwd(x, out, lse, d_out, causal=causal, scale=scale)
    ref, tol = lu.bwd_ref(x["q"], x["k"], x["v"], x["k_rope"], out, lse, d_out, x["cu_q"],
                          x["cu_k"], causal, sc)
    for name, t in zip(("dq", "dk", "dv", "dr"), got):
        if t is not None:
            lu.check(name, t, ref[name], tol[name])


LENGTHS = [([1], [1]), ([5, 0, 130, 64], [5, 7, 130, 257]), ([127, 128, 129], [127, 128, 129]),
           ([1, 2, 300], [1000, 3, 700]), ([255, 65], [255, 63]), ([10, 40], [4, 0])]


@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("lens", LENGTHS)
def test_lengths(lens, dr):
    check_both(_problem(*lens, H=3, dr=dr))


@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("lens", [([5, 0, 130, 64], [5, 7, 130, 257]), ([200, 10], [3, 321])])
def test_not_causal(lens, dr):
    check_both(_problem(*lens, H=2, dr=dr), causal=False)


@pytest.mark.parametrize("layout", ["heads", "plain"])
@pytest.mark.parametrize("H", [1, 5])
def test_layouts(layout, H):
    check_both(_problem([70, 150], [70, 210], H=H, dr=64, layout=layout))


def test_many_short_sequences():
    lens = [(7 * i) % 40 for i in range(75)]
    check_both(_problem(lens, lens, H=2, dr=0))


def test_long_sequence():
    check_both(_problem([1500], [1700], H=1, dr=64))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("lens", [([3], [5000]), ([300, 1], [2500, 4100]), ([257], [1100])])
def test_few_queries_over_many_keys(lens, dr, causal):
    """Few work items: their keys are shared out over several CTAs and joined."""
    check_both(_problem(*lens, H=2, dr=dr), causal=causal)


@pytest.mark.parametrize("n", [31, 32, 33, 700, 2500])
def test_sequence_counts(n):
    """Up to 32 sequences are found in a warp's lanes, more through a table."""
    lens_q = [(5 * i) % 13 for i in range(n)]
    lens_k = [q + (3 * i) % 7 for i, q in enumerate(lens_q)]
    lens_q[n // 2], lens_k[n // 2] = 300, 420
    check_both(_problem(lens_q, lens_k, H=1, dr=64 if n % 2 else 0))


def test_graph_of_both_directions():
    x = _problem([100, 300], [100, 300], H=2, dr=64)
    d_out = _randn(400, 2, 128, seed=3)
    want = _fwd(x)
    want_g = _bwd(x, *want, d_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = _fwd(x)
        grads = _bwd(x, out, lse, d_out)
    for t in (out, lse, *grads):
        t.zero_()
    graph.replay()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for a, b in zip(want_g, grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [0.5, 1e-3, 3.0])
def test_scales(scale):
    check_both(_problem([130, 200], [130, 400], H=2, dr=64), scale=scale)


def test_growing_scores():
    """Every later key raises the running maximum by far."""
    x = _problem([40, 300], [500, 300], H=2, dr=0)
    ramp = torch.linspace(0.02, 12, 800, device=DEV).view(-1, 1, 1)
    x["k"] = (x["q"][:1].float() * ramp).bfloat16() + x["k"]
    check_both(x)


def test_one_sequence_without_cu():
    x = _problem([90], [90], H=2, dr=64)
    a = _fwd(x)
    b = pkg.kda_latent_fwd(x["q"], x["k"], x["v"], x["k_rope"])
    c = pkg.kda_latent_fwd(x["q"], x["k"], x["v"], x["k_rope"], x["cu_q"].cpu(), x["cu_k"].cpu())
    for y in (b, c):
        assert torch.equal(a[0], y[0]) and torch.equal(a[1], y[1])


def test_no_tokens():
    x = _problem([0], [5], H=2, dr=64)
    out, lse = _fwd(x)
    assert out.shape == (0, 2, 128)
    got = _bwd(x, out, lse, out)
    assert all(float(t.float().abs().sum()) == 0 for t in got)
    x = _problem([5], [0], H=2, dr=0)
    out, lse = _fwd(x)
    assert float(out.float().abs().sum()) == 0 and bool((lse == -math.inf).all())
    assert float(_bwd(x, out, lse, out)[0].float().abs().sum()) == 0


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_other_sequences_never_matter(poison):
    """A sequence of NaN or infinities between two others leaves them as they are."""
    lens_q, lens_k = [70, 20, 100], [75, 33, 100]
    x = _problem(lens_q, lens_k, H=2, dr=64)
    d_out = _randn(190, 2, 128, seed=9)
    out, lse = _fwd(x)
    grads = _bwd(x, out, lse, d_out)
    y = {n: t.clone() if t is not None else None for n, t in x.items()}
    for n in ("k", "v", "k_rope"):
        y[n][75:108] = poison
    y["q"][70:90] = poison
    out2, lse2 = _fwd(y)
    d2 = d_out.clone()
    d2[70:90] = poison
    grads2 = _bwd(y, out2, lse2, d2)
    for a, b in ((out, out2), (lse, lse2), (grads[0], grads2[0])):
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[90:], b[90:])
    for a, b in zip(grads[1:], grads2[1:]):
        assert torch.equal(a[:75], b[:75]) and torch.equal(a[108:], b[108:])


def test_gradients_do_not_vary_and_fit_strided_outputs():
    x = _problem([300, 200], [300, 333], H=4, dr=64)
    out, lse = _fwd(x)
    d_out = _randn(*out.shape, seed=4)
    a = _bwd(x, out, lse, d_out)
    g = torch.full((633, 4, 256), 7.0, device=DEV).bfloat16()
    b = _bwd(x, out, lse, d_out, d_k=g[..., :128], d_v=g[..., 128:])
    assert b[1].data_ptr() == g.data_ptr()
    for s, t in zip(a, b):
        assert torch.equal(s, t)


def test_bad_cu_seqlens_are_reported():
    from gated_delta_rule_13_gb300 import kda
    x = _problem([30, 40], [30, 40], H=2, dr=0)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    out = torch.full((70, 2, 128), 3.0, device=DEV).bfloat16()
    x["cu_q"] = torch.tensor([0, 80, 70], dtype=torch.int32, device=DEV)
    _fwd(x, out=out, workspace=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_ERR_INVALID_ARG
    assert bool((out == 3.0).all())
    x["cu_q"] = x["cu_q"].cpu()
    with pytest.raises(pkg.KDAError):
        _fwd(x, out=out, workspace=ws)


@pytest.mark.parametrize("n", [5, 100])
@pytest.mark.parametrize("which", ["cu_q", "cu_k"])
@pytest.mark.parametrize("how", ["first", "order", "last", "past"])
def test_malformed_cu_seqlens(n, which, how):
    from gated_delta_rule_13_gb300 import kda
    x = _problem([7] * n, [7] * n, H=2, dr=64)
    out, lse = _fwd(x)
    bad = x[which].clone()
    if how == "first":
        bad[0] = 1
    elif how == "order":
        bad[3] = 7 * n
    elif how == "last":
        bad[n] -= 1
    else:
        bad[n // 2] = 1 << 30
    y = dict(x, **{which: bad})
    ws = torch.empty(1 << 25, dtype=torch.uint8, device=DEV)
    keep = torch.full_like(out, 3.0)
    _fwd(y, out=keep, workspace=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_ERR_INVALID_ARG
    assert bool((keep == 3.0).all())
    g = torch.full((2, 7 * n, 2, 128), 3.0, device=DEV).bfloat16()
    _bwd(y, out, lse, out, d_k=g[0], d_v=g[1], workspace=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_ERR_INVALID_ARG
    assert bool((g == 3.0).all())
    _fwd(x, workspace=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_OK


def test_keys_past_two_to_the_31_elements():
    n, H = 90000, 96
    kv = torch.zeros(n, H, 256, dtype=torch.bfloat16, device=DEV)
    kv[-200:] = _randn(200, H, 256, seed=1)
    q = _randn(3, H, 128, seed=2)
    heads = [0, 50, 95]
    out, lse = pkg.kda_latent_fwd(q, kv[..., :128], kv[..., 128:], None, _cu([3]), _cu([n]))
    ref = lu.fwd_ref(q[:, heads], kv[:, heads, :128], kv[:, heads, 128:], None, _cu([3]), _cu([n]),
                     True, 1 / math.sqrt(128))
    lu.check("out", out[:, heads], ref[0], ref[2])
    lu.check("lse", lse[:, heads], ref[1], ref[3])


# ------------------------------------------------------------------ absorbed form
def _decode_problem(lens, T, H, dr, page, seed=0, tree=False):
    cache, table = lu.paged(lens, page, 512 + dr, DEV, seed=seed)
    return dict(q=_randn(len(lens), T, H, 512 + dr, seed=seed + 1), cache=cache, table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                mask=lu.tree_masks(len(lens), T, seed).to(DEV) if tree else None)


def check_decode(x, scale=None):
    B, T, H, W = x["q"].shape
    lse = torch.empty(B, T, H, device=DEV)
    out = pkg.kda_latent_decode(x["q"], x["cache"], x["table"], x["lens"], tree_mask=x["mask"],
                                scale=scale, lse=lse)
    r_out, r_lse, t_out, t_lse = lu.decode_ref(x["q"], x["cache"], x["table"], x["lens"],
                                               x["mask"], scale or 1 / math.sqrt(W - 384))
    lu.check("out", out, r_out, t_out)
    lu.check("lse", lse, r_lse, t_lse)
    return out


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]


@pytest.mark.parametrize("dr", [0, 64])
@pytest.mark.parametrize("page", [16, 48, 64, 128, 512])
def test_decode_lengths(page, dr):
    check_decode(_decode_problem(EDGES, 1, 5, dr, page))


@pytest.mark.parametrize("H", [1, 7, 16, 33, 64, 96, 97, 128])
def test_decode_heads(H):
    check_decode(_decode_problem([200, 5, 1000], 1, H, 64, 64))


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("T,H", [(2, 96), (3, 7), (8, 16), (24, 5), (64, 2)])
def test_decode_drafts(T, H, tree):
    lens = [T, T + 1, 130, 500, 128 + T // 2, 257]
    check_decode(_decode_problem([max(n, T) for n in lens], T, H, 64, 64, tree=tree))


def test_more_drafts_than_a_mask_holds():
    check_decode(_decode_problem([70, 300], 70, 3, 0, 16))


def test_decode_rows_that_see_nothing():
    """Shorter sequences than drafts, and masks that leave rows empty."""
    x = _decode_problem([3, 8, 0, 40], 8, 4, 64, 16)
    check_decode(x)
    x["mask"] = torch.zeros(4, 8, dtype=torch.int64, device=DEV)
    x["mask"][1, 3] = 1 << 5
    x["mask"][3, 2] = -1    # every bit, also those past the T drafts
    check_decode(x)


def test_decode_growing_scores():
    x = _decode_problem([700, 90], 2, 16, 0, 64)
    ramp = torch.linspace(0.02, 3, 700, device=DEV)
    for b, n in enumerate((700, 90)):
        pos = torch.arange(n, device=DEV)
        page, at = x["table"][b].long()[pos // 64], pos % 64
        x["cache"][page, at] = (x["cache"][page, at].float()
                                + ramp[:n, None] * x["q"][b, 0, 0].float()).bfloat16()
    check_decode(x)


@pytest.mark.parametrize("scale", [0.5, 1e-3])
def test_decode_scales(scale):
    check_decode(_decode_problem([200, 31], 2, 16, 64, 64), scale=scale)


def test_decode_long_and_short_together():
    check_decode(_decode_problem([9000, 1, 17, 4000, 300], 1, 16, 64, 64))


def test_decode_one_long_sequence():
    check_decode(_decode_problem([20000], 1, 96, 0, 512))


def test_decode_many_sequences():
    lens = [(37 * i) % 400 for i in range(333)]
    check_decode(_decode_problem(lens, 1, 4, 0, 16))


def test_decode_pool_past_two_to_the_31_elements():
    page, n_pages = 512, 8200                       # 2.4e9 elements
    cache = torch.empty(n_pages, page, 576, dtype=torch.bfloat16, device=DEV)
    cache[-3:] = _randn(3, page, 576, seed=3)
    table = torch.tensor([[n_pages - 1, n_pages - 3, n_pages - 2]], dtype=torch.int32, device=DEV)
    check_decode(dict(q=_randn(1, 1, 8, 576, seed=5), cache=cache, table=table, mask=None,
                      lens=torch.tensor([1300], dtype=torch.int32, device=DEV)))


def test_decode_bad_lengths_and_pages_are_reported():
    from gated_delta_rule_13_gb300 import kda
    x = _decode_problem([100, 200, 50], 1, 16, 64, 64)
    ref = check_decode(x)
    ws = torch.empty(pkg.kda_latent_decode_workspace_size(3, 1, 16, dr=64), dtype=torch.uint8,
                     device=DEV)

    def run():
        return pkg.kda_latent_decode(x["q"], x["cache"], x["table"], x["lens"], workspace=ws)

    run()
    assert kda.kda_read_device_status(ws) == kda.KDA_OK
    for bad in (-1, 1 << 30):
        x["lens"][1] = bad
        out = run()
        assert kda.kda_read_device_status(ws) == kda.KDA_ERR_INVALID_ARG
        assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
    x["lens"][1] = 200
    for bad in (-1, 1 << 30, x["cache"].shape[0]):
        x["table"][1, 1] = bad
        out = run()
        assert kda.kda_read_device_status(ws) == kda.KDA_ERR_INVALID_ARG
        assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])


def test_graph_replay_on_new_lengths():
    """One captured call serves every step: lengths, pages and queries are data."""
    x = _decode_problem([100, 700, 50], 2, 16, 64, 64)
    out = torch.empty(3, 2, 16, 512, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(pkg.kda_latent_decode_workspace_size(3, 2, 16, dr=64), dtype=torch.uint8,
                     device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkg.kda_latent_decode(x["q"], x["cache"], x["table"], x["lens"], out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.kda_latent_decode(x["q"], x["cache"], x["table"], x["lens"], out=out, workspace=ws)
    for lens in ([100, 700, 50], [2, 333, 0]):
        x["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        x["q"].copy_(_randn(*x["q"].shape, seed=sum(lens)))
        graph.replay()
        ref = lu.decode_ref(x["q"], x["cache"], x["table"], x["lens"], None, 1 / math.sqrt(192))
        lu.check("out", out, ref[0], ref[2])


def test_another_stream():
    x = _problem([300], [300], H=2, dr=64)
    want = _fwd(x)
    d = _decode_problem([300, 20], 1, 16, 0, 64)
    want_d = check_decode(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _fwd(x, stream=side)
    got_d = pkg.kda_latent_decode(d["q"], d["cache"], d["table"], d["lens"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert torch.equal(want_d, got_d)


def test_absorbed_form_matches_the_expanded_one():
    """The same attention computed both ways, through the same projections, within
    the sum of what each way rounds."""
    H, n, dr = 8, 333, 64
    c, r = _randn(n, 512, seed=1), _randn(n, dr, seed=2)
    wk = (_randn(H, 128, 512, seed=3).float() / 22.6).bfloat16()
    q = _randn(1, H, 192, seed=4)
    k = torch.einsum("hdc,nc->nhd", wk.double(), c.double())
    qa = torch.cat([torch.einsum("bhd,hdc->bhc", q[..., :128].double(), wk.double()),
                    q[..., 128:].double()], -1)
    kb, qb = k.bfloat16(), qa.bfloat16()
    _, lse = pkg.kda_latent_fwd(q, kb, kb, r, _cu([1]), _cu([n]))
    cache = torch.zeros(6, 64, 576, dtype=torch.bfloat16, device=DEV)
    cache.view(-1, 576)[:n] = torch.cat([c, r], 1)
    lse2 = torch.empty(1, 1, H, device=DEV)
    pkg.kda_latent_decode(qb.unsqueeze(1).contiguous(), cache,
                          torch.arange(6, dtype=torch.int32, device=DEV).view(1, 6),
                          torch.tensor([n], dtype=torch.int32, device=DEV), lse=lse2)
    # a score is off by the rounding of k in one form and of the query in the other
    sc = 1 / math.sqrt(192)
    e = lu.U * sc * (torch.einsum("bhd,nhd->bhn", q[..., :128].double().abs(), k.abs())
                     + torch.einsum("bhc,nc->bhn", qa[..., :512].abs(), c.double().abs()))
    assert bool(((lse - lse2[:, 0]).abs() <= e.amax(-1) + 1e-4).all())
