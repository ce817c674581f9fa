"""A run of the operators around a cached row as they are used: rows normalised, turned
and cached, decode steps, the weights they give, eviction, and decode over what is left."""
from __future__ import annotations

import torch
import pytest

import gated_delta_rule_13_gb300 as kda
import rows_util as ru

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def test_serving_under_a_budget():
    """Decode over the evicted cache equals attention, in 64 bits, over the rows that
    should be left."""
    g = torch.Generator(device=DEV).manual_seed(0)
    B, H, DC, DR, PAGE, n0, budget, first, recent = 3, 16, 512, 64, 16, 90, 64, 4, 12
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    freq = kda.kda_rope_inv_freq(DR, device=DEV)
    gamma = 1 + 0.1 * randn(DC)
    host = torch.Generator().manual_seed(1)
    table, n_pages = ru.pages([n0 + 40] * B, PAGE, host)
    table = table.to(DEV)
    cache = torch.zeros(n_pages, PAGE, DC + DR, dtype=BF, device=DEV)
    cap = table.shape[1] * PAGE
    weights = torch.zeros(B, cap, device=DEV)

    def new_rows(pos):
        raw = randn(B, pos.shape[1], DC + DR).to(BF)
        rows = raw.clone()
        kda.kda_norm_fwd(raw[..., :DC], gamma, center=False, out=rows[..., :DC], stats=False)
        q = randn(B, pos.shape[1], H, DC + DR).to(BF)
        kda.kda_rope(q[..., DC:], pos, freq, k=rows[..., DC:], out=q[..., DC:], k_out=rows[..., DC:])
        want = ru.norm_ref(raw[..., :DC], gamma, None, False, 1e-5)[0]
        tol = ru.norm_bounds(raw[..., :DC], gamma, None, False, 1e-5, BF)[0]
        assert ((rows[..., :DC].double() - want).abs() <= tol).all()
        return q, rows

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    prompt = torch.arange(n0, dtype=torch.int32, device=DEV).expand(B, n0).contiguous()
    q, rows = new_rows(prompt)
    kda.kda_cache_write(cache, rows, table, i32([0] * B))
    # the rows each sequence should hold, in the cache's order
    held = [rows[b] for b in range(B)]
    lens = i32([n0] * B)
    # the prompt's last 32 tokens give the first weights
    last = q[:, -32:].contiguous()
    lse = torch.empty(B, 32, H, device=DEV)
    kda.kda_latent_decode(last, cache, table, lens, lse=lse)
    kda.kda_latent_weights(last, cache, table, lens, lse, weights)
    assert ((weights.sum(1) - 32 * H).abs() < 32 * H * 3e-4).all()
    scale = (128 + DR) ** -0.5
    for step in range(30):
        pos = torch.full((B, 1), n0 + step, dtype=torch.int32, device=DEV)
        q, rows = new_rows(pos)
        kda.kda_cache_write(cache, rows, table, lens)
        lens = lens + 1
        lse = torch.empty(B, 1, H, device=DEV)
        out = kda.kda_latent_decode(q, cache, table, lens, lse=lse)
        kda.kda_latent_weights(q, cache, table, lens, lse, weights, decay=0.9)
        for b in range(B):
            held[b] = torch.cat([held[b], rows[b]])
            c = held[b].double()
            p = torch.softmax(q[b, 0].double() @ c.T * scale, -1)
            want = p @ c[:, :DC]
            # probabilities and the result round to bf16, 2^-8 each, relative to the
            # values' root mean square under p
            size = torch.sqrt(p @ (c[:, :DC] ** 2))
            assert ((out[b, 0].double() - want).abs() <= 2.2 * 2 ** -8 * size + 1e-3).all()
        before = weights.cpu().clone()
        n = lens.tolist()
        lens, origin = kda.kda_cache_evict(cache, table, lens, weights, budget, first=first, recent=recent)
        for b in range(B):
            want = ru.evict_ref(before[b].tolist(), n[b], budget, first, recent)
            assert origin[b].tolist() == want + [-1] * (budget - len(want))
            held[b] = held[b][torch.tensor(want, device=DEV)]
            assert torch.equal(ru.rows_of(cache, table, b, len(want)), held[b])
        assert lens.tolist() == [budget] * B


def test_training_around_the_attention():
    """Gradients through norm, rotation and latent attention against automatic
    differentiation of the same formulas in 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(2)
    n, H, DR, D = 70, 2, 64, 128
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    raw_q, raw_k = randn(n, H, D + DR).to(BF), randn(n, DR).to(BF)
    kv, gamma = randn(n, H, 2 * D).to(BF), 1 + 0.1 * randn(2 * D)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    freq = kda.kda_rope_inv_freq(DR, device=DEV)
    d_out = randn(n, H, D).to(BF)

    q = raw_q.clone()
    _, k_rope = kda.kda_rope(q[..., D:], pos, freq, k=raw_k, out=q[..., D:])
    z, mean, rstd = kda.kda_norm_fwd(kv, gamma)
    out, lse = kda.kda_latent_fwd(q, z[..., :D], z[..., D:], k_rope)
    d_z = torch.empty_like(z)
    dq, _, _, d_rope = kda.kda_latent_bwd(q, z[..., :D], z[..., D:], k_rope, out, lse, d_out,
                                          d_k=d_z[..., :D], d_v=d_z[..., D:])
    kda.kda_rope(dq[..., D:], pos, freq, k=d_rope, out=dq[..., D:], k_out=d_rope, transpose=True)
    d_kv, d_gamma, _ = kda.kda_norm_bwd(d_z, kv, gamma, mean, rstd)

    leaves = [t.double().requires_grad_() for t in (raw_q, raw_k, kv, gamma)]
    a, b, c, w = leaves
    turn = lambda t: ru.rope_ref(t, pos, freq, True, 1.0, False)  # noqa: E731
    z64 = ru.norm_ref(c, w, None, True, 1e-5)[0]
    q64 = torch.cat([a[..., :D], turn(a[..., D:])], -1)
    s = torch.einsum("ihd,jhd->hij", q64[..., :D], z64[..., :D]) \
        + torch.einsum("ihd,jd->hij", q64[..., D:], turn(b))
    s = (s * (D + DR) ** -0.5).masked_fill(torch.ones(n, n, device=DEV).triu(1).bool(), float("-inf"))
    o = torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), z64[..., D:])
    want = torch.autograd.grad(o, leaves, d_out.double())
    # five roundings to bf16 on the way (rotated, normalised, probabilities, their gradient,
    # results), half a step each, adding up as independent ones: 2^-8 sqrt 5 < 0.9 %
    for name, x, y in zip(("q", "k_rope", "kv", "gamma"), (dq, d_rope, d_kv, d_gamma), want):
        err = ((x.double() - y).norm() / y.norm()).item()
        assert err < 0.009, f"{name}: {err}"


def test_two_streams_at_once():
    """Every operator on two streams, with workspaces of their own, gives what it gives alone."""
    g = torch.Generator(device=DEV).manual_seed(11)

    def data(k):
        B, n_pages = 4 + k, 200
        lens = torch.randint(500, 1500, (B,), generator=g, device=DEV).to(torch.int32)
        return dict(q=torch.randn(B, 2, 96, 576, generator=g, device=DEV).to(BF),
                    cache=torch.randn(n_pages, 64, 576, generator=g, device=DEV).to(BF),
                    table=torch.randperm(n_pages, generator=g, device=DEV)[:B * 24].to(torch.int32).view(B, 24),
                    lens=lens, w=torch.rand(B, 24 * 64, generator=g, device=DEV),
                    x=torch.randn(9000, 512, generator=g, device=DEV).to(BF),
                    weight=torch.rand(512, generator=g, device=DEV),
                    pos=torch.arange(9000, dtype=torch.int32, device=DEV),
                    freq=kda.kda_rope_inv_freq(64, device=DEV))

    def run(d):
        cache, w = d["cache"].clone(), d["w"].clone()
        lse = torch.empty(d["q"].shape[:3], device=DEV)
        out = kda.kda_latent_decode(d["q"], cache, d["table"], d["lens"], lse=lse)
        kda.kda_latent_weights(d["q"], cache, d["table"], d["lens"], lse, w, decay=0.5)
        weights = w.clone()
        evicted = kda.kda_cache_evict(cache, d["table"], d["lens"], w, 400, first=4, recent=64)
        y, mean, rstd = kda.kda_norm_fwd(d["x"], d["weight"])
        back = kda.kda_norm_bwd(d["x"], y, d["weight"], mean, rstd, bias=True)
        turned = kda.kda_rope(d["x"].view(9000, 8, 64), d["pos"], d["freq"])
        return [out, lse, weights, w, cache, *evicted, y, mean, rstd, *back, turned]

    both = [data(0), data(1)]
    want = [run(d) for d in both]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k] = run(both[k])
    torch.cuda.synchronize()
    graphs = []
    for k in (0, 1):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[k]):
            captured = run(both[k])
        graphs.append((graph, captured))
    for _ in range(3):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                graphs[k][0].replay()
    torch.cuda.synchronize()
    for k in (0, 1):
        for a, b, c in zip(want[k], got[k], graphs[k][1]):
            a, b, c = (a, b, c) if torch.is_tensor(a) else (a[0], b[0], c[0])
            assert torch.equal(a, b) and torch.equal(a, c)
