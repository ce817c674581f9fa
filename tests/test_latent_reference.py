"""The 64-bit reference of latent attention itself (CPU): gradients against
central differences, the absorbed form against the expanded one, tree masks
against the linear order."""
from __future__ import annotations

import pytest
import torch

import latent_util as lu


def _problem(lens_q, lens_k, H, dr, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    cu = lambda x: torch.tensor([0] + list(torch.tensor(x).cumsum(0)), dtype=torch.int32)  # noqa
    nq, nk = sum(lens_q), sum(lens_k)
    return dict(q=r(nq, H, 6 + dr), k=r(nk, H, 6), v=r(nk, H, 6),
                k_rope=r(nk, dr) if dr else None, cu_q=cu(lens_q), cu_k=cu(lens_k))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dr", [0, 2])
def test_gradients_against_differences(causal, dr):
    x = _problem([3, 0, 2, 3], [3, 2, 5, 2], H=2, dr=dr)
    g = torch.Generator().manual_seed(9)
    w = torch.randn(8, 2, 6, generator=g, dtype=torch.float64)

    def loss():
        return (lu.fwd_ref(**x, causal=causal, scale=0.7)[0] * w).sum()

    out, lse, _, _ = lu.fwd_ref(**x, causal=causal, scale=0.7)
    grads, _ = lu.bwd_ref(x["q"], x["k"], x["v"], x["k_rope"], out, lse, w, x["cu_q"], x["cu_k"],
                          causal, 0.7)
    h = 1e-5
    for name, got in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("k_rope", "dr")):
        if x[name] is None:
            continue
        flat, want = x[name].view(-1), torch.zeros(x[name].numel(), dtype=torch.float64)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss()
            flat[i] = keep - h
            want[i] = (up - loss()) / (2 * h)
            flat[i] = keep
        # a central difference is off by about h^2 of the third derivative and eps / h
        assert torch.allclose(grads[got].reshape(-1), want, rtol=0, atol=1e-8), name


def test_absorbed_equals_expanded():
    g = torch.Generator().manual_seed(3)
    H, n, dr = 3, 21, 64
    c = torch.randn(n, 512, generator=g, dtype=torch.float64)
    r = torch.randn(n, dr, generator=g, dtype=torch.float64)
    wk = torch.randn(H, 128, 512, generator=g, dtype=torch.float64) / 22
    wv = torch.randn(H, 128, 512, generator=g, dtype=torch.float64) / 22
    q = torch.randn(1, H, 192, generator=g, dtype=torch.float64)
    one = torch.tensor([0, 1]), torch.tensor([0, n])
    k, v = torch.einsum("hdc,nc->nhd", wk, c), torch.einsum("hdc,nc->nhd", wv, c)
    want, lse, _, _ = lu.fwd_ref(q, k, v, r, *one, True, 0.1)
    qa = torch.cat([torch.einsum("bhd,hdc->bhc", q[..., :128], wk), q[..., 128:]], -1)
    cache = torch.cat([c, r], 1)
    cache = torch.cat([cache, torch.full((11, 576), float("nan"), dtype=torch.float64)])
    got, lse2, _, _ = lu.decode_ref(qa.unsqueeze(1), cache.view(2, 16, 576),
                                    torch.tensor([[0, 1]]), torch.tensor([n]), None, 0.1)
    got = torch.einsum("bthc,hdc->bthd", got, wv)
    assert torch.allclose(got[:, 0], want, atol=1e-12)
    assert torch.allclose(lse2[:, 0], lse, atol=1e-12)


def test_chain_tree_is_the_linear_order():
    cache, table = lu.paged([9, 30], 16, 512, "cpu")
    q = torch.randn(2, 4, 2, 512, generator=torch.Generator().manual_seed(1))
    lens = torch.tensor([9, 30])
    chain = torch.tensor([[1, 3, 7, 15]] * 2)
    a = lu.decode_ref(q, cache, table, lens, None, 0.1)
    b = lu.decode_ref(q, cache, table, lens, chain, 0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_that_see_nothing():
    out, lse, _, _ = lu.fwd_ref(**_problem([4], [2], H=1, dr=0), causal=True, scale=1.0)
    assert torch.equal(out[:2], torch.zeros(2, 1, 6, dtype=torch.float64))
    assert lse[:2].isinf().all() and lse[2:].isfinite().all()
