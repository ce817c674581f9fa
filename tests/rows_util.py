"""Plain 64-bit forms of the operators around a cached latent row, and inputs for them."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24          # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ rotation
def rope_ref(x, positions, inv_freq, interleaved, scale, transpose):
    """x [*tokens, (H,) dr] in fp64: the rotation of each pair as a 2 x 2 matrix."""
    x, dr = x.double(), x.shape[-1]
    t = positions.double()[..., None] * inv_freq.double()
    if x.dim() == positions.dim() + 2:
        t = t[..., None, :]
    c, s = torch.cos(t) * scale, torch.sin(t) * scale
    if transpose:
        s = -s
    i = torch.arange(dr // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + dr // 2)
    a, b = x[..., ia], x[..., ib]
    out = torch.empty_like(x)
    out[..., ia] = c * a - s * b
    out[..., ib] = s * a + c * b
    return out


def rope_bound(x, interleaved, scale, dtype, want):
    """Half a step of t / pi in fp32, 2^-25, is pi 2^-25 = 1.6 u of angle; sine and cosine
    are off by at most 2 of their steps, 4 u; their product with the scale, the two
    products and the sum round four times, u each: 10 u times the pair's length.  Then the
    result's own rounding."""
    x, dr = x.double(), x.shape[-1]
    i = torch.arange(dr // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + dr // 2)
    length = torch.hypot(x[..., ia], x[..., ib]) * abs(scale)
    tol = torch.empty_like(x)
    tol[..., ia] = tol[..., ib] = 10 * U * length
    return tol + half_step(dtype) * (want.abs() + tol) + 1e-38


# ------------------------------------------------------------------ norm
def norm_ref(x, weight, bias, center, eps):
    x = x.double()
    m = x.mean(-1, keepdim=True) if center else torch.zeros_like(x[..., :1])
    d = x - m
    r = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    y = d * r
    if weight is not None:
        y = y * weight.double()
    if bias is not None:
        y = y + bias.double()
    return y, m[..., 0], r[..., 0]


def norm_grad_ref(g, x, weight, mean, rstd):
    g, x, r = g.double(), x.double(), rstd.double()[..., None]
    z = (x - mean.double()[..., None]) * r if mean is not None else x * r
    e = g * weight.double() if weight is not None else g
    d = e - z * (e * z).mean(-1, keepdim=True)
    if mean is not None:
        d = d - e.mean(-1, keepdim=True)
    rows = tuple(range(g.dim() - 1))
    return d * r, (g * z).sum(rows), g.sum(rows)


# A sum over a row: at most 32 terms by a thread, then 5 + 5 steps of a tree; rounded up.
ROW = 48 * U


def norm_bounds(x, weight, bias, center, eps, dtype):
    """(out, mean, rstd) bounds: the mean's sum; the variance's, and the mean's error in
    it; the reciprocal root, 2 steps; then the result's four roundings."""
    y, m, r = norm_ref(x, weight, bias, center, eps)
    x = x.double()
    dm = ROW * x.abs().mean(-1) if center else torch.zeros_like(m)
    dr = r * ((ROW + 4 * U) / 2 + 4 * U + (dm * r) ** 2)
    w = 1.0 if weight is None else weight.double().abs()
    z = (x - m[..., None]).abs() * r[..., None]
    tol = w * (z * (dr / r)[..., None] + (dm * r)[..., None] + 4 * U * z)
    if bias is not None:
        tol = tol + U * (y.abs() + tol)
    return tol + half_step(dtype) * (y.abs() + tol) + 1e-38, dm + U * m.abs(), dr


def norm_grad_bounds(g, x, weight, mean, rstd, dtype):
    """Bounds of (d_x, d_weight, d_bias).  z rounds twice, its products once more each; a
    sum over rows has at most as many terms as rows, and 72 from the joins."""
    want, dw, db = norm_grad_ref(g, x, weight, mean, rstd)
    g, x, r = g.double(), x.double(), rstd.double()[..., None]
    z = ((x - mean.double()[..., None]) if mean is not None else x).abs() * r
    e = (g * weight.double() if weight is not None else g).abs()
    tol = r * (z * (ROW + 8 * U) * (e * z).mean(-1, keepdim=True) + 6 * U * e
               + 6 * U * z * (e * z).mean(-1, keepdim=True))
    if mean is not None:
        tol = tol + r * (ROW + 4 * U) * e.mean(-1, keepdim=True)
    rows = tuple(range(g.dim() - 1))
    terms = (math.prod(g.shape[:-1]) + 72) * U
    return (tol + half_step(dtype) * (want.abs() + tol) + 1e-38,
            (terms + 4 * U) * (g * z).abs().sum(rows) + 1e-38,
            terms * g.abs().sum(rows) + 1e-38)


# ------------------------------------------------------------------ paged cache
def pages(lens, page, g, extra=2, width=None):
    """(table [B, width], n_pages): each sequence's pages drawn from a shuffled pool;
    entries behind its last page are out of range (they must not be read)."""
    need = [(n + page - 1) // page for n in lens]
    width = max(1, max(need, default=1)) if width is None else width
    n_pages = sum(need) + extra
    order = torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((len(lens), width), 1 << 28, dtype=torch.int32)
    for b, k in enumerate(need):
        for i in range(k):
            table[b, i] = order.pop()
    return table, n_pages


def rows_of(cache, table, b, n):
    """The n cached rows of sequence b."""
    page = cache.shape[-2]
    pos = torch.arange(n, device=cache.device)
    return cache[..., table[b].long()[pos // page], pos % page, :]


def seen_by(b, t, n, T, mask):
    """Positions token t of sequence b looks at."""
    if mask is None:
        return list(range(max(0, n - T + t + 1)))
    word = int(mask[b, t])
    return [j for j in range(n) if j < n - T or word >> (j - (n - T)) & 1]


def weights_ref(q, cache, table, lens, lse, old, mask, scale, decay):
    """The weights in fp64."""
    B, T, H, _ = q.shape
    out = old.double().clone()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        rows = rows_of(cache, table, b, n).double()
        new = torch.zeros(n, dtype=torch.float64, device=q.device)
        for t in range(T):
            see = torch.tensor(seen_by(b, t, n, T, mask), dtype=torch.long, device=q.device)
            if len(see) == 0:
                continue
            s = q[b, t].double() @ rows[see].T * scale
            p = torch.exp(s - lse[b, t].double()[:, None])
            new[see] += p[torch.isfinite(lse[b, t])].sum(0)
        out[b, :n] = (decay * out[b, :n] if decay else 0) + new
    return out


def evict_ref(w, n, budget, first, recent):
    """Former positions of the rows at 0, 1, ... after a sequence's eviction."""
    if n <= budget:
        return list(range(n))
    last = budget - recent
    key = [-math.inf if v != v else v for v in w]
    nan = [v != v for v in w]
    order = sorted(range(first, n - recent), key=lambda j: (nan[j], -key[j], j))
    kept = set(range(first)) | set(order[:budget - first - recent])
    movers = sorted(j for j in kept if j >= last)
    out = []
    for j in range(last):
        out.append(j if j in kept else movers.pop(0))
    assert not movers
    return out + list(range(n - recent, n))
