"""Latent attention in 64 bits from its definition, and the error bounds of the
bf16 kernels, for the tests.

Bounds.  A rounding to bf16 is off by at most half a step, U = 2^-8 of the value.
The kernels compute scores and sums in fp32 from exact bf16 products.  The
matrix units may cut instead of round an addend, so a sum of n products is taken
to be off by at most n 2^-23 times the sum of the products' magnitudes:
  e_s   = (W + 4) 2^-23 * scale * max_j sum_c |q_c k_jc| + 2^-20   (a score; the
          2^-20 covers exp2, log and the change of base)
  out   : probabilities are rounded to bf16 before their product with the values,
          and the result is rounded:  U (A + |o|) + 2 e_s A + (n + 8) 2^-23 A,
          A = sum_j p_j |v_j|
  lse   : e_s + n 2^-24 (a sum of n positive fp32 terms, relative)
  grads : p is off by (U + e_p) p as an operand, ds by U |ds| + e_p |ds| + p e_d,
          e_p = 2 e_s + 2^-20, e_d the error of d_out.v - delta in fp32; each is
          carried through the sum it enters, plus U of the result.
"""
from __future__ import annotations

import math

import torch

U = torch.finfo(torch.bfloat16).eps / 2
E = 2.0 ** -23


def seqs(cu):
    cu = cu.tolist()
    return list(zip(cu[:-1], cu[1:]))


def _keys(k, k_rope, h):
    x = k[:, h].double()
    return x if k_rope is None else torch.cat([x, k_rope.double()], dim=1)


def allowed(nq, nk, causal, device):
    i = torch.arange(nq, device=device).unsqueeze(1)
    j = torch.arange(nk, device=device).unsqueeze(0)
    return j <= i + nk - nq if causal else torch.ones(nq, nk, dtype=torch.bool, device=device)


def softmax_rows(z, ok):
    """(p, lse) of scores under a mask; a row that sees nothing: p = 0, lse = -inf."""
    z = z.masked_fill(~ok, -math.inf)
    some = ok.any(-1, keepdim=True)
    m = torch.where(some, z.amax(-1, keepdim=True) if z.shape[-1] else torch.zeros_like(
        z.sum(-1, keepdim=True)), torch.zeros((), dtype=z.dtype, device=z.device))
    e = torch.where(ok, torch.exp(z - m), torch.zeros_like(z))
    l = e.sum(-1, keepdim=True)
    p = e / torch.where(some, l, torch.ones_like(l))
    lse = torch.where(some, m + torch.log(l), torch.full_like(l, -math.inf)).squeeze(-1)
    return p, lse


def fwd_ref(q, k, v, k_rope, cu_q, cu_k, causal, scale):
    """out, lse in fp64 and the elementwise bounds of both."""
    nq, H, W = q.shape
    dev = q.device
    out = torch.zeros(nq, H, v.shape[2], dtype=torch.float64, device=dev)
    lse = torch.full((nq, H), -math.inf, dtype=torch.float64, device=dev)
    t_out, t_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for (a, b), (c, d) in zip(seqs(cu_q), seqs(cu_k)):
        if b == a or d == c:
            continue
        ok = allowed(b - a, d - c, causal, dev)
        for h in range(H):
            kk = _keys(k[c:d], None if k_rope is None else k_rope[c:d], h)
            qq, vv = q[a:b, h].double(), v[c:d, h].double()
            p, l = softmax_rows(qq @ kk.T * scale, ok)
            e_s = (W + 4) * E * scale * (qq.abs() @ kk.abs().T).amax(1) + 2.0 ** -20
            out[a:b, h], lse[a:b, h] = p @ vv, l
            A = p @ vv.abs()
            t_out[a:b, h] = (U * (A + out[a:b, h].abs())
                             + (2 * e_s.unsqueeze(1) + (d - c + 8) * E) * A)
            t_lse[a:b, h] = e_s + (d - c) * 2.0 ** -24
    return out, lse, t_out, t_lse


def bwd_ref(q, k, v, k_rope, out, lse, d_out, cu_q, cu_k, causal, scale):
    """Gradients in fp64 for the given out and lse, and their bounds."""
    nq, H, W = q.shape
    nk, D = k.shape[0], k.shape[2]
    dev = q.device
    z = dict(dtype=torch.float64, device=dev)
    g = dict(dq=torch.zeros(nq, H, W, **z), dk=torch.zeros(nk, H, D, **z),
             dv=torch.zeros(nk, H, D, **z), dr=torch.zeros(nk, W - D, **z))
    t = {n: torch.zeros_like(x) for n, x in g.items()}
    for (a, b), (c, d) in zip(seqs(cu_q), seqs(cu_k)):
        if b == a or d == c:
            continue
        ok = allowed(b - a, d - c, causal, dev)
        for h in range(H):
            kk = _keys(k[c:d], None if k_rope is None else k_rope[c:d], h)
            qq, vv = q[a:b, h].double(), v[c:d, h].double()
            go, oo = d_out[a:b, h].double(), out[a:b, h].double()
            l = lse[a:b, h].double().unsqueeze(1)
            p = torch.where(ok, torch.exp(qq @ kk.T * scale - l), torch.zeros((), **z))
            e_s = (W + 4) * E * scale * (qq.abs() @ kk.abs().T).amax(1, keepdim=True) + 2.0 ** -20
            # the base change of lse is one fp32 rounding of a value of its size
            e_p = 2 * e_s + 2.0 ** -20 + torch.where(l.isfinite(), l.abs(), torch.zeros_like(l)) * E
            delta = (go * oo).sum(1, keepdim=True)
            ds = p * (go @ vv.T - delta)
            e_d = (D + 8) * E * (go.abs() @ vv.abs().T + (go * oo).abs().sum(1, keepdim=True))
            t_ds = (U + e_p) * ds.abs() + p * e_d
            n_sum = (b - a + d - c) * E
            g["dv"][c:d, h] = p.T @ go
            t["dv"][c:d, h] = ((U + e_p + n_sum) * p).T @ go.abs()
            g["dq"][a:b, h] = scale * (ds @ kk)
            t["dq"][a:b, h] = scale * ((t_ds + n_sum * ds.abs()) @ kk.abs())
            gk = scale * (ds.T @ qq)
            tk = scale * ((t_ds + n_sum * ds.abs()).T @ qq.abs())
            g["dk"][c:d, h], t["dk"][c:d, h] = gk[:, :D], tk[:, :D]
            g["dr"][c:d] += gk[:, D:]
            t["dr"][c:d] += tk[:, D:] + H * E * gk[:, D:].abs()
    for n in g:
        t[n] += U * g[n].abs()
    return g, t


def decode_rows(cache, table_row, n):
    """The n cached rows of a sequence, through its block table."""
    page = cache.shape[1]
    pos = torch.arange(n, device=cache.device)
    return cache[table_row.long()[pos // page], pos % page]


def decode_ref(q, cache, table, lens, mask, scale):
    B, T, H, W = q.shape
    dev = q.device
    out = torch.zeros(B, T, H, 512, dtype=torch.float64, device=dev)
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device=dev)
    t_out, t_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens.tolist()):
        if n == 0:
            continue
        x = decode_rows(cache, table[b], n).double()
        for t in range(T):
            ok = torch.zeros(n, dtype=torch.bool, device=dev)
            ok[:max(0, n - T)] = True
            for j in range(T):
                if n - T + j >= 0:
                    ok[n - T + j] = (j <= t) if mask is None else bool(int(mask[b, t]) >> j & 1)
            if not ok.any():
                continue
            qq = q[b, t].double()
            p, l = softmax_rows(qq @ x.T * scale, ok.unsqueeze(0).expand(H, n))
            e_s = (W + 4) * E * scale * (qq.abs() @ x[ok].abs().T).amax(1) + 2.0 ** -20
            out[b, t], lse[b, t] = p @ x[:, :512], l
            A = p @ x[:, :512].abs()
            t_out[b, t] = U * (A + out[b, t].abs()) + (2 * e_s.unsqueeze(1) + (n + 8) * E) * A
            t_lse[b, t] = e_s + n * 2.0 ** -24
    return out, lse, t_out, t_lse


def check(name, got, ref, tol):
    """Every element within its bound; -inf and 0 where the reference has them."""
    got = got.double()
    inf = ref.isinf()
    assert torch.equal(got.isinf(), inf), f"{name}: infinities differ"
    err = torch.where(inf, torch.zeros_like(ref), (got - ref).abs())
    bad = ~(err <= tol + 1e-30)   # a NaN is bad
    if bad.any():
        at = tuple(int(x) for x in torch.nonzero(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} elements off, first at "
                             f"{at}: got {got[at].item()}, want {ref[at].item()} "
                             f"+- {tol[at].item()}")


def paged(lens, page, width, device, seed=0, spare=2, dtype=torch.bfloat16, max_pages=None):
    """(cache, table) with the sequences' pages shuffled over a pool.  Rows and
    table entries no sequence uses hold NaN and out-of-range ids."""
    g = torch.Generator().manual_seed(seed)
    need = [(n + page - 1) // page for n in lens]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    width_t = max_pages or max(need + [1]) + 1
    table = torch.full((len(lens), width_t), -7, dtype=torch.int32)
    cache = torch.full((n_pages, page, width), float("nan"), dtype=dtype)
    at = 0
    for b, (n, k) in enumerate(zip(lens, need)):
        table[b, :k] = order[at:at + k]
        rows = torch.randn(n, width, generator=g).to(dtype)
        for i in range(k):
            piece = rows[i * page:(i + 1) * page]
            cache[order[at + i].long(), :piece.shape[0]] = piece
        at += k
    return cache.to(device), table.to(device)


def tree_masks(B, T, seed=0):
    g = torch.Generator().manual_seed(seed)
    out = torch.zeros(B, T, dtype=torch.int64)
    for b in range(B):
        words = []
        for i in range(T):
            up = words[int(torch.randint(0, i, (1,), generator=g))] if i else 0
            words.append(up | (1 << i))
        # bit 63 is the sign of an int64
        out[b] = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words])
    return out
