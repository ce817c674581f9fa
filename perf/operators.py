"""Workloads of the latent-attention operators and of the paged cache behind them.

Each case is one call of one operator, at sizes from the smallest a user makes
(a ragged handful of tokens, one token of one sequence) to the largest (a
training batch, a prompt's chunk over a long prefix, a full serving batch).
With ``own`` false the operators run in a plain form of elementary torch
operations in 32 bits; with ``own`` true they run through the package.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda:0"
D = 128       # head dimension (keys without positions, values)
DC = 512      # latent channels of a cached row


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few short packed requests of a scheduler step: latency counts
        dict(name="fwd_ragged", kind="fwd", lens_q="1,17,130,64,509", lens_k="1,17,130,64,509",
             H=8, dr=64),
        # one training layer: 4 sequences of 4096 tokens, 16 heads
        dict(name="fwd_train", kind="fwd", lens_q="4096,4096,4096,4096",
             lens_k="4096,4096,4096,4096", H=16, dr=64),
        # a prompt's last chunk over the keys of its long prefix, 96 heads, no rotary part
        dict(name="fwd_chunk", kind="fwd", lens_q="2048", lens_k="32768", H=96, dr=0),
        # gradients of a small ragged fine-tuning batch
        dict(name="bwd_ragged", kind="bwd", lens_q="33,200,513,1024,77",
             lens_k="33,200,513,1024,77", H=16, dr=64),
        # gradients of the training layer above
        dict(name="bwd_train", kind="bwd", lens_q="4096,4096,4096,4096",
             lens_k="4096,4096,4096,4096", H=16, dr=64),
        # one token of one interactive request: latency counts
        dict(name="decode_single", kind="decode", B=1, T=1, H=96, dr=0, lo=3001, hi=3001,
             page=64, tree=False),
        # one token for each of a serving batch of ragged lengths
        dict(name="decode_batch", kind="decode", B=128, T=1, H=96, dr=64, lo=1, hi=16384,
             page=64, tree=False),
        # verification of a tree of 16 drafts for each of 32 requests
        dict(name="tree_batch", kind="decode", B=32, T=16, H=96, dr=64, lo=3000, hi=16000,
             page=512, tree=True),
        # the new token's latent of one layer, 64 requests
        dict(name="append_token", kind="write", B=64, T=1, L=1, dr=64, hi=4096, page=64,
             compact=False),
        # the accepted path of 16 drafts moved together, 256 requests, 24 layers at once
        dict(name="compact_drafts", kind="write", B=256, T=16, L=24, dr=64, hi=170, page=64,
             compact=True),
        # fork of a request: its last, partly filled page gets a private copy in 24 layers
        dict(name="fork_page", kind="copy", n=1, pages=64, L=24, elems=64 * 576, fp32=False),
        # cached recurrent states of 16 requests copied to private running states (96 heads)
        dict(name="copy_states", kind="copy", n=16, pages=40, L=3, elems=96 * 128 * 128, fp32=True),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "bwd", "bwd", "decode", "decode", "decode", "write", "copy"])
    dr = rng.choice([0, 64])
    if kind in ("fwd", "bwd"):
        n = rng.randint(1, 6)
        H = rng.choice([1, 3, 8, 16, 24, 32, 96])
        cap = (4096 if kind == "fwd" else 2048) if H <= 32 else 1024
        lq = [_logint(rng, 1, cap) for _ in range(n)]
        lk = list(lq)
        if rng.random() < 0.4:  # continue from prefixes
            lk = [a + rng.randint(0, 2 * cap) for a in lq]
        return dict(kind=kind, lens_q=",".join(map(str, lq)), lens_k=",".join(map(str, lk)),
                    H=H, dr=dr)
    if kind == "decode":
        tree = rng.random() < 0.5
        T = rng.randint(2, 24) if tree else rng.choice([1, 1, 2, 4, 5])
        H = rng.choice([1, 5, 16, 40, 64, 96, 128])
        B = _logint(rng, 1, 64)
        lo = T + _logint(rng, 1, 4096)
        hi = lo + _logint(rng, 1, 8192)
        return dict(kind=kind, B=B, T=T, H=H, dr=dr, lo=lo, hi=hi,
                    page=rng.choice([16, 48, 64, 128, 512]), tree=tree)
    if kind == "write":
        return dict(kind=kind, B=_logint(rng, 1, 256), T=rng.randint(1, 24), L=rng.randint(1, 12),
                    dr=dr, hi=rng.randint(100, 500), page=rng.choice([16, 48, 64, 512]),
                    compact=rng.random() < 0.5)
    pages = rng.randint(8, 200)
    return dict(kind="copy", n=rng.randint(1, pages // 2), pages=pages, L=rng.randint(1, 24),
                elems=8 * _logint(rng, 64, 16384), fp32=rng.random() < 0.5)


def _ints(text):
    return [int(x) for x in text.split(",")]


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=DEV)


def _lengths(case, seed):
    g = torch.Generator()
    g.manual_seed(seed + 1)
    return torch.randint(case["lo"], case["hi"] + 1, (case["B"],), generator=g).tolist()


def _tables(lens, page, seed, most):
    """Block tables of sequences of these lengths (``most`` at the most), their
    pages spread over a shuffled pool that has room for all of them at their longest."""
    need = [(n + page - 1) // page for n in lens]
    n_pages = len(lens) * ((most + page - 1) // page) + 3
    g = torch.Generator()
    g.manual_seed(seed + 2)
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.zeros(len(lens), (most + page - 1) // page, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, n_pages


def _tree(B, T, seed):
    """Ancestor masks of random draft trees (a node sees itself and its ancestors)."""
    g = torch.Generator()
    g.manual_seed(seed + 3)
    out = torch.zeros(B, T, dtype=torch.int64)
    pick = torch.rand(B, T, generator=g)
    for b in range(B):
        words = []
        for i in range(T):
            up = words[int(pick[b, i] * i)] if i else 0
            words.append(up | (1 << i))
        out[b] = torch.tensor(words, dtype=torch.int64)
    return out


def prepare(case, seed):
    kind = case["kind"]
    g = _gen(seed)
    if kind in ("fwd", "bwd"):
        lq, lk, H, dr = _ints(case["lens_q"]), _ints(case["lens_k"]), case["H"], case["dr"]
        kv = _randn(g, sum(lk), H, 2 * D)      # one projection holds keys and values of a head
        s = dict(case=case, lq=lq, lk=lk, cu_q=_cu(lq), cu_k=_cu(lk),
                 q=_randn(g, sum(lq), H, D + dr), k=kv[..., :D], v=kv[..., D:],
                 k_rope=_randn(g, sum(lk), dr) if dr else None)
        if kind == "bwd":  # what the forward pass left, and the gradient that comes in
            s["d_out"] = _randn(g, sum(lq), H, D)
            s["out"], s["lse"] = _plain_fwd(s)
        return s
    if kind == "decode":
        lens = _lengths(case, seed)
        table, n_pages = _tables(lens, case["page"], seed, case["hi"])
        W = DC + case["dr"]
        s = dict(case=case, lens=lens, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 table=table.to(DEV), cache=_randn(g, n_pages, case["page"], W),
                 q=_randn(g, case["B"], case["T"], case["H"], W), mask=None)
        if case["tree"]:
            s["mask"] = _tree(case["B"], case["T"], seed).to(DEV)
        return s
    if kind == "write":
        B, T, L, page, W = case["B"], case["T"], case["L"], case["page"], DC + case["dr"]
        h = torch.Generator()
        h.manual_seed(seed + 1)
        start = torch.randint(0, case["hi"] + 1, (B,), generator=h)
        table, n_pages = _tables([int(x) + T for x in start], page, seed, case["hi"] + T)
        s = dict(case=case, cache=_randn(g, L, n_pages, page, W), table=table.to(DEV),
                 start=start.to(torch.int32).to(DEV), rows=None, path=None, count=None)
        if case["compact"]:
            # Accepted nodes stay where they are or come from behind the accepted
            # prefix, so a pass repeated on the same cache gives the same rows.
            count = torch.randint(1, T // 2 + 2, (B,), generator=h).clamp(max=T)
            path = torch.zeros(B, T, dtype=torch.int64)
            for b in range(B):
                n = int(count[b])
                keep = int(torch.randint(0, n + 1, (1,), generator=h))
                keep = max(keep, 2 * n - T)
                far = torch.randperm(T - n, generator=h)[:n - keep].sort().values + n
                path[b, :keep] = torch.arange(keep)
                path[b, keep:n] = far
            s["path"] = path.to(torch.int32).to(DEV)
            s["count"] = count.to(torch.int32).to(DEV)
        else:
            s["rows"] = _randn(g, L, B, T, W)
        return s
    dtype = torch.float32 if case["fp32"] else torch.bfloat16
    h = torch.Generator()
    h.manual_seed(seed + 1)
    ids = torch.randperm(case["pages"], generator=h)[:2 * case["n"]].to(torch.int32).to(DEV)
    pool = torch.randn(case["L"], case["pages"], case["elems"], generator=g, device=DEV,
                       dtype=torch.float32).to(dtype)
    return dict(case=case, pool=pool, src=ids[:case["n"]].clone(), dst=ids[case["n"]:].clone())


# ------------------------------------------------------------------ plain forms
def _head_step(nq, nk, H):
    """Heads at a time, so that a score matrix stays within about 2 GB."""
    return max(1, min(H, (1 << 29) // max(1, nq * nk)))


def _plain_scores(s, b0, bk, nq, nk, h0, h1):
    D_ = s["q"].shape[-1]
    q = s["q"][b0:b0 + nq, h0:h1].float().transpose(0, 1)
    k = s["k"][bk:bk + nk, h0:h1].float().transpose(0, 1)
    if s["k_rope"] is not None:
        r = s["k_rope"][bk:bk + nk].float()
        k = torch.cat([k, r.unsqueeze(0).expand(h1 - h0, nk, r.shape[-1])], dim=-1)
    x = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(D_))
    seen = (torch.arange(nk, device=DEV).unsqueeze(0)
            <= torch.arange(nq, device=DEV).unsqueeze(1) + (nk - nq))
    return q, k, x.masked_fill_(~seen, float("-inf"))


def _plain_fwd(s):
    Nq, H = s["q"].shape[:2]
    out = torch.empty(Nq, H, D, dtype=s["q"].dtype, device=DEV)
    lse = torch.empty(Nq, H, dtype=torch.float32, device=DEV)
    b0 = bk = 0
    for nq, nk in zip(s["lq"], s["lk"]):
        step = _head_step(nq, nk, H)
        for h0 in range(0, H, step):
            h1 = min(H, h0 + step)
            _, _, x = _plain_scores(s, b0, bk, nq, nk, h0, h1)
            m = x.amax(dim=-1, keepdim=True)
            p = torch.exp(x.sub_(m))
            l = p.sum(dim=-1, keepdim=True)
            v = s["v"][bk:bk + nk, h0:h1].float().transpose(0, 1)
            o = torch.matmul(p, v) / l
            out[b0:b0 + nq, h0:h1] = o.transpose(0, 1).to(out.dtype)
            lse[b0:b0 + nq, h0:h1] = (m + torch.log(l)).squeeze(-1).transpose(0, 1)
        b0 += nq
        bk += nk
    return out, lse


def _plain_bwd(s):
    Nq, H, Dq = s["q"].shape
    Nk = s["k"].shape[0]
    dt = s["q"].dtype
    scale = 1.0 / math.sqrt(Dq)
    dq = torch.empty(Nq, H, Dq, dtype=dt, device=DEV)
    dk = torch.empty(Nk, H, D, dtype=dt, device=DEV)
    dv = torch.empty(Nk, H, D, dtype=dt, device=DEV)
    dr = torch.zeros(Nk, Dq - D, dtype=torch.float32, device=DEV) if Dq > D else None
    b0 = bk = 0
    for nq, nk in zip(s["lq"], s["lk"]):
        step = _head_step(nq, nk, H)
        for h0 in range(0, H, step):
            h1 = min(H, h0 + step)
            q, k, x = _plain_scores(s, b0, bk, nq, nk, h0, h1)
            rows = slice(b0, b0 + nq)
            p = torch.exp(x.sub_(s["lse"][rows, h0:h1].t().unsqueeze(-1)))
            g = s["d_out"][rows, h0:h1].float().transpose(0, 1)
            o = s["out"][rows, h0:h1].float().transpose(0, 1)
            v = s["v"][bk:bk + nk, h0:h1].float().transpose(0, 1)
            delta = (g * o).sum(dim=-1, keepdim=True)
            dv[bk:bk + nk, h0:h1] = torch.matmul(p.transpose(1, 2), g).transpose(0, 1).to(dt)
            ds = torch.matmul(g, v.transpose(1, 2)).sub_(delta).mul_(p).mul_(scale)
            dq[rows, h0:h1] = torch.matmul(ds, k).transpose(0, 1).to(dt)
            gk = torch.matmul(ds.transpose(1, 2), q)
            dk[bk:bk + nk, h0:h1] = gk[..., :D].transpose(0, 1).to(dt)
            if dr is not None:
                dr[bk:bk + nk] += gk[..., D:].sum(dim=0)
        b0 += nq
        bk += nk
    return (dq, dk, dv) if dr is None else (dq, dk, dv, dr.to(dt))


def _plain_decode(s):
    c = s["case"]
    B, T, H, W = s["q"].shape
    scale = 1.0 / math.sqrt(D + c["dr"])
    out = torch.empty(B, T, H, DC, dtype=s["q"].dtype, device=DEV)
    bit = torch.arange(T, device=DEV)
    for b, n in enumerate(s["lens"]):
        used = (n + c["page"] - 1) // c["page"]
        rows = s["cache"][s["table"][b, :used].long()].reshape(-1, W)[:n].float()
        x = torch.matmul(s["q"][b].float(), rows.t()) * scale        # [T, H, n]
        if T > 1:
            t0 = n - T
            if s["mask"] is not None:
                seen = ((s["mask"][b].unsqueeze(1) >> bit) & 1).bool()
            else:
                seen = bit.unsqueeze(0) <= bit.unsqueeze(1)
            x[:, :, t0:].masked_fill_(~seen.unsqueeze(1), float("-inf"))
        p = torch.exp(x - x.amax(dim=-1, keepdim=True))
        p = p / p.sum(dim=-1, keepdim=True)
        out[b] = torch.matmul(p, rows[:, :DC]).to(out.dtype)
    return out


def _plain_write(s):
    c = s["case"]
    cache, T = s["cache"], c["T"]
    L, n_pages, page, W = cache.shape
    i = torch.arange(T, device=DEV).unsqueeze(0)
    start = s["start"].long().unsqueeze(1)

    def slot(pos):
        return torch.gather(s["table"].long(), 1, pos // page) * page + pos % page

    flat = cache.view(L, n_pages * page, W)
    to = slot(start + i)
    if c["compact"]:
        live = i < s["count"].unsqueeze(1)
        rows = flat[:, slot(start + s["path"].long())[live]]
        flat[:, to[live]] = rows
    else:
        flat[:, to.reshape(-1)] = s["rows"].reshape(L, -1, W)
    return cache


def _plain_copy(s):
    s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
    return s["pool"]


def run(state):
    s = state
    kind = s["case"]["kind"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "decode": _plain_decode,
                "write": _plain_write, "copy": _plain_copy}[kind](s)
    import gated_delta_rule_13_gb300 as kda
    if kind == "fwd":
        return kda.kda_latent_fwd(s["q"], s["k"], s["v"], s["k_rope"], s["cu_q"], s["cu_k"])
    if kind == "bwd":
        got = kda.kda_latent_bwd(s["q"], s["k"], s["v"], s["k_rope"], s["out"], s["lse"],
                                 s["d_out"], s["cu_q"], s["cu_k"])
        return got if s["k_rope"] is not None else got[:3]
    if kind == "decode":
        return kda.kda_latent_decode(s["q"], s["cache"], s["table"], s["seq_lens"],
                                     tree_mask=s["mask"])
    if kind == "write":
        return kda.kda_cache_write(s["cache"], s["rows"], s["table"], s["start"],
                                   path=s["path"], n_write=s["count"])
    return kda.kda_cache_copy_pages(s["pool"], s["src"], s["dst"])


# ------------------------------------------------------------------ work
def _pairs(case):
    """Allowed (query, key) pairs of a causal case, per head."""
    return sum(nq * nk - nq * (nq - 1) // 2
               for nq, nk in zip(_ints(case["lens_q"]), _ints(case["lens_k"])))


def work(case):
    kind = case["kind"]
    if kind in ("fwd", "bwd"):
        nq, nk = sum(_ints(case["lens_q"])), sum(_ints(case["lens_k"]))
        H, dr = case["H"], case["dr"]
        dq = D + dr
        q, kv, r, o = nq * H * dq * 2, nk * H * 2 * D * 2, nk * dr * 2, nq * H * D * 2
        lse = nq * H * 4
        if kind == "fwd":
            return {"bytes": q + kv + r + o + lse, "flops": 2 * _pairs(case) * H * (dq + D)}
        return {"bytes": 2 * (q + kv + r) + 2 * o + lse,
                "flops": 2 * _pairs(case) * H * (3 * dq + 2 * D)}
    if kind == "decode":
        mean = (case["lo"] + case["hi"]) / 2
        W = DC + case["dr"]
        B, T, H = case["B"], case["T"], case["H"]
        return {"bytes": int(B * mean * W * 2 + B * T * H * (W + DC) * 2),
                "flops": int(2 * B * T * H * mean * (W + DC))}
    if kind == "write":
        rows = case["B"] * case["T"]
        if case["compact"]:   # at most half of the drafts and one are accepted, from one on
            rows = case["B"] * (1 + min(case["T"], case["T"] // 2 + 1)) / 2
        return {"bytes": int(2 * rows * case["L"] * (DC + case["dr"]) * 2), "flops": 0}
    return {"bytes": 2 * case["n"] * case["L"] * case["elems"] * (4 if case["fp32"] else 2),
            "flops": 0}


# ------------------------------------------------------------------ 64 bits
def _exact_rows(s, seq, h, i0, i1):
    """Scores of query rows i0 .. i1 of a sequence and head, from the definition."""
    bq, bk = sum(s["lq"][:seq]), sum(s["lk"][:seq])
    nq, nk = s["lq"][seq], s["lk"][seq]
    last = nk - nq + i1                       # keys the block's last row sees
    q = s["q"][bq + i0:bq + i1, h].double()
    k = s["k"][bk:bk + last, h].double()
    z = q[:, :D] @ k.T
    if s["k_rope"] is not None:
        z = z + q[:, D:] @ s["k_rope"][bk:bk + last].double().T
    z = z / math.sqrt(q.shape[1])
    i = torch.arange(i0, i1, device=DEV)[:, None] + (nk - nq)
    z[torch.arange(last, device=DEV)[None, :] > i] = -math.inf
    return q, k, z, bq, bk, last


def _exact_blocks(s, rows=2048):
    for seq, nq in enumerate(s["lq"]):
        for h in range(s["q"].shape[1]):
            for i0 in range(0, nq, rows):
                i1 = min(nq, i0 + rows)
                yield (h, i0, i1) + _exact_rows(s, seq, h, i0, i1)


def _exact_fwd(s):
    Nq, H = s["q"].shape[:2]
    out = torch.zeros(Nq, H, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(Nq, H, dtype=torch.float64, device=DEV)
    for h, i0, i1, q, k, z, bq, bk, last in _exact_blocks(s):
        l = torch.logsumexp(z, dim=1)
        lse[bq + i0:bq + i1, h] = l
        out[bq + i0:bq + i1, h] = torch.exp(z - l[:, None]) @ s["v"][bk:bk + last, h].double()
    return out, lse


def _exact_bwd(s):
    Nq, H, Dq = s["q"].shape
    Nk = s["k"].shape[0]
    z64 = dict(dtype=torch.float64, device=DEV)
    dq, dk, dv = (torch.zeros(Nq, H, Dq, **z64), torch.zeros(Nk, H, D, **z64),
                  torch.zeros(Nk, H, D, **z64))
    dr = torch.zeros(Nk, Dq - D, **z64)
    for h, i0, i1, q, k, z, bq, bk, last in _exact_blocks(s):
        rows, keys = slice(bq + i0, bq + i1), slice(bk, bk + last)
        p = torch.exp(z - s["lse"][rows, h].double()[:, None])
        g = s["d_out"][rows, h].double()
        dv[keys, h] += p.T @ g
        delta = torch.einsum("id,id->i", g, s["out"][rows, h].double())
        e = p * (g @ s["v"][keys, h].double().T - delta[:, None]) / math.sqrt(Dq)
        dq[rows, h, :D] = e @ k
        dk[keys, h] += e.T @ q[:, :D]
        if Dq > D:
            dq[rows, h, D:] = e @ s["k_rope"][keys].double()
            dr[keys] += e.T @ q[:, D:]
    return (dq, dk, dv, dr) if Dq > D else (dq, dk, dv)


def _exact_decode(s):
    c = s["case"]
    B, T, H, W = s["q"].shape
    out = torch.zeros(B, T, H, DC, dtype=torch.float64, device=DEV)
    mask = None if s["mask"] is None else s["mask"].cpu().tolist()
    for b, n in enumerate(s["lens"]):
        pos = torch.arange(n, device=DEV)
        page = s["table"][b].long()[torch.div(pos, c["page"], rounding_mode="floor")]
        x = s["cache"][page, pos % c["page"]].double()
        for t in range(T):
            if mask is None:
                keys = pos[:n - T + t + 1]
            else:
                keys = torch.cat([pos[:n - T], torch.tensor(
                    [n - T + j for j in range(T) if mask[b][t] >> j & 1], device=DEV,
                    dtype=torch.long)])
            y = x if len(keys) == n else x[keys]
            w = torch.softmax(s["q"][b, t].double() @ y.T / math.sqrt(D + c["dr"]), dim=1)
            out[b, t] = w @ y[:, :DC]
    return out


def _exact_write(s):
    c = s["case"]
    new = s["cache"].clone()
    table, start = s["table"].cpu().tolist(), s["start"].cpu().tolist()
    path = None if s["path"] is None else s["path"].cpu().tolist()
    count = None if s["count"] is None else s["count"].cpu().tolist()
    to, frm = [], []
    for b in range(c["B"]):
        for i in range(c["T"] if count is None else count[b]):
            p = start[b] + i
            to.append((table[b][p // c["page"]], p % c["page"]))
            f = start[b] + path[b][i] if path is not None else p
            frm.append((table[b][f // c["page"]], f % c["page"]))
    tp, tr = (torch.tensor(x, device=DEV) for x in zip(*to))
    if c["compact"]:
        fp, fr = (torch.tensor(x, device=DEV) for x in zip(*frm))
        new[:, tp, tr] = s["cache"][:, fp, fr]
    else:
        new[:, tp, tr] = s["rows"].flatten(1, 2)
    return new.double()


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "copy":
        new = s["pool"].clone()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            new[:, b] = s["pool"][:, a]
        return new.double()
    return {"fwd": _exact_fwd, "bwd": _exact_bwd, "decode": _exact_decode,
            "write": _exact_write}[kind](s)
