"""Workloads of the operators around a cached latent row: the norm before its
projections, the rotation of its positions, the attention weight it has been given,
and its eviction from a full cache.

Each case is one call of one operator, from the smallest a user makes (one token of
each request of a decode step) to the largest (a training batch, a full serving
batch).  With ``own`` false the operators run in a plain form of elementary torch
operations in 32 bits; with ``own`` true they run through the package.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda:0"
DC = 512      # latent channels of a cached row
D = 128       # channels of a head without positions


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the new token of 64 requests: rotary channels of 96 heads and of the shared key
        dict(name="rope_token", kind="rope", n=64, H=96, dr=64, key=True, interleaved=True,
             far=131072, factor=1.0, transpose=False, fp32=False),
        # a training batch of 4 x 4096 tokens, 16 heads
        dict(name="rope_train", kind="rope", n=16384, H=16, dr=64, key=True, interleaved=False,
             far=4096, factor=1.0, transpose=False, fp32=False),
        # the gradient of a chunk of a long prompt, 96 heads, positions scaled to 1 M tokens
        dict(name="rope_grad_long", kind="rope", n=8192, H=96, dr=64, key=False, interleaved=True,
             far=1048576, factor=32.0, transpose=True, fp32=True),
        # the hidden states of a decode step, 64 requests, no mean taken off
        dict(name="norm_token", kind="norm", n=64, W=7168, stride=7168, center=False, bias=False,
             fp32=False),
        # the hidden states of a training batch of 16384 tokens
        dict(name="norm_train", kind="norm", n=16384, W=7168, stride=7168, center=True, bias=True,
             fp32=False),
        # gradients of the latents' norm: 512 channels of rows of 576, fp32
        dict(name="norm_grad_latent", kind="norm_grad", n=16384, W=512, stride=576, center=False,
             bias=False, fp32=True),
        # gradients of the hidden states' norm of the training batch
        dict(name="norm_grad_train", kind="norm_grad", n=16384, W=7168, stride=7168, center=True,
             bias=True, fp32=False),
        # weights given by one token of one interactive request: latency counts
        dict(name="weights_single", kind="weights", B=1, T=1, H=96, dr=0, lo=3001, hi=3001,
             page=64, tree=False, decay=1.0),
        # by one token of each of a serving batch of ragged lengths
        dict(name="weights_batch", kind="weights", B=128, T=1, H=96, dr=64, lo=1, hi=16384,
             page=64, tree=False, decay=1.0),
        # by a tree of 16 drafts of each of 32 requests
        dict(name="weights_tree", kind="weights", B=32, T=16, H=96, dr=64, lo=3000, hi=16000,
             page=512, tree=True, decay=0.97),
        # a full cache takes a step's row: one row of each of 16 requests leaves, one layer
        dict(name="evict_step", kind="evict", L=1, B=16, dr=64, lo=2049, hi=2049, budget=2048,
             first=4, recent=64, page=64),
        # prompts of 8 requests cut to a budget, 24 layers at once
        dict(name="evict_prompt", kind="evict", L=24, B=8, dr=64, lo=3000, hi=8192, budget=2048,
             first=4, recent=256, page=64),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "norm", "norm", "norm_grad", "norm_grad", "weights",
                       "weights", "evict", "evict"])
    if kind == "rope":
        dr = rng.choice([64, 64, 64, 128, 32, 16, 2 * rng.randint(1, 64)])
        H = rng.choice([1, 3, 8, 16, 24, 40, 96, 128])
        return dict(kind=kind, n=_logint(rng, 1, min(32768, (1 << 25) // (H * dr))), H=H, dr=dr,
                    key=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                    far=_logint(rng, 1000, 1048576), factor=rng.choice([1.0, 4.0, 32.0]),
                    transpose=rng.random() < 0.4, fp32=rng.random() < 0.4)
    if kind in ("norm", "norm_grad"):
        W = rng.choice([128, 512, 3584, 7168, _logint(rng, 16, 16384), _logint(rng, 16, 16384)])
        return dict(kind=kind, n=_logint(rng, 1, min(32768, 58_000_000 // W)), W=W,
                    stride=W + rng.choice([0, 0, 0, 1, 8, 64]), center=rng.random() < 0.5,
                    bias=rng.random() < 0.5, fp32=rng.random() < 0.4)
    if kind == "weights":
        tree = rng.random() < 0.4
        T = rng.randint(2, 24) if tree else rng.choice([1, 1, 1, 2, 4, 5, 70])
        H = rng.choice([1, 5, 16, 40, 64, 96, 128])
        lo = T + _logint(rng, 1, 4096)
        hi = lo + _logint(rng, 1, 8192)
        most = max(1, min(64, 400_000_000 // (T * H * hi)))
        return dict(kind=kind, B=_logint(rng, 1, most), T=T, H=H, dr=rng.choice([0, 64]), lo=lo,
                    hi=hi, page=rng.choice([16, 48, 64, 128, 512]), tree=tree,
                    decay=rng.choice([0.0, 0.9, 1.0]))
    budget = _logint(rng, 1, 3000)
    recent = rng.randint(0, budget // 2)
    lo = _logint(rng, 1, 4096)
    return dict(kind=kind, L=rng.randint(1, 12), B=_logint(rng, 1, 12), dr=rng.choice([0, 64]),
                lo=lo, hi=lo + _logint(rng, 1, 6000), budget=budget,
                first=rng.randint(0, min(8, budget - recent)), recent=recent,
                page=rng.choice([16, 48, 64, 128, 512]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _host(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _inv_freq(case):
    """Angle per position of every channel pair: base 10000, slowed down by the factor
    by which the context has grown."""
    i = torch.arange(case["dr"] // 2, dtype=torch.float64)
    return 10000.0 ** (-2.0 * i / case["dr"]) / case["factor"]


def _tables(lens, page, seed, most):
    """Block tables of sequences of these lengths (``most`` at the most), their pages
    spread over a shuffled pool that has room for all of them at their longest."""
    width = (most + page - 1) // page
    need = torch.tensor([(n + page - 1) // page for n in lens])
    n_pages = len(lens) * width + 3
    order = torch.randperm(n_pages, generator=_host(seed + 2)).to(torch.int32)
    used = torch.arange(width)[None, :] < need[:, None]
    table = torch.zeros(len(lens), width, dtype=torch.int32)
    table[used] = order[:int(need.sum())]
    return table.to(DEV), n_pages


def _tree(B, T, seed):
    """Ancestor masks of random draft trees (a node sees itself and its ancestors)."""
    pick = torch.rand(B, T, generator=_host(seed + 3))
    out = torch.zeros(B, T, dtype=torch.int64)
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
    if kind == "rope":
        n, H, dr = case["n"], case["H"], case["dr"]
        dt = torch.float32 if case["fp32"] else torch.bfloat16
        pos = torch.randint(0, case["far"], (n,), generator=g, device=DEV).to(torch.int32)
        # heads of 128 + dr channels and rows of 512 + dr, the last dr rotary; the queries
        # go to those of another buffer of the same layout
        return dict(case=case, pos=pos, freq=_inv_freq(case).to(DEV),
                    scale=0.1 * math.log(case["factor"]) + 1.0,
                    q=_randn(g, n, H, D + dr, dtype=dt),
                    to=torch.zeros(n, H, D + dr, dtype=dt, device=DEV),
                    rows=_randn(g, n, DC + dr, dtype=dt) if case["key"] else None)
    if kind in ("norm", "norm_grad"):
        n, W, stride = case["n"], case["W"], case["stride"]
        dt = torch.float32 if case["fp32"] else torch.bfloat16
        base = _randn(g, n, stride, dtype=dt)
        x = base.mul_(1.5).add_(0.3)[:, :W]
        s = dict(case=case, x=x, weight=1 + 0.2 * _randn(g, W, dtype=torch.float32),
                 bias=0.1 * _randn(g, W, dtype=torch.float32) if case["bias"] else None)
        if kind == "norm_grad":
            s["g"] = _randn(g, n, stride, dtype=dt)[:, :W]
            s["mean"], s["rstd"] = _stats(x, case["center"])
        return s
    lens = torch.randint(case["lo"], case["hi"] + 1, (case["B"],), generator=_host(seed + 1)).tolist()
    table, n_pages = _tables(lens, case["page"], seed, case["hi"])
    W, cap = DC + case["dr"], table.shape[1] * case["page"]
    s = dict(case=case, lens=lens, seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
             table=table)
    live = torch.arange(cap, device=DEV)[None, :] < s["seq_lens"][:, None]
    if kind == "weights":
        s.update(cache=_randn(g, n_pages, case["page"], W),
                 q=_randn(g, case["B"], case["T"], case["H"], W), mask=None,
                 weights=torch.rand(case["B"], cap, generator=g, device=DEV) * live)
        if case["tree"]:
            s["mask"] = _tree(case["B"], case["T"], seed).to(DEV)
        s["lse"] = _lse(s)
        return s
    # what rows have been given by many steps spreads over some powers of ten
    spread = torch.randn(case["L"], case["B"], cap, generator=g, device=DEV).mul_(2.0).exp_()
    s.update(weights=spread * live, after=torch.zeros_like(spread),
             cache=torch.empty(case["L"], n_pages, case["page"], W, dtype=torch.bfloat16, device=DEV))
    for layer in s["cache"]:
        layer.copy_(_randn(g, n_pages, case["page"], W))
    return s


# ------------------------------------------------------------------ plain forms
def _turn(x, angle, scale, interleaved, transpose):
    c, t = (torch.cos(angle) * scale).float(), (torch.sin(angle) * scale).float()
    if transpose:
        t = -t
    half = x.shape[-1] // 2
    y = x.float()
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :half], y[..., half:])
    u, v = a * c - b * t, b * c + a * t
    out = torch.stack([u, v], dim=-1).flatten(-2) if interleaved else torch.cat([u, v], dim=-1)
    return out.to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    dr = c["dr"]
    angle = s["pos"].double()[:, None] * s["freq"]
    s["to"][..., D:] = _turn(s["q"][..., D:], angle[:, None], s["scale"], c["interleaved"],
                             c["transpose"])
    if not c["key"]:
        return s["to"][..., D:]
    return s["to"][..., D:], _turn(s["rows"][:, DC:], angle, s["scale"], c["interleaved"],
                                   c["transpose"])


def _stats(x, center, eps=1e-5):
    y = x.float()
    mean = y.mean(dim=-1) if center else None
    if center:
        y = y - mean[:, None]
    return mean, torch.rsqrt((y * y).mean(dim=-1) + eps)


def _plain_norm(s):
    mean, rstd = _stats(s["x"], s["case"]["center"])
    y = s["x"].float()
    if mean is not None:
        y = y - mean[:, None]
    y = y * rstd[:, None] * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    y = y.to(s["x"].dtype)
    return (y, rstd) if mean is None else (y, mean, rstd)


def _plain_norm_grad(s):
    g, y = s["g"].float(), s["x"].float()
    if s["mean"] is not None:
        y = y - s["mean"][:, None]
    y = y * s["rstd"][:, None]
    d_weight, d_bias = (g * y).sum(dim=0), g.sum(dim=0)
    g = g * s["weight"]
    d = g - y * (g * y).mean(dim=-1, keepdim=True)
    if s["mean"] is not None:
        d = d - g.mean(dim=-1, keepdim=True)
    d = (d * s["rstd"][:, None]).to(s["x"].dtype)
    return (d, d_weight, d_bias) if s["case"]["bias"] else (d, d_weight)


def _scores(s, b0, b1):
    """[b, T, H, cap] scores of sequences b0 .. b1, -inf where a token does not look."""
    c = s["case"]
    page, T, W = c["page"], c["T"], s["q"].shape[-1]
    rows = s["cache"][s["table"][b0:b1].long()].reshape(b1 - b0, -1, W).float()
    q = s["q"][b0:b1].reshape(b1 - b0, -1, W).float()
    x = torch.matmul(q, rows.transpose(1, 2)).mul_(1.0 / math.sqrt(D + c["dr"]))
    cap = rows.shape[1]
    pos = torch.arange(cap, device=DEV)
    n = s["seq_lens"][b0:b1].long()[:, None, None]
    draft = pos - (n - T)                                       # [b, 1, cap]
    t = torch.arange(T, device=DEV)[None, :, None]
    if s["mask"] is None:
        seen = draft <= t
    else:
        bits = s["mask"][b0:b1, :, None] >> draft.clamp(0, 63)
        seen = (draft < 0) | ((draft < T) & ((bits & 1) == 1))
    x = x.view(b1 - b0, T, -1, cap)
    return x.masked_fill_(~(seen & (pos < n))[:, :, None, :], float("-inf"))


def _pieces(s):
    c = s["case"]
    step = max(1, (1 << 29) // (c["T"] * c["H"] * s["table"].shape[1] * c["page"]))
    return [(b, min(c["B"], b + step)) for b in range(0, c["B"], step)]


def _lse(s):
    return torch.cat([torch.logsumexp(_scores(s, b0, b1), dim=-1) for b0, b1 in _pieces(s)])


def _plain_weights(s):
    w, decay = s["weights"], s["case"]["decay"]
    live = torch.arange(w.shape[1], device=DEV)[None, :] < s["seq_lens"][:, None]
    given = torch.cat([torch.exp(_scores(s, b0, b1) - s["lse"][b0:b1, ..., None]).sum(dim=(1, 2))
                       for b0, b1 in _pieces(s)])
    w.copy_(torch.where(live, w * decay + given, w))
    return w


def _plain_evict(s):
    """Kept rows from behind the places that stay go to the places that fall free, in
    order; the last rows move up together."""
    c = s["case"]
    L, B, cap = s["weights"].shape
    budget, recent = c["budget"], c["recent"]
    n = s["seq_lens"].long()[None, :, None]                     # [1, B, 1]
    pos = torch.arange(cap, device=DEV)[None, None, :]
    full = n > budget
    front = (pos < c["first"]) | ~full
    middle = (pos >= c["first"]) & (pos < n - recent) & full
    key = torch.where(middle, s["weights"], torch.full_like(s["weights"], -1.0))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order)
    rank.scatter_(-1, order, pos.expand(L, B, cap))
    stay = (front | (middle & (rank < budget - c["first"] - recent))) & (pos < n)
    last = budget - recent
    hole = full & ~stay & (pos < last)
    mover = full & stay & (pos >= last) & (pos < n - recent)
    # the i-th hole takes the i-th mover
    take = torch.cumsum(hole, dim=-1) - 1
    movers = torch.sort((~mover).to(torch.int8), dim=-1, stable=True).indices
    origin = torch.where(hole, torch.gather(movers, -1, take.clamp(min=0)), pos)
    origin = torch.where(full & (pos >= last), pos + (n - budget), origin)
    origin = torch.nn.functional.pad(origin, (0, max(0, budget - cap)))[..., :budget]
    at = torch.arange(budget, device=DEV)[None, None, :]
    new_lens = torch.clamp(s["seq_lens"], max=budget)
    origin = torch.where(at < new_lens[None, :, None], origin, torch.full_like(origin, -1))
    live = origin >= 0
    s["after"].zero_()
    keep = min(budget, cap)
    s["after"][..., :keep] = (torch.gather(s["weights"], -1, origin.clamp(min=0)) * live)[..., :keep]
    move = live & (origin != at)
    l, b, i = torch.nonzero(move, as_tuple=True)
    page = c["page"]
    src, table = origin[l, b, i], s["table"].long()
    s["cache"][l, table[b, i // page], i % page] = s["cache"][l, table[b, src // page], src % page]
    return new_lens, origin.to(torch.int32), s["after"], s["cache"]


def run(state):
    s = state
    c = s["case"]
    kind = c["kind"]
    if not own:
        return {"rope": _plain_rope, "norm": _plain_norm, "norm_grad": _plain_norm_grad,
                "weights": _plain_weights, "evict": _plain_evict}[kind](s)
    import gated_delta_rule_13_gb300 as kda
    if kind == "rope":
        return kda.kda_rope(s["q"][..., D:], s["pos"], s["freq"], out=s["to"][..., D:],
                            k=s["rows"][:, DC:] if c["key"] else None,
                            interleaved=c["interleaved"], scale=s["scale"],
                            transpose=c["transpose"])
    if kind == "norm":
        y, mean, rstd = kda.kda_norm_fwd(s["x"], s["weight"], s["bias"], center=c["center"])
        return (y, rstd) if mean is None else (y, mean, rstd)
    if kind == "norm_grad":
        got = kda.kda_norm_bwd(s["g"], s["x"], s["weight"], s["mean"], s["rstd"], bias=c["bias"])
        return got if c["bias"] else got[:2]
    if kind == "weights":
        return kda.kda_latent_weights(s["q"], s["cache"], s["table"], s["seq_lens"], s["lse"],
                                      s["weights"], tree_mask=s["mask"], decay=c["decay"])
    new_lens, origin = kda.kda_cache_evict(s["cache"], s["table"], s["seq_lens"], s["weights"],
                                           c["budget"], first=c["first"], recent=c["recent"],
                                           weights_out=s["after"])
    return new_lens, origin, s["after"], s["cache"]


# ------------------------------------------------------------------ work
def work(case):
    kind = case["kind"]
    if kind == "rope":
        esz = 4 if case["fp32"] else 2
        rows = case["n"] * (case["H"] + (1 if case["key"] else 0))
        return {"bytes": 2 * rows * case["dr"] * esz + case["n"] * 4,
                "flops": 3 * rows * case["dr"]}
    if kind in ("norm", "norm_grad"):
        n, W, esz = case["n"], case["W"], 4 if case["fp32"] else 2
        stats = n * 4 * (2 if case["center"] else 1)
        vectors = W * 4 * (2 if case["bias"] else 1)
        if kind == "norm":
            return {"bytes": 2 * n * W * esz + vectors + stats, "flops": 8 * n * W}
        return {"bytes": 3 * n * W * esz + vectors + W * 4 + stats, "flops": 14 * n * W}
    mean = (case["lo"] + case["hi"]) / 2
    B, W = case["B"], DC + case["dr"]
    if kind == "weights":
        R = case["T"] * case["H"]
        old = 1 if case["decay"] else 0
        return {"bytes": int(B * mean * (W * 2 + 4 * (1 + old)) + B * R * (W * 2 + 4)),
                "flops": int(2 * B * R * mean * W)}
    # of the kept rows of the middle, as many lie behind their final places as chance has it
    budget, recent, first = case["budget"], case["recent"], case["first"]
    over = max(0.0, mean - budget)
    middle = max(1.0, mean - recent - first)
    rows = case["L"] * B * ((budget - recent - first) * over / middle + recent if over else 0)
    cap = (case["hi"] + case["page"] - 1) // case["page"] * case["page"]
    return {"bytes": int(2 * rows * W * 2 + case["L"] * B * (mean * 4 + cap * 4 + budget * 4)),
            "flops": 0}


# ------------------------------------------------------------------ 64 bits
def _exact_rope(s):
    c = s["case"]

    def turned(x, lead):
        z = x.double()
        z = z.unflatten(-1, (-1, 2)) if c["interleaved"] else z.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_complex(z.contiguous())
        phi = torch.outer(s["pos"].double(), s["freq"])
        by = torch.polar(torch.full_like(phi, s["scale"]), -phi if c["transpose"] else phi)
        z = torch.view_as_real(z * (by[:, None, :] if lead else by))
        return z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)

    q = turned(s["q"][..., D:], True)
    return (q, turned(s["rows"][:, DC:], False)) if c["key"] else q


def _exact_norm(s):
    x = s["x"].double()
    if s["case"]["center"]:
        var, mean = torch.var_mean(x, dim=1, correction=0)
    else:
        var, mean = x.square().mean(dim=1), None
    sd = torch.sqrt(var + 1e-5)
    y = (x if mean is None else x.sub_(mean[:, None])).div_(sd[:, None])
    y = torch.addcmul(torch.zeros((), dtype=torch.float64, device=DEV) if s["bias"] is None
                      else s["bias"].double(), y, s["weight"].double())
    return (y, 1 / sd) if mean is None else (y, mean, 1 / sd)


def _exact_norm_grad(s):
    g, x = s["g"].double(), s["x"].double()
    W, r = x.shape[1], s["rstd"].double()[:, None]
    z = (x if s["mean"] is None else x - s["mean"].double()[:, None]) * r
    d_weight, d_bias = torch.einsum("nw,nw->w", g, z), g.sum(0)
    e = g * s["weight"].double()
    d = e - z * (torch.einsum("nw,nw->n", e, z) / W)[:, None]
    if s["mean"] is not None:
        d -= (e.sum(1) / W)[:, None]
    d *= r
    return (d, d_weight, d_bias) if s["case"]["bias"] else (d, d_weight)


def _exact_weights(s):
    c = s["case"]
    T = c["T"]
    out = s["weights"].double()
    mask = None if s["mask"] is None else s["mask"].cpu().tolist()
    for b, n in enumerate(s["lens"]):
        at = torch.arange(n, device=DEV)
        y = s["cache"][s["table"][b].long()[at // c["page"]], at % c["page"]].double()
        w = torch.zeros(n, dtype=torch.float64, device=DEV)
        for t in range(T):
            z = s["q"][b, t].double() @ y.T / math.sqrt(D + c["dr"]) - s["lse"][b, t].double()[:, None]
            p = torch.exp(z).sum(0)
            if mask is None:
                p[n - T + t + 1:] = 0
            else:
                for j in range(T):
                    if not mask[b][t] >> j & 1:
                        p[n - T + j] = 0
            w += p
        out[b, :n] = c["decay"] * out[b, :n] + w
    return out


def _exact_evict(s):
    c = s["case"]
    L, B, cap = s["weights"].shape
    budget, recent, first, page = c["budget"], c["recent"], c["first"], c["page"]
    host = s["weights"].cpu().tolist()
    table = s["table"].cpu().tolist()
    origin = torch.full((L, B, budget), -1, dtype=torch.int32)
    after = torch.zeros(L, B, cap, dtype=torch.float64)
    cache = s["cache"].clone()
    for layer in range(L):
        to, frm = [], []
        for b, n in enumerate(s["lens"]):
            w = host[layer][b]
            if n <= budget:
                new = list(range(n))
            else:
                best = sorted(range(first, n - recent), key=lambda j: (-w[j], j))
                kept = set(best[:budget - first - recent]) | set(range(first))
                behind = sorted(j for j in kept if j >= budget - recent)
                new = [j if j in kept else None for j in range(budget - recent)]
                behind.reverse()
                new = [behind.pop() if j is None else j for j in new] + list(range(n - recent, n))
            for i, j in enumerate(new):
                origin[layer, b, i] = j
                after[layer, b, i] = w[j]
                if i != j:
                    to.append(table[b][i // page] * page + i % page)
                    frm.append(table[b][j // page] * page + j % page)
        if to:
            flat = cache[layer].view(-1, cache.shape[-1])
            flat[torch.tensor(to, device=DEV)] = s["cache"][layer].view(-1, cache.shape[-1])[
                torch.tensor(frm, device=DEV)]
    new_lens = torch.tensor([min(n, budget) for n in s["lens"]], dtype=torch.int32, device=DEV)
    return new_lens, origin.to(DEV), after.to(DEV), cache.double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "norm": _exact_norm, "norm_grad": _exact_norm_grad,
            "weights": _exact_weights, "evict": _exact_evict}[case["kind"]](s)
