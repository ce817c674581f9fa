"""A hybrid stack's two kinds of layer served together: one recurrent (KDA) layer
and one latent-attention layer, two requests, a prompt, a tree of drafted tokens, the
accepted path, and a fork.

    python examples/hybrid_serving.py

What happens to the latent layer:
  prompt      expanded form (kda_latent_fwd); its latent rows go to the paged cache
              (kda_cache_write)
  drafts      rows appended to the cache, absorbed form with the tree's masks
              (kda_latent_decode)
  acceptance  the accepted rows move together in the cache (kda_cache_write, no rows)
  fork        the last, partly filled page gets a private copy (kda_cache_copy_pages)
and to the recurrent layer: kda_chunk_fwd over the prompt, kda_decode_replay over the
accepted tokens, its state copied for the fork (kda_cache_copy_pages).

Every step's attention output is compared with the expanded form over the tokens the
step stands for.  A training step of the latent layer (kda_latent_fwd and
kda_latent_bwd around the projections) closes the example.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_13_gb300 as kda  # noqa: E402

DEV = "cuda:0"
D_MODEL, H, DC, DR, DH = 256, 8, 512, 64, 128
PAGE, PAGES = 64, 12


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).bfloat16()


class LatentLayer:
    """Latent attention between its projections (plain matrix products)."""

    def __init__(self, g):
        self.w_q = randn(g, D_MODEL, H * (DH + DR), std=D_MODEL ** -0.5)
        self.w_c = randn(g, D_MODEL, DC + DR, std=D_MODEL ** -0.5)
        self.w_kv = randn(g, DC, H * 2 * DH, std=DC ** -0.5)
        up = self.w_kv.view(DC, H, 2 * DH)
        self.w_uk, self.w_uv = up[..., :DH], up[..., DH:]

    def queries(self, x):
        return (x @ self.w_q).view(*x.shape[:-1], H, DH + DR)

    def rows(self, x):
        """The cached row of every token: latent and rotary channels."""
        return x @ self.w_c

    def expanded(self, x, cu):
        rows = self.rows(x)
        kv = (rows[:, :DC] @ self.w_kv).view(-1, H, 2 * DH)
        return kda.kda_latent_fwd(self.queries(x), kv[..., :DH], kv[..., DH:],
                                  rows[:, DC:].contiguous(), cu)

    def absorbed(self, x, cache, table, lens, tree=None):
        """x [B, T, D]: attention outputs [B, T, H, 128] of the last T tokens."""
        q = self.queries(x)
        q = torch.cat([torch.einsum("bthd,chd->bthc", q[..., :DH], self.w_uk), q[..., DH:]], -1)
        o = kda.kda_latent_decode(q.contiguous(), cache, table, lens, tree_mask=tree)
        return torch.einsum("bthc,chd->bthd", o, self.w_uv)


def compare(what, got, want):
    """Both ways round to bf16 at different places; outputs are of order 1."""
    err = (got.float() - want.float()).norm() / want.float().norm()
    print(f"{what:44s} relative difference {err:.4f}")
    if not err < 0.02:
        raise AssertionError(f"{what}: {err}")


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


def serve(g):
    layer, n = LatentLayer(g), 100
    B = 2
    prompt = randn(g, B, n, D_MODEL)
    cache = torch.zeros(PAGES, PAGE, DC + DR, device=DEV).bfloat16()
    table = i32([[3, 0, 7], [1, 9, 4]])

    # prompt: both requests packed, expanded form; latent rows into the cache
    cu = i32([0, n, 2 * n])
    out, _ = layer.expanded(prompt.view(-1, D_MODEL), cu)
    kda.kda_cache_write(cache, layer.rows(prompt), table, i32([0, 0]))

    # the recurrent layer of the same requests
    k = randn(g, B, n, 3, H, DH)
    unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).bfloat16()  # noqa: E731
    gates = torch.rand(2, B, n, H, DH, generator=g, device=DEV)
    flat = lambda t: t.reshape(B * n, *t.shape[2:]).contiguous()  # noqa: E731
    _, state = kda.kda_chunk_fwd(flat(unit(k[:, :, 0])), flat(unit(k[:, :, 1])),
                                 flat(k[:, :, 2]), flat(-5 * gates[0]),
                                 flat(gates[1][..., 0]), None, cu)
    pool = torch.zeros(1, 4, H, DH, DH, device=DEV)     # running states and snapshots
    pool[0, :B] = state

    # a tree of six drafts for each request:  0 - 1 - 3,  0 - 2 - 4 - 5
    parent = [-1, 0, 0, 1, 2, 4]
    words, paths = [], []
    for i, p in enumerate(parent):
        words.append((words[p] if p >= 0 else 0) | 1 << i)
        paths.append((paths[p] if p >= 0 else []) + [i])
    T = len(parent)
    drafts = randn(g, B, T, D_MODEL)
    kda.kda_cache_write(cache, layer.rows(drafts), table, i32([n, n]))
    tree = torch.tensor([words] * B, device=DEV)
    got = layer.absorbed(drafts, cache, table, i32([n + T] * B), tree)
    for i in (0, 3, 5):
        tokens = torch.cat([prompt, drafts[:, paths[i]]], 1)
        m = tokens.shape[1]
        want, _ = layer.expanded(tokens.reshape(-1, D_MODEL), i32([0, m, 2 * m]))
        compare(f"draft {i}, its path of {len(paths[i])}", got[:, i], want.view(B, m, H, DH)[:, -1])

    # request 0 accepts 0 - 2 - 4, request 1 accepts 0 - 1
    accepted, count = [[0, 2, 4], [0, 1]], i32([3, 2])
    path = i32([p + [0] * (T - len(p)) for p in accepted])
    kda.kda_cache_write(cache, None, table, i32([n, n]), path=path, n_write=count)
    pick = path.long()[:, :4].clamp(min=0)
    kd = randn(g, B, T, 3, H, DH)
    gd = torch.rand(2, B, T, H, DH, generator=g, device=DEV)
    at = torch.arange(B, device=DEV)[:, None]
    take = lambda t: t[at, pick].contiguous()  # noqa: E731
    running = pool[0, :B].contiguous()
    kda.kda_decode_replay(running, take(unit(kd[:, :, 0])), take(unit(kd[:, :, 1])),
                          take(kd[:, :, 2]), take(-5 * gd[0]), take(gd[1][..., 0]), count)
    pool[0, :B] = running

    # request 0 is forked: a private copy of its partly filled page and of its state
    lens = [n + 3, n + 2]
    last = lens[0] // PAGE
    fork_page, fork_state = 11, 2
    kda.kda_cache_copy_pages(cache.unsqueeze(0), i32([int(table[0, last])]), i32([fork_page]))
    kda.kda_cache_copy_pages(pool, i32([0]), i32([fork_state]))
    assert torch.equal(pool[0, 0], pool[0, fork_state])
    table = torch.cat([table, table[:1]])
    table[2, last] = fork_page

    # one more token for each of the three, one step
    step = randn(g, 3, 1, D_MODEL)
    lens = i32(lens + lens[:1])
    kda.kda_cache_write(cache, layer.rows(step), table, lens)
    got = layer.absorbed(step, cache, table, lens + 1)
    for b in range(3):
        r = b % 2 if b < 2 else 0
        tokens = torch.cat([prompt[r], drafts[r, accepted[r]], step[b]])
        want, _ = layer.expanded(tokens, None)
        compare(f"request {b}, the token after acceptance", got[b, 0], want[-1])
    return out


def train(g):
    """Gradients of the latent layer's weights for a packed batch; the loss goes down
    along them by what they predict."""
    layer = LatentLayer(g)
    lens = [70, 130, 40]
    cu = i32([0, 70, 200, 240])
    x, target = randn(g, sum(lens), D_MODEL), randn(g, sum(lens), H, DH)

    def forward():
        q, rows = layer.queries(x), layer.rows(x)
        kv = (rows[:, :DC] @ layer.w_kv).view(-1, H, 2 * DH)
        rope = rows[:, DC:].contiguous()
        out, lse = kda.kda_latent_fwd(q, kv[..., :DH], kv[..., DH:], rope, cu)
        diff = out.float() - target.float()
        return q, rows, kv, rope, out, lse, diff, 0.5 * float((diff * diff).mean())

    q, rows, kv, rope, out, lse, diff, before = forward()
    scale = 1024.0                                       # keeps bf16 gradients in range
    d_out = (diff * (scale / diff.numel())).bfloat16()
    d_kv = torch.empty_like(kv)
    dq, _, _, d_rope = kda.kda_latent_bwd(q, kv[..., :DH], kv[..., DH:], rope, out, lse, d_out, cu,
                                          d_k=d_kv[..., :DH], d_v=d_kv[..., DH:])
    d_kv = d_kv.view(sum(lens), -1)
    d_rows = torch.cat([d_kv @ layer.w_kv.t(), d_rope], 1)
    grads = [(layer.w_q, x.t() @ dq.view(sum(lens), -1)), (layer.w_c, x.t() @ d_rows),
             (layer.w_kv, rows[:, :DC].t() @ d_kv)]
    grads = [(w, d.float() / scale) for w, d in grads]
    square = sum(float((d * d).sum()) for _, d in grads)
    step = 0.02 * before / square                        # a first-order drop of 2 %
    for w, d in grads:
        w.copy_((w.float() - step * d).bfloat16())
    after = forward()[-1]
    print(f"training step: loss {before:.5f} -> {after:.5f}")
    if not 0.005 * before < before - after < 0.04 * before:
        raise AssertionError("the step did not lower the loss as its gradients predict")


def main():
    g = torch.Generator(device=DEV).manual_seed(0)
    serve(g)
    train(g)
    torch.cuda.synchronize()
    print("ok")


if __name__ == "__main__":
    main()
