"""The attention weight of cached rows against its 64-bit form."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_13_gb300 as kda
import rows_util as ru

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32

# A score is a sum of 512 or 576 products in 32 to 36 steps of the tensor cores, each off by
# at most 2^-22 of the largest partial sum; with scores of deviation 1.7 a partial sum stays
# below 12: 36 x 2^-22 x 12 = 1e-4 in the exponent, where the last bits of lse (2^-23 of at
# most 12) and of the exponential are lost beside it.
REL = 1.1e-4


def _data(lens, T, H, dr, page, seed=0, tree=False, spare=0, wild=True):
    g = torch.Generator().manual_seed(seed)
    B, W = len(lens), 512 + dr
    width = max(1, max((n + page - 1) // page for n in lens)) + spare
    table, n_pages = ru.pages(lens, page, g, width=width)
    cache = torch.randn(n_pages, page, W, generator=g).to(BF).to(DEV)
    if wild:                                  # what lies behind a sequence is anything
        used = torch.zeros(n_pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for i in range(n):
                used[table[b, i // page], i % page] = True
        cache[~used.to(DEV)] = float("nan")
    q = torch.randn(B, T, H, W, generator=g).to(BF).to(DEV)
    mask = None
    if tree:
        mask = torch.zeros(B, T, dtype=torch.int64)
        for b in range(B):
            words = []
            for i in range(T):
                up = words[int(torch.randint(0, i, (1,), generator=g))] if i else 0
                words.append(up | 1 << i)
            # as 64-bit words: the last draft's bit may be the sign
            mask[b] = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words])
        mask = mask.to(DEV)
    old = torch.rand(B, width * page, generator=g).to(DEV)
    return dict(q=q, cache=cache, table=table.to(DEV), lens=lens, mask=mask, old=old,
                seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                scale=(128 + dr) ** -0.5)


def _lse(d):
    lse = torch.full(d["q"].shape[:3], 7.0, device=DEV)
    kda.kda_latent_decode(d["q"], d["cache"], d["table"], d["seq_lens"], tree_mask=d["mask"], lse=lse)
    return lse


def _run(d, lse, decay=1.0, **kw):
    w = d["old"].clone()
    got = kda.kda_latent_weights(d["q"], d["cache"], d["table"], d["seq_lens"], lse, w,
                                 tree_mask=d["mask"], decay=decay, **kw)
    assert got is w
    return w


def _check(got, d, lse, decay=1.0):
    mask = None if d["mask"] is None else d["mask"].cpu()
    want = ru.weights_ref(d["q"], d["cache"], d["table"], d["lens"], lse, d["old"], mask, d["scale"],
                          decay)
    R = d["q"].shape[1] * d["q"].shape[2]
    # sums of R terms, fp32; then the old weights' product and sum
    tol = (REL + (R + 8) * ru.U) * (want - decay * d["old"].double()).abs() \
        + 2 * ru.U * want.abs() + 1e-30
    for b, n in enumerate(d["lens"]):
        assert torch.equal(got[b, n:], d["old"][b, n:])
        err = (got[b, :n].double() - want[b, :n]).abs()
        assert (err <= tol[b, :n]).all(), f"{b}: {(err / tol[b, :n]).max().item():.3g} of the bound"


@pytest.mark.parametrize("lens,T,H,dr,page,tree", [
    ([1], 1, 1, 0, 16, False), ([1], 1, 96, 64, 64, False), ([3001], 1, 96, 0, 64, False),
    ([0, 1, 5, 128, 129, 1000], 1, 96, 64, 64, False), ([127, 0, 300], 1, 5, 64, 16, False),
    ([513, 77, 256], 1, 128, 64, 512, False), ([700, 31], 1, 40, 0, 48, False),
    ([2, 3, 200, 1], 4, 16, 64, 64, False), ([500, 64, 333], 5, 96, 64, 48, False),
    ([1000, 129], 70, 3, 64, 64, False), ([640, 200, 90], 16, 96, 64, 64, True),
    ([300, 24, 150], 24, 40, 0, 128, True), ([64, 65, 200], 64, 8, 64, 16, True),
    ([257], 2, 129, 64, 64, False), ([1025], 1, 300, 64, 64, False),
    ([300], 70, 128, 64, 64, False), ([255, 256, 257, 0, 512, 1], 2, 96, 0, 16, False),
    ([40000, 3, 9000], 1, 130, 64, 512, False), ([30000, 0, 700], 1, 96, 64, 64, False)])
def test_against_64_bits(lens, T, H, dr, page, tree):
    d = _data(lens, T, H, dr, page, tree=tree)
    lse = _lse(d)
    _check(_run(d, lse), d, lse)


@pytest.mark.parametrize("T,H", [(1, 8), (2, 80)])
def test_many_short_sequences(T, H):
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 300, (500,), generator=g).tolist()
    d = _data(lens, T, H, 64, 16)
    lse = _lse(d)
    _check(_run(d, lse), d, lse)


@pytest.mark.parametrize("decay", [0.0, 0.5])
@pytest.mark.parametrize("lens,T,H,dr,tree", [
    ([100], 64, 128, 64, False), ([30, 0, 700], 70, 200, 0, False), ([5000] * 4, 16, 96, 64, True),
    ([9000, 1, 256], 5, 128, 64, False), ([200] * 50, 3, 100, 0, False), ([64], 64, 5, 64, True)])
def test_few_tiles_in_parts(lens, T, H, dr, tree, decay):
    """Keys whose query rows are shared out over pairs, in one round and in several."""
    d = _data(lens, T, H, dr, 64, tree=tree, spare=1)
    lse = _lse(d)
    ws = torch.empty(kda.kda_latent_weights_workspace_size(len(lens), T, H, dr=dr), dtype=torch.uint8,
                     device=DEV)
    want = _run(d, lse, decay, workspace=ws)
    _check(want, d, lse, decay)
    ws.fill_(255)                             # no call relies on what the last one left
    for _ in range(3):
        assert torch.equal(_run(d, lse, decay, workspace=ws), want)


def test_sequences_that_share_pages():
    """A prefix held once: the same rows, weights of each sequence's own."""
    d = _data([500, 500, 64], 1, 96, 64, 64)
    d["table"][1, :6] = d["table"][0, :6]
    lse = _lse(d)
    _check(_run(d, lse), d, lse)


@pytest.mark.parametrize("T,H", [(1, 96), (2, 96)])
def test_a_pool_past_two_to_the_31_elements(T, H):
    """The same rows and pages' order from a small pool and from a large one's ends."""
    d = _data([700, 300], T, H, 64, 64, wild=False)
    lse = _lse(d)
    want = _run(d, lse)
    n = d["cache"].shape[0]
    far = torch.arange(n, device=DEV) * 7 + 60000 - 7 * n
    pool = torch.empty(60000, 64, 576, dtype=BF, device=DEV)
    pool[far] = d["cache"]
    d["cache"], d["table"] = pool, far.to(torch.int32)[d["table"].clamp(0, n - 1).long()].contiguous()
    assert torch.equal(_run(d, lse), want)


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0, 3.0])
def test_decay(decay):
    d = _data([100, 300, 0], 2, 16, 64, 64, spare=1)
    if decay == 0.0:
        d["old"][0, 50] = float("nan")            # not read
    lse = _lse(d)
    got = _run(d, lse, decay)
    if decay == 0.0:
        d["old"][0, 50] = 0.0
    _check(got, d, lse, decay)


@pytest.mark.parametrize("T,H", [(1, 96), (4, 96), (8, 16)])
def test_a_row_of_probabilities_sums_to_one(T, H):
    d = _data([2, 1000, 4000, 0, 17], T, H, 64, 64)
    lse = _lse(d)
    d["old"].zero_()
    got = _run(d, lse)
    rows = torch.isfinite(lse).sum((1, 2)).double()
    # 2^-8 no longer enters: probabilities are not rounded to bf16 here
    assert ((got.double().sum(1) - rows).abs() <= 2 * REL * rows).all()


@pytest.mark.parametrize("H", [96, 200])
@pytest.mark.parametrize("dr", [0, 64])
def test_cut_off_sums_are_made_up_for(H, dr):
    """Scores of deviation 6, against 64 bits, by the mean over heads: a score that comes out
    too near to zero by a part c of itself takes c times the mean score from lse, and from the
    weights by an exact lse.  The tensor cores' c is about W / 16 steps x 2^-26, in decode, which
    adds two halves of the channels, half as much.  A call makes up for it but for a quarter
    (measured over operands 7 to 10 units of 2^-24 where the steps give 8 and 9).  A head's lse,
    of about 22, is rounded in steps of 2^-18 (as a logarithm to the base 2) and 2^-19, each
    off by a third of a step in the mean square, and with its sum's roundings by no more than
    1.5e-6; the mean of H of them by six times that over sqrt H at most.  A factor left out, or
    one taken for the other, is off by the whole or the half."""
    n, W = 3000, 512 + dr
    d = _data([n], 1, H, dr, 64, seed=11)
    d["scale"] = 6.0 / W ** 0.5
    scale = float(torch.tensor(d["scale"], dtype=F32))            # as the call has it
    s = d["q"][0, 0].double() @ ru.rows_of(d["cache"], d["table"], 0, n).double().T * scale
    exact = torch.logsumexp(s, -1)
    cut = W / 16 * 2.0 ** -26 * (torch.exp(s - exact[:, None]) * s).sum(-1).mean().item()
    rounded = 6 * 1.5e-6 / H ** 0.5
    assert cut > 6 * rounded
    lse = torch.empty(1, 1, H, device=DEV)
    kda.kda_latent_decode(d["q"], d["cache"], d["table"], d["seq_lens"], scale=scale, lse=lse)
    off = (lse[0, 0].double() - exact).mean().item()
    assert abs(off) <= cut / 8 + rounded, f"lse {off:.3g} of {cut:.3g}"
    d["old"].zero_()
    for lse, more in ((exact.float()[None, None], 0.0), (lse, cut / 8 + rounded)):
        given = torch.exp(exact - lse[0, 0].double()).sum().item()  # by this lse, rounded as it is
        total = _run(d, lse, scale=scale)[0, :n].double().sum().item()
        assert abs(total - given) / H <= cut / 4 + rounded / 3, f"{(total - given) / H:.3g} of {cut:.3g}"
        assert abs(total / H - 1) <= cut / 4 + more + rounded


def test_tokens_left_out():
    """A draft of lse +inf gives nothing, whatever the others do; so does one of -inf."""
    d = _data([400, 90], 6, 16, 64, 64, tree=True)
    lse = _lse(d)
    lse[0, 2] = float("inf")
    lse[0, 5] = float("-inf")
    lse[1, 0, 3] = float("inf")
    _check(_run(d, lse), d, lse)
    lse.fill_(float("inf"))
    d["old"].mul_(2.0)
    assert torch.equal(_run(d, lse), d["old"])


def test_scale_and_far_apart_scores():
    d = _data([600], 1, 32, 64, 64)
    d["q"] = d["q"] * 4
    d["scale"] = 0.25
    lse = torch.empty(1, 1, 32, device=DEV)
    kda.kda_latent_decode(d["q"], d["cache"], d["table"], d["seq_lens"], scale=0.25, lse=lse)
    got = _run(d, lse, scale=0.25)
    want = ru.weights_ref(d["q"], d["cache"], d["table"], d["lens"], lse, d["old"], None, 0.25, 1.0)
    # scores of deviation 24: partial sums reach 14 times as far as above
    tol = 14 * REL * (want - d["old"].double()).abs() + 4 * ru.U * want.abs()
    assert ((got.double() - want).abs()[0, :600] <= tol[0, :600]).all()


def test_a_row_that_is_no_number_keeps_to_itself():
    d = _data([200, 100], 1, 96, 64, 64)
    lse = _lse(d)
    bad = d["cache"][d["table"][0, 1].item(), 3]      # position 67
    bad[5] = float("nan")
    got = _run(d, lse)
    nan = torch.isnan(got).nonzero().tolist()
    assert nan == [[0, 67]]


def test_bad_lengths_and_pages_are_refused():
    d = _data([200, 100, 300], 1, 16, 64, 64, wild=False)
    lse = _lse(d)
    want = _run(d, lse)
    ws = torch.empty(kda.kda_latent_weights_workspace_size(3, 1, 16, dr=64), dtype=torch.uint8,
                     device=DEV)
    for n in (-1, 321, -2 ** 31, 2 ** 31 - 1):
        lens = torch.tensor([200, n, 300], dtype=torch.int32, device=DEV)
        w = d["old"].clone()
        kda.kda_latent_weights(d["q"], d["cache"], d["table"], lens, lse, w, workspace=ws)
        assert kda.kda_read_device_status(ws) == 1
        assert torch.equal(w[[0, 2]], want[[0, 2]]) and torch.equal(w[1], d["old"][1])
    for page in (-1, d["cache"].shape[0], 2 ** 31 - 1):
        table = d["table"].clone()
        table[2, 1] = page
        w = d["old"].clone()
        kda.kda_latent_weights(d["q"], d["cache"], table, d["seq_lens"], lse, w, workspace=ws)
        assert kda.kda_read_device_status(ws) == 1
        assert torch.equal(w[:2], want[:2])
    _run(d, lse, workspace=ws)
    assert kda.kda_read_device_status(ws) == 0


def test_the_same_bits_again_streams_and_graphs():
    d = _data([3000, 1, 0, 700, 2000], 3, 96, 64, 64)
    lse = _lse(d)
    want = _run(d, lse)
    assert torch.equal(_run(d, lse), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w = d["old"].clone()
    torch.cuda.synchronize()
    kda.kda_latent_weights(d["q"], d["cache"], d["table"], d["seq_lens"], lse, w, stream=s)
    s.synchronize()
    assert torch.equal(w, want)
    w = d["old"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_latent_weights(d["q"], d["cache"], d["table"], d["seq_lens"], lse, w)
    w.copy_(d["old"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w, want)
    # shorter sequences with the same graph
    d["lens"] = [100, 1, 0, 64, 1999]
    d["seq_lens"].copy_(torch.tensor(d["lens"], dtype=torch.int32))
    lse.copy_(_lse(d))
    w.copy_(d["old"])
    graph.replay()
    torch.cuda.synchronize()
    _check(w, d, lse)


def test_refusals():
    d = _data([100], 1, 8, 64, 64)
    lse = _lse(d)
    base = dict(q=d["q"], cache=d["cache"], block_table=d["table"], seq_lens=d["seq_lens"], lse=lse,
                weights=d["old"])
    for bad in (dict(q=d["q"].float()), dict(q=d["q"][..., :100]), dict(cache=d["cache"][..., :512]),
                dict(block_table=d["table"].long()), dict(seq_lens=d["seq_lens"].long()),
                dict(lse=lse.double()), dict(lse=lse[..., :4]), dict(weights=d["old"][:, :64]),
                dict(weights=d["old"].double()), dict(decay=-1.0), dict(decay=float("nan")),
                dict(scale=-1.0), dict(tree_mask=torch.zeros(1, 2, dtype=torch.int64, device=DEV)),
                dict(q=d["q"].cpu())):
        args = dict(base)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            kda.kda_latent_weights(**args)
    with pytest.raises(kda.KDAError):
        kda.kda_latent_weights(**base, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
