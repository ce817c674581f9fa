"""Eviction of cached rows against its plain form: whole numbers and bytes, equal."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_13_gb300 as kda
import rows_util as ru

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _data(lens, page, L=1, W=64, dtype=torch.bfloat16, seed=0, values=None, spare=0):
    g = torch.Generator().manual_seed(seed)
    width = max(1, max((n + page - 1) // page for n in lens)) + spare
    table, n_pages = ru.pages(lens, page, g, width=width)
    if dtype.is_floating_point:
        cache = torch.randn(L, n_pages, page, W, generator=g).to(dtype)
    else:
        cache = torch.randint(-100, 100, (L, n_pages, page, W), generator=g).to(dtype)
    w = torch.randn(L, len(lens), width * page, generator=g).exp()
    if values is not None:                    # few values, so that many are equal
        pick = torch.randint(0, len(values), w.shape, generator=g)
        w = torch.tensor(values)[pick]
    for b, n in enumerate(lens):
        w[:, b, n:] = 99.0                    # not looked at
    return dict(cache=cache.to(DEV), table=table.to(DEV), weights=w.to(DEV), lens=lens,
                seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), page=page)


def _check(d, budget, first, recent, in_place=False, layered=True):
    cache, w = d["cache"].clone(), d["weights"].clone()
    L, B, cap = w.shape
    out = w if in_place else torch.full_like(w, -7.0)
    args = (cache, w, out) if layered else (cache[0], w[0], out[0])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    new_lens, origin = kda.kda_cache_evict(args[0], d["table"], d["seq_lens"], args[1], budget,
                                           first=first, recent=recent, status=status,
                                           weights_out=None if in_place else args[2])
    torch.cuda.synchronize()
    assert status.item() == 0
    assert new_lens.tolist() == [min(n, budget) for n in d["lens"]]
    assert origin.shape == ((L, B, budget) if layered else (B, budget))
    origin = origin.view(L, B, budget).cpu()
    want_cache, old = d["cache"].cpu().clone(), d["cache"].cpu()
    table, weights = d["table"].cpu(), d["weights"].cpu()
    want_w = torch.zeros(L, B, cap)
    page = d["page"]
    for l in range(L):
        for b, n in enumerate(d["lens"]):
            want = ru.evict_ref(weights[l, b].tolist(), n, budget, first, recent)
            assert origin[l, b].tolist() == want + [-1] * (budget - len(want)), (l, b)
            if not want:
                continue
            src = torch.tensor(want)
            dst = torch.arange(len(want))
            want_w[l, b, :len(want)] = weights[l, b, src]
            moved = src != dst
            s, t = src[moved], dst[moved]
            want_cache[l, table[b].long()[t // page], t % page] = \
                old[l, table[b].long()[s // page], s % page]
    assert torch.equal(cache.cpu().view(torch.uint8), want_cache.view(torch.uint8))
    got = out.cpu()
    assert torch.equal(got.nan_to_num(-1.0), want_w.nan_to_num(-1.0))
    if not in_place:
        assert torch.equal(w.nan_to_num(-1.0), d["weights"].nan_to_num(-1.0))


@pytest.mark.parametrize("lens,page,budget,first,recent", [
    ([1], 16, 1, 0, 0), ([2], 16, 1, 0, 0), ([2], 16, 1, 1, 0), ([2], 16, 1, 0, 1),
    ([0, 1, 17, 16, 15], 16, 16, 0, 0), ([40, 100, 7], 16, 30, 4, 8), ([100, 200, 300], 64, 99, 0, 99),
    ([100, 200, 300], 64, 99, 99, 0), ([100, 200], 64, 60, 30, 30), ([2049, 2048, 2047], 64, 2048, 4, 64),
    ([1000, 5000, 33, 4096], 48, 700, 3, 100), ([1500], 512, 1499, 0, 700), ([777, 1200], 7, 333, 5, 300),
    ([5, 600], 64, 2000, 1, 1), ([40000], 64, 5000, 10, 1000), ([4080, 4000], 16, 4050, 1, 4040),
    ([4080, 4000], 16, 2020, 0, 2020), ([4080], 16, 2000, 5, 1990), ([300] * 40, 16, 100, 4, 30),
    ([17000, 16385, 100], 64, 16380, 0, 9), ([20000], 16, 3, 1, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_against_the_plain_form(lens, page, budget, first, recent, in_place):
    _check(_data(lens, page, spare=1), budget, first, recent, in_place, layered=False)


@pytest.mark.parametrize("values", [[1.0], [0.0, -0.0, 1e-40, -1.0], [3.0, float("nan"), 2.0],
                                    [float("inf"), float("-inf"), 0.5, float("nan")]])
@pytest.mark.parametrize("in_place", [False, True])
def test_equal_weights_and_no_numbers(values, in_place):
    d = _data([300, 1025, 64, 129], 16, L=2, values=values)
    for budget, first, recent in ((100, 0, 0), (64, 2, 30), (128, 0, 128), (1, 0, 0)):
        _check(d, budget, first, recent, in_place)


@pytest.mark.parametrize("L,W,dtype", [(3, 576, torch.bfloat16), (24, 8, torch.float32),
                                       (2, 48, torch.uint8), (5, 16, torch.int64), (1, 1000, torch.bfloat16)])
def test_layers_and_row_sizes(L, W, dtype):
    d = _data([333, 90, 512, 700], 64, L=L, W=W, dtype=dtype)
    _check(d, 128, 4, 20)
    _check(d, 400, 0, 150, in_place=True)


def test_one_sequence_shares_its_moves_out():
    """Few columns and many moves: they are shared out over blocks, the last rows follow."""
    _check(_data([9000], 64, W=576), 4000, 4, 500, layered=False)
    _check(_data([9000], 64, W=8), 4000, 4, 3999 - 4, layered=False)
    _check(_data([3000, 10], 64, W=64), 1100, 0, 1100, layered=False)


@pytest.mark.parametrize("lens,budget", [([49000, 30, 20000], 9000), ([60000, 12000], 300), ([49153], 49000)])
def test_long_sequences(lens, budget):
    """Candidates that shared memory holds, and more than it does."""
    d = _data(lens, 64, W=8)
    _check(d, budget, 3, 100, layered=False)
    _check(_data(lens, 64, W=8, values=[1.0, 0.5, float("nan")]), budget, 0, 0, True, layered=False)


def test_many_sequences():
    _check(_data([20 + i % 50 for i in range(300)], 16, L=2, W=8), 32, 1, 5, in_place=True)


def test_bad_lengths_and_pages_are_left_alone():
    d = _data([100, 200, 150], 16, L=2, spare=1)
    for what, b in (("len", 1), ("len", 0), ("page", 2), ("page", 1)):
        lens, table = d["seq_lens"].clone(), d["table"].clone()
        for bad in ((-1, 225, 2 ** 31 - 1) if what == "len" else (-1, d["cache"].shape[1])):
            if what == "len":
                lens[b] = bad
            else:
                table[b, 3] = bad
            cache, out = d["cache"].clone(), torch.full_like(d["weights"], -7.0)
            status = torch.zeros(1, dtype=torch.int32, device=DEV)
            new_lens, origin = kda.kda_cache_evict(cache, table, lens, d["weights"], 50, first=1,
                                                   recent=9, weights_out=out, status=status)
            assert status.item() == 1
            assert new_lens[b] == lens[b] and (origin[:, b] == -1).all()
            n = out.shape[2] if what == "len" else d["lens"][b]
            assert torch.equal(out[:, b], d["weights"][:, b]) and n
            for p in d["table"][b, :(d["lens"][b] + 15) // 16].tolist():
                assert torch.equal(cache[:, p], d["cache"][:, p])
            other = (b + 1) % 3
            assert (origin[:, other] >= 0).all()


@pytest.mark.parametrize("in_place", [False, True])
def test_a_pool_past_two_to_the_32_bytes(in_place):
    """Two layers of 4.4 GB each, one sequence's pages at their ends."""
    n_pages, page, W, n, budget, first, recent = 60000, 64, 576, 700, 300, 4, 30
    cache = torch.empty(2, n_pages, page, W, dtype=torch.bfloat16, device=DEV)
    ids = torch.tensor([59999, 0, 58000, 30000, 59998, 59001, 58999, 1, 2, 59000, 45000],
                       dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(3)
    rows = torch.randn(2, len(ids), page, W, generator=g).to(torch.bfloat16).to(DEV)
    cache[:, ids.long()] = rows
    w = torch.rand(2, 1, len(ids) * page, generator=g).to(DEV)
    before, out = w.clone(), w if in_place else torch.empty_like(w)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    new, origin = kda.kda_cache_evict(cache, ids[None], lens, w, budget, first=first, recent=recent,
                                      weights_out=out)      # in place by name as well
    assert new.tolist() == [budget]
    for l in range(2):
        want = torch.tensor(ru.evict_ref(before[l, 0].tolist(), n, budget, first, recent))
        assert origin[l, 0].tolist() == want.tolist()
        got, old = cache[l, ids.long()].view(-1, W), rows[l].view(-1, W)
        assert torch.equal(got[:budget], old[want.to(DEV)])
        assert torch.equal(got[n:], old[n:])
        assert torch.equal(out[l, 0, :budget], before[l, 0, want.to(DEV)])


def test_again_on_what_is_left():
    """A budget kept up step by step: rows come and go, the weights follow them."""
    d = _data([64, 64], 16, W=8, spare=2)
    cache, w = d["cache"][0], d["weights"][0]
    w[:, 64:] = 0
    g = torch.Generator().manual_seed(9)
    # every row carries a number of its own, to be followed
    ids = torch.zeros(2, 96, dtype=torch.int64)
    seq, table = d["seq_lens"].clone(), d["table"].clone()
    spare = [p for p in range(cache.shape[0]) if p not in set(table[:, :4].flatten().tolist())]
    table[0, 4], table[1, 4] = spare[0], spare[1]
    nxt = 0
    for b in range(2):
        for i in range(64):
            ids[b, i] = nxt
            cache[table[b, i // 16], i % 16] = float(nxt)
            nxt += 1
    for step in range(40):
        for b in range(2):
            i = int(seq[b])
            ids[b, i] = 200 + step
            cache[table[b, i // 16], i % 16] = float(200 + step)
        seq += 1
        w += torch.rand(w.shape, generator=g).to(DEV) * (torch.arange(w.shape[1], device=DEV) < seq[:, None])
        before = w.cpu().clone()
        new, origin = kda.kda_cache_evict(cache, table, seq, w, 60, first=2, recent=10)
        for b in range(2):
            want = ru.evict_ref(before[b].tolist(), int(seq[b]), 60, 2, 10)
            assert origin[b].tolist() == want
            ids[b, :60] = ids[b, torch.tensor(want)]
            rows = ru.rows_of(cache, table, b, 60)
            assert torch.equal(rows.cpu().float(), ids[b, :60, None].bfloat16().float().expand(60, 8))
            assert ids[b, 59] == 200 + step
        seq = new


def test_streams_and_graphs():
    d = _data([500, 300], 64, L=2)
    cache, out = d["cache"].clone(), torch.empty_like(d["weights"])
    new, origin = kda.kda_cache_evict(cache, d["table"], d["seq_lens"], d["weights"], 128, first=2,
                                      recent=16, weights_out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cache2, out2 = d["cache"].clone(), torch.empty_like(out)
    torch.cuda.synchronize()
    got = kda.kda_cache_evict(cache2, d["table"], d["seq_lens"], d["weights"], 128, first=2,
                              recent=16, weights_out=out2, stream=s)
    s.synchronize()
    assert torch.equal(got[0], new) and torch.equal(got[1], origin)
    assert torch.equal(cache2, cache) and torch.equal(out2, out)
    graph = torch.cuda.CUDAGraph()
    cache2.copy_(d["cache"])
    with torch.cuda.graph(graph):
        got = kda.kda_cache_evict(cache2, d["table"], d["seq_lens"], d["weights"], 128, first=2,
                                  recent=16, weights_out=out2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[1], origin) and torch.equal(cache2, cache) and torch.equal(out2, out)


def test_refusals():
    d = _data([100], 16)
    base = dict(cache=d["cache"], block_table=d["table"], seq_lens=d["seq_lens"], weights=d["weights"],
                budget=50)
    for bad in (dict(budget=0), dict(first=-1), dict(recent=60), dict(first=30, recent=21),
                dict(weights=d["weights"][0]), dict(weights=d["weights"].double()),
                dict(weights=d["weights"][..., :16]), dict(weights_out=d["weights"][0]),
                dict(seq_lens=d["seq_lens"].long()), dict(block_table=d["table"][0]),
                dict(cache=d["cache"].transpose(1, 2)), dict(cache=d["cache"].cpu()),
                dict(status=torch.zeros(2, dtype=torch.int32, device=DEV))):
        args = dict(base)
        args.update(bad)
        with pytest.raises((TypeError, ValueError)):
            kda.kda_cache_evict(**args)
    big = torch.zeros(2, *d["weights"].shape, device=DEV).flatten()
    n = d["weights"].numel()
    with pytest.raises(kda.KDAError):                      # meets the weights
        kda.kda_cache_evict(**dict(base, weights=big[:n].view_as(d["weights"]),
                                   weights_out=big[16:16 + n].view_as(d["weights"])))
    with pytest.raises(kda.KDAError):                      # rows of 4 bytes
        kda.kda_cache_evict(d["cache"][..., :2].contiguous(), d["table"], d["seq_lens"], d["weights"], 50)
