"""Moves of the paged cache: bytes in, the same bytes out."""
from __future__ import annotations

import pytest
import torch

import gated_delta_rule_13_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _pool(L, n_pages, page, W, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(L, n_pages, page, W, generator=g, device=DEV)
    return (100 * x).to(dtype)


def _tables(start, T, page, seed=0):
    need = [(s + T + page - 1) // page for s in start]
    order = torch.randperm(sum(need) + 3, generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(start), max(need) + 1), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, sum(need) + 3


def _expect(cache, rows, table, start, path, n):
    new = cache.clone()
    page = cache.shape[2]
    at = lambda b, p: (int(table[b, p // page]), p % page)  # noqa: E731
    for b in range(len(start)):
        for i in range(n[b]):
            j = int(path[b][i]) if path is not None else i
            p, r = at(b, start[b] + i)
            if rows is None:
                p2, r2 = at(b, start[b] + j)
                new[:, p, r] = cache[:, p2, r2]
            else:
                new[:, p, r] = rows[:, b, j]
    return new


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.uint8])
@pytest.mark.parametrize("page,W", [(16, 576), (5, 16), (64, 2048), (1, 512)])
@pytest.mark.parametrize("T", [1, 7])
def test_append(dtype, page, W, T):
    start = [0, 1, page - 1, 3 * page + 2, 77]
    table, n_pages = _tables(start, T, page)
    cache = _pool(2, n_pages, page, W, dtype)
    rows = _pool(2, 5, T, W, dtype, seed=1)
    want = _expect(cache, rows, table, start, None, [T] * 5)
    got = pkg.kda_cache_write(cache, rows, table.to(DEV), _i32(start))
    assert got.data_ptr() == cache.data_ptr() and torch.equal(cache, want)


def test_append_a_layer_of_strided_rows_through_a_path():
    start, T, page = [3, 60, 17], 6, 16
    table, n_pages = _tables(start, T, page)
    cache = _pool(1, n_pages, page, 576, torch.bfloat16)
    wide = _pool(1, 3, T, 1024, torch.bfloat16, seed=1)
    rows = wide[..., 64:640]
    path, n = torch.tensor([[5, 0, 2, 2, 9, -4], [1, 3, 5, 0, 0, 0], [0] * 6]), [4, 9, 0]
    want = _expect(cache, rows, table, start, [[5, 0, 2, 2], [1, 3, 5, 0, 0, 0], []], [4, 6, 0])
    pkg.kda_cache_write(cache[0], rows[0], table.to(DEV), _i32(start), path=_i32(path),
                        n_write=_i32(n))
    assert torch.equal(cache, want)


@pytest.mark.parametrize("T", [1, 4, 16, 40])
@pytest.mark.parametrize("page", [5, 16, 64])
def test_compaction(T, page):
    g = torch.Generator().manual_seed(T)
    B, L = 9, 3
    start = [0, 1, 15, 16, 40, 63, 64, 100, 7]
    table, n_pages = _tables(start, T, page)
    n = [int(torch.randint(0, T + 1, (1,), generator=g)) for _ in range(B)]
    n[0], n[1] = T, 0
    path = torch.zeros(B, T, dtype=torch.int64)
    for b in range(B):
        path[b, :n[b]] = torch.randperm(T, generator=g)[:n[b]].sort().values
    cache = _pool(L, n_pages, page, 576, torch.bfloat16)
    want = _expect(cache, None, table, start, path, n)
    pkg.kda_cache_write(cache, None, table.to(DEV), _i32(start), path=_i32(path), n_write=_i32(n))
    assert torch.equal(cache, want)


def test_refused_sequences_move_nothing():
    start, T, page = [3, 20, 40, 9, 5], 4, 16
    table, n_pages = _tables(start, T, page)
    cache = _pool(2, n_pages, page, 64, torch.float32)
    path = torch.tensor([[1, 2, 3, 3], [1, 1, 2, 3], [0, 2, 4, 0], [-1, 2, 3, 0], [2, 3, 0, 0]])
    n = [3, 2, 3, 2, 2]
    good = {0, 4}
    want = _expect(cache, None, table, start, path.clamp(0, 3),
                   [k if b in good else 0 for b, k in enumerate(n)])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = dict(path=_i32(path), n_write=_i32(n))
    pkg.kda_cache_write(cache, None, table.to(DEV), _i32(start), status=status, **args)
    assert torch.equal(cache, want) and int(status) == 1
    # positions outside the table, pages outside the pool
    keep = cache.clone()
    for bad_start, bad_page in (([-1] * 5, None), ([10 ** 6] * 5, None), ([0] * 5, -1),
                                ([0] * 5, n_pages), ([2 ** 31 - 1] * 5, None)):
        t = table.to(DEV) if bad_page is None else torch.full_like(table, bad_page).to(DEV)
        status.zero_()
        pkg.kda_cache_write(cache, None, t, _i32(bad_start), path=_i32([[0, 1, 2, 3]] * 5),
                            status=status)
        assert torch.equal(cache, keep) and int(status) == 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 9, 8), (3, 20, 16, 576), (2, 12, 3, 128, 128), (5, 7, 8200)])
def test_copy_pages(shape, dtype):
    x = _pool(1, 1, 1, 1, dtype).new_empty(shape)
    x.copy_(torch.randn(shape, device=DEV))
    ids = torch.randperm(shape[1], generator=torch.Generator().manual_seed(2))
    n = shape[1] // 2
    src, dst = ids[:n].clone(), ids[n:2 * n].clone()
    src[1] = src[0]                      # one page forked twice
    want = x.clone()
    want[:, dst] = x[:, src]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkg.kda_cache_copy_pages(x, _i32(src), _i32(dst), status=status)
    assert torch.equal(x, want) and int(status) == 0
    # out of range on either side, and a page onto itself: nothing moves
    pkg.kda_cache_copy_pages(x, _i32([-1, 0, 2]), _i32([1, shape[1], 2]), status=status)
    assert torch.equal(x, want) and int(status) == 1


def test_nothing_to_do():
    x = _pool(1, 4, 16, 64, torch.float32)
    want = x.clone()
    pkg.kda_cache_copy_pages(x, _i32([]), _i32([]))
    pkg.kda_cache_write(x, x.new_zeros(1, 0, 2, 64), torch.zeros(0, 2, dtype=torch.int32,
                                                                 device=DEV), _i32([]))
    assert torch.equal(x, want)
