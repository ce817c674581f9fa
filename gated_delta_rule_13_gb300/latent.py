"""Binding of the latent-attention and paged-cache entry points of libkda.

Like ``kda``: every function has the name of the C entry point it wraps
(include/kda.h), checks shapes, dtypes and devices, allocates what the caller
did not pass, and forwards pointers with the current CUDA stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from .kda import (HEAD_DIM, KDA_BF16, _check, _need_cuda, _ptr, _stream_handle, library)

LATENT_DIM = 512    # latent channels of a cached row
ROPE_DIM = 64       # rotary channels of a row, or none


def _view3(name, t, shape):
    """A bf16 ``[N, H, 128]`` view with contiguous rows; its token and head strides."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    # torch leaves the strides of a dimension of size 1 (or 0) open
    ts = t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]
    hs = t.stride(1) if t.shape[1] > 1 else t.shape[2]
    return ts, hs


def _on(stream):
    """What a call allocates belongs to the stream it runs on, so that the caching
    allocator hands the memory on in that stream's order."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _cu(name, cu):
    if not isinstance(cu, torch.Tensor) or cu.dtype != torch.int32 or cu.dim() != 1 \
            or cu.shape[0] < 2 or not cu.is_contiguous():
        raise TypeError(f"{name} must be a contiguous 1-D int32 tensor of n_seqs + 1 entries")
    return cu


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.is_cuda and t.device != device:
            raise ValueError(f"{name} is on {t.device}, q on {device}")


def _scale(scale, dim):
    scale = 1.0 / math.sqrt(dim) if scale is None else float(scale)
    if not (scale > 0.0 and math.isfinite(scale)):
        raise ValueError(f"scale must be finite and positive, got {scale}")
    return scale


def _expanded(q, k, v, k_rope, cu_seqlens_q, cu_seqlens_k, scale):
    """The checked arguments both directions share."""
    _need_cuda("q", q, torch.bfloat16)
    if q.dim() != 3 or q.shape[2] not in (HEAD_DIM, HEAD_DIM + ROPE_DIM):
        raise ValueError(f"q must be [n_q, H, 128] or [n_q, H, 192], got {tuple(q.shape)}")
    n_q, H, width = q.shape
    dr = width - HEAD_DIM
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be [n_k, H, 128]")
    n_k = k.shape[0]
    ks = _view3("k", k, (n_k, H, HEAD_DIM))
    vs = _view3("v", v, (n_k, H, HEAD_DIM))
    if (k_rope is not None) != (dr > 0):
        raise ValueError("k_rope is given if and only if q has its 64 rotary channels")
    if k_rope is not None:
        _need_cuda("k_rope", k_rope, torch.bfloat16, (n_k, dr))
    cu_q, cu_k = cu_seqlens_q, cu_seqlens_k
    if cu_k is None and (cu_q is None or n_q == n_k):
        cu_k = cu_q
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_seqlens_q and cu_seqlens_k are both needed when there are not as "
                         "many keys as queries")
    n_seqs = 1
    if cu_q is not None:
        n_seqs = _cu("cu_seqlens_q", cu_q).shape[0] - 1
        if _cu("cu_seqlens_k", cu_k).shape != cu_q.shape:
            raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    _same_device(q.device, k=k, v=v, k_rope=k_rope, cu_seqlens_q=cu_q, cu_seqlens_k=cu_k)
    head = (_ptr(q), _ptr(k), _ptr(v), _ptr(k_rope), *ks, *vs, _ptr(cu_q), _ptr(cu_k), n_seqs,
            n_q, n_k, H, HEAD_DIM, dr, HEAD_DIM, KDA_BF16)
    return head, _scale(scale, width), (n_seqs, n_q, n_k, H, dr)


def _workspace(workspace, size, device, stream):
    if workspace is None:
        with _on(stream):
            return torch.empty(size, dtype=torch.uint8, device=device)
    _need_cuda("workspace", workspace)
    _same_device(device, workspace=workspace)
    return workspace


def _size(fn, *args):
    out = ctypes.c_size_t(0)
    _check(getattr(library(), fn)(*args, ctypes.byref(out)), fn)
    return out.value


def kda_latent_fwd_workspace_size(n_seqs, n_q, n_k, H, dk=HEAD_DIM, dr=0, dv=HEAD_DIM,
                                  dtype=KDA_BF16) -> int:
    return _size("kda_latent_fwd_workspace_size", n_seqs, n_q, n_k, H, dk, dr, dv, dtype)


def kda_latent_bwd_workspace_size(n_seqs, n_q, n_k, H, dk=HEAD_DIM, dr=0, dv=HEAD_DIM,
                                  dtype=KDA_BF16) -> int:
    return _size("kda_latent_bwd_workspace_size", n_seqs, n_q, n_k, H, dk, dr, dv, dtype)


def kda_latent_decode_workspace_size(B, T, H, dc=LATENT_DIM, dr=0, dtype=KDA_BF16) -> int:
    return _size("kda_latent_decode_workspace_size", B, T, H, dc, dr, dtype)


def kda_latent_fwd(q, k, v, k_rope=None, cu_seqlens_q=None, cu_seqlens_k=None, *, causal=True,
                   scale=None, out=None, lse=None, workspace=None, stream=None):
    """Latent attention in its expanded form, over packed sequences.

    q ``[n_q, H, 128 (+ 64)]``, k and v ``[n_k, H, 128]`` (bf16; k and v may be
    strided views of one projection), k_rope ``[n_k, 64]`` shared by the heads
    (given if and only if q has the 64 rotary channels).  ``cu_seqlens_q`` /
    ``cu_seqlens_k``: int32 prefix sums (CUDA or CPU), None for one sequence; with as
    many keys as queries a missing ``cu_seqlens_k`` is ``cu_seqlens_q``.  With ``causal`` the queries are
    the last tokens of their sequence's keys.  ``scale`` defaults to
    1 / sqrt(128 + dr).  Returns ``(out [n_q, H, 128], lse [n_q, H])``."""
    head, sc, (n_seqs, n_q, n_k, H, dr) = _expanded(q, k, v, k_rope, cu_seqlens_q, cu_seqlens_k,
                                                    scale)
    with _on(stream):
        if out is None:
            out = torch.empty(n_q, H, HEAD_DIM, dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty(n_q, H, dtype=torch.float32, device=q.device)
    _need_cuda("out", out, q.dtype, (n_q, H, HEAD_DIM))
    _need_cuda("lse", lse, torch.float32, (n_q, H))
    ws = _workspace(workspace, kda_latent_fwd_workspace_size(n_seqs, n_q, n_k, H, dr=dr),
                    q.device, stream)
    _same_device(q.device, out=out, lse=lse)
    _check(library().kda_latent_fwd(*head, sc, int(bool(causal)), _ptr(out), _ptr(lse), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream_handle(stream)),
           "kda_latent_fwd")
    return out, lse


def kda_latent_bwd(q, k, v, k_rope, out, lse, d_out, cu_seqlens_q=None, cu_seqlens_k=None, *,
                   causal=True, scale=None, d_k=None, d_v=None, workspace=None, stream=None):
    """Gradients of ``kda_latent_fwd`` for the output gradient ``d_out``; ``out``
    and ``lse`` are what it returned.  Returns ``(dq, d_k, d_v, d_k_rope)`` in the
    layouts of the inputs (d_k_rope None without a rotary part).  ``d_k`` and
    ``d_v`` may be given as strided views, as k and v may."""
    head, sc, (n_seqs, n_q, n_k, H, dr) = _expanded(q, k, v, k_rope, cu_seqlens_q, cu_seqlens_k,
                                                    scale)
    _need_cuda("out", out, q.dtype, (n_q, H, HEAD_DIM))
    _need_cuda("lse", lse, torch.float32, (n_q, H))
    _need_cuda("d_out", d_out, q.dtype, (n_q, H, HEAD_DIM))
    with _on(stream):
        dq = torch.empty_like(q)
        if d_k is None:
            d_k = torch.empty(n_k, H, HEAD_DIM, dtype=q.dtype, device=q.device)
        if d_v is None:
            d_v = torch.empty(n_k, H, HEAD_DIM, dtype=q.dtype, device=q.device)
        d_rope = torch.empty(n_k, dr, dtype=q.dtype, device=q.device) if dr else None
    dks = _view3("d_k", d_k, (n_k, H, HEAD_DIM))
    dvs = _view3("d_v", d_v, (n_k, H, HEAD_DIM))
    ws = _workspace(workspace, kda_latent_bwd_workspace_size(n_seqs, n_q, n_k, H, dr=dr),
                    q.device, stream)
    _same_device(q.device, out=out, lse=lse, d_out=d_out, d_k=d_k, d_v=d_v)
    _check(library().kda_latent_bwd(*head, sc, int(bool(causal)), _ptr(out), _ptr(lse),
                                    _ptr(d_out), _ptr(dq), _ptr(d_k), _ptr(d_v), _ptr(d_rope),
                                    *dks, *dvs, _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream_handle(stream)), "kda_latent_bwd")
    return dq, d_k, d_v, d_rope


def kda_latent_decode(q, cache, block_table, seq_lens, *, tree_mask=None, scale=None, out=None,
                      lse=None, workspace=None, stream=None):
    """Latent attention in its absorbed form: the last T tokens of each sequence
    over its rows of a paged cache.

    q ``[B, T, H, 512 (+ 64)]`` and cache ``[n_pages, page_size, 512 (+ 64)]``
    (bf16, page_size a multiple of 16), block_table ``[B, max_pages]`` and
    seq_lens ``[B]`` int32 on the device (lengths with the T new rows included).
    tree_mask ``[B, T]`` int64: bit j of a token's mask lets it see the j-th of the
    T new rows; None: the new rows are consecutive tokens.  ``scale`` defaults to
    1 / sqrt(128 + dr), the expanded form's.  ``lse`` (``[B, T, H]`` fp32) is
    written when given.  Returns out ``[B, T, H, 512]``."""
    _need_cuda("q", q, torch.bfloat16)
    if q.dim() != 4 or q.shape[3] not in (LATENT_DIM, LATENT_DIM + ROPE_DIM):
        raise ValueError(f"q must be [B, T, H, 512] or [B, T, H, 576], got {tuple(q.shape)}")
    B, T, H, width = q.shape
    dr = width - LATENT_DIM
    _need_cuda("cache", cache, torch.bfloat16)
    if cache.dim() != 3 or cache.shape[2] != width:
        raise ValueError(f"cache must be [n_pages, page_size, {width}], got {tuple(cache.shape)}")
    _need_cuda("block_table", block_table, torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    _need_cuda("seq_lens", seq_lens, torch.int32, (B,))
    if tree_mask is not None:
        _need_cuda("tree_mask", tree_mask, torch.int64, (B, T))
    if out is None:
        with _on(stream):
            out = torch.empty(B, T, H, LATENT_DIM, dtype=q.dtype, device=q.device)
    _need_cuda("out", out, q.dtype, (B, T, H, LATENT_DIM))
    if lse is not None:
        _need_cuda("lse", lse, torch.float32, (B, T, H))
    sc = _scale(scale, HEAD_DIM + dr)
    ws = _workspace(workspace, kda_latent_decode_workspace_size(B, T, H, dr=dr),
                    q.device, stream)
    _same_device(q.device, cache=cache, block_table=block_table, seq_lens=seq_lens,
                 tree_mask=tree_mask, out=out, lse=lse)
    _check(library().kda_latent_decode(
        _ptr(q), _ptr(cache), _ptr(block_table), _ptr(seq_lens), _ptr(tree_mask), B, T, H,
        LATENT_DIM, dr, cache.shape[0], cache.shape[1], block_table.shape[1], KDA_BF16, sc,
        _ptr(out), _ptr(lse), _ptr(ws), ws.numel() * ws.element_size(), _stream_handle(stream)),
        "kda_latent_decode")
    return out


def _status_arg(status, device):
    if status is not None:
        _need_cuda("status", status, torch.int32, (1,))
        _same_device(device, status=status)
    return _ptr(status)


def kda_cache_write(cache, rows, block_table, start, *, path=None, n_write=None, status=None,
                    stream=None):
    """Rows written into a paged cache ``[n_pages, page_size, W]`` or, all layers in
    one call, ``[L, n_pages, page_size, W]`` (any dtype), in place.

    rows ``[B, T, W]`` (``[L, B, T, W]``): row ``path[b, i]`` (row i without path)
    goes to position ``start[b] + i`` for i < ``n_write[b]`` (all T without it).
    rows None: the cached rows ``start[b] + path[b, i]`` are moved to
    ``start[b] + i`` (the accepted path of a draft tree, strictly increasing).
    block_table ``[B, max_pages]``, start ``[B]``, path ``[B, T]``, n_write ``[B]``:
    int32 on the device.  ``status`` (int32 ``[1]`` on the device) receives an
    error code if a sequence's positions or path are refused.  Returns cache."""
    _need_cuda("cache", cache)
    if cache.dim() not in (3, 4):
        raise ValueError("cache must be [n_pages, page_size, W] or [L, n_pages, page_size, W]")
    layers = cache.shape[0] if cache.dim() == 4 else 1
    n_pages, page, W = cache.shape[-3:]
    esz = cache.element_size()
    _need_cuda("block_table", block_table, torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    _need_cuda("start", start, torch.int32, (B,))
    if path is not None:
        _need_cuda("path", path, torch.int32)
        if path.dim() != 2 or path.shape[0] != B:
            raise ValueError("path must be [B, T]")
    if n_write is not None:
        _need_cuda("n_write", n_write, torch.int32, (B,))
    if rows is None:
        if path is None:
            raise ValueError("compaction (rows None) needs path")
        T, strides = path.shape[1], (0, 0, 0)
    else:
        if not isinstance(rows, torch.Tensor) or not rows.is_cuda or rows.dtype != cache.dtype:
            raise TypeError(f"rows must be a CUDA tensor of {cache.dtype}")
        if rows.dim() != cache.dim():
            raise ValueError("rows must be [B, T, W], or [L, B, T, W] for a cache with layers")
        T = rows.shape[-2]
        want = ((layers,) if cache.dim() == 4 else ()) + (B, T, W)
        if tuple(rows.shape) != want or (path is not None and path.shape[1] != T):
            raise ValueError(f"rows must have shape {want} and path [B, T]")
        if W > 1 and rows.stride(-1) != 1:
            raise ValueError("rows must have contiguous channels")
        # torch leaves the strides of a dimension of size 1 open
        strides = tuple(0 if n == 1 else st * esz for n, st in
                        zip(((1,) if rows.dim() == 3 else ()) + tuple(rows.shape[:-1]),
                            ((0,) if rows.dim() == 3 else ()) + tuple(rows.stride()[:-1])))
    for name, t in dict(rows=rows, block_table=block_table, start=start, path=path,
                        n_write=n_write).items():
        if t is not None and t.device != cache.device:
            raise ValueError(f"{name} is on {t.device}, cache on {cache.device}")
    if layers == 0 or B == 0 or T == 0:
        return cache
    _check(library().kda_cache_write(
        _ptr(cache), _ptr(rows), *strides, _ptr(block_table), _ptr(start), _ptr(path),
        _ptr(n_write), layers, n_pages, page, W * esz, B, T, max_pages,
        _status_arg(status, cache.device), _stream_handle(stream)), "kda_cache_write")
    return cache


def kda_cache_copy_pages(cache, src, dst, *, status=None, stream=None):
    """Page ``dst[i]`` of every layer of the pool ``[L, n_pages, ...]`` becomes a
    copy of page ``src[i]``, in place (any dtype; a page is all that lies behind the
    first two dimensions).  src, dst: int32 ``[n]`` on the device; the dst pages are
    distinct and none is a src.  Returns cache."""
    _need_cuda("cache", cache)
    if cache.dim() < 3:
        raise ValueError("cache must be [L, n_pages, ...]")
    _need_cuda("src", src, torch.int32)
    if src.dim() != 1:
        raise ValueError("src must be one-dimensional")
    _need_cuda("dst", dst, torch.int32, src.shape)
    for name, t in dict(src=src, dst=dst).items():
        if t.device != cache.device:
            raise ValueError(f"{name} is on {t.device}, cache on {cache.device}")
    L, n_pages = cache.shape[:2]
    if L == 0 or src.shape[0] == 0:
        return cache
    page_bytes = math.prod(cache.shape[2:]) * cache.element_size()
    _check(library().kda_cache_copy_pages(
        _ptr(cache), _ptr(src), _ptr(dst), src.shape[0], L, n_pages, page_bytes,
        _status_arg(status, cache.device), _stream_handle(stream)), "kda_cache_copy_pages")
    return cache
