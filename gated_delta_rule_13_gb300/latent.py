"""Binding of the latent-attention and paged-cache entry points of libkda.

Like ``kda``: every function has the name of the C entry point it wraps
(include/kda.h), checks shapes, dtypes and devices, allocates what the caller
did not pass, and forwards pointers with the current CUDA stream.

The smallest calls take a few microseconds on the device, so the checks are one
expression per tensor; the reason for a refusal is worked out only when there is
one.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from .kda import HEAD_DIM, KDA_BF16, _check, _need_cuda, library

LATENT_DIM = 512    # latent channels of a cached row
ROPE_DIM = 64       # rotary channels of a row, or none

_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def _refuse(name, t, dtype, shape, device):
    _need_cuda(name, t, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, not on {device}")


def _tensor(name, t, dtype, shape, device):
    """A contiguous tensor of this dtype and shape (None: any) on the device."""
    try:
        good = (t.dtype is dtype and t.device == device and t.is_contiguous()
                and (shape is None or t.shape == shape))
    except AttributeError:
        good = False
    if not good:
        _refuse(name, t, dtype, shape, device)


def _view(name, t, n, H, device):
    """Token and head strides of a bf16 ``[n, H, 128]`` view with contiguous rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.shape != (n, H, HEAD_DIM):
        raise ValueError(f"{name} must have shape {(n, H, HEAD_DIM)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    ts, hs, one = t.stride()
    if one != 1:
        raise ValueError(f"{name} must have contiguous rows")
    # torch leaves the strides of a dimension of size 1 (or 0) open
    return ts if n > 1 else H * HEAD_DIM, hs if H > 1 else HEAD_DIM


def _cu(name, cu, device):
    if not isinstance(cu, torch.Tensor) or cu.dtype is not _I32 or cu.dim() != 1 \
            or cu.shape[0] < 2 or not cu.is_contiguous():
        raise TypeError(f"{name} must be a contiguous 1-D int32 tensor of n_seqs + 1 entries")
    if cu.is_cuda and cu.device != device:
        raise ValueError(f"{name} is on {cu.device}, not on {device}")
    return cu.data_ptr()


def _new(stream, shape, dtype, device):
    """A tensor that belongs to the stream of the call, so that the caching allocator
    hands its memory on in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _stream(stream, device):
    """The raw stream of a call.  The kernels launch on the current device, and what is
    asked of a device (its SMs, whether a kernel fits) is asked of that one."""
    current = torch._C._cuda_getDevice()   # the tensors exist: CUDA is initialised
    if current != device.index:
        raise ValueError(f"the tensors are on {device}, but the current device is "
                         f"cuda:{current} (torch.cuda.set_device)")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    return stream.cuda_stream


def _scale(scale, dim):
    scale = 1.0 / math.sqrt(dim) if scale is None else float(scale)
    if not (scale > 0.0 and math.isfinite(scale)):
        raise ValueError(f"scale must be finite and positive, got {scale}")
    return scale


def _expanded(q, k, v, k_rope, cu_q, cu_k, scale):
    """The checked arguments both directions share: those of the C call, then sizes."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor")
    dev = q.device
    _tensor("q", q, _BF16, None, dev)
    if q.dim() != 3 or q.shape[2] not in (HEAD_DIM, HEAD_DIM + ROPE_DIM):
        raise ValueError(f"q must be [n_q, H, 128] or [n_q, H, 192], got {tuple(q.shape)}")
    n_q, H, width = q.shape
    dr = width - HEAD_DIM
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("k must be [n_k, H, 128]")
    n_k = k.shape[0]
    k_ts, k_hs = _view("k", k, n_k, H, dev)
    v_ts, v_hs = _view("v", v, n_k, H, dev)
    if (k_rope is not None) != (dr > 0):
        raise ValueError("k_rope is given if and only if q has its 64 rotary channels")
    rope = None
    if k_rope is not None:
        _tensor("k_rope", k_rope, _BF16, (n_k, dr), dev)
        rope = k_rope.data_ptr()
    if cu_k is None and (cu_q is None or n_q == n_k):
        cu_k = cu_q
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_seqlens_q and cu_seqlens_k are both needed when there are not as "
                         "many keys as queries")
    n_seqs, at_q, at_k = 1, None, None
    if cu_q is not None:
        at_q, at_k = _cu("cu_seqlens_q", cu_q, dev), _cu("cu_seqlens_k", cu_k, dev)
        n_seqs = cu_q.shape[0] - 1
        if cu_k.shape[0] != n_seqs + 1:
            raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    head = (q.data_ptr(), k.data_ptr(), v.data_ptr(), rope, k_ts, k_hs, v_ts, v_hs, at_q, at_k,
            n_seqs, n_q, n_k, H, HEAD_DIM, dr, HEAD_DIM, KDA_BF16, _scale(scale, width))
    return head, (n_seqs, n_q, n_k, H, dr), dev


def _workspace(workspace, size, device, stream):
    if workspace is None:
        return _new(stream, size, torch.uint8, device)
    _need_cuda("workspace", workspace)
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, not on {device}")
    return workspace


def _device():
    """Index of the current device; without one in use, a number of its own."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -1


@functools.lru_cache(maxsize=1024)
def _size(fn, device, *args):
    """A workspace size: it follows from the sizes and the SM count of the current
    device, whose index is ``device``."""
    out = ctypes.c_size_t(0)
    _check(getattr(library(), fn)(*args, ctypes.byref(out)), fn)
    return out.value


def kda_latent_fwd_workspace_size(n_seqs, n_q, n_k, H, dk=HEAD_DIM, dr=0, dv=HEAD_DIM,
                                  dtype=KDA_BF16) -> int:
    return _size("kda_latent_fwd_workspace_size", _device(), n_seqs, n_q, n_k, H, dk, dr, dv,
                 dtype)


def kda_latent_bwd_workspace_size(n_seqs, n_q, n_k, H, dk=HEAD_DIM, dr=0, dv=HEAD_DIM,
                                  dtype=KDA_BF16) -> int:
    return _size("kda_latent_bwd_workspace_size", _device(), n_seqs, n_q, n_k, H, dk, dr, dv,
                 dtype)


def kda_latent_decode_workspace_size(B, T, H, dc=LATENT_DIM, dr=0, dtype=KDA_BF16) -> int:
    return _size("kda_latent_decode_workspace_size", _device(), B, T, H, dc, dr, dtype)


def kda_latent_fwd(q, k, v, k_rope=None, cu_seqlens_q=None, cu_seqlens_k=None, *, causal=True,
                   scale=None, out=None, lse=None, workspace=None, stream=None):
    """Latent attention in its expanded form, over packed sequences.

    q ``[n_q, H, 128 (+ 64)]``, k and v ``[n_k, H, 128]`` (bf16; k and v may be
    strided views of one projection), k_rope ``[n_k, 64]`` shared by the heads
    (given if and only if q has the 64 rotary channels).  ``cu_seqlens_q`` /
    ``cu_seqlens_k``: int32 prefix sums (CUDA or CPU), None for one sequence; with as
    many keys as queries a missing ``cu_seqlens_k`` is ``cu_seqlens_q``.  With
    ``causal`` the queries are the last tokens of their sequence's keys.  ``scale``
    defaults to 1 / sqrt(128 + dr).  Returns ``(out [n_q, H, 128], lse [n_q, H])``."""
    head, sizes, dev = _expanded(q, k, v, k_rope, cu_seqlens_q, cu_seqlens_k, scale)
    n_seqs, n_q, n_k, H, dr = sizes
    raw = _stream(stream, dev)
    if out is None:
        out = _new(stream, (n_q, H, HEAD_DIM), _BF16, dev)
    else:
        _tensor("out", out, _BF16, (n_q, H, HEAD_DIM), dev)
    if lse is None:
        lse = _new(stream, (n_q, H), _F32, dev)
    else:
        _tensor("lse", lse, _F32, (n_q, H), dev)
    ws = _workspace(workspace, _size("kda_latent_fwd_workspace_size", dev.index, n_seqs, n_q, n_k,
                                     H, HEAD_DIM, dr, HEAD_DIM, KDA_BF16), dev, stream)
    _check(library().kda_latent_fwd(*head, 1 if causal else 0, out.data_ptr(), lse.data_ptr(),
                                    ws.data_ptr(), ws.nbytes, raw),
           "kda_latent_fwd")
    return out, lse


def kda_latent_bwd(q, k, v, k_rope, out, lse, d_out, cu_seqlens_q=None, cu_seqlens_k=None, *,
                   causal=True, scale=None, d_k=None, d_v=None, workspace=None, stream=None):
    """Gradients of ``kda_latent_fwd`` for the output gradient ``d_out``; ``out``
    and ``lse`` are what it returned.  Returns ``(dq, d_k, d_v, d_k_rope)`` in the
    layouts of the inputs (d_k_rope None without a rotary part).  ``d_k`` and
    ``d_v`` may be given as strided views, as k and v may."""
    head, sizes, dev = _expanded(q, k, v, k_rope, cu_seqlens_q, cu_seqlens_k, scale)
    n_seqs, n_q, n_k, H, dr = sizes
    raw = _stream(stream, dev)
    _tensor("out", out, _BF16, (n_q, H, HEAD_DIM), dev)
    _tensor("lse", lse, _F32, (n_q, H), dev)
    _tensor("d_out", d_out, _BF16, (n_q, H, HEAD_DIM), dev)
    dq = _new(stream, q.shape, _BF16, dev)
    k_strides = v_strides = (H * HEAD_DIM, HEAD_DIM)
    if d_k is None:
        d_k = _new(stream, (n_k, H, HEAD_DIM), _BF16, dev)
    else:
        k_strides = _view("d_k", d_k, n_k, H, dev)
    if d_v is None:
        d_v = _new(stream, (n_k, H, HEAD_DIM), _BF16, dev)
    else:
        v_strides = _view("d_v", d_v, n_k, H, dev)
    d_rope = _new(stream, (n_k, dr), _BF16, dev) if dr else None
    ws = _workspace(workspace, _size("kda_latent_bwd_workspace_size", dev.index, n_seqs, n_q, n_k,
                                     H, HEAD_DIM, dr, HEAD_DIM, KDA_BF16), dev, stream)
    _check(library().kda_latent_bwd(*head, 1 if causal else 0, out.data_ptr(), lse.data_ptr(),
                                    d_out.data_ptr(), dq.data_ptr(), d_k.data_ptr(),
                                    d_v.data_ptr(), d_rope.data_ptr() if dr else None,
                                    *k_strides, *v_strides, ws.data_ptr(), ws.nbytes, raw),
           "kda_latent_bwd")
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
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor")
    dev = q.device
    raw = _stream(stream, dev)
    _tensor("q", q, _BF16, None, dev)
    if q.dim() != 4 or q.shape[3] not in (LATENT_DIM, LATENT_DIM + ROPE_DIM):
        raise ValueError(f"q must be [B, T, H, 512] or [B, T, H, 576], got {tuple(q.shape)}")
    B, T, H, width = q.shape
    dr = width - LATENT_DIM
    _tensor("cache", cache, _BF16, None, dev)
    if cache.dim() != 3 or cache.shape[2] != width:
        raise ValueError(f"cache must be [n_pages, page_size, {width}], got {tuple(cache.shape)}")
    _tensor("block_table", block_table, _I32, None, dev)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    _tensor("seq_lens", seq_lens, _I32, (B,), dev)
    if tree_mask is not None:
        _tensor("tree_mask", tree_mask, _I64, (B, T), dev)
    if out is None:
        out = _new(stream, (B, T, H, LATENT_DIM), _BF16, dev)
    else:
        _tensor("out", out, _BF16, (B, T, H, LATENT_DIM), dev)
    if lse is not None:
        _tensor("lse", lse, _F32, (B, T, H), dev)
    ws = _workspace(workspace, _size("kda_latent_decode_workspace_size", dev.index, B, T, H,
                                     LATENT_DIM, dr, KDA_BF16), dev, stream)
    _check(library().kda_latent_decode(
        q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        None if tree_mask is None else tree_mask.data_ptr(), B, T, H, LATENT_DIM, dr,
        cache.shape[0], cache.shape[1], block_table.shape[1], KDA_BF16,
        _scale(scale, HEAD_DIM + dr), out.data_ptr(), None if lse is None else lse.data_ptr(),
        ws.data_ptr(), ws.nbytes, raw), "kda_latent_decode")
    return out


def kda_latent_test_timeout(workspace, block: int, tile: int = 0, wait_us: int = 1000):
    """Test control of the bounded waits (see include/kda.h): the next latent-attention
    call with ``workspace`` waits at most ``wait_us`` for anything, and block ``block``
    withholds tile ``tile``; ``block < 0`` disarms."""
    _need_cuda("workspace", workspace)
    _check(library().kda_latent_test_timeout(workspace.data_ptr(), int(block), int(tile),
                                             int(wait_us)), "kda_latent_test_timeout")


def _status(status, device):
    if status is None:
        return None
    _tensor("status", status, _I32, (1,), device)
    return status.data_ptr()


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
    if not isinstance(cache, torch.Tensor) or not cache.is_cuda:
        raise TypeError("cache must be a CUDA tensor")
    dev, dtype = cache.device, cache.dtype
    raw = _stream(stream, dev)
    _tensor("cache", cache, dtype, None, dev)
    layered = cache.dim() == 4
    if not layered and cache.dim() != 3:
        raise ValueError("cache must be [n_pages, page_size, W] or [L, n_pages, page_size, W]")
    L = cache.shape[0] if layered else 1
    n_pages, page, W = cache.shape[-3:]
    esz = cache.element_size()
    _tensor("block_table", block_table, _I32, None, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    _tensor("start", start, _I32, (B,), dev)
    at_path = at_n = None
    if path is not None:
        _tensor("path", path, _I32, None, dev)
        if path.dim() != 2 or path.shape[0] != B:
            raise ValueError("path must be [B, T]")
        at_path = path.data_ptr()
    if n_write is not None:
        _tensor("n_write", n_write, _I32, (B,), dev)
        at_n = n_write.data_ptr()
    at_status = _status(status, dev)
    if rows is None:
        if path is None:
            raise ValueError("compaction (rows None) needs path")
        T, ls, bs, ts, at_rows = path.shape[1], 0, 0, 0, None
    else:
        if not isinstance(rows, torch.Tensor) or not rows.is_cuda or rows.dtype is not dtype:
            raise TypeError(f"rows must be a CUDA tensor of {dtype}")
        if rows.device != dev:
            raise ValueError(f"rows is on {rows.device}, not on {dev}")
        if rows.dim() != cache.dim():
            raise ValueError("rows must be [B, T, W], or [L, B, T, W] for a cache with layers")
        T = rows.shape[-2]
        if rows.shape != ((L, B, T, W) if layered else (B, T, W)) \
                or (path is not None and path.shape[1] != T):
            raise ValueError(f"rows must be {'[L, ' if layered else '['}{B}, T, {W}] and path "
                             f"[{B}, T], got {tuple(rows.shape)}")
        stride = rows.stride()
        if W > 1 and stride[-1] != 1:
            raise ValueError("rows must have contiguous channels")
        # torch leaves the strides of a dimension of size 1 open
        ls = stride[0] * esz if L > 1 else 0
        bs = stride[-3] * esz if B > 1 else 0
        ts = stride[-2] * esz if T > 1 else 0
        at_rows = rows.data_ptr()
    if L == 0 or B == 0 or T == 0:
        return cache
    _check(library().kda_cache_write(
        cache.data_ptr(), at_rows, ls, bs, ts, block_table.data_ptr(), start.data_ptr(), at_path,
        at_n, L, n_pages, page, W * esz, B, T, max_pages, at_status, raw),
        "kda_cache_write")
    return cache


def kda_cache_copy_pages(cache, src, dst, *, status=None, stream=None):
    """Page ``dst[i]`` of every layer of the pool ``[L, n_pages, ...]`` becomes a
    copy of page ``src[i]``, in place (any dtype; a page is all that lies behind the
    first two dimensions).  src, dst: int32 ``[n]`` on the device; the dst pages are
    distinct and none is a src.  Returns cache."""
    if not isinstance(cache, torch.Tensor) or not cache.is_cuda:
        raise TypeError("cache must be a CUDA tensor")
    dev = cache.device
    raw = _stream(stream, dev)
    _tensor("cache", cache, cache.dtype, None, dev)
    if cache.dim() < 3:
        raise ValueError("cache must be [L, n_pages, ...]")
    _tensor("src", src, _I32, None, dev)
    if src.dim() != 1:
        raise ValueError("src must be one-dimensional")
    n = src.shape[0]
    _tensor("dst", dst, _I32, (n,), dev)
    at_status = _status(status, dev)
    L, n_pages = cache.shape[:2]
    if L == 0 or n == 0:
        return cache
    page_bytes = math.prod(cache.shape[2:]) * cache.element_size()
    _check(library().kda_cache_copy_pages(cache.data_ptr(), src.data_ptr(), dst.data_ptr(), n, L,
                                          n_pages, page_bytes, at_status, raw),
           "kda_cache_copy_pages")
    return cache
