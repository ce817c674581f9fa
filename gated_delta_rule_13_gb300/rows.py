"""Binding of the entry points around a cached latent row: its norm, the rotation of its
positions, the attention weight it has been given, its eviction.

Like ``latent``: every function has the name of the C entry point it wraps
(include/kda.h), checks shapes, dtypes and devices, allocates what the caller did not
pass, and forwards pointers with the current CUDA stream.
"""
from __future__ import annotations

import math

import torch

from .kda import HEAD_DIM, KDA_BF16, KDA_F32, _check, library
from .latent import (_BF16, _F32, _I32, _I64, LATENT_DIM, _device, _new, _scale, _size, _status,
                     _stream, _tensor, _workspace)

_F64 = torch.float64
_CODE = {_BF16: KDA_BF16, _F32: KDA_F32}


def _code(name, t):
    """A CUDA tensor's dtype code."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return code


def _like(name, t, dtype, device, shape):
    """A tensor of this dtype and shape on the device, with any strides."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device:
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not dtype:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _step(name, shape, stride, lead):
    """Stride between the rows of a view whose first ``lead`` dimensions are one dimension
    of rows, as of a slice of a contiguous tensor; its rows must be contiguous."""
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if lead == 1 and shape[0] > 1:
        return stride[0]
    step = None
    for i in range(lead - 1, -1, -1):
        if shape[i] == 0:
            return shape[-1]
        if shape[i] == 1:                   # torch leaves its stride open
            continue
        if step is None:
            first = stride[i]
        elif stride[i] != step * n:
            raise ValueError(f"{name}: rows of {tuple(shape)} must be evenly spaced, "
                             f"got strides {stride}")
        step, n = stride[i], shape[i]
    return math.prod(shape[lead:]) if step is None else first


def kda_rope_inv_freq(dim, base=10000.0, *, scaling=None, factor=1.0, original=None,
                      beta_fast=32.0, beta_slow=1.0, device=None):
    """Angles per position of the ``dim // 2`` channel pairs of ``kda_rope``, fp64:
    ``base ** (-2 i / dim)``, for a context longer than the trained one scaled by

    ``"linear"``  every angle divided by ``factor``;
    ``"base"``    the base raised so that the slowest pair turns ``factor`` times slower
                  and the fastest as before;
    ``"ramp"``    pairs that turn more than ``beta_fast`` times over the ``original``
                  context as before, those that turn less than ``beta_slow`` times
                  divided by ``factor``, those between in proportion to their index
                  (such models multiply by ``0.1 log(factor) + 1``: ``kda_rope``'s scale).

    "ramp" is the method of Peng, Quesnelle, Fan and Shippole, "YaRN: Efficient Context
    Window Extension of Large Language Models" (2023), with the borders rounded outwards and
    held to 0 and ``dim - 1``, as models trained with it have them."""
    if dim < 2 or dim % 2:
        raise ValueError(f"dim must be even and positive, got {dim}")
    if not (base > 1.0 and math.isfinite(base)):
        raise ValueError(f"base must be finite and above 1, got {base}")
    if not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError(f"factor must be finite and at least 1, got {factor}")
    i = torch.arange(dim // 2, dtype=_F64)
    if scaling == "base" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    freq = base ** (-2.0 * i / dim)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "ramp":
        if original is None or original <= 0 or not beta_fast > beta_slow > 0:
            raise ValueError("ramp scaling needs the original context's length and "
                             "beta_fast > beta_slow > 0")

        def index(turns):                   # of the pair that turns so often
            return dim * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))

        low = max(0, math.floor(index(beta_fast)))
        high = min(dim - 1, math.ceil(index(beta_slow)))
        slow = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        freq = freq * (1.0 - slow) + freq / factor * slow
    elif scaling not in (None, "base"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'ramp', got {scaling!r}")
    return freq.to(device) if device is not None else freq


def kda_rope(x, positions, inv_freq, *, k=None, interleaved=True, scale=1.0, transpose=False,
             out=None, k_out=None, stream=None):
    """The channel pairs of ``x`` turned by ``positions * inv_freq`` and scaled.

    x ``[*tokens, H, dr]`` or, without heads, ``[*tokens, dr]`` (bf16 or fp32), a view
    of the rotary channels of wider heads as it may be; positions int32 ``[*tokens]``;
    inv_freq fp64 ``[dr // 2]`` (``kda_rope_inv_freq``), both on the device.  Pairs are
    neighbours (``interleaved``) or channel i and i + dr // 2.  ``k`` ``[*tokens, dr]``
    is the key the heads share, turned in the same launch.  ``transpose`` turns back:
    the gradient of the call without it.  ``out`` and ``k_out`` may be views, and x and
    k themselves (in place).  Returns ``out``, with ``k`` ``(out, k_out)``."""
    code = _code("x", x)
    dev, shape, dtype = x.device, x.shape, x.dtype
    raw = _stream(stream, dev)
    _tensor("positions", positions, _I32, None, dev)
    lead, tokens = positions.dim(), positions.shape
    heads = len(shape) == lead + 2
    if shape[:lead] != tokens or not (heads or len(shape) == lead + 1):
        raise ValueError(f"x must be [*tokens, H, dr] or [*tokens, dr] with positions "
                         f"{tuple(tokens)}, got {tuple(shape)}")
    H, dr = shape[-2] if heads else 1, shape[-1]
    _tensor("inv_freq", inv_freq, _F64, None, dev)
    if dr % 2 or dr == 0 or inv_freq.shape != (dr // 2,):
        raise ValueError(f"x has {dr} rotary channels: inv_freq must be [{dr // 2}] and "
                         f"the channels pairs, got {tuple(inv_freq.shape)}")
    scale = float(scale)
    if not math.isfinite(scale):
        raise ValueError(f"scale must be finite, got {scale}")
    if out is None:
        out = _new(stream, shape, dtype, dev)
    else:
        _like("out", out, dtype, dev, shape)
    x_st, o_st = x.stride(), out.stride()
    x_ts, o_ts = _step("x", shape, x_st, lead), _step("out", shape, o_st, lead)
    x_hs, o_hs = (x_st[-2], o_st[-2]) if heads and H > 1 else (dr, dr)
    at_k = at_ko = None
    k_ts = ko_ts = dr
    if k is not None:
        k_shape = (*tokens, dr)
        _like("k", k, dtype, dev, k_shape)
        if k_out is None:
            k_out = _new(stream, k_shape, dtype, dev)
        else:
            _like("k_out", k_out, dtype, dev, k_shape)
            ko_ts = _step("k_out", k_shape, k_out.stride(), lead)
        k_ts = _step("k", k_shape, k.stride(), lead)
        at_k, at_ko = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out is given without k")
    n = positions.numel()
    if n > 0 and H > 0:
        _check(library().kda_rope(
            x.data_ptr(), x_ts, x_hs, out.data_ptr(), o_ts, o_hs, at_k, k_ts, at_ko, ko_ts,
            positions.data_ptr(), inv_freq.data_ptr(), n, H, dr, interleaved, scale, transpose,
            code, raw), "kda_rope")
    elif n > 0 and k is not None:
        raise ValueError("x has no heads")
    return out if k is None else (out, k_out)


def kda_norm_fwd(x, weight=None, bias=None, *, center=True, eps=1e-5, out=None, stats=True,
                 stream=None):
    """Each row of ``x`` ``[*rows, W]`` (bf16 or fp32, rows evenly spaced, W at most
    16384) without its mean (``center``; else as it is) over its root mean square, times
    ``weight``, plus ``bias`` (fp32 ``[W]`` or None).  ``out`` may be a view, and x itself.
    Returns ``(out, mean, rstd)``: fp32 ``[*rows]`` for ``kda_norm_bwd``, mean None without
    ``center``, both None without ``stats``."""
    code = _code("x", x)
    dev, shape, dtype = x.device, x.shape, x.dtype
    raw = _stream(stream, dev)
    lead = len(shape) - 1
    if lead < 0:
        raise ValueError("x must be [*rows, W]")
    W, rows = shape[-1], shape[:-1]
    n = rows[0] if lead == 1 else math.prod(rows)
    x_rs = _step("x", shape, x.stride(), lead)
    if weight is not None:
        _tensor("weight", weight, _F32, (W,), dev)
    if bias is not None:
        _tensor("bias", bias, _F32, (W,), dev)
    eps = float(eps)
    if not (eps > 0.0 and math.isfinite(eps)):
        raise ValueError(f"eps must be finite and positive, got {eps}")
    if out is None:
        out, out_rs = _new(stream, shape, dtype, dev), W
    else:
        _like("out", out, dtype, dev, shape)
        out_rs = _step("out", shape, out.stride(), lead)
    mean = _new(stream, rows, _F32, dev) if stats and center else None
    rstd = _new(stream, rows, _F32, dev) if stats else None
    _check(library().kda_norm_fwd(
        x.data_ptr(), x_rs, None if weight is None else weight.data_ptr(),
        None if bias is None else bias.data_ptr(), n, W, code, center, eps,
        out.data_ptr(), out_rs, None if mean is None else mean.data_ptr(),
        None if rstd is None else rstd.data_ptr(), raw), "kda_norm_fwd")
    return out, mean, rstd


def kda_norm_bwd_workspace_size(n, W, dtype=KDA_BF16) -> int:
    return _size("kda_norm_bwd_workspace_size", _device(), n, W, dtype)


def kda_norm_bwd(d_out, x, weight, mean, rstd, *, bias=False, d_x=None, workspace=None,
                 stream=None):
    """Gradients of ``kda_norm_fwd`` for the output gradient ``d_out``; ``mean`` (None: a
    norm without its mean) and ``rstd`` are what it returned.  Returns ``(d_x, d_weight,
    d_bias)``, the sums in fp32, d_weight None without ``weight``, d_bias None without
    ``bias``.  ``d_x`` may be given as a view, and be d_out or x itself."""
    code = _code("x", x)
    dev, shape, dtype = x.device, x.shape, x.dtype
    raw = _stream(stream, dev)
    lead = len(shape) - 1
    if lead < 0:
        raise ValueError("x must be [*rows, W]")
    W, rows = shape[-1], shape[:-1]
    n = rows[0] if lead == 1 else math.prod(rows)
    x_rs = _step("x", shape, x.stride(), lead)
    _like("d_out", d_out, dtype, dev, shape)
    g_rs = _step("d_out", shape, d_out.stride(), lead)
    if weight is not None:
        _tensor("weight", weight, _F32, (W,), dev)
    if mean is not None:
        _tensor("mean", mean, _F32, rows, dev)
    _tensor("rstd", rstd, _F32, rows, dev)
    if d_x is None:
        d_x, dx_rs = _new(stream, shape, dtype, dev), W
    else:
        _like("d_x", d_x, dtype, dev, shape)
        dx_rs = _step("d_x", shape, d_x.stride(), lead)
    d_weight = _new(stream, (W,), _F32, dev) if weight is not None else None
    d_bias = _new(stream, (W,), _F32, dev) if bias else None
    at_ws, ws_bytes = None, 0
    if weight is not None or bias:
        ws = _workspace(workspace, _size("kda_norm_bwd_workspace_size", dev.index, n, W, code),
                        dev, stream)
        at_ws, ws_bytes = ws.data_ptr(), ws.nbytes
    _check(library().kda_norm_bwd(
        d_out.data_ptr(), g_rs, x.data_ptr(), x_rs, None if weight is None else weight.data_ptr(),
        None if mean is None else mean.data_ptr(), rstd.data_ptr(), n, W, code, d_x.data_ptr(),
        dx_rs, None if d_weight is None else d_weight.data_ptr(),
        None if d_bias is None else d_bias.data_ptr(), at_ws, ws_bytes, raw), "kda_norm_bwd")
    return d_x, d_weight, d_bias


def kda_latent_weights_workspace_size(B, T, H, dc=LATENT_DIM, dr=0, dtype=KDA_BF16) -> int:
    return _size("kda_latent_weights_workspace_size", _device(), B, T, H, dc, dr, dtype)


def kda_latent_weights(q, cache, block_table, seq_lens, lse, weights, *, tree_mask=None,
                       scale=None, decay=1.0, workspace=None, stream=None):
    """``weights`` (fp32 ``[B, max_pages * page_size]``, in place) times ``decay`` plus the
    probabilities that the last T tokens of each sequence gave its cached rows, summed
    over tokens and heads.

    The other arguments are those of ``kda_latent_decode``, ``lse`` (fp32 ``[B, T, H]``) what
    it wrote; a row of infinite lse gives nothing (+inf leaves a rejected draft out).
    Places from a sequence's length on stay as they are.  Returns weights."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor")
    dev = q.device
    raw = _stream(stream, dev)
    _tensor("q", q, _BF16, None, dev)
    if q.dim() != 4 or q.shape[3] not in (LATENT_DIM, LATENT_DIM + 64):
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
    _tensor("lse", lse, _F32, (B, T, H), dev)
    _tensor("weights", weights, _F32, (B, block_table.shape[1] * cache.shape[1]), dev)
    if tree_mask is not None:
        _tensor("tree_mask", tree_mask, _I64, (B, T), dev)
    decay = float(decay)
    if not (decay >= 0.0 and math.isfinite(decay)):
        raise ValueError(f"decay must be finite and not negative, got {decay}")
    ws = _workspace(workspace, _size("kda_latent_weights_workspace_size", dev.index, B, T, H,
                                     LATENT_DIM, dr, KDA_BF16), dev, stream)
    _check(library().kda_latent_weights(
        q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        None if tree_mask is None else tree_mask.data_ptr(), lse.data_ptr(), B, T, H, LATENT_DIM,
        dr, cache.shape[0], cache.shape[1], block_table.shape[1], KDA_BF16,
        _scale(scale, HEAD_DIM + dr), decay, weights.data_ptr(), ws.data_ptr(), ws.nbytes, raw),
        "kda_latent_weights")
    return weights


def kda_cache_evict_workspace_size(L, B, budget) -> int:
    return _size("kda_cache_evict_workspace_size", _device(), L, B, budget)


def kda_cache_evict(cache, block_table, seq_lens, weights, budget, *, first=0, recent=0,
                    weights_out=None, workspace=None, status=None, stream=None):
    """Sequences of more than ``budget`` cached rows cut to it, in place: the ``first``
    first and ``recent`` last rows stay and, of those between, the ones of the greatest
    weight.

    cache ``[n_pages, page_size, W]`` with weights fp32 ``[B, max_pages * page_size]``, or
    all layers in one call ``[L, n_pages, page_size, W]`` with ``[L, B, ...]`` (any dtype;
    each layer by its own weights).  Rows kept in front of ``budget - recent`` stay in
    place, the places that fall free there take the kept rows from behind, the last rows
    move up.  ``weights_out`` (None: weights) receives the kept rows' weights at their new
    places and zeros behind them.  ``status`` (int32 ``[1]`` on the device) receives an error
    code if a sequence's length or pages are refused.  Returns ``(new_lens [B], origin)``,
    origin int32 ``[B, budget]`` (``[L, B, budget]``): where the row now at a place was
    before, -1 behind the last."""
    if not isinstance(cache, torch.Tensor) or not cache.is_cuda:
        raise TypeError("cache must be a CUDA tensor")
    dev = cache.device
    raw = _stream(stream, dev)
    _tensor("cache", cache, cache.dtype, None, dev)
    layered = cache.dim() == 4
    if not layered and cache.dim() != 3:
        raise ValueError("cache must be [n_pages, page_size, W] or [L, n_pages, page_size, W]")
    L = cache.shape[0] if layered else 1
    n_pages, page, W = cache.shape[-3:]
    _tensor("block_table", block_table, _I32, None, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    _tensor("seq_lens", seq_lens, _I32, (B,), dev)
    budget, first, recent = int(budget), int(first), int(recent)
    if budget < 1 or first < 0 or recent < 0 or first + recent > budget:
        raise ValueError(f"budget must be positive and hold first and recent, got {budget}, "
                         f"{first}, {recent}")
    lead = (L, B) if layered else (B,)
    _tensor("weights", weights, _F32, (*lead, max_pages * page), dev)
    if weights_out is None:
        weights_out = weights
    else:
        _tensor("weights_out", weights_out, _F32, weights.shape, dev)
    at_status = _status(status, dev)
    new_lens = _new(stream, (B,), _I32, dev)
    origin = _new(stream, (*lead, budget), _I32, dev)
    if B == 0:
        return new_lens, origin
    ws = _workspace(workspace, _size("kda_cache_evict_workspace_size", dev.index, L, B, budget),
                    dev, stream)
    _check(library().kda_cache_evict(
        cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), weights.data_ptr(),
        weights_out.data_ptr(), L, n_pages, page, W * cache.element_size(), B, max_pages, budget,
        first, recent, new_lens.data_ptr(), origin.data_ptr(), ws.data_ptr(), ws.nbytes,
        at_status, raw), "kda_cache_evict")
    return new_lens, origin
