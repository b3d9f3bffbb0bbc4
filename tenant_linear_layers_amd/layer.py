"""Decoder-layer operators beside the linears: the norm of the residual
stream, the paged key/value cache and attention over it (include/bitdelta.h).

Argument checks and marshalling only, as in bitdelta.py.  These calls are made
for single tokens too, where the host's time is most of a call's (a launch by
itself takes it 3.7 us), so each asks in one expression whether its tensors are
as they usually are, and looks at them one by one, for what to allow or to
refuse, only where they are not.  Outputs come from empty_like and new_empty,
which read no keywords (1.2 and 1.4 us against 1.7 of torch.empty).
"""

from __future__ import annotations

import contextlib
import math

import torch

from . import bitdelta as _bd

_BF16, _I32 = torch.bfloat16, torch.int32
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_raw_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice
_NONE = contextlib.nullcontext()
_ROWS = torch.contiguous_format


def _device(t, name: str) -> int:
    """The HIP device index of a call's first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (HIP) tensor")
    return t.get_device()


def _is(t, name: str, dtype, dev: int, contiguous: bool = True) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected device {dev}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _fail(status: int, where: str) -> None:
    raise _bd.BitDeltaError(status, where)


def _at(dev: int, stream):
    """The context that makes dev and the caller's stream current: tensors made
    in it belong to the stream that the kernels run on."""
    if stream is not None:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        return torch.cuda.stream(stream)
    return _NONE if dev == _current() else torch.cuda.device(dev)


# ------------------------------------------------------------------ norm
def _rows(t, name: str, shape, dev: int):
    """The stride of the rows of a bf16 tensor [..., cols]: any in two
    dimensions, that of contiguous rows otherwise."""
    _is(t, name, _BF16, dev, contiguous=False)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have x's shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.shape[-1]
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be contiguous, or two-dimensional with contiguous rows")
    return t.stride(0)


def _norm_checks(x, weight, residual, y, h, mx):
    """(x stride, residual stride) of tensors that are not all contiguous, or
    what is wrong with them."""
    dev = _device(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., cols]")
    shape, cols = x.shape, x.shape[-1]
    if mx and cols % 32:
        raise ValueError(f"cols must be a multiple of 32 for an 8-bit output, got {cols}")
    xs = _rows(x, "x", None, dev)
    _is(weight, "weight", _BF16, dev)
    if weight.numel() != cols:
        raise ValueError(f"weight must hold {cols} elements, got {weight.numel()}")
    rs = 0
    if residual is not None:
        rs = _rows(residual, "residual", shape, dev)
    elif h is not None:
        raise ValueError("h is written with a residual only")
    for t, name in ((y, "y"), (h, "h")):
        if t is not None:
            _is(t, name, _BF16, dev)
            if t.shape != shape:
                raise ValueError(f"{name} must have x's shape")
    return xs, rs


def _norm(x, weight, eps, residual, y, h, stream, mx):
    try:
        shape = x.shape
        xs = rs = cols = shape[-1]
        dev = x.get_device()
        usual = (cols > 0 and dev >= 0 and x.dtype is _BF16 and x.is_contiguous() and
                 weight.dtype is _BF16 and weight.get_device() == dev and
                 weight.numel() == cols and weight.is_contiguous() and
                 y is None and h is None and not (mx and cols % 32) and
                 (residual is None or residual.dtype is _BF16 and residual.shape == shape and
                  residual.get_device() == dev and residual.is_contiguous()))
    except (AttributeError, IndexError):
        usual = False
    if not usual:
        xs, rs = _norm_checks(x, weight, residual, y, h, mx)
    with _at(dev, stream):
        if mx:
            y = x.new_empty(shape, dtype=_E4M3)
            scale = x.new_empty((*shape[:-1], cols // 32), dtype=_E8M0)
        elif y is None:
            y = torch.empty_like(x, memory_format=_ROWS)
        rp = hp = None
        if residual is not None:
            rp = residual.data_ptr()
            if h is None:
                h = torch.empty_like(x, memory_format=_ROWS)
            hp = h.data_ptr()
        rows = x.numel() // cols
        if mx:
            st = _bd.lib().bitdelta_rms_norm_mx(
                x.data_ptr(), xs, rp, rs, weight.data_ptr(), eps, rows, cols, hp, y.data_ptr(),
                scale.data_ptr(), _raw_stream(dev))
        else:
            st = _bd.lib().bitdelta_rms_norm(
                x.data_ptr(), xs, rp, rs, weight.data_ptr(), eps, rows, cols, hp, y.data_ptr(),
                _raw_stream(dev))
    if st:
        _fail(st, "bitdelta_rms_norm_mx" if mx else "bitdelta_rms_norm")
    return (y, scale, h) if mx else (y, h)


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual=None, y=None, h=None,
             stream=None):
    """(y, h): h = x + residual (None without one), y = h / sqrt(mean(h^2) + eps) * weight.
    x, residual: bf16 [..., cols]; weight: bf16 [cols]."""
    return _norm(x, weight, eps, residual, y, h, stream, False)


def rms_norm_mx(x: torch.Tensor, weight: torch.Tensor, eps: float, residual=None, h=None,
                stream=None):
    """(q, scale, h): rms_norm with its output in e4m3 [..., cols] and one
    e8m0 scale per 32 values [..., cols / 32]: the smallest power of two under
    which none of them passes 448, so that no value saturates (the OCP MX text
    takes the maximum's logarithm rounded down)."""
    return _norm(x, weight, eps, residual, None, h, stream, True)


# ------------------------------------------------------------------ cache
def _cache_checks(k_cache, v_cache, k_scale, v_scale, dev: int):
    """What is wrong with a cache."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a tensor [pages, heads, page, dim]")
    q8 = k_cache.dtype is _E4M3
    kind = _E4M3 if q8 else _BF16
    _is(k_cache, "k_cache", kind, dev)
    _is(v_cache, "v_cache", kind, dev)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be of one shape")
    if not q8:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
    elif k_scale is None or v_scale is None:
        raise ValueError("an e4m3 cache needs k_scale and v_scale")
    else:
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _is(t, name, _E8M0, dev)
            if t.shape != shape[:3]:
                raise ValueError(f"{name} must be [pages, heads, page]")
    raise ValueError("a cache has pages, heads, dim 64 or 128 and pages of a multiple of 16 rows, "
                     f"got {tuple(shape)}")


def _cache(k_cache, v_cache, k_scale, v_scale, dev: int):
    """(pages, heads, page, dim, k_scale pointer, v_scale pointer) of a cache."""
    try:
        shape, kind = k_cache.shape, k_cache.dtype
        pages, heads, page, dim = shape
        good = (v_cache.dtype is kind and v_cache.shape == shape and
                k_cache.get_device() == dev and v_cache.get_device() == dev and
                k_cache.is_contiguous() and v_cache.is_contiguous() and
                (dim == 128 or dim == 64) and not page % 16 and 16 <= page <= 65536 and
                pages > 0 and heads > 0 and
                (k_scale is None and v_scale is None if kind is _BF16 else
                 kind is _E4M3 and k_scale.dtype is _E8M0 and v_scale.dtype is _E8M0 and
                 k_scale.get_device() == dev and v_scale.get_device() == dev and
                 k_scale.shape == v_scale.shape == (pages, heads, page) and
                 k_scale.is_contiguous() and v_scale.is_contiguous()))
    except (AttributeError, ValueError):
        good = False
    if not good:
        _cache_checks(k_cache, v_cache, k_scale, v_scale, dev)
    if k_scale is None:
        return pages, heads, page, dim, None, None
    return pages, heads, page, dim, k_scale.data_ptr(), v_scale.data_ptr()


def _heads(t, name: str, dev: int, heads, dim: int):
    """The strides of a bf16 [tokens, heads, dim] view with contiguous dims."""
    try:
        shape, s = t.shape, t.stride()
        if (t.dtype is _BF16 and t.get_device() == dev and len(s) == 3 and s[2] == 1 and
                shape[2] == dim and (heads is None or shape[1] == heads)):
            return s
    except AttributeError:
        pass
    _is(t, name, _BF16, dev, contiguous=False)
    if t.dim() != 3 or t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {dim}], "
                         f"got {tuple(t.shape)}")
    raise ValueError(f"{name}'s last dimension must be contiguous")


def _ints(t, name: str, dev: int) -> int:
    """The number of values of an int32 tensor."""
    try:
        if t.dtype is _I32 and t.get_device() == dev and t.is_contiguous():
            return t.numel()
    except AttributeError:
        pass
    _is(t, name, _I32, dev)


def kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
             v_cache: torch.Tensor, k_scale=None, v_scale=None, stream=None) -> None:
    """Put k and v (bf16 [tokens, heads, dim], any token and head strides) into
    the cache rows slots (int32 [tokens]; negative: passed over), in bf16 or,
    for an e4m3 cache, in 8 bits with a scale per row."""
    dev = _device(k, "k")
    pages, heads, page, dim, ks, vs = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    sk = _heads(k, "k", dev, heads, dim)
    sv = _heads(v, "v", dev, heads, dim)
    tokens = _ints(slots, "slots", dev)
    if k.shape[0] != tokens or v.shape[0] != tokens:
        raise ValueError("k, v and slots must have one entry per token")
    with _at(dev, stream):
        st = _bd.lib().bitdelta_kv_write(
            k.data_ptr(), v.data_ptr(), sk[0], sk[1], sv[0], sv[1], slots.data_ptr(), tokens,
            heads, dim, pages, page, k_cache.data_ptr(), v_cache.data_ptr(), ks, vs,
            _raw_stream(dev))
    if st:
        _fail(st, "bitdelta_kv_write")


def kv_read(slots: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale=None,
            v_scale=None, stream=None):
    """(k, v): the cache rows slots as bf16 [tokens, heads, dim]."""
    dev = _device(slots, "slots")
    tokens = _ints(slots, "slots", dev)
    pages, heads, page, dim, ks, vs = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    with _at(dev, stream):
        k = slots.new_empty((tokens, heads, dim), dtype=_BF16)
        v = torch.empty_like(k)
        st = _bd.lib().bitdelta_kv_read(
            slots.data_ptr(), tokens, heads, dim, pages, page, k_cache.data_ptr(),
            v_cache.data_ptr(), ks, vs, k.data_ptr(), v.data_ptr(), _raw_stream(dev))
    if st:
        _fail(st, "bitdelta_kv_read")
    return k, v


# ------------------------------------------------------------------ attention
def paged_attention_workspace_size(tokens: int, seqs: int, max_q: int, heads: int, kv_heads: int,
                                   dim: int, width: int, page: int) -> int:
    return int(_bd.lib().bitdelta_paged_attention_workspace_size(tokens, seqs, max_q, heads,
                                                                 kv_heads, dim, width, page))


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor, max_q: int,
                    k_scale=None, v_scale=None, window: int = 0, scale=None, out=None,
                    workspace=None, stream=None) -> torch.Tensor:
    """Causal attention of new tokens over the paged cache, bf16 [tokens, heads, dim].

    q: bf16 [tokens, heads, dim], any token and head strides; table: int32
    [seqs, width] page ids; cu_q: int32 [seqs + 1], the sequences' rows of q;
    kv_len: int32 [seqs], cached keys of each, the new tokens' among them;
    max_q: the most rows of a sequence, or more (a sequence of more than max_q
    may be left out); window: keys a row sees, 0 for all;
    scale: of the scores, above 0, 1 / sqrt(dim) by default.  A row that sees no key
    gives zeros."""
    dev = _device(q, "q")
    pages, kv_heads, page, dim, ks, vs = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    s = _heads(q, "q", dev, None, dim)
    tokens, heads, _ = q.shape
    if heads % kv_heads or not 1 <= heads // kv_heads <= 64:
        raise ValueError(f"{heads} query heads do not share {kv_heads} key/value heads")
    seqs = _ints(kv_len, "kv_len", dev)
    _ints(table, "table", dev)
    if (_ints(cu_q, "cu_q", dev) != seqs + 1 or table.dim() != 2 or table.shape[0] != seqs):
        raise ValueError("table must be [seqs, width], cu_q [seqs + 1] and kv_len [seqs]")
    if window < 0 or max_q < 0:
        raise ValueError("window and max_q must not be negative")
    width = table.shape[1]
    L = _bd.lib()
    with _at(dev, stream):
        if out is None:
            out = torch.empty_like(q, memory_format=_ROWS)
        else:
            _is(out, "out", _BF16, dev)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
        wp, wn = None, 0
        if workspace is None:
            wn = L.bitdelta_paged_attention_workspace_size(tokens, seqs, max_q, heads, kv_heads,
                                                           dim, width, page)
            if wn:
                workspace = kv_len.new_empty((wn + 3) // 4)
                wp = workspace.data_ptr()
        else:
            if workspace.get_device() != dev or not workspace.is_contiguous():
                raise ValueError("workspace must be a contiguous tensor on q's device")
            wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        st = L.bitdelta_paged_attention(
            q.data_ptr(), s[0], s[1], k_cache.data_ptr(), v_cache.data_ptr(), ks, vs,
            table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), tokens, seqs, max_q, heads,
            kv_heads, dim, pages, page, width, 1.0 / math.sqrt(dim) if scale is None else scale,
            window, out.data_ptr(), wp, wn, _raw_stream(dev))
    if st:
        _fail(st, "bitdelta_paged_attention")
    return out
