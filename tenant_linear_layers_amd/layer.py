"""Decoder-layer operators beside the linears: the norms of the residual
stream, rotary positions, the paged key/value cache and attention over it
(include/bitdelta.h).

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
_E4M3, _E8M0, _E2M1 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.float4_e2m1fn_x2
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


def _gate(gate, shape, dev: int):
    """(the gate, its row stride): bf16 of x's shape, or one row [cols]."""
    _is(gate, "gate", _BF16, dev, contiguous=False)
    if gate.dim() == 1 and gate.shape[0] == shape[-1] and gate.is_contiguous():
        return 0
    return _rows(gate, "gate", shape, dev)


def _block_checks(x, residual, post_weight, weight, gate, scale, y, h):
    """(device, row strides of x, residual and gate) of a block norm's tensors,
    or what is wrong with them."""
    dev = _device(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., cols]")
    shape, cols = x.shape, x.shape[-1]
    xs = _rows(x, "x", None, dev)
    rs = _rows(residual, "residual", shape, dev)
    for t, name in ((post_weight, "post_weight"), (weight, "weight")):
        if t is not None or name == "weight":
            _is(t, name, _BF16, dev)
            if t.numel() != cols:
                raise ValueError(f"{name} must hold {cols} elements, got {t.numel()}")
    gs = 0 if gate is None else _gate(gate, shape, dev)
    for t, name in ((y, "y"), (h, "h")):
        if t is not None:
            _is(t, name, _BF16, dev)
            if t.shape != shape:
                raise ValueError(f"{name} must have x's shape")
    if not math.isfinite(scale):
        raise ValueError(f"scale must be finite, got {scale}")
    return dev, xs, rs, gs


def rms_norm_block(x: torch.Tensor, residual: torch.Tensor, post_weight, weight: torch.Tensor,
                   eps: float, gate=None, scale: float = 1.0, y=None, h=None, stream=None):
    """(y, h) of a block's output x, around its end and before the next block:

        u = x / sqrt(mean(x^2) + eps) * post_weight     (post_weight None: u = x)
        h = residual + scale * gate * u                 (gate None: 1)
        y = h / sqrt(mean(h^2) + eps) * weight

    x, residual, y, h: bf16 [..., cols]; gate: bf16 of that shape or [cols];
    post_weight, weight: bf16 [cols]; scale: finite.  The sums of squares are
    float32: of a row whose sum passes 2^128 the norm is zeros."""
    gs = 0
    try:
        shape = x.shape
        xs = rs = cols = shape[-1]
        dev = x.get_device()
        usual = (cols > 0 and dev >= 0 and x.dtype is _BF16 and x.is_contiguous() and
                 residual.dtype is _BF16 and residual.shape == shape and
                 residual.get_device() == dev and residual.is_contiguous() and
                 weight.dtype is _BF16 and weight.get_device() == dev and
                 weight.numel() == cols and weight.is_contiguous() and
                 (post_weight is None or post_weight.dtype is _BF16 and
                  post_weight.get_device() == dev and post_weight.numel() == cols and
                  post_weight.is_contiguous()) and
                 gate is None and y is None and h is None and math.isfinite(scale))
    except (AttributeError, IndexError, TypeError):
        usual = False
    if not usual:
        dev, xs, rs, gs = _block_checks(x, residual, post_weight, weight, gate, scale, y, h)
        cols = x.shape[-1]
    with _at(dev, stream):
        y = torch.empty_like(x, memory_format=_ROWS) if y is None else y
        h = torch.empty_like(x, memory_format=_ROWS) if h is None else h
        st = _bd.lib().bitdelta_rms_norm_block(
            x.data_ptr(), xs, None if post_weight is None else post_weight.data_ptr(),
            None if gate is None else gate.data_ptr(), gs, scale, residual.data_ptr(), rs,
            weight.data_ptr(), eps, x.numel() // cols, cols, h.data_ptr(), y.data_ptr(),
            _raw_stream(dev))
    if st:
        _fail(st, "bitdelta_rms_norm_block")
    return y, h


# ------------------------------------------------------------------ rotary positions
def rotary_frequencies(rot: int, base: float = 10000.0, factor: float = 1.0,
                       method: str = "linear", original_length: int = 0, fast: float = 32.0,
                       slow: float = 1.0):
    """(frequencies, magnitude) for rotary_table: float64 [rot / 2], radians a position.

    Without scaling (factor 1) pair i turns by base^(-2 i / rot).  For contexts
    factor times as long as those of training:
      "linear"  every frequency over factor (positions interpolated);
      "base"    the base times factor^(rot / (rot - 2)): the slowest pair is
                stretched by factor, the fastest not at all;
      "ramp"    by the turns that a pair makes within original_length: those of
                more than `fast` turns stay, of fewer than `slow` are stretched by
                factor, with a linear ramp over the pair's index between; the
                magnitude 0.1 ln(factor) + 1 goes into the table, so that scores
                grow by its square;
      "smooth"  the same two borders, with the ramp over the number of turns and
                no magnitude."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2, got {rot}")
    if not base > 1 or not factor > 0:
        raise ValueError("base must be above 1 and factor above 0")
    if method not in ("linear", "base", "ramp", "smooth"):
        raise ValueError(f"no such method: {method!r}")
    if method in ("ramp", "smooth") and (original_length < 1 or not fast > slow > 0):
        raise ValueError(f"{method!r} needs original_length and fast > slow > 0")
    if method == "base" and factor != 1:
        if rot < 4:
            raise ValueError("the base of a single pair cannot be scaled")
        base *= factor ** (rot / (rot - 2))
    f = torch.pow(base, torch.arange(0, rot, 2, dtype=torch.float64) / -rot)
    if method == "base" or factor == 1:
        return f, 1.0
    if method == "linear":
        return f / factor, 1.0
    if method == "smooth":
        turns = f * (original_length / (2 * math.pi))
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        return f / factor * (1 - keep) + f * keep, 1.0
    # the pair that makes this many turns within original_length
    lo, hi = (rot * math.log(original_length / (n * 2 * math.pi)) / (2 * math.log(base))
              for n in (fast, slow))
    lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
    stretch = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return (f / factor * stretch + f * (1 - stretch),
            0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0)


def rotary_table(frequencies: torch.Tensor, length: int, first: int = 0, magnitude: float = 1.0,
                 device=None, stream=None) -> torch.Tensor:
    """float32 [length, pairs, 2]: cosine and sine of position * frequency, times
    magnitude, for the positions first .. first + length - 1; angles are taken in
    64 bits.  frequencies: float64 [pairs], on a device or on the host, from
    where they go to `device` (the current one); the table is on that device."""
    if not isinstance(frequencies, torch.Tensor) or frequencies.dtype is not torch.float64 or \
            frequencies.dim() != 1:
        raise TypeError("frequencies must be a float64 tensor [pairs]")
    pairs = frequencies.shape[0]
    if length < 0 or first < 0 or pairs < 1:
        raise ValueError("length and first must not be negative, and there must be a pair")
    want = torch.device("cuda" if device is None else device)
    if want.type != "cuda":
        raise ValueError(f"device must be a HIP device, got {want}")
    if frequencies.is_cuda:
        dev = frequencies.get_device()
        if want.index is not None and want.index != dev:
            raise ValueError(f"frequencies are on {frequencies.device}, device is {want}")
    else:
        dev = _current() if want.index is None else want.index
    with _at(dev, stream):
        frequencies = frequencies.to(f"cuda:{dev}").contiguous()
        table = torch.empty((length, pairs, 2), dtype=torch.float32, device=frequencies.device)
        st = _bd.lib().bitdelta_rotary_table(frequencies.data_ptr(), pairs, first, length,
                                             magnitude, table.data_ptr(), _raw_stream(dev))
    if st:
        _fail(st, "bitdelta_rotary_table")
    return table


def _table(table, dim: int, dev: int):
    """(length, rotated dims) of a table of cosines and sines."""
    try:
        length, pairs, two = table.shape
        if (table.dtype is torch.float32 and table.get_device() == dev and two == 2 and
                table.is_contiguous() and 0 < 2 * pairs <= dim and length > 0):
            return length, 2 * pairs
    except (AttributeError, ValueError):
        pass
    _is(table, "table", torch.float32, dev)
    raise ValueError(f"table must be [positions, pairs, 2] with at most {dim // 2} pairs, "
                     f"got {tuple(table.shape)}")


def rotary(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor,
           interleaved: bool = False, out=None, stream=None) -> torch.Tensor:
    """x (bf16 [tokens, heads, dim], any token and head strides) with the first
    rot = 2 pairs dims of each head turned by the angles of the tokens'
    positions (int32 [tokens]): the pairs (i, i + rot / 2), or (2 i, 2 i + 1)
    interleaved; the other dims as they are.  table: float32 [positions, pairs,
    2] (rotary_table).  A position outside it makes the turned dims NaN.  out:
    of x's shape, any strides under which its rows lie apart; x itself turns it
    in place."""
    dev = _device(x, "x")
    s = _heads(x, "x", dev, None, None)
    tokens, heads, dim = x.shape
    if _ints(positions, "positions", dev) != tokens:
        raise ValueError("positions must have one entry per token")
    length, rot = _table(table, dim, dev)
    with _at(dev, stream):
        if out is None:
            out = torch.empty_like(x, memory_format=_ROWS)
            o = (heads * dim, dim)
        else:
            o = _heads(out, "out", dev, heads, dim)
            if out.shape != x.shape:
                raise ValueError("out must have x's shape")
        st = _bd.lib().bitdelta_rotary(
            x.data_ptr(), s[0], s[1], positions.data_ptr(), table.data_ptr(), length, rot,
            interleaved, tokens, heads, dim, out.data_ptr(), o[0], o[1], _raw_stream(dev))
    if st:
        _fail(st, "bitdelta_rotary")
    return out


# ------------------------------------------------------------------ cache
def _cache_checks(k_cache, v_cache, k_scale, v_scale, dev: int):
    """What is wrong with a cache."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a tensor [pages, heads, page, dim]")
    kind = k_cache.dtype if k_cache.dtype in (_E4M3, _E2M1) else _BF16
    _is(k_cache, "k_cache", kind, dev)
    _is(v_cache, "v_cache", kind, dev)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be of one shape")
    if kind is _BF16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
    elif k_scale is None or v_scale is None:
        raise ValueError(f"an {'e4m3' if kind is _E4M3 else 'e2m1'} cache needs k_scale and v_scale")
    else:
        want = shape[:3] if kind is _E4M3 else (*shape[:3], shape[3] // 16)
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _is(t, name, _E8M0, dev)
            if t.shape != want:
                raise ValueError(f"{name} must be [pages, heads, page"
                                 f"{']' if kind is _E4M3 else ', dim / 32]'}")
    raise ValueError("a cache has pages, heads, dim 64 or 128 (e2m1: half as many bytes) and pages "
                     f"of a multiple of 16 rows, got {tuple(shape)}")


def _cache(k_cache, v_cache, k_scale, v_scale, dev: int):
    """(pages, heads, page, dim, k_scale pointer, v_scale pointer, bits of a value) of a cache."""
    bits = 16
    try:
        shape, kind = k_cache.shape, k_cache.dtype
        pages, heads, page, dim = shape
        if kind is not _BF16:
            bits = 8 if kind is _E4M3 else 4
            scales = shape[:3] if bits == 8 else (pages, heads, page, dim // 16)
            if bits == 4:
                dim *= 2
        good = (v_cache.dtype is kind and v_cache.shape == shape and
                k_cache.get_device() == dev and v_cache.get_device() == dev and
                k_cache.is_contiguous() and v_cache.is_contiguous() and
                (dim == 128 or dim == 64) and not page % 16 and 16 <= page <= 65536 and
                pages > 0 and heads > 0 and
                (k_scale is None and v_scale is None if bits == 16 else
                 (bits == 8 or kind is _E2M1) and k_scale.dtype is _E8M0 and
                 v_scale.dtype is _E8M0 and
                 k_scale.get_device() == dev and v_scale.get_device() == dev and
                 k_scale.shape == scales and v_scale.shape == scales and
                 k_scale.is_contiguous() and v_scale.is_contiguous()))
    except (AttributeError, ValueError):
        good = False
    if not good:
        _cache_checks(k_cache, v_cache, k_scale, v_scale, dev)
    if k_scale is None:
        return pages, heads, page, dim, None, None, bits
    return pages, heads, page, dim, k_scale.data_ptr(), v_scale.data_ptr(), bits


def _heads(t, name: str, dev: int, heads, dim: int):
    """The strides of a bf16 [tokens, heads, dim] view with contiguous dims."""
    try:
        shape, s = t.shape, t.stride()
        if (t.dtype is _BF16 and t.get_device() == dev and len(s) == 3 and s[2] == 1 and
                (dim is None or shape[2] == dim) and (heads is None or shape[1] == heads)):
            return s
    except AttributeError:
        pass
    _is(t, name, _BF16, dev, contiguous=False)
    if t.dim() != 3 or (dim is not None and t.shape[2] != dim) or \
            (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {dim or 'dim'}], "
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
    for an e4m3 cache, in 8 bits with a scale per row, for an e2m1 cache (two
    values a byte, [pages, heads, page, dim / 2]) in 4 bits with a scale per 32
    dims."""
    dev = _device(k, "k")
    pages, heads, page, dim, ks, vs, bits = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    sk = _heads(k, "k", dev, heads, dim)
    sv = _heads(v, "v", dev, heads, dim)
    tokens = _ints(slots, "slots", dev)
    if k.shape[0] != tokens or v.shape[0] != tokens:
        raise ValueError("k, v and slots must have one entry per token")
    with _at(dev, stream):
        call = _bd.lib().bitdelta_kv_write_4bit if bits == 4 else _bd.lib().bitdelta_kv_write
        st = call(
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
    pages, heads, page, dim, ks, vs, bits = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    with _at(dev, stream):
        k = slots.new_empty((tokens, heads, dim), dtype=_BF16)
        v = torch.empty_like(k)
        call = _bd.lib().bitdelta_kv_read_4bit if bits == 4 else _bd.lib().bitdelta_kv_read
        st = call(
            slots.data_ptr(), tokens, heads, dim, pages, page, k_cache.data_ptr(),
            v_cache.data_ptr(), ks, vs, k.data_ptr(), v.data_ptr(), _raw_stream(dev))
    if st:
        _fail(st, "bitdelta_kv_read")
    return k, v


def kv_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
              table: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
              v_cache: torch.Tensor, k_scale=None, v_scale=None, interleaved: bool = False,
              q_out=None, stream=None) -> torch.Tensor:
    """q turned by its tokens' positions (as rotary does; bf16 [tokens, heads,
    dim], q_out where it is given), with k, turned alike, and v put into the
    cache rows slots (as kv_write does): in one pass, k rounded once to the
    cache's type.  The queries of tokens whose slot is outside the cache are
    turned too."""
    dev = _device(q, "q")
    pages, kv_heads, page, dim, ks, vs, bits = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    sq = _heads(q, "q", dev, None, dim)
    sk = _heads(k, "k", dev, kv_heads, dim)
    sv = _heads(v, "v", dev, kv_heads, dim)
    length, rot = _table(table, dim, dev)
    tokens, heads, _ = q.shape
    if not (tokens == k.shape[0] == v.shape[0] == _ints(slots, "slots", dev) ==
            _ints(positions, "positions", dev)):
        raise ValueError("q, k, v, positions and slots must have one entry per token")
    with _at(dev, stream):
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=_ROWS)
        else:
            _is(q_out, "q_out", _BF16, dev)
            if q_out.shape != q.shape:
                raise ValueError("q_out must have q's shape")
        st = _bd.lib().bitdelta_kv_append(
            q.data_ptr(), sq[0], sq[1], k.data_ptr(), sk[0], sk[1], v.data_ptr(), sv[0], sv[1],
            positions.data_ptr(), table.data_ptr(), length, rot, interleaved, slots.data_ptr(),
            tokens, heads, kv_heads, dim, pages, page, bits, k_cache.data_ptr(),
            v_cache.data_ptr(), ks, vs, q_out.data_ptr(), _raw_stream(dev))
    if st:
        _fail(st, "bitdelta_kv_append")
    return q_out


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
    pages, kv_heads, page, dim, ks, vs, bits = _cache(k_cache, v_cache, k_scale, v_scale, dev)
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
        call = L.bitdelta_paged_attention_4bit if bits == 4 else L.bitdelta_paged_attention
        st = call(
            q.data_ptr(), s[0], s[1], k_cache.data_ptr(), v_cache.data_ptr(), ks, vs,
            table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), tokens, seqs, max_q, heads,
            kv_heads, dim, pages, page, width, 1.0 / math.sqrt(dim) if scale is None else scale,
            window, out.data_ptr(), wp, wn, _raw_stream(dev))
    if st:
        _fail(st, "bitdelta_paged_attention")
    return out
