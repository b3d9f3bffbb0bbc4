"""The decoder-layer operators on the GPU against their float64 oracle.

Tolerances, each derived from the roundings on the way (half a step: 2^-8 of
the value in bf16, 2^-4 in e4m3, 2^-24 in float32):

* h: one float32 addition and a rounding to bf16, 2^-8 + 2^-24 of the value.
* y in bf16: that rounding and float32 steps before it (a sum of squares whose
  relative error is below 2^-18, a root, two products): 2^-8 + 2^-17.
* y in 8 bits: half an e4m3 step, 2^-4 of the value or, among the subnormals,
  2^-10 of the scale; plus 2^-17 of the value.  A scale may be the other
  neighbour only where the group's largest value is within 2^-17 of a border.
* the cache is exact: a division by a power of two and one rounding.
* attention: the probabilities are rounded to bf16 (2^-8 of each), scores and
  sums are float32 (below 2^-13 in the probabilities for the sizes here), the
  output to bf16: 2^-8 |o| + (2^-8 + 2^-12) sum_j p_j |v_j|.
"""

import numpy as np
import pytest
import torch

import oracle.layer as OL
import tenant_linear_layers_amd as T
from helpers import bits16

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    T.lib()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, seed, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=_gen(seed), device=DEV) * std).to(dtype)


def _f64(t):
    return OL.bf16_values(bits16(t))


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


# ------------------------------------------------------------------ norm
NORM_SHAPES = [(1, 1), (3, 7), (5, 8), (2, 33), (7, 100), (4, 511), (9, 512), (3, 520), (2, 1023),
               (5, 1024), (3, 1032), (4, 2048), (2, 2049), (3, 4096), (2, 4097), (3, 8191),
               (1, 8192), (2, 8193), (700, 8192), (2, 16384), (2, 16385), (1, 30001),
               (1030, 96), (1500, 2056)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_rms_norm(rows, cols, residual):
    x = _randn((rows, cols), rows + cols, 1.4)
    w = _randn((cols,), 3, 0.1) + 1.0
    r = _randn((rows, cols), 5, 3.0) if residual else None
    y, h = T.rms_norm(x, w, EPS, r)
    ref, href = OL.rms_norm(_f64(x), _f64(w), EPS, _f64(r) if residual else None)
    assert np.all(np.abs(_f64(y) - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -17))
    if residual:
        assert np.all(np.abs(_f64(h) - href) <= np.abs(href) * (2.0 ** -8 + 2.0 ** -24))
    else:
        assert h is None


def _check_mx(q, scale, ref):
    rows, cols = ref.shape
    g = ref.reshape(rows, -1, 32)
    sb = _bytes(scale).reshape(rows, -1)
    amax = np.abs(g).max(-1)
    lo = OL.scale_exponent(amax * (1 - 2.0 ** -17)) + 127
    hi = OL.scale_exponent(amax * (1 + 2.0 ** -17)) + 127
    assert np.all((sb == lo) | (sb == hi))
    got = OL.dequantise(_bytes(q).reshape(g.shape), sb)
    step = np.exp2(sb.astype(np.float64) - 127)[..., None]
    tol = np.maximum(np.abs(g) * 2.0 ** -4, step * 2.0 ** -10) + np.abs(g) * 2.0 ** -17
    assert np.all(np.abs(got - g) <= tol)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (5, 480), (2, 544), (3, 1024), (2, 2080),
                                       (3, 4096), (1, 8192), (600, 8192), (2, 16384), (2, 16416),
                                       (1030, 96)])
def test_rms_norm_mx(rows, cols, residual):
    x = _randn((rows, cols), rows * 3 + cols, 1.4)
    w = _randn((cols,), 4, 0.1) + 1.0
    r = _randn((rows, cols), 6, 3.0) if residual else None
    q, scale, h = T.rms_norm_mx(x, w, EPS, r)
    assert q.dtype == torch.float8_e4m3fn and scale.dtype == torch.float8_e8m0fnu
    assert scale.shape == (rows, cols // 32)
    ref, href = OL.rms_norm(_f64(x), _f64(w), EPS, _f64(r) if residual else None)
    _check_mx(q, scale, ref)
    if residual:
        assert np.all(np.abs(_f64(h) - href) <= np.abs(href) * (2.0 ** -8 + 2.0 ** -24))


def test_rms_norm_mx_groups_of_zero_and_of_very_different_size():
    x = _randn((2, 256), 8)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    w[32:64] = 0.0
    w[64:96] = 2.0 ** -100
    w[96:128] = 2.0 ** 100
    q, scale, _ = T.rms_norm_mx(x, w, EPS)
    ref, _ = OL.rms_norm(_f64(x), _f64(w), EPS)
    _check_mx(q, scale, ref)
    assert np.all(_bytes(scale)[:, 1] == 7) and np.all(_bytes(q)[:, 32:64] & 127 == 0)


def test_rms_norm_strided_rows_and_leading_dims():
    big = _randn((9, 3 * 1024 + 40), 9)
    x, r = big[:, 8:1032], big[:, 1033:2057]            # the second starts on an odd element
    w = _randn((1024,), 10, 0.1) + 1.0
    y, h = T.rms_norm(x, w, EPS, r)
    y2, h2 = T.rms_norm(x.contiguous(), w, EPS, r.contiguous())
    assert torch.equal(y, y2) and torch.equal(h, h2)
    y3, h3 = T.rms_norm(x.contiguous().view(3, 3, 1024), w, EPS, r.contiguous().view(3, 3, 1024))
    assert y3.shape == (3, 3, 1024) and torch.equal(y3.view(9, 1024), y)
    q, s, _ = T.rms_norm_mx(x, w, EPS, r)
    q2, s2, _ = T.rms_norm_mx(x.contiguous(), w, EPS, r.contiguous())
    assert np.array_equal(_bytes(q), _bytes(q2)) and np.array_equal(_bytes(s), _bytes(s2))


def test_rms_norm_no_rows_outputs_given_and_refusals():
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    x = _randn((4, 64), 11)
    y, h = T.rms_norm(x[:0], w, EPS, x[:0])
    assert y.shape == (0, 64) and h.shape == (0, 64)
    y, h = torch.empty_like(x), torch.empty_like(x)
    y1, h1 = T.rms_norm(x, w, EPS, x.clone(), y=y, h=h)
    assert y1 is y and h1 is h
    for bad, kind in ((lambda: T.rms_norm(x, w[:32], EPS), ValueError),
                      (lambda: T.rms_norm(x, w.float(), EPS), TypeError),
                      (lambda: T.rms_norm(x, w, EPS, x[:2]), ValueError),
                      (lambda: T.rms_norm(x.t(), w[:4], EPS), ValueError),
                      (lambda: T.rms_norm(x, w, EPS, h=h), ValueError),
                      (lambda: T.rms_norm(x, w, EPS, x.clone(), h=x), T.BitDeltaError),
                      (lambda: T.rms_norm_mx(x[:, :48], w[:48], EPS), ValueError)):
        with pytest.raises(kind):
            bad()


def test_rms_norm_non_finite_rows_stay_their_own():
    x = _randn((4, 4096), 12)
    x[1, 17] = float("nan")
    x[2, 18] = float("inf")
    w = torch.ones(4096, dtype=torch.bfloat16, device=DEV)
    y, _ = T.rms_norm(x, w, EPS)
    ref, _ = OL.rms_norm(_f64(x[[0, 3]]), _f64(w), EPS)
    assert np.all(np.abs(_f64(y[[0, 3]]) - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -17))
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[2, 18]))


# ------------------------------------------------------------------ cache
def _empty_cache(pages, heads, page, dim, q8, fill=0):
    if not q8:
        c = [torch.full((pages, heads, page, dim), float(fill), dtype=torch.bfloat16, device=DEV)
             for _ in range(2)]
        return (*c, None, None)
    c = [torch.full((pages, heads, page, dim), fill, dtype=torch.uint8, device=DEV)
         .view(torch.float8_e4m3fn) for _ in range(2)]
    s = [torch.full((pages, heads, page), fill, dtype=torch.uint8, device=DEV)
         .view(torch.float8_e8m0fnu) for _ in range(2)]
    return (*c, *s)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 1, 64, 16), (1, 8, 128, 64), (37, 3, 64, 48),
                                                   (65, 8, 128, 16), (300, 2, 128, 128)])
def test_kv_write_and_read(tokens, heads, dim, page, q8):
    pages = tokens * 5 // (4 * page) + 2
    row = _randn((tokens, (2 * heads + 1) * dim + 3), tokens + dim, 1.4)
    k = row[:, 3:3 + heads * dim].unflatten(1, (heads, dim))       # rows of an odd alignment
    v = row[:, 3 + heads * dim:3 + 2 * heads * dim].unflatten(1, (heads, dim))
    slots = torch.randperm(pages * page, generator=_gen(1), device=DEV)[:tokens].int()
    if tokens > 4:
        slots[2], slots[3] = -1, pages * page                        # passed over
    cache = _empty_cache(pages, heads, page, dim, q8, fill=3)
    before = [None if c is None else _bytes(c).copy() for c in cache]
    T.kv_write(k, v, slots, *cache)
    want = [None if c is None else c.copy() for c in before]
    src = (_f64(k), _f64(v))
    raw = (bits16(k), bits16(v))
    for t, s in enumerate(slots.cpu().tolist()):
        if not 0 <= s < pages * page:
            continue
        p, at = OL.cache_row(s, page)
        for c in range(2):
            if q8:
                q, sb = OL.quantise(src[c][t])
                want[c][p, :, at], want[2 + c][p, :, at] = q, sb
            else:
                want[c].view(np.uint16)[p, :, at] = raw[c][t]
    for got, exp in zip(cache, want):
        if got is not None:
            assert np.array_equal(_bytes(got), exp)
    back = T.kv_read(slots, *cache)
    for c in range(2):
        for t, s in enumerate(slots.cpu().tolist()):
            if not 0 <= s < pages * page:
                assert bool(torch.isnan(back[c][t]).all())
                continue
            if q8:
                p, at = OL.cache_row(s, page)
                ref = OL.dequantise(want[c][p, :, at], want[2 + c][p, :, at])
                assert np.array_equal(_f64(back[c][t]), ref)
            else:
                assert torch.equal(back[c][t], (k, v)[c][t])


def test_kv_write_8bit_borders():
    """Rows at the scale's borders, of zeros, infinities and NaN, the type's
    smallest and largest values."""
    big = torch.finfo(torch.bfloat16).max
    rows = [torch.zeros(64), torch.full((64,), 448.0), torch.full((64,), 450.0),
            torch.full((64,), 2.0 ** -133), torch.full((64,), big),
            torch.linspace(-1, 1, 64), torch.linspace(-1e-30, 1e30, 64)]
    for bad in (float("inf"), float("-inf"), float("nan")):
        r = torch.linspace(-2, 3, 64)
        r[7] = bad
        rows.append(r)
    k = torch.stack(rows).to(torch.bfloat16).to(DEV).unsqueeze(1)
    n = k.shape[0]
    cache = _empty_cache(1, 1, 16, 64, True)
    T.kv_write(k, k, torch.arange(n, dtype=torch.int32, device=DEV), *cache)
    q, sb = OL.quantise(_f64(k))
    got = _bytes(cache[0])[0, :, :n].transpose(1, 0, 2)
    assert np.array_equal(_bytes(cache[2])[0, :, :n].transpose(1, 0), sb)
    nan = (q & 127) == 127
    assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], q[~nan])


def test_kv_refusals():
    c = _empty_cache(2, 2, 16, 64, False)
    e = _empty_cache(2, 2, 16, 64, True)
    k = _randn((3, 2, 64), 1)
    s = torch.zeros(3, dtype=torch.int32, device=DEV)
    for bad, kind in ((lambda: T.kv_write(k, k, s.long(), *c), TypeError),
                      (lambda: T.kv_write(k, k[:2], s, *c), ValueError),
                      (lambda: T.kv_write(k[:, :1], k, s, *c), ValueError),
                      (lambda: T.kv_write(k, k, s, c[0], c[1], e[2], e[3]), ValueError),
                      (lambda: T.kv_write(k, k, s, e[0], e[1]), ValueError),
                      (lambda: T.kv_write(k, k, s, c[0], e[1]), TypeError),
                      (lambda: T.kv_read(s, c[0].transpose(1, 2), c[1]), ValueError),
                      (lambda: T.kv_read(s, c[0], c[1].transpose(1, 2)), ValueError),
                      (lambda: T.kv_read(s, c[0][..., :32].contiguous(), c[1]), ValueError),
                      (lambda: T.kv_read(s, c[0][:, :, :8].contiguous(), c[1]), ValueError)):
        with pytest.raises(kind):
            bad()
    k0, v0 = T.kv_read(s[:0], *c)
    assert k0.shape == (0, 2, 64) and v0.shape == (0, 2, 64)
    T.kv_write(k[:0], k[:0], s[:0], *c)


# ------------------------------------------------------------------ attention
def _problem(new, kv, heads, kv_heads, dim, page, q8, seed=0, std=1.36, spare=3):
    """A filled cache whose unused rows hold NaN (and, in 8 bits, scales of
    any size), and a page table whose unused entries are out of range."""
    need = [-(-m // page) for m in kv]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=_gen(seed), device=DEV).int().cpu()
    width = max(max(need), 1) + 1
    table = torch.full((len(kv), width), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = _empty_cache(pages, kv_heads, page, dim, q8, fill=float("nan") if not q8 else 0xFF)
    slots = torch.tensor([int(table[b, j // page]) * page + j % page
                          for b, m in enumerate(kv) for j in range(m)],
                         dtype=torch.int32, device=DEV)
    k = _randn((len(slots), kv_heads, dim), seed + 1, std)
    v = _randn((len(slots), kv_heads, dim), seed + 2, std)
    T.kv_write(k, v, slots, *cache)
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
    q = _randn((sum(new), heads, dim), seed + 3, std)
    return dict(q=q, cache=cache, table=table, cu=cu, kv=torch.tensor(kv, dtype=torch.int32),
                max_q=max(new))


def _call(p, **more):
    return T.paged_attention(p["q"], p["cache"][0], p["cache"][1], p["table"].to(DEV),
                             p["cu"].to(DEV), p["kv"].to(DEV), p["max_q"],
                             k_scale=p["cache"][2], v_scale=p["cache"][3], **more)


def _stored(cache):
    out = []
    for c in range(2):
        if cache[2] is None:
            out.append(_f64(cache[c]))
        else:
            out.append(OL.dequantise(_bytes(cache[c]), _bytes(cache[2 + c])))
    return out


def _check(p, out, **more):
    k, v = _stored(p["cache"])
    ref, mag = OL.paged_attention(_f64(p["q"]), k, v, p["table"].numpy(), p["cu"].tolist(),
                                  p["kv"].tolist(), **more)
    got = _f64(out)
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * mag
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} values off, the first at "
                           f"{np.argwhere(bad)[0].tolist()}: {got[bad][0]} for {ref[bad][0]}")


ATTEND = [
    # new tokens, cached keys, heads, kv_heads, dim, page, window
    ([1], [1], 1, 1, 64, 16, 0),
    ([1], [1], 8, 1, 128, 16, 0),
    ([1, 1, 1], [15, 16, 17], 8, 2, 128, 16, 0),
    ([1, 1, 1, 1], [31, 32, 33, 127], 4, 2, 64, 16, 0),
    ([1, 1], [128, 129], 16, 2, 128, 64, 0),
    ([1, 1, 1], [700, 3, 2500], 8, 1, 128, 32, 0),
    ([1, 1], [1000, 77], 14, 2, 64, 48, 0),
    ([1, 1, 1], [500, 501, 40], 8, 2, 128, 16, 100),
    ([1, 1], [64, 65], 8, 2, 64, 64, 1),
    ([2, 1, 5], [2, 300, 90], 8, 1, 128, 16, 0),
    ([3, 4], [200, 201], 7, 1, 64, 32, 0),
    ([17], [17], 8, 2, 128, 16, 0),
    ([64], [64], 8, 2, 64, 16, 0),
    ([100], [228], 8, 1, 128, 64, 0),
    ([130, 1, 33], [130, 400, 600], 4, 1, 128, 32, 0),
    ([40, 90], [400, 90], 8, 2, 64, 16, 50),
    ([65, 1], [300, 299], 16, 4, 128, 16, 17),
    ([257], [300], 2, 2, 128, 128, 0),
    ([33], [700], 64, 1, 64, 16, 0),
    ([1, 0, 2], [20, 33, 40], 8, 2, 128, 16, 0),       # a sequence with no new tokens
    ([4, 1], [2, 0], 8, 2, 128, 16, 0),                # rows that see no key
    ([40, 3], [25, 0], 4, 1, 64, 16, 8),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("new,kv,heads,kv_heads,dim,page,window", ATTEND)
def test_paged_attention(new, kv, heads, kv_heads, dim, page, window, q8):
    p = _problem(new, kv, heads, kv_heads, dim, page, q8, seed=sum(kv) + heads)
    out = _call(p, window=window)
    assert out.shape == p["q"].shape and out.dtype == torch.bfloat16
    _check(p, out, window=window)


@pytest.mark.parametrize("q8", [False, True])
def test_paged_attention_large_scores(q8):
    """Scores of some hundred: one key takes all the weight of most rows, and
    the running maximum moves often."""
    p = _problem([1, 20], [900, 333], 8, 1, 128, 16, q8, seed=5, std=6.0)
    _check(p, _call(p))
    p = _problem([70], [700], 8, 2, 64, 16, q8, seed=6, std=6.0)
    _check(p, _call(p, window=333), window=333)


def test_paged_attention_given_scale_strides_output_and_workspace():
    p = _problem([1, 9], [100, 200], 8, 2, 128, 16, False, seed=7)
    wide = _randn((10, 8 * 128 + 5 + 64), 8)
    p["q"] = wide[:, 5:5 + 1024].unflatten(1, (8, 128))           # rows of an odd alignment
    out = torch.empty((10, 8, 128), dtype=torch.bfloat16, device=DEV)
    n = T.paged_attention_workspace_size(10, 2, 9, 8, 2, 128, p["table"].shape[1], 16)
    ws = torch.full((n + 16,), 0xFF, dtype=torch.uint8, device=DEV)
    assert _call(p, scale=0.05, out=out, workspace=ws) is out
    _check(p, out, scale=0.05)
    by_head = _randn((8, 10, 128), 9).transpose(0, 1)               # heads outermost
    p["q"] = by_head
    _check(p, _call(p))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("new", [1, 40])
def test_paged_attention_bad_page_is_that_sequences_nan(q8, new):
    p = _problem([new, new, new], [200, 200, 200], 8, 2, 128, 16, q8, seed=11)
    _check(p, _call(p))
    for bad in (-1, p["cache"][0].shape[0], 2 ** 31 - 1):
        table = p["table"].clone()
        table[1, 3] = bad
        out = _call(dict(p, table=table))
        first = _call(p)
        assert torch.equal(out[:new], first[:new]) and torch.equal(out[2 * new:], first[2 * new:])
        assert bool(torch.isnan(out[new:2 * new]).all())


def test_paged_attention_lengths_past_the_table_are_held():
    p = _problem([1], [64], 8, 2, 64, 16, False, seed=12)
    p["table"] = p["table"][:, :4].contiguous()
    want = _call(p)
    p["kv"] = torch.tensor([10 ** 9], dtype=torch.int32)
    assert torch.equal(_call(p), want)


def test_paged_attention_repeats_bit_for_bit_and_in_a_graph():
    p = _problem([1, 1, 30], [3000, 100, 900], 16, 2, 128, 16, True, seed=13)
    args = (p["q"], p["cache"][0], p["cache"][1], p["table"].to(DEV), p["cu"].to(DEV),
            p["kv"].to(DEV), p["max_q"])
    more = dict(k_scale=p["cache"][2], v_scale=p["cache"][3])
    first = T.paged_attention(*args, **more)
    for _ in range(3):
        assert torch.equal(T.paged_attention(*args, **more), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        T.paged_attention(*args, **more)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = T.paged_attention(*args, **more)
    for i in range(4):
        p["q"].copy_(_randn(tuple(p["q"].shape), 20 + i))
        want = T.paged_attention(*args, **more)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = T.paged_attention(*args, stream=other, **more)
    other.synchronize()
    assert torch.equal(got, want)


def test_paged_attention_refusals():
    p = _problem([1, 1], [20, 20], 4, 2, 64, 16, False, seed=14)
    q, c = p["q"], p["cache"]
    t, cu, kv = p["table"].to(DEV), p["cu"].to(DEV), p["kv"].to(DEV)
    for bad, kind in ((lambda: T.paged_attention(q.float(), c[0], c[1], t, cu, kv, 1), TypeError),
                      (lambda: T.paged_attention(q[:, :3], c[0], c[1], t, cu, kv, 1), ValueError),
                      (lambda: T.paged_attention(q, c[0], c[1], t[:1], cu, kv, 1), ValueError),
                      (lambda: T.paged_attention(q, c[0], c[1], t, cu[:2], kv, 1), ValueError),
                      (lambda: T.paged_attention(q, c[0], c[1], t.long(), cu, kv, 1), TypeError),
                      (lambda: T.paged_attention(q, c[0], c[1], t, cu, kv, -1), ValueError),
                      (lambda: T.paged_attention(q, c[0], c[1], t, cu, kv, 1, window=-1),
                       ValueError),
                      (lambda: T.paged_attention(q, c[0], c[1], t, cu, kv, 1, out=q),
                       T.BitDeltaError),
                      (lambda: T.paged_attention(q[..., ::2], c[0], c[1], t, cu, kv, 1),
                       ValueError)):
        with pytest.raises(kind):
            bad()
    none = T.paged_attention(q[:0], c[0], c[1], t[:0], cu[:1], kv[:0], 0)
    assert none.shape == (0, 4, 64)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 40, 64, 31, 32])
def test_paged_attention_windows_wider_than_any_sequence(window):
    """A window hides nothing from a sequence that does not fill it, also where
    the sequence's first rows stand before key 0 and see none."""
    p = _problem([4, 40, 1], [2, 25, 31], 8, 2, 64, 16, False, seed=15)
    _check(p, _call(p, window=window), window=min(window, 10 ** 6))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("new,kv,heads,kv_heads,dim,page,window,key", [
    ([3, 2], [40, 9], 4, 1, 64, 16, 0, 38),
    ([3, 2], [40, 9], 4, 1, 128, 16, 0, 39),
    ([4, 1], [300, 70], 4, 2, 128, 16, 100, 198),
    ([40, 5], [40, 20], 8, 2, 128, 16, 0, 17),
    ([40, 5], [40, 20], 8, 2, 64, 16, 0, 31),
    ([70], [700], 8, 2, 64, 64, 0, 650),
    ([70, 1], [400, 3], 8, 1, 128, 32, 90, 300),
    ([260], [300], 16, 16, 128, 16, 50, 250),
])
def test_paged_attention_non_finite_rows_stay_with_those_who_see_them(new, kv, heads, kv_heads,
                                                                      dim, page, window, key, q8):
    """NaN and infinities in a value row reach the rows that see its key, in
    their dims, and NaN in a key row the rows that see it: no others."""
    p = _problem(new, kv, heads, kv_heads, dim, page, q8, seed=21)
    at = (int(p["table"][0, key // page]), key % page)
    pos = np.concatenate([np.arange(n) + m - n for n, m in zip(new, kv)])
    first = np.arange(sum(new)) < new[0]
    sees = first & (key <= pos) & ((pos - key < window) if window else True)
    assert sees.any() and not sees.all()
    nan8 = torch.tensor([0x7F], dtype=torch.uint8, device=DEV)

    def poison(c, dims, value):
        if q8:
            c.view(torch.uint8)[at[0], :, at[1], dims] = nan8
        else:
            c[at[0], :, at[1], dims] = value

    def check(out, dims):
        k, v = _stored(p["cache"])
        k, v = np.nan_to_num(k, nan=0.0, posinf=0.0, neginf=0.0), np.nan_to_num(
            v, nan=0.0, posinf=0.0, neginf=0.0)
        ref, mag = OL.paged_attention(_f64(p["q"]), k, v, p["table"].numpy(), p["cu"].tolist(),
                                      p["kv"].tolist(), window=window)
        got = _f64(out)
        hit = np.zeros(got.shape, bool)
        hit[np.ix_(np.flatnonzero(sees), np.arange(heads), dims)] = True
        assert not np.isfinite(got[hit]).any()
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * mag
        bad = ~hit & ~(np.abs(got - ref) <= tol)
        assert not bad.any(), f"{int(bad.sum())} values off, first {np.argwhere(bad)[0].tolist()}"

    clean = [c.clone() if c is not None else None for c in p["cache"]]
    for value in (float("nan"), float("inf"), float("-inf")):
        poison(p["cache"][1], slice(5, dim - 3), value)
        check(_call(p, window=window), np.arange(5, dim - 3))
    p["cache"] = tuple(clean)
    poison(p["cache"][0], slice(7, 9), float("nan"))
    check(_call(p, window=window), np.arange(dim))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("new,kv,heads,kv_heads,dim,page,window", [
    ([1], [9000], 2, 1, 64, 16, 0),                          # more pieces than a join reads at once
    ([1], [5000], 64, 1, 128, 64, 0),                        # one token of more rows than 16
    ([1] * 150, [(37 * i) % 211 + 1 for i in range(150)], 4, 1, 64, 16, 0),
    ([1] * 70, [(97 * i) % 900 + 1 for i in range(69)] + [6000], 2, 1, 128, 16, 0),
    ([1 + i % 3 for i in range(130)], [(53 * i) % 300 + 3 for i in range(130)], 4, 2, 64, 32, 40),
    ([40 * (i % 9 == 0) + i % 2 for i in range(100)],
     [40 + (71 * i) % 400 for i in range(100)], 2, 1, 128, 16, 0),
    ([300], [3000], 1, 1, 128, 16, 1700),
])
def test_paged_attention_long_and_many_sequences(new, kv, heads, kv_heads, dim, page, window, q8):
    p = _problem(new, kv, heads, kv_heads, dim, page, q8, seed=31)
    _check(p, _call(p, window=window), window=window)


@pytest.mark.parametrize("q8", [False, True])
def test_cache_rows_and_query_strides_past_32_bits(q8):
    """Rows of a cache that lie beyond 2^32 bytes, queries beyond 2^31 elements."""
    heads, page, dim = 8, 64, 128
    pages = 2 ** 32 // (heads * page * dim * (1 if q8 else 2)) + 40
    kind = torch.float8_e4m3fn if q8 else torch.bfloat16
    cache = [torch.empty((pages, heads, page, dim), dtype=kind, device=DEV) for _ in range(2)]
    cache += [torch.empty((pages, heads, page), dtype=torch.float8_e8m0fnu, device=DEV)
              for _ in range(2)] if q8 else [None, None]
    new, kv = [1, 40], [150, 90]
    small = _problem(new, kv, 8, heads, dim, page, q8, seed=41)
    table = pages - 1 - torch.arange(small["table"].numel(), dtype=torch.int32).view(
        small["table"].shape)
    for b, m in enumerate(kv):
        def slots(t):
            t = t[b].to(DEV)
            j = torch.arange(m, device=DEV)
            return (t[j // page] * page + j % page).int()
        k, v = T.kv_read(slots(small["table"]), *small["cache"])
        T.kv_write(k, v, slots(table), *cache)
        k2, v2 = T.kv_read(slots(table), *cache)
        assert torch.equal(k, k2) and torch.equal(v, v2)
    want = _call(small)
    _check(small, want)
    assert torch.equal(_call(dict(small, cache=cache, table=table)), want)
    stride = 2 ** 31 // 40 + 8
    q = torch.empty(40 * stride + 8 * dim, dtype=torch.bfloat16, device=DEV)
    q = q.as_strided((41, 8, dim), (stride, dim, 1))
    q.copy_(small["q"])
    assert torch.equal(_call(dict(small, q=q)), want)


def test_rms_norm_of_more_than_2_to_31_values():
    rows, cols = 2 ** 31 // 8192 + 3, 8192
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    x[-5:] = _randn((5, cols), 51, 1.4)
    w = _randn((cols,), 52, 0.1) + 1.0
    for call in (lambda x: T.rms_norm(x, w, EPS, x)[:2],
                 lambda x: [t.view(torch.uint8) for t in T.rms_norm_mx(x, w, EPS)[:2]]):
        for big, few in zip(call(x), call(x[-5:].clone())):
            assert torch.equal(big[-5:], few)


def test_paged_attention_of_no_sequences_or_rows():
    p = _problem([2, 1], [20, 20], 16, 1, 64, 16, False, seed=61)
    q, c = p["q"], p["cache"]
    t, cu, kv = p["table"].to(DEV), p["cu"].to(DEV), p["kv"].to(DEV)
    out = torch.full_like(q, 3.0)
    for args in ((t[:0], cu[:1], kv[:0], 2), (t, cu, kv, 0)):
        assert T.paged_attention(q, c[0], c[1], *args, out=out) is out
        assert bool((out == 3.0).all())                     # rows that no sequence has


def test_caches_of_no_heads_or_pages_are_refused():
    s = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = _randn((1, 4, 64), 62)
    for shape in ((2, 0, 16, 64), (0, 2, 16, 64)):
        c = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
        with pytest.raises(ValueError):
            T.kv_read(s, c, c.clone())
        with pytest.raises(ValueError):
            T.paged_attention(q, c, c.clone(), s.view(1, 1), torch.zeros(2, dtype=torch.int32,
                                                                         device=DEV), s, 1)
