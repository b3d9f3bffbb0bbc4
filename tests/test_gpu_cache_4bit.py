"""The paged cache in 4 bits and attention over it, on the GPU against float64.

The cache is exact: a division by a power of two and one rounding.

Attention's tolerance: the probabilities are rounded to bf16 (2^-8 of each) and
the output too (2^-8 |o|).  The sums are float32.  A score's error is that of the
product, which loses up to 2^-18 of its largest term with each term (together
about 2^-14 of it; terms are below 6 here, 2^-11.4), and of the split of a query
into two 8-bit parts (2^-20 of its largest value to each of its values).  The
probabilities' roundings are within half of 2^-8 on average, and a score's part
is the mean of many keys': 2^-8 |o| + (2^-8 + 2^-12) sum_j p_j |v_j|."""

import threading

import numpy as np
import pytest
import torch

import oracle.layer as OL
import tenant_linear_layers_amd as T
from helpers import bits16

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    T.lib()
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, seed, std=1.36):
    return (torch.randn(shape, generator=_gen(seed), device=DEV) * std).to(torch.bfloat16)


def _f64(t):
    return OL.bf16_values(bits16(t))


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _empty(pages, heads, page, dim, fill=0):
    def raw(*shape):
        return torch.full(shape, fill, dtype=torch.uint8, device=DEV)
    rows = (pages, heads, page)
    return [raw(*rows, dim // 2).view(torch.float4_e2m1fn_x2) for _ in range(2)] + \
        [raw(*rows, dim // 32).view(torch.float8_e8m0fnu) for _ in range(2)]


def _stored(cache):
    return [OL.dequantise4(_bytes(cache[c]), _bytes(cache[2 + c])) for c in range(2)]


# ------------------------------------------------------------------ write, read
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 1, 64, 16), (1, 8, 128, 64), (37, 3, 64, 48),
                                                   (65, 8, 128, 16), (300, 2, 128, 128),
                                                   (2048, 8, 64, 64)])
def test_write_and_read(tokens, heads, dim, page):
    pages = tokens * 5 // (4 * page) + 2
    row = _randn((tokens, (2 * heads + 1) * dim + 3), tokens + dim)
    k = row[:, 3:3 + heads * dim].unflatten(1, (heads, dim))       # rows of an odd alignment
    v = row[:, 3 + heads * dim:3 + 2 * heads * dim].unflatten(1, (heads, dim))
    slots = torch.randperm(pages * page, generator=_gen(1), device=DEV)[:tokens].int()
    if tokens > 4:
        slots[2], slots[3] = -1, pages * page                        # passed over
    cache = _empty(pages, heads, page, dim, fill=0x53)
    want = [_bytes(c).copy() for c in cache]
    T.kv_write(k, v, slots, *cache)
    live = [(t, *OL.cache_row(s, page)) for t, s in enumerate(slots.cpu().tolist())
            if 0 <= s < pages * page]
    ts, p, at = (np.array(i) for i in zip(*live))
    for c, src in enumerate((k, v)):
        want[c][p, :, at], want[2 + c][p, :, at] = OL.quantise4(_f64(src)[ts])
    for got, exp in zip(cache, want):
        assert np.array_equal(_bytes(got), exp)
    back = T.kv_read(slots, *cache)
    for c, rows in enumerate(_stored(cache)):
        assert np.array_equal(_f64(back[c])[ts], rows[p, :, at])
    if tokens > 4:
        assert all(bool(torch.isnan(b[2:4]).all()) for b in back)


def test_write_borders():
    """Groups at the scale's borders, of zeros, infinities and NaN, the type's
    smallest and largest values."""
    big = torch.finfo(torch.bfloat16).max
    rows = [torch.zeros(64), torch.full((64,), -0.0), torch.full((64,), 6.0),
            torch.full((64,), 6.03125), torch.full((64,), 2.0 ** -133), torch.full((64,), big),
            torch.full((64,), -(2.0 ** 122)), torch.linspace(-1, 1, 64),
            torch.linspace(-1e-30, 1e30, 64), torch.linspace(-7.96875, 7.96875, 64)]
    for bad in (float("inf"), float("-inf"), float("nan"), -float("nan")):
        r = torch.linspace(-2, 3, 64)
        r[7] = bad
        rows.append(r)
    k = torch.stack(rows).to(torch.bfloat16).to(DEV).unsqueeze(1)
    n = k.shape[0]
    cache = _empty(1, 1, 16, 64)
    T.kv_write(k, k, torch.arange(n, dtype=torch.int32, device=DEV), *cache)
    q, sb = OL.quantise4(_f64(k))
    assert np.array_equal(_bytes(cache[2])[0, :, :n].transpose(1, 0, 2), sb)
    assert np.array_equal(_bytes(cache[0])[0, :, :n].transpose(1, 0, 2), q)
    back, _ = T.kv_read(torch.arange(n, dtype=torch.int32, device=DEV), *cache)
    assert bool(torch.isnan(back[-1, 0, :32]).all()) and bool(torch.isfinite(back[-1, 0, 32:]).all())
    assert bool(torch.isfinite(back[:-2]).all())


def test_every_value_between_the_codes():
    """All bf16 magnitudes between 2^-4 and 8 beside one value that sets the scale."""
    bits = torch.arange(0x3D80, 0x40C1, dtype=torch.int16)
    x = bits.view(torch.bfloat16)
    x = torch.cat([x, -x, torch.zeros(-2 * len(x) % 31, dtype=torch.bfloat16)]).view(-1, 31)
    x = torch.cat([torch.full((len(x), 1), 6.0, dtype=torch.bfloat16), x], 1)
    x = x.repeat(1, 2).to(DEV).unsqueeze(1)
    pages = -(-len(x) // 16)
    cache = _empty(pages, 1, 16, 64)
    T.kv_write(x, x, torch.arange(len(x), dtype=torch.int32, device=DEV), *cache)
    q, s = OL.quantise4(_f64(x))
    assert np.array_equal(_bytes(cache[1]).reshape(-1, 1, 32)[:len(x)], q) and np.all(s == 127)


@pytest.mark.parametrize("scale", [0, 1, 6, 127, 200, 254, 255])
def test_read_of_bytes_of_other_writers(scale):
    """Every code under every kind of scale byte, as e8m0 says; below bf16's
    smallest value within half of its step."""
    cache = _empty(1, 1, 16, 64)
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).view(1, 1, 8, 32)
    for c in range(2):
        cache[c].view(torch.uint8)[:, :, :8] = codes
        cache[2 + c].view(torch.uint8).fill_(scale)
    k, v = T.kv_read(torch.arange(8, dtype=torch.int32, device=DEV), *cache)
    ref = _stored(cache)[0][0, 0, :8]
    got = _f64(k)[:, 0]
    if scale == 255:
        assert np.isnan(got).all()
    elif scale == 254:                       # 4 and 6 times 2^127 are past bf16's range
        over = np.abs(ref) >= 2.0 ** 128
        assert np.array_equal(got[~over], ref[~over]) and np.isinf(got[over]).all()
    else:
        assert np.all(np.abs(got - ref) <= 2.0 ** -134)
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))


def test_cache_refusals():
    e = _empty(2, 2, 16, 64)
    b = [torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    f = [torch.zeros((2, 2, 16, 32), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
         for _ in range(2)]
    k = _randn((3, 2, 64), 1)
    s = torch.zeros(3, dtype=torch.int32, device=DEV)
    half = [t.view(torch.uint8)[..., :1].contiguous().view(torch.float8_e8m0fnu) for t in e[2:]]
    rows = [t.view(torch.uint8)[..., 0].contiguous().view(torch.float8_e8m0fnu) for t in e[2:]]
    for bad, kind in ((lambda: T.kv_write(k, k, s, *e[:2]), ValueError),
                      (lambda: T.kv_write(k, k, s, *e[:2], e[2]), ValueError),
                      (lambda: T.kv_write(k, k, s, *e[:2], *half), ValueError),
                      (lambda: T.kv_write(k, k, s, *e[:2], *rows), ValueError),
                      (lambda: T.kv_write(k, k, s, e[0], b[1], *e[2:]), TypeError),
                      (lambda: T.kv_write(k, k, s, *b, *e[2:]), ValueError),
                      (lambda: T.kv_write(k, k, s, *f, *e[2:]), ValueError),
                      (lambda: T.kv_write(k, k, s, *(t.view(torch.uint8) for t in e[:2]), *e[2:]),
                       TypeError),
                      (lambda: T.kv_write(k, k, s, *e[:2], *(t.view(torch.uint8) for t in e[2:])),
                       TypeError),
                      (lambda: T.kv_write(_randn((3, 2, 32), 1), k, s, *e), ValueError),
                      (lambda: T.kv_read(s, e[0].transpose(1, 2), e[1], *e[2:]), ValueError),
                      (lambda: T.kv_read(s.long(), *e), TypeError)):
        with pytest.raises(kind):
            bad()
    k0, v0 = T.kv_read(s[:0], *e)
    assert k0.shape == (0, 2, 64) and v0.shape == (0, 2, 64)


# ------------------------------------------------------------------ attention
def _problem(new, kv, heads, kv_heads, dim, page, seed=0, std=1.36, spare=3):
    """A filled cache whose unused rows hold NaN, and a page table whose unused
    entries are out of range."""
    need = [-(-m // page) for m in kv]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((len(kv), max(max(need), 1) + 1), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = _empty(pages, kv_heads, page, dim, fill=0xFF)
    slots = torch.tensor([int(table[b, j // page]) * page + j % page
                          for b, m in enumerate(kv) for j in range(m)], dtype=torch.int32,
                         device=DEV)
    T.kv_write(_randn((len(slots), kv_heads, dim), seed + 1, std),
               _randn((len(slots), kv_heads, dim), seed + 2, std), slots, *cache)
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
    return dict(q=_randn((sum(new), heads, dim), seed + 3, std), cache=cache, table=table, cu=cu,
                kv=torch.tensor(kv, dtype=torch.int32), max_q=max(new))


def _call(p, **more):
    return T.paged_attention(p["q"], p["cache"][0], p["cache"][1], p["table"].to(DEV),
                             p["cu"].to(DEV), p["kv"].to(DEV), p["max_q"],
                             k_scale=p["cache"][2], v_scale=p["cache"][3], **more)


def _reference(p, k=None, v=None, **more):
    if k is None:
        k, v = _stored(p["cache"])
    ref, mag = OL.paged_attention(_f64(p["q"]), k, v, p["table"].numpy(), p["cu"].tolist(),
                                  p["kv"].tolist(), **more)
    # A weight below float32's smallest normal number, 2^-126, may be taken for 0: where
    # the heaviest keys' values are 0, as many of 4 bits are, that is all there is.
    least = 2.0 ** -126 * p["kv"].max().item() * np.max(np.abs(v), initial=0.0,
                                                       where=np.isfinite(v))
    return ref, 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * mag + least


def _check(p, out, **more):
    ref, tol = _reference(p, **more)
    got = _f64(out)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.size} values off, the first at "
                           f"{np.argwhere(bad)[0].tolist()}: {got[bad][0]} for {ref[bad][0]}")


ATTEND = [
    # new tokens, cached keys, heads, kv_heads, dim, page, window
    ([1], [1], 1, 1, 64, 16, 0),
    ([1], [1], 8, 1, 128, 16, 0),
    ([1, 1, 1], [15, 16, 17], 8, 2, 128, 16, 0),
    ([1, 1, 1, 1], [31, 32, 33, 127], 4, 2, 64, 16, 0),
    ([1, 1, 1, 1], [63, 64, 65, 97], 4, 2, 128, 16, 0),
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
    ([1], [9000], 2, 1, 64, 16, 0),                    # many pieces of a row
    ([1], [5000], 64, 1, 128, 64, 0),                  # one token of more rows than 16
    ([1] * 150, [(37 * i) % 211 + 1 for i in range(150)], 4, 1, 64, 16, 0),
    ([1] * 70, [(97 * i) % 900 + 1 for i in range(69)] + [6000], 2, 1, 128, 16, 0),
    ([1 + i % 3 for i in range(130)], [(53 * i) % 300 + 3 for i in range(130)], 4, 2, 64, 32, 40),
    ([40 * (i % 9 == 0) + i % 2 for i in range(100)],
     [40 + (71 * i) % 400 for i in range(100)], 2, 1, 128, 16, 0),
    ([300], [3000], 1, 1, 128, 16, 1700),
]


@pytest.mark.parametrize("new,kv,heads,kv_heads,dim,page,window", ATTEND)
def test_attention(new, kv, heads, kv_heads, dim, page, window):
    p = _problem(new, kv, heads, kv_heads, dim, page, seed=sum(kv) + heads)
    out = _call(p, window=window)
    assert out.shape == p["q"].shape and out.dtype == torch.bfloat16
    _check(p, out, window=window)


def test_attention_large_scores():
    """Scores of some hundred: one key takes all the weight of most rows, and
    the running maximum moves often."""
    p = _problem([1, 20], [900, 333], 8, 1, 128, 16, seed=5, std=6.0)
    _check(p, _call(p))
    p = _problem([70], [700], 8, 2, 64, 16, seed=6, std=6.0)
    _check(p, _call(p, window=333), window=333)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_query_of_very_different_values(dim, new):
    """Dims of a query 2^16 apart, the small ones against keys that are large
    there: what is left of the smallest values after the split still counts."""
    p = _problem([new], [200], 4, 2, dim, 16, seed=8, std=1.0)
    size = torch.ones(dim, device=DEV)
    size[dim // 2:] = 2.0 ** -12
    p["q"] = (p["q"].float() * size).bfloat16()
    k, v = _randn((200, 2, dim), 9, 1.0), _randn((200, 2, dim), 10, 1.0)
    k[:, :, dim // 2:] *= 2.0 ** 12
    j = torch.arange(200, device=DEV)
    slots = (p["table"][0].to(DEV)[j // 16] * 16 + j % 16).int()
    T.kv_write(k, v, slots, *p["cache"])
    # the split leaves 2^-20 of a row's largest value (5) to each of dim / 2 values against
    # keys of up to 2^12 * 5: 2^-20 * 5 * dim / 2 * 2^12 * 5 / sqrt(dim) is the score's error
    score = 2.0 ** -20 * 5 * dim / 2 * 2.0 ** 12 * 5 / dim ** 0.5
    ref, tol = _reference(p)
    _, mag = OL.paged_attention(_f64(p["q"]), *_stored(p["cache"]), p["table"].numpy(),
                                p["cu"].tolist(), p["kv"].tolist())
    assert np.all(np.abs(_f64(_call(p)) - ref) <= tol + np.expm1(2 * score) * mag)


def test_attention_given_scale_strides_output_and_workspace():
    p = _problem([1, 9], [100, 200], 8, 2, 128, 16, seed=7)
    wide = _randn((10, 8 * 128 + 5 + 64), 8)
    p["q"] = wide[:, 5:5 + 1024].unflatten(1, (8, 128))           # rows of an odd alignment
    out = torch.empty((10, 8, 128), dtype=torch.bfloat16, device=DEV)
    n = T.paged_attention_workspace_size(10, 2, 9, 8, 2, 128, p["table"].shape[1], 16)
    ws = torch.full((n + 16,), 0xFF, dtype=torch.uint8, device=DEV)
    assert _call(p, scale=0.05, out=out, workspace=ws) is out
    _check(p, out, scale=0.05)
    p["q"] = _randn((8, 10, 128), 9).transpose(0, 1)               # heads outermost
    _check(p, _call(p))


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_bad_page_is_that_sequences_nan(new, dim):
    p = _problem([new, new, new], [200, 200, 200], 8, 2, dim, 16, seed=11)
    first = _call(p)
    _check(p, first)
    for bad in (-1, p["cache"][0].shape[0], 2 ** 31 - 1):
        table = p["table"].clone()
        table[1, 3] = bad
        out = _call(dict(p, table=table))
        assert torch.equal(out[:new], first[:new]) and torch.equal(out[2 * new:], first[2 * new:])
        assert bool(torch.isnan(out[new:2 * new]).all())


def test_attention_lengths_past_the_table_are_held():
    p = _problem([1], [64], 8, 2, 64, 16, seed=12)
    p["table"] = p["table"][:, :4].contiguous()
    want = _call(p)
    p["kv"] = torch.tensor([10 ** 9], dtype=torch.int32)
    assert torch.equal(_call(p), want)


def test_attention_rows_behind_the_last_sequence_stay():
    p = _problem([1, 20], [40, 50], 8, 2, 128, 16, seed=16)
    out = torch.full_like(p["q"], 3.0)
    p["cu"] = torch.tensor([0, 1, 12], dtype=torch.int32)
    _call(p, out=out)
    assert bool((out[12:] == 3.0).all()) and not bool((out[:12] == 3.0).all())


def test_attention_repeats_bit_for_bit_and_in_a_graph():
    p = _problem([1, 1, 30], [3000, 100, 900], 16, 2, 128, 16, seed=13)
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


def test_attention_refusals():
    p = _problem([1, 1], [20, 20], 4, 2, 64, 16, seed=14)
    q, c = p["q"], p["cache"]
    t, cu, kv = p["table"].to(DEV), p["cu"].to(DEV), p["kv"].to(DEV)
    for bad, kind in ((lambda: T.paged_attention(q, *c[:2], t, cu, kv, 1), ValueError),
                      (lambda: T.paged_attention(q, *c[:2], t, cu, kv, 1, c[2]), ValueError),
                      (lambda: T.paged_attention(q[..., :32], *c[:2], t, cu, kv, 1, *c[2:]),
                       ValueError),
                      (lambda: T.paged_attention(q.float(), *c[:2], t, cu, kv, 1, *c[2:]),
                       TypeError),
                      (lambda: T.paged_attention(q, *c[:2], t, cu, kv, 1, *c[2:], out=q),
                       T.BitDeltaError),
                      (lambda: T.paged_attention(q, *c[:2], t, cu, kv, 1, *c[2:], scale=0.0),
                       T.BitDeltaError)):
        with pytest.raises(kind):
            bad()
    assert T.paged_attention(q[:0], *c[:2], t[:0], cu[:1], kv[:0], 0, *c[2:]).shape == (0, 4, 64)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 40, 64, 31, 32])
def test_attention_windows_wider_than_any_sequence(window):
    p = _problem([4, 40, 1], [2, 25, 31], 8, 2, 64, 16, seed=15)
    _check(p, _call(p, window=window), window=min(window, 10 ** 6))


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
def test_attention_nan_groups_stay_with_those_who_see_them(new, kv, heads, kv_heads, dim, page,
                                                           window, key):
    """A group of a value row that is NaN reaches the rows that see its key, in
    its dims, one of a key row the rows that see it: no others."""
    p = _problem(new, kv, heads, kv_heads, dim, page, seed=21)
    at = (int(p["table"][0, key // page]), key % page)
    pos = np.concatenate([np.arange(n) + m - n for n, m in zip(new, kv)])
    first = np.arange(sum(new)) < new[0]
    sees = first & (key <= pos) & ((pos - key < window) if window else True)
    assert sees.any() and not sees.all()
    for which, dims in ((1, np.arange(32, 64)), (0, np.arange(dim))):
        s = p["cache"][2 + which].view(torch.uint8)
        was = s.clone()
        s[at[0], :, at[1], 1] = 255
        k, v = (np.nan_to_num(x, nan=0.0) for x in _stored(p["cache"]))
        ref, tol = _reference(p, k, v, window=window)
        got = _f64(_call(p, window=window))
        hit = np.zeros(got.shape, bool)
        hit[np.ix_(np.flatnonzero(sees), np.arange(heads), dims)] = True
        assert np.isnan(got[hit]).all()
        bad = ~hit & ~(np.abs(got - ref) <= tol)
        assert not bad.any(), f"{int(bad.sum())} values off, first {np.argwhere(bad)[0].tolist()}"
        s.copy_(was)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_queries_that_are_not_finite_are_their_rows_own(new, dim):
    p = _problem([new, new], [100, 90], 8, 2, dim, 16, seed=23)
    want = _call(p)
    for value in (float("nan"), float("inf")):
        q = p["q"].clone()
        q[0, 3, 5] = value
        got = _call(dict(p, q=q))
        hit = torch.zeros(got.shape[:2], dtype=torch.bool, device=DEV)
        hit[0, 3] = True
        assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("k_scale,v_scale", [(0, 0), (7, 200), (127, 0), (100, 247), (0, 254)])
def test_attention_over_scales_of_other_writers(new, dim, k_scale, v_scale):
    """Scale bytes that this library's writes seldom or never make; weights of
    zero stay zero whatever the value's scale is.  bf16's smallest step, 2^-133, is
    what a value below its normal range may be off by."""
    p = _problem([new], [50], 4, 2, dim, 16, seed=24)
    for c, b in ((2, k_scale), (3, v_scale)):
        live = p["cache"][c].view(torch.uint8)
        live[live != 255] = b
    got = _f64(_call(p))
    k, v = _stored(p["cache"])
    if v_scale == 254:
        v = np.where(np.abs(v) >= 2.0 ** 128, np.sign(v) * np.inf, v)
        assert not np.isfinite(got).all()
        return
    ref, tol = _reference(p)
    assert np.all(np.abs(got - ref) <= tol + 2.0 ** -133)


def _definition(p):
    """(out, sum of probability times |v|) in float64, a sequence and head at a
    time, from the values that the cache holds."""
    q, heads, dim, page = p["q"].double(), p["q"].shape[1], p["q"].shape[2], p["cache"][0].shape[2]
    kv_heads, table = p["cache"][0].shape[1], p["table"].to(DEV)
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    for b, m in enumerate(p["kv"].tolist()):
        first, last = p["cu"][b:b + 2].tolist()
        j = torch.arange(m, device=DEV)
        slots = (table[b][j // page] * page + j % page).int()
        k, v = (x.double() for x in T.kv_read(slots, *p["cache"]))
        i = torch.arange(m - (last - first), m, device=DEV).unsqueeze(1)
        for h in range(heads):
            kk, vv = (x[:, h * kv_heads // heads].contiguous() for x in (k, v))
            z = (q[first:last, h].contiguous() @ kk.t().contiguous()) / dim ** 0.5
            w = torch.softmax(z.masked_fill(j > i, float("-inf")), 1)
            out[first:last, h] = w @ vv
            mag[first:last, h] = w @ vv.abs()
    return out, mag


@pytest.mark.parametrize("new,kv,heads,kv_heads,dim", [
    ([1600], [1600], 16, 2, 128),
    ([1000], [2100], 32, 8, 64),
    ([700, 900], [700, 900], 16, 2, 64),
    ([2048], [2048], 32, 4, 128),
    ([2048], [2048], 64, 8, 64),
    ([2011], [2011], 64, 8, 128),
    ([509], [6000], 64, 8, 128),
    ([1] * 40, [8000 - 150 * i for i in range(40)], 64, 8, 128),
])
def test_attention_of_rounds_of_tiles(new, kv, heads, kv_heads, dim):
    p = _problem(new, kv, heads, kv_heads, dim, 16, seed=25)
    ref, mag = _definition(p)
    bad = (_call(p).double() - ref).abs() > \
        2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * mag
    assert not bool(bad.any()), f"{int(bad.sum())} values off"


@pytest.mark.parametrize("new,kv,heads,kv_heads,dim", [
    ([1] * 20, [100 + 37 * i for i in range(20)], 8, 2, 128),
    ([1, 1, 2], [4000, 1500, 90], 8, 4, 64),
    ([40, 70], [300, 900], 8, 2, 128),
    ([200], [1000], 8, 1, 64),
])
def test_attention_over_one_value_gives_that_value(new, kv, heads, kv_heads, dim):
    """The weights, as the product with V takes them, add up to one (float32's
    roundings are far below half a step of 1.5); scores of some tens."""
    p = _problem(new, kv, heads, kv_heads, dim, 16, seed=91)
    p["q"] = (p["q"].float() * 8).to(torch.bfloat16)
    p["cache"][1].view(torch.uint8).fill_(0x33)            # 1.5
    p["cache"][3].view(torch.uint8).fill_(127)
    off = _call(p) != 1.5
    assert not bool(off.any()), f"{int(off.sum())} of {off.numel()} values off"


@pytest.mark.parametrize("new,kv,heads,kv_heads,dim", [
    ([1, 1, 1], [3000, 700, 5], 8, 2, 128),
    ([1] * 90, [300 + 40 * i for i in range(90)], 4, 4, 64),
    ([33], [4000], 8, 2, 128),
    ([200], [5000], 8, 1, 64),
    ([1, 90, 1, 3, 300, 17], [2500, 900, 40, 3000, 2048, 1000], 8, 2, 128),
])
def test_attention_keeps_to_a_workspace_of_the_size_asked_for(new, kv, heads, kv_heads, dim):
    p = _problem(new, kv, heads, kv_heads, dim, 16, seed=11)
    n = T.paged_attention_workspace_size(len(p["q"]), len(kv), p["max_q"], heads, kv_heads, dim,
                                         p["table"].shape[1], 16)
    assert n > 0
    big = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
    out = _call(p, workspace=big[4096:4096 + n])
    assert torch.equal(out, _call(p))
    assert bool((big[:4096] == 0xA5).all()) and bool((big[4096 + n:] == 0xA5).all())
    with pytest.raises(T.BitDeltaError):
        _call(p, workspace=big[4096:4096 + n - 16])


def test_cache_rows_and_query_strides_past_32_bits():
    """Rows of a cache that lie beyond 2^32 bytes, scales beyond 2^28, queries
    beyond 2^31 elements."""
    heads, page, dim = 8, 64, 128
    pages = 2 ** 32 // (heads * page * dim // 2) + 40
    cache = [torch.empty((pages, heads, page, dim // 2), dtype=torch.uint8, device=DEV)
             .view(torch.float4_e2m1fn_x2) for _ in range(2)]
    cache += [torch.empty((pages, heads, page, 4), dtype=torch.uint8, device=DEV)
              .view(torch.float8_e8m0fnu) for _ in range(2)]
    new, kv = [1, 40], [150, 90]
    small = _problem(new, kv, 8, heads, dim, page, seed=41)
    table = pages - 1 - torch.arange(small["table"].numel(), dtype=torch.int32).view(
        small["table"].shape)
    for b, m in enumerate(kv):
        def slots(t):
            t = t[b].to(DEV)
            j = torch.arange(m, device=DEV)
            return (t[j // page] * page + j % page).int()
        k, v = T.kv_read(slots(small["table"]), *small["cache"])
        T.kv_write(k, v, slots(table), *cache)
        for x, y in zip((k, v), T.kv_read(slots(table), *cache)):
            assert torch.equal(x, y)
    want = _call(small)
    _check(small, want)
    # Rows written from the values read have those values, but where a group's
    # largest code was 3 or less in other codes under half the scale, and the
    # product that adds them rounds otherwise: bits are compared for rows of the
    # same bytes.
    _check(small, _call(dict(small, cache=cache, table=table)))
    for b, m in enumerate(kv):
        j = torch.arange(-(-m // page))
        near, far = small["table"][b, j].to(DEV), table[b, j].to(DEV)
        for x, y in zip(small["cache"], cache):
            y.view(torch.uint8)[far.long()] = x.view(torch.uint8)[near.long()]
    assert torch.equal(_call(dict(small, cache=cache, table=table)), want)
    stride = 2 ** 31 // 40 + 8
    q = torch.empty(40 * stride + 8 * dim, dtype=torch.bfloat16, device=DEV)
    q = q.as_strided((41, 8, dim), (stride, dim, 1))
    q.copy_(small["q"])
    assert torch.equal(_call(dict(small, q=q)), want)


def test_calls_on_streams_of_several_threads_at_once():
    problems = [_problem([1, 40, 3], [700, 400, 2000], 8, 2, d, 16, seed=s)
                for d, s in ((128, 71), (64, 81), (128, 91))]
    want = [_call(p) for p in problems]
    torch.cuda.synchronize()
    got = [None] * len(problems)

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got[i] = [_call(problems[i]) for _ in range(5)]
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(problems))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for many, w in zip(got, want):
        assert all(torch.equal(g, w) for g in many)
