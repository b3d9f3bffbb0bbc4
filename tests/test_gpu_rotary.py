"""Rotary positions and the append that rotates on the way into the cache, on
the GPU.

Tolerance of a turned value against 64 bits: two products and a sum in float32
(2^-24 of each), cosine and sine rounded once to float32 (2^-24 more of each
product) and the rounding to bf16, 2^-8 of the value:
2^-8 |r| + 2^-22 (|a| + |b|).  Everything else is compared bit for bit: the
rotation's float32 steps are the plain ones, one rounding each, and a cache's
rows are their one rounding to its type."""

import numpy as np
import pytest
import torch

import oracle.layer as OL
import tenant_linear_layers_amd as T
from helpers import bits16

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
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


def _ints(n, most, seed):
    return torch.randint(0, most, (n,), generator=_gen(seed), device=DEV).int()


def _f64(t):
    return OL.bf16_values(bits16(t))


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _plain(x, positions, table, interleaved):
    """float32 rows by elementary operations, each rounded by itself."""
    x, half = x.float(), table.shape[1]
    c, s = table[positions.long()].unsqueeze(1).unbind(3)
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else \
        (x[..., :half], x[..., half:2 * half])
    first, second = a * c - b * s, b * c + a * s
    turned = torch.stack([first, second], 3).flatten(2) if interleaved else \
        torch.cat([first, second], 2)
    return torch.cat([turned, x[..., 2 * half:]], 2)


# ------------------------------------------------------------------ table
@pytest.mark.parametrize("pairs,first,length,magnitude", [(1, 0, 1, 1.0), (64, 0, 5000, 1.0),
                                                          (37, 131000, 100, 1.2),
                                                          (20, 2 ** 31 - 50, 50, 1.0),
                                                          (32768, 7, 3, 0.5)])
def test_table(pairs, first, length, magnitude):
    """numpy's cosine and sine of the same float64 angle, each within a unit of
    float64's last place, rounded to float32: at most one float32 step apart."""
    f, _ = T.rotary_frequencies(2 * pairs)
    got = T.rotary_table(f, length, first, magnitude).cpu().numpy()
    assert got.shape == (length, pairs, 2) and got.dtype == np.float32
    angle = (first + np.arange(length, dtype=np.float64))[:, None] * f.numpy()
    for k, want in enumerate((np.cos(angle), np.sin(angle))):
        want = want * magnitude
        assert np.all(np.abs(got[..., k] - want) <= np.abs(want) * 2.0 ** -24 * 1.001 + 2e-16)


def test_table_on_the_device_of_a_stream_and_of_no_positions():
    f, _ = T.rotary_frequencies(64)
    want = T.rotary_table(f, 100)
    s = torch.cuda.Stream()
    got = T.rotary_table(f.to(DEV), 100, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(T.rotary_table(f, 30, first=70), want[70:])
    assert T.rotary_table(f, 0).shape == (0, 32, 2)
    with pytest.raises(ValueError):
        T.rotary_table(f, -1)


# ------------------------------------------------------------------ rotation
SHAPES = [
    # tokens, heads, dim, rot
    (1, 1, 2, 2), (1, 64, 128, 128), (3, 2, 128, 64), (5, 3, 80, 80), (7, 1, 96, 24), (2, 5, 64, 2),
    (4, 3, 64, 46), (9, 2, 18, 6), (33, 28, 128, 128), (1, 1, 512, 510), (65, 8, 256, 256),
    (6, 2, 130, 66), (2001, 8, 128, 32), (700, 64, 128, 128), (4096, 64, 64, 64), (3, 2, 65536, 40),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rot", SHAPES)
def test_rotary(tokens, heads, dim, rot, interleaved):
    x = _randn((tokens, heads, dim), tokens + dim + rot)
    f, _ = T.rotary_frequencies(rot)
    table = T.rotary_table(f, 5000)
    pos = _ints(tokens, 5000, rot)
    out = T.rotary(x, pos, table, interleaved)
    assert out.shape == x.shape and out.is_contiguous()
    assert torch.equal(out, _plain(x, pos, table, interleaved).bfloat16())
    n = min(tokens, 200)
    ref = OL.rotary(_f64(x[:n]), pos[:n].cpu().numpy()[:, None] * f.numpy(), interleaved)
    a, half = np.abs(_f64(x[:n])), rot // 2
    both = a.copy()
    u, v = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half),
                                                                     slice(half, rot))
    both[..., u] = both[..., v] = a[..., u] + a[..., v]
    assert np.all(np.abs(_f64(out[:n]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * both)
    # in place, and into a given output
    assert torch.equal(T.rotary(x, pos, table, interleaved, out=torch.empty_like(x)), out)
    assert T.rotary(x, pos, table, interleaved, out=x) is x and torch.equal(x, out)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 32), (80, 60), (64, 14)])
def test_rotary_strided(dim, rot, interleaved):
    """Views of fused rows, heads outermost, rows of an odd alignment; in place
    their neighbours stay as they are."""
    tokens, heads = 19, 6
    table = T.rotary_table(T.rotary_frequencies(rot)[0], 300)
    pos = _ints(tokens, 300, 1)
    wide = _randn((tokens, 3 + (heads + 2) * dim), 2)
    view = wide[:, 3:3 + heads * dim].unflatten(1, (heads, dim))
    want = T.rotary(view.contiguous(), pos, table, interleaved)
    assert torch.equal(T.rotary(view, pos, table, interleaved), want)
    by_head = view.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(T.rotary(by_head, pos, table, interleaved), want)
    out = torch.zeros((heads, tokens, dim), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    assert torch.equal(T.rotary(view, pos, table, interleaved, out=out), want)
    before = wide.clone()
    T.rotary(view, pos, table, interleaved, out=view)
    assert torch.equal(view, want)
    assert torch.equal(wide[:, :3], before[:, :3])
    assert torch.equal(wide[:, 3 + heads * dim:], before[:, 3 + heads * dim:])


def test_rotary_positions_outside_the_table_and_values_that_are_not_finite():
    table = T.rotary_table(T.rotary_frequencies(64)[0], 100)
    x = _randn((6, 2, 128), 3)
    x[5, 1, 3], x[5, 0, 70] = float("inf"), float("nan")
    pos = torch.tensor([0, -1, 100, 99, 2 ** 31 - 1, 5], dtype=torch.int32, device=DEV)
    for inter in (False, True):
        out = T.rotary(x, pos, table, inter)
        assert torch.equal(out[:5, :, 64:], x[:5, :, 64:])
        for t in (1, 2, 4):
            assert bool(torch.isnan(out[t, :, :64]).all())
        for t in (0, 3):
            assert bool(torch.isfinite(out[t]).all())
        bad = ~torch.isfinite(out[5])
        assert bad[1, :64].sum() == 2 and bad[0, :64].sum() == 0 and bad[0, 64:].sum() == 1


def test_rotary_turns_by_differences():
    """Products of turned rows depend on the distance of their positions alone:
    (R_p q) . (R_r k) = (R_(p-r) q) . k, within the roundings to bf16 (2^-8 of each
    product's factors)."""
    f, _ = T.rotary_frequencies(128)
    table = T.rotary_table(f, 4000)
    q, k = _randn((50, 1, 128), 4), _randn((50, 1, 128), 5)
    p, r = _ints(50, 2000, 6) + 2000, _ints(50, 2000, 7)
    a, b = T.rotary(q, p, table), T.rotary(k, r, table)
    c = OL.rotary(_f64(q), (p - r).cpu().numpy()[:, None] * f.numpy())
    size = np.linalg.norm(_f64(q), axis=2) * np.linalg.norm(_f64(k), axis=2)
    off = np.abs((_f64(a) * _f64(b)).sum(2) - (c * _f64(k)).sum(2))
    assert np.all(off <= 2 * (2.0 ** -8 + 2.0 ** -16) * size)


def test_rotary_refusals():
    table = torch.zeros((10, 32, 2), device=DEV)
    x, pos = _randn((3, 2, 64), 1), torch.zeros(3, dtype=torch.int32, device=DEV)
    for bad, kind in ((lambda: T.rotary(x.float(), pos, table), TypeError),
                      (lambda: T.rotary(x[0], pos, table), ValueError),
                      (lambda: T.rotary(x, pos[:2], table), ValueError),
                      (lambda: T.rotary(x, pos.long(), table), TypeError),
                      (lambda: T.rotary(x, pos, table.double()), TypeError),
                      (lambda: T.rotary(x, pos, table[:, :, 0]), ValueError),
                      (lambda: T.rotary(x, pos, table[:0]), ValueError),
                      (lambda: T.rotary(x[..., :62], pos, table), ValueError),
                      (lambda: T.rotary(x, pos, table.cpu()), ValueError),
                      (lambda: T.rotary(x[..., ::2], pos, table), ValueError),
                      (lambda: T.rotary(x, pos, table, out=x[:2]), ValueError),
                      (lambda: T.rotary(x[1:], pos[1:], table, out=x[:2]), T.BitDeltaError),
                      (lambda: T.rotary(x, pos, table, out=x[:1].expand(3, 2, 64)),
                       T.BitDeltaError)):
        with pytest.raises(kind):
            bad()
    assert T.rotary(x[:0], pos[:0], table).shape == (0, 2, 64)


# ------------------------------------------------------------------ append
def _empty(pages, heads, page, dim, bits, fill=3):
    def raw(*shape):
        return torch.full(shape, fill, dtype=torch.uint8, device=DEV)
    rows = (pages, heads, page)
    if bits == 16:
        return [raw(*rows, 2 * dim).view(torch.bfloat16) for _ in range(2)] + [None, None]
    if bits == 8:
        return [raw(*rows, dim).view(torch.float8_e4m3fn) for _ in range(2)] + \
            [raw(*rows).view(torch.float8_e8m0fnu) for _ in range(2)]
    return [raw(*rows, dim // 2).view(torch.float4_e2m1fn_x2) for _ in range(2)] + \
        [raw(*rows, dim // 32).view(torch.float8_e8m0fnu) for _ in range(2)]


APPEND = [
    # tokens, heads, kv_heads, dim, rot, page
    (1, 1, 1, 64, 64, 16), (1, 64, 8, 128, 128, 64), (64, 64, 8, 128, 128, 64),
    (37, 6, 3, 64, 32, 48), (65, 8, 8, 128, 2, 16), (50, 7, 1, 128, 46, 16), (20, 2, 2, 64, 18, 32),
    (9, 4, 2, 128, 34, 16), (2048, 64, 8, 128, 128, 16), (301, 16, 2, 64, 62, 128),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("tokens,heads,kv_heads,dim,rot,page", APPEND)
def test_append(tokens, heads, kv_heads, dim, rot, page, bits, interleaved):
    pages = tokens * 5 // (4 * page) + 2
    row = _randn((tokens, 3 + (heads + 2 * kv_heads) * dim), tokens + dim + rot)
    q, k, v = (t.unflatten(1, (-1, dim)) for t in
               row[:, 3:].split([heads * dim, kv_heads * dim, kv_heads * dim], 1))
    table = T.rotary_table(T.rotary_frequencies(rot)[0], 3000)
    pos = _ints(tokens, 3000, 8)
    slots = torch.randperm(pages * page, generator=_gen(9), device=DEV)[:tokens].int()
    if tokens > 4:
        slots[2], slots[3] = -1, pages * page                        # passed over
        pos[4] = 3000                                                # no such position
    cache, before = _empty(pages, kv_heads, page, dim, bits), _empty(pages, kv_heads, page, dim,
                                                                     bits)
    out = T.kv_append(q, k, v, pos, table, slots, *cache, interleaved=interleaved)
    assert out.is_contiguous()
    want = T.rotary(q, pos, table, interleaved)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) or \
        torch.equal(torch.nan_to_num(out, nan=7.0), torch.nan_to_num(want, nan=7.0))
    safe = pos.clamp(max=2999)
    turned = _plain(k, safe, table, interleaved)
    turned[pos > 2999, :, :rot] = float("nan")
    src = [turned.cpu().double().numpy(), _f64(v)]
    want = [None if c is None else _bytes(c).copy() for c in before]
    live = [(t, s) for t, s in enumerate(slots.cpu().tolist()) if 0 <= s < pages * page]
    ts, p, at = (np.array(i) for i in zip(*[(t, *OL.cache_row(s, page)) for t, s in live]))
    for c in range(2):
        rows = src[c][ts]
        if bits == 16:
            rows = torch.from_numpy(rows).float().bfloat16().view(torch.uint8).numpy()
            want[c][p, :, at] = rows
        else:
            x, s = OL.quantise(rows) if bits == 8 else OL.quantise4(rows)
            want[c][p, :, at], want[2 + c][p, :, at] = x, s
    for c, (got, exp) in enumerate(zip(cache, want)):
        if got is None:
            continue
        got = _bytes(got)
        if bits == 16:
            nan = np.isnan(OL.bf16_values(exp.view(np.uint16)))
            got, exp = got.view(np.uint16), exp.view(np.uint16)
            assert np.isnan(OL.bf16_values(got[nan])).all()
            got, exp = got[~nan], exp[~nan]
        elif bits == 8 and c < 2:
            got, exp = np.where(got & 127 == 127, 127, got), np.where(exp & 127 == 127, 127, exp)
        assert np.array_equal(got, exp)


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_append_without_a_turn_is_a_write(bits):
    """At position 0 nothing turns: the cache is that of kv_write, q is itself."""
    q, k, v = (_randn((33, h, 128), i) for i, h in enumerate((8, 2, 2)))
    table = T.rotary_table(T.rotary_frequencies(128)[0], 1)
    zero = torch.zeros(33, dtype=torch.int32, device=DEV)
    slots = torch.arange(33, dtype=torch.int32, device=DEV)
    one, two = _empty(3, 2, 16, 128, bits), _empty(3, 2, 16, 128, bits)
    assert torch.equal(T.kv_append(q, k, v, zero, table, slots, *one), q)
    T.kv_write(k, v, slots, *two)
    for a, b in zip(one, two):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append_on_streams_and_in_a_graph():
    table = T.rotary_table(T.rotary_frequencies(128)[0], 500)
    q, k, v = (_randn((40, h, 128), i) for i, h in enumerate((8, 2, 2)))
    pos, slots = _ints(40, 500, 3), torch.arange(40, dtype=torch.int32, device=DEV)
    cache = _empty(3, 2, 16, 128, 4)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert T.kv_append(q, k, v, pos, table, slots, *cache, q_out=out, stream=s) is out
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.kv_append(q, k, v, pos, table, slots, *cache, q_out=out)
        turned = T.rotary(q, pos, table, True)
        back = T.kv_read(slots, *cache)
    for i in range(4):
        for t, x in ((q, 10 + i), (k, 20 + i), (v, 30 + i)):
            t.copy_(_randn(tuple(t.shape), x))
        pos.copy_(_ints(40, 500, 40 + i))
        graph.replay()
        torch.cuda.synchronize()
        two = _empty(3, 2, 16, 128, 4)
        assert torch.equal(out, T.kv_append(q, k, v, pos, table, slots, *two))
        assert torch.equal(turned, T.rotary(q, pos, table, True))
        for a, b in zip(back, T.kv_read(slots, *two)):
            assert torch.equal(a, b)


def test_append_refusals():
    table = torch.zeros((10, 32, 2), device=DEV)
    q, k = _randn((3, 4, 64), 1), _randn((3, 2, 64), 2)
    i = torch.zeros(3, dtype=torch.int32, device=DEV)
    c = _empty(2, 2, 16, 64, 16)
    e = _empty(2, 2, 16, 64, 4)
    for bad, kind in ((lambda: T.kv_append(q, k, k, i[:2], table, i, *c), ValueError),
                      (lambda: T.kv_append(q, k, k, i, table, i[:2], *c), ValueError),
                      (lambda: T.kv_append(q[:2], k, k, i, table, i, *c), ValueError),
                      (lambda: T.kv_append(q, k, k[:, :1], i, table, i, *c), ValueError),
                      (lambda: T.kv_append(q, k, k, i.long(), table, i, *c), TypeError),
                      (lambda: T.kv_append(q, k, k, i, table.half(), i, *c), TypeError),
                      (lambda: T.kv_append(q, k, k, i, table, i, *e[:2]), ValueError),
                      (lambda: T.kv_append(q, k, k, i, table, i, *c[:2], *e[2:]), ValueError),
                      (lambda: T.kv_append(q, k, k, i, table, i, *c, q_out=q), T.BitDeltaError),
                      (lambda: T.kv_append(q, k, k, i, table, i, *c, q_out=q[:1]), ValueError),
                      (lambda: T.kv_append(q, k, k, i, torch.zeros((10, 33, 2), device=DEV), i,
                                           *c), ValueError)):
        with pytest.raises(kind):
            bad()
    assert T.kv_append(q[:0], k[:0], k[:0], i[:0], table, i[:0], *e).shape == (0, 4, 64)
