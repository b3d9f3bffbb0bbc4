"""The decoder-layer operators on the GPU where their sizes meet a limit: calls
of more threads than one launch takes, workspaces of exactly the size asked
for, tiles in about one round of the card, and calls that run beside each other.

Where no tolerance is given bits are compared: what a row holds, or how a
sequence is cut, does not depend on what the test changes."""

import threading

import pytest
import torch

import tenant_linear_layers_amd as T

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-5


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    T.lib()
    yield
    torch.cuda.empty_cache()          # these tests hold up to 90 GB


def _randn(shape, seed, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


# ------------------------------------------------------------------ launches
def _picked(rows, part):
    """Rows at the ends of the parts that a call's rows are launched in."""
    at = {0, 1, rows - 2, rows - 1}
    for p in range(part, rows, part):
        at |= {p - 1, p, p + 1}
    return torch.tensor(sorted(at), device=DEV)


@pytest.mark.parametrize("rows,cols,threads", [(2 ** 26 + 5, 32, 64), (2 ** 22 + 3, 4128, 1024)])
def test_rms_norm_of_more_rows_than_a_launch_takes(rows, cols, threads):
    """threads * rows passes 2^32.  Whole numbers: their squares add up exactly,
    in whatever order the threads of a row take them."""
    at = _picked(rows, 2 ** 31 // threads)
    w = _randn((cols,), 2, 0.1) + 1.0
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    x[at] = _randn((len(at), cols), 3, 1.4).round()
    y, _ = T.rms_norm(x, w, EPS)
    want, _ = T.rms_norm(x[at], w, EPS)
    assert torch.equal(y[at], want)
    del y
    few = T.rms_norm_mx(x[at], w, EPS, x[at])
    for got, want in zip(T.rms_norm_mx(x, w, EPS, x), few):
        assert torch.equal(got.view(torch.uint8)[at], want.view(torch.uint8))


@pytest.mark.parametrize("q8", [False, True])
def test_cache_calls_of_more_tokens_than_a_launch_takes(q8):
    """Eight values a thread: 2 * tokens * heads * dim / 8 passes 2^32.  The rows
    of neighbouring tokens overlap in memory, and all but a few of the tokens are
    passed over."""
    heads, dim, page, step = 1024, 128, 16, 8
    part = 2 ** 31 // (2 * heads * dim // 8)
    tokens = 2 * part + 5
    at = _picked(tokens, part)
    n = len(at)
    kind = torch.float8_e4m3fn if q8 else torch.bfloat16
    cache = [torch.zeros((1, heads, page, dim), dtype=kind, device=DEV) for _ in range(2)]
    cache += [torch.zeros((1, heads, page), dtype=torch.uint8, device=DEV)
              .view(torch.float8_e8m0fnu) for _ in range(2)] if q8 else [None, None]
    k, v = (_randn((tokens * step + heads * dim,), i, 1.4)
            .as_strided((tokens, heads, dim), (step, dim, 1)) for i in (4, 5))
    slots = torch.full((tokens,), -1, dtype=torch.int32, device=DEV)
    slots[at] = torch.arange(n, dtype=torch.int32, device=DEV)
    T.kv_write(k, v, slots, *cache)
    few = [None if c is None else torch.zeros_like(c) for c in cache]
    T.kv_write(k[at], v[at], slots[at], *few)
    for got, want in zip(cache, few):
        if got is not None:
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    want = T.kv_read(slots[at], *cache)
    for got, exp in zip(T.kv_read(slots, *cache), want):
        assert torch.equal(got[at], exp)
        assert bool(torch.isnan(got[at[1] + 1]).all())        # a slot outside the cache


@pytest.mark.parametrize("q8", [False, True])
def test_attention_of_more_pieces_than_a_launch_takes(q8):
    """A workgroup of 256 threads per sequence and head: more than 2^32 threads.
    All sequences read the same few pages; lengths of one page are never cut."""
    heads, dim, page = 1024, 64, 16
    part = 2 ** 31 // 256 // heads
    seqs = 2 * part + 5
    pages = 7
    kind = torch.float8_e4m3fn if q8 else torch.bfloat16
    cache = [torch.zeros((pages, heads, page, dim), dtype=kind, device=DEV) for _ in range(2)]
    cache += [torch.zeros((pages, heads, page), dtype=torch.uint8, device=DEV)
              .view(torch.float8_e8m0fnu) for _ in range(2)] if q8 else [None, None]
    rows = pages * page
    T.kv_write(_randn((rows, heads, dim), 6), _randn((rows, heads, dim), 7),
               torch.arange(rows, dtype=torch.int32, device=DEV), *cache)
    at = _picked(seqs, part)
    q = _randn((seqs, heads, dim), 8)
    i = torch.arange(seqs, device=DEV, dtype=torch.int32)
    table, kv = (i % pages).unsqueeze(1), 1 + i * 5 % page
    cu = torch.arange(seqs + 1, device=DEV, dtype=torch.int32)
    out = T.paged_attention(q, *cache[:2], table, cu, kv, 1, *cache[2:])
    want = T.paged_attention(q[at], *cache[:2], table[at], cu[:len(at) + 1], kv[at], 1, *cache[2:])
    assert torch.equal(out[at], want)


# ------------------------------------------------------------------ workspaces
def _serving(new, kv, heads, kv_heads, dim, page, q8, seed):
    """The arguments of a call over a filled cache."""
    need = [-(-m // page) for m in kv]
    table = torch.full((len(kv), max(need)), -1, dtype=torch.int32)
    order, at = torch.randperm(sum(need), generator=torch.Generator().manual_seed(seed)), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    rows = sum(need) * page
    shape = (sum(need), kv_heads, page, dim)
    kind = torch.float8_e4m3fn if q8 else torch.bfloat16
    cache = [torch.empty(shape, dtype=kind, device=DEV) for _ in range(2)]
    cache += [torch.empty(shape[:3], dtype=torch.float8_e8m0fnu, device=DEV)
              for _ in range(2)] if q8 else [None, None]
    T.kv_write(_randn((rows, kv_heads, dim), seed, 1.4), _randn((rows, kv_heads, dim), seed + 1),
               torch.arange(rows, dtype=torch.int32, device=DEV), *cache)
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEV)
    return dict(q=_randn((sum(new), heads, dim), seed + 2, 1.4), k_cache=cache[0],
                v_cache=cache[1], table=table.to(DEV), cu_q=cu,
                kv_len=torch.tensor(kv, dtype=torch.int32, device=DEV), max_q=max(new),
                k_scale=cache[2], v_scale=cache[3])


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("new,kv,heads,kv_heads,dim", [
    ([1, 1, 1], [3000, 700, 5], 8, 2, 128),                  # few rows
    ([1] * 90, [300 + 40 * i for i in range(90)], 4, 4, 64),
    ([33], [4000], 8, 2, 128),                               # many rows, tiles of 64 and of 128
    ([200], [5000], 8, 1, 64),
    ([1, 90, 1, 3, 300, 17], [2500, 900, 40, 3000, 2048, 1000], 8, 2, 128),    # both in a call
])
def test_attention_keeps_to_a_workspace_of_the_size_asked_for(new, kv, heads, kv_heads, dim, q8):
    p = _serving(new, kv, heads, kv_heads, dim, 16, q8, 11)
    n = T.paged_attention_workspace_size(len(p["q"]), len(kv), p["max_q"], heads, kv_heads, dim,
                                         p["table"].shape[1], 16)
    assert n > 0
    big = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
    out = T.paged_attention(**p, workspace=big[4096:4096 + n])
    assert torch.equal(out, T.paged_attention(**p))
    assert bool((big[:4096] == 0xA5).all()) and bool((big[4096 + n:] == 0xA5).all())
    with pytest.raises(T.BitDeltaError):
        T.paged_attention(**p, workspace=big[4096:4096 + n - 16])


# ------------------------------------------------------------------ tiles of many rows
def _definition(p):
    """(out, sum of probability times |v|) in float64, a sequence and head at a
    time, from the values that the cache holds."""
    q, heads, dim = p["q"].double(), p["q"].shape[1], p["q"].shape[2]
    _, kv_heads, page, _ = p["k_cache"].shape
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    for b, m in enumerate(p["kv_len"].tolist()):
        first, last = p["cu_q"][b:b + 2].tolist()
        j = torch.arange(m, device=DEV)
        slots = (p["table"][b][j // page] * page + j % page).int()
        k, v = (x.double() for x in T.kv_read(slots, p["k_cache"], p["v_cache"], p["k_scale"],
                                              p["v_scale"]))
        i = torch.arange(m - (last - first), m, device=DEV).unsqueeze(1)
        for h in range(heads):
            kk, vv = (x[:, h * kv_heads // heads].contiguous() for x in (k, v))
            z = (q[first:last, h].contiguous() @ kk.t().contiguous()) / dim ** 0.5
            w = torch.softmax(z.masked_fill(j > i, float("-inf")), 1)
            out[first:last, h] = w @ vv
            mag[first:last, h] = w @ vv.abs()
    return out, mag


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("new,kv,heads,kv_heads,dim", [
    ([1600], [1600], 16, 2, 128),        # tiles of 64 rows, cut: 200 tiles of 128, half a round
    ([1000], [2100], 32, 8, 64),         # the same where the new tokens are just half of the keys
    ([700, 900], [700, 900], 16, 2, 64),
    ([2048], [2048], 32, 4, 128),        # tiles of 64 rows, not cut: two rounds of them
    ([2048], [2048], 32, 4, 64),
    ([2048], [2048], 64, 8, 64),         # tiles of 128 rows, not cut
    ([2011], [2011], 64, 8, 128),        # and a little short of that
])
def test_attention_of_rounds_of_tiles(new, kv, heads, kv_heads, dim, q8):
    """Tolerance: probabilities rounded to bf16 (2^-8 of each), scores and sums in
    float32 (below 2^-13 of the probabilities), the output rounded to bf16."""
    p = _serving(new, kv, heads, kv_heads, dim, 16, q8, 21)
    ref, mag = _definition(p)
    bad = (T.paged_attention(**p).double() - ref).abs() > \
        2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * mag
    assert not bool(bad.any()), f"{int(bad.sum())} values off"


# ------------------------------------------------------------------ calls beside each other
def _layer_calls(seed, q8):
    """What a layer does between its linears, as a function of a stream."""
    p = _serving([1, 40, 3], [700, 400, 2000], 8, 2, 128, 16, q8, seed)
    x, r = _randn((44, 1024), seed + 3, 1.4), _randn((44, 1024), seed + 4, 3.0)
    w = _randn((1024,), seed + 5, 0.1) + 1.0
    k, v = _randn((44, 2, 128), seed + 6), _randn((44, 2, 128), seed + 7)
    cache = [c if c is None else torch.zeros_like(c[:4])
             for c in (p["k_cache"], p["v_cache"], p["k_scale"], p["v_scale"])]
    slots = torch.randperm(64, generator=torch.Generator().manual_seed(seed))[:44].int().to(DEV)

    def run(stream=None):
        y, h = T.rms_norm(x, w, EPS, r, stream=stream)
        q, s, _ = T.rms_norm_mx(x, w, EPS, r, stream=stream)
        T.kv_write(k, v, slots, *cache, stream=stream)
        back = T.kv_read(slots, *cache, stream=stream)
        o = T.paged_attention(**p, stream=stream)
        return [t.view(torch.uint8) for t in (y, h, q, s, *back, o)]

    return run


def test_calls_on_two_streams_at_once():
    runs = [_layer_calls(31, False), _layer_calls(51, True)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [[run(s) for run, s in zip(runs, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for one in got:
        for a, b in zip(one, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_calls_from_several_threads_at_once():
    runs = [_layer_calls(71 + 20 * i, i % 2 == 1) for i in range(4)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    got = [None] * len(runs)

    def work(i):
        s = torch.cuda.Stream()
        got[i] = [runs[i](s) for _ in range(5)]
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(runs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for many, b in zip(got, want):
        for a in many:
            assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------ weights
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("new,kv,heads,kv_heads,dim", [
    ([1] * 20, [100 + 37 * i for i in range(20)], 8, 2, 128),      # few rows
    ([1, 1, 2], [4000, 1500, 90], 8, 4, 64),                       # cut into pieces
    ([40, 70], [300, 900], 8, 2, 128),                             # many rows
    ([200], [1000], 8, 1, 64),
])
def test_attention_over_one_value_gives_that_value(new, kv, heads, kv_heads, dim, q8):
    """The weights, as the product with V takes them, add up to one: float32's
    roundings are far below half a step of the result, which is next to a power of
    two, where the steps are smallest.  Scores of some tens, so that of most rows
    one key has most of the weight, and seldom a weight of one."""
    p = _serving(new, kv, heads, kv_heads, dim, 16, q8, 91)
    p["q"] = (p["q"].float() * 8).to(torch.bfloat16)
    value = 1.875 if q8 else 1.9921875
    rows = p["v_cache"].shape[0] * 16
    T.kv_write(_randn((rows, kv_heads, dim), 91, 1.4),
               torch.full((rows, kv_heads, dim), value, dtype=torch.bfloat16, device=DEV),
               torch.arange(rows, dtype=torch.int32, device=DEV), p["k_cache"], p["v_cache"],
               p["k_scale"], p["v_scale"])
    out = T.paged_attention(**p)
    off = out != value
    assert not bool(off.any()), f"{int(off.sum())} of {off.numel()} values off"
