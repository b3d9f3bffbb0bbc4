"""Rotary positions, the rotating append and the 4-bit cache where a call has more
threads than one launch takes, and calls that run beside each other.  Bits are
compared: what a row holds does not depend on what the test changes."""

import pytest
import torch

import tenant_linear_layers_amd as T

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    T.lib()
    yield
    torch.cuda.empty_cache()          # these tests hold up to 40 GB


def _randn(shape, seed, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _picked(rows, part):
    """Rows at the ends of the parts that a call's rows are launched in."""
    at = {0, 1, rows - 2, rows - 1}
    for p in range(part, rows, part):
        at |= {p - 1, p, p + 1}
    return torch.tensor(sorted(at), device=DEV)


def _empty(pages, heads, page, dim):
    rows = (pages, heads, page)
    return [torch.zeros((*rows, dim // 2), dtype=torch.uint8, device=DEV)
            .view(torch.float4_e2m1fn_x2) for _ in range(2)] + \
        [torch.zeros((*rows, dim // 32), dtype=torch.uint8, device=DEV)
         .view(torch.float8_e8m0fnu) for _ in range(2)]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_of_more_tokens_than_a_launch_takes(interleaved):
    """A thread a token, 2^30 in a launch.  The rows of neighbouring tokens
    overlap in memory."""
    tokens = 2 ** 30 + 5
    at = _picked(tokens, 2 ** 30)
    flat = _randn((tokens // 2 ** 10 + 2,), 1)
    x = flat.repeat(2 ** 10)[:tokens + 1].as_strided((tokens, 1, 2), (1, 2, 1))
    pos = torch.zeros((tokens,), dtype=torch.int32, device=DEV)
    pos[at] = torch.arange(len(at), dtype=torch.int32, device=DEV) * 3
    table = T.rotary_table(T.rotary_frequencies(2)[0], 100)
    out = T.rotary(x, pos, table, interleaved)
    assert torch.equal(out[at], T.rotary(x[at], pos[at], table, interleaved))
    assert torch.equal(out[5:1000], x[5:1000])            # position 0


def test_append_of_more_tokens_than_a_launch_takes():
    """Eight threads a token.  All but a few of the tokens' slots are passed over."""
    tokens, dim = 2 ** 27 + 5, 64
    at = _picked(tokens, 2 ** 27)
    n = len(at)
    q, k, v = (_randn((2 ** 17 + dim,), i, 1.4).repeat(2 ** 10)[:tokens + dim]
               .as_strided((tokens, 1, dim), (1, dim, 1)) for i in (2, 3, 4))
    slots = torch.full((tokens,), -1, dtype=torch.int32, device=DEV)
    slots[at] = torch.arange(n, dtype=torch.int32, device=DEV)
    pos = torch.arange(tokens, device=DEV, dtype=torch.int32) % 500
    table = T.rotary_table(T.rotary_frequencies(dim)[0], 500)
    cache, few = _empty(1, 1, 16, dim), _empty(1, 1, 16, dim)
    out = T.kv_append(q, k, v, pos, table, slots, *cache)
    want = T.kv_append(q[at], k[at], v[at], pos[at], table, slots[at], *few)
    assert torch.equal(out[at], want)
    for a, b in zip(cache, few):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_attention_of_more_pieces_than_a_launch_takes():
    """A workgroup of 256 threads per sequence and head: more than 2^32 threads.
    All sequences read the same few pages; lengths of one page are never cut."""
    heads, dim, page, pages = 1024, 64, 16, 7
    part = 2 ** 31 // 256 // heads
    seqs = 2 * part + 5
    cache = _empty(pages, heads, page, dim)
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


def test_cache_calls_of_more_tokens_than_a_launch_takes():
    heads, dim, step = 1024, 128, 8
    part = 2 ** 30 // (heads * dim // 8)
    tokens = 2 * part + 5
    at = _picked(tokens, part)
    k, v = (_randn((tokens * step + heads * dim,), i, 1.4)
            .as_strided((tokens, heads, dim), (step, dim, 1)) for i in (4, 5))
    slots = torch.full((tokens,), -1, dtype=torch.int32, device=DEV)
    slots[at] = torch.arange(len(at), dtype=torch.int32, device=DEV)
    cache, few = _empty(1, heads, 16, dim), _empty(1, heads, 16, dim)
    T.kv_write(k, v, slots, *cache)
    T.kv_write(k[at], v[at], slots[at], *few)
    for a, b in zip(cache, few):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for got, want in zip(T.kv_read(slots, *cache), T.kv_read(slots[at], *cache)):
        assert torch.equal(got[at], want)
        assert bool(torch.isnan(got[at[1] + 1]).all())        # a slot outside the cache


def _layer_calls(seed, dim, heads, kv_heads):
    """What a layer does between its linears, as a function of a stream."""
    n = 90
    q, k, v = (_randn((n, h, dim), seed + i, 1.4)
               for i, h in enumerate((heads, kv_heads, kv_heads)))
    x, r, g = (_randn((n, 1024), seed + 3 + i, 1.4) for i in range(3))
    w = _randn((1024,), seed + 6, 0.1) + 1.0
    table = T.rotary_table(T.rotary_frequencies(dim)[0], 200)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    cache = _empty(6, kv_heads, 16, dim)
    pages = torch.arange(6, dtype=torch.int32, device=DEV).unsqueeze(0)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    kv = torch.tensor([n], dtype=torch.int32, device=DEV)

    def run(stream=None):
        a = T.kv_append(q, k, v, pos, table, pos, *cache, stream=stream)
        back = T.kv_read(pos, *cache, stream=stream)
        o = T.paged_attention(a, *cache[:2], pages, cu, kv, n, *cache[2:], stream=stream)
        t = T.rotary(k, pos, table, True, stream=stream)
        y, h = T.rms_norm_block(x, r, w, w, 1e-5, g, 0.5, stream=stream)
        return [a, *back, o, t, y, h]

    return run


def test_calls_on_two_streams_at_once():
    runs = [_layer_calls(31, 128, 16, 2), _layer_calls(51, 64, 64, 64)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [[run(s) for run, s in zip(runs, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for one in got:
        for a, b in zip(one, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_step_in_a_graph():
    run = _layer_calls(71, 128, 64, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
