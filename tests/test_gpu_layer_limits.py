"""The decoder-layer operators on the GPU where their sizes meet a limit: calls
of more threads than one launch takes, workspaces of exactly the size asked
for, and calls that run beside each other.

Comparisons are of bits: a row, or a sequence's plan, does not depend on what
the test changes."""

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
    torch.cuda.empty_cache()          # these tests hold up to 70 GB


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
