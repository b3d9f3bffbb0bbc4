"""Attention over the 4-bit cache where a call's rows are many: more than 192 tiles
of 16 rows and key/value heads, so that sequences of more than 32 rows (new tokens
times the query heads of a key/value head) take tiles of 64 or 128 rows, beside
those of fewer in the same launch.  Problems, tolerances and the meaning of each
test are those of test_gpu_cache_4bit.py."""

import numpy as np
import pytest
import torch

import test_gpu_cache_4bit as base
from test_gpu_cache_4bit import DEV, _call, _check, _definition, _f64, _gpu, _problem  # noqa: F401

import tenant_linear_layers_amd as T

pytestmark = pytest.mark.gpu

ATTEND = [
    # new tokens, cached keys, heads, kv_heads, dim, page, window
    ([33], [33], 128, 128, 64, 16, 0),
    ([40], [340], 128, 128, 128, 16, 0),
    ([64, 1], [64, 70], 128, 64, 64, 16, 0),
    ([100], [228], 64, 64, 128, 64, 0),
    ([130, 1, 33], [130, 400, 600], 64, 32, 128, 32, 0),
    ([40, 90], [400, 90], 128, 64, 64, 16, 50),
    ([65, 1], [300, 299], 128, 64, 128, 16, 17),
    ([257], [300], 32, 32, 128, 128, 0),
    ([257], [300], 32, 32, 64, 16, 0),
    ([33, 2, 1], [700, 31, 65], 256, 16, 64, 16, 0),
    ([40, 0, 50], [60, 33, 50], 64, 64, 128, 16, 0),   # a sequence with no new tokens
    ([40, 3], [25, 0], 128, 64, 64, 16, 8),            # rows that see no key
    ([40, 3], [25, 0], 128, 64, 128, 16, 0),
    ([40 * (i % 9 == 0) + i % 2 for i in range(100)],
     [40 + (71 * i) % 400 for i in range(100)], 8, 4, 128, 16, 0),
    ([300], [3000], 16, 16, 128, 16, 1700),
    ([300], [3000], 16, 16, 64, 16, 0),
]


@pytest.mark.parametrize("new,kv,heads,kv_heads,dim,page,window", ATTEND)
def test_attention(new, kv, heads, kv_heads, dim, page, window):
    p = _problem(new, kv, heads, kv_heads, dim, page, seed=sum(kv) + heads)
    _check(p, _call(p, window=window), window=window)


def test_attention_large_scores():
    p = _problem([70, 1], [700, 90], 64, 64, 64, 16, seed=6, std=6.0)
    _check(p, _call(p, window=333), window=333)
    p = _problem([70, 1], [300, 90], 64, 64, 128, 16, seed=7, std=6.0)
    _check(p, _call(p))


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_bad_page_is_that_sequences_nan(dim):
    new = 40
    p = _problem([new, new, new], [200, 200, 200], 64, 64, dim, 16, seed=11)
    first = _call(p)
    _check(p, first)
    for bad in (-1, p["cache"][0].shape[0], 2 ** 31 - 1):
        table = p["table"].clone()
        table[1, 3] = bad
        out = _call(dict(p, table=table))
        assert torch.equal(out[:new], first[:new]) and torch.equal(out[2 * new:], first[2 * new:])
        assert bool(torch.isnan(out[new:2 * new]).all())


def test_attention_rows_behind_the_last_sequence_stay():
    p = _problem([1, 60], [40, 80], 64, 64, 128, 16, seed=16)
    out = torch.full_like(p["q"], 3.0)
    p["cu"] = torch.tensor([0, 1, 52], dtype=torch.int32)
    _call(p, out=out)
    assert bool((out[52:] == 3.0).all()) and not bool((out[:52] == 3.0).all())


def test_attention_repeats_bit_for_bit_and_in_a_graph():
    p = _problem([1, 1, 60], [3000, 100, 900], 64, 32, 128, 16, seed=13)
    args = (p["q"], p["cache"][0], p["cache"][1], p["table"].to(DEV), p["cu"].to(DEV),
            p["kv"].to(DEV), p["max_q"])
    more = dict(k_scale=p["cache"][2], v_scale=p["cache"][3])
    first = T.paged_attention(*args, **more)
    for _ in range(3):
        assert torch.equal(T.paged_attention(*args, **more), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = T.paged_attention(*args, **more)
    for i in range(4):
        p["q"].copy_(base._randn(tuple(p["q"].shape), 20 + i))
        want = T.paged_attention(*args, **more)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 64, 31, 32])
def test_attention_windows_wider_than_any_sequence(window):
    p = _problem([4, 60, 1], [2, 45, 31], 64, 64, 64, 16, seed=15)
    _check(p, _call(p, window=window), window=min(window, 10 ** 6))


@pytest.mark.parametrize("new,kv,heads,kv_heads,dim,page,window,key", [
    ([40, 5], [40, 20], 64, 64, 128, 16, 0, 17),
    ([40, 5], [40, 20], 64, 64, 64, 16, 0, 31),
    ([70], [700], 64, 64, 64, 64, 0, 650),
    ([70, 1], [400, 3], 64, 32, 128, 32, 90, 300),
    ([260], [300], 16, 16, 128, 16, 50, 250),
    ([260], [300], 16, 16, 64, 16, 0, 270),
])
def test_attention_nan_groups_stay_with_those_who_see_them(new, kv, heads, kv_heads, dim, page,
                                                           window, key):
    base.test_attention_nan_groups_stay_with_those_who_see_them(new, kv, heads, kv_heads, dim,
                                                                page, window, key)


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_queries_that_are_not_finite_are_their_rows_own(dim):
    p = _problem([60, 40], [100, 90], 64, 64, dim, 16, seed=23)
    want = _call(p)
    for value in (float("nan"), float("inf")):
        q = p["q"].clone()
        q[0, 3, 5] = value
        got = _call(dict(p, q=q))
        hit = torch.zeros(got.shape[:2], dtype=torch.bool, device=DEV)
        hit[0, 3] = True
        assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("k_scale,v_scale", [(0, 0), (7, 200), (127, 0), (100, 247)])
def test_attention_over_scales_of_other_writers(dim, k_scale, v_scale):
    p = _problem([50], [60], 64, 64, dim, 16, seed=24)
    for c, b in ((2, k_scale), (3, v_scale)):
        live = p["cache"][c].view(torch.uint8)
        live[live != 255] = b
    got = _f64(_call(p))
    ref, tol = base._reference(p)
    assert np.all(np.abs(got - ref) <= tol + 2.0 ** -133)


@pytest.mark.parametrize("new,kv,heads,kv_heads,dim", [
    ([40, 70, 3], [300, 900, 50], 64, 64, 128),
    ([200], [1000], 64, 16, 64),
    ([200], [1000], 64, 16, 128),
])
def test_attention_over_one_value_gives_that_value(new, kv, heads, kv_heads, dim):
    base.test_attention_over_one_value_gives_that_value(new, kv, heads, kv_heads, dim)


@pytest.mark.parametrize("new,kv,heads,kv_heads,dim", [
    ([33], [4000], 128, 64, 128),
    ([200], [5000], 64, 16, 64),
    ([1, 90, 1, 3, 300, 17], [2500, 900, 40, 3000, 2048, 1000], 64, 16, 128),
    ([4] * 30, [900 + 100 * i for i in range(30)], 64, 8, 128),   # 32 rows each
    ([3, 100, 4], [900, 2000, 700], 64, 8, 64),
])
def test_attention_keeps_to_a_workspace_of_the_size_asked_for(new, kv, heads, kv_heads, dim):
    base.test_attention_keeps_to_a_workspace_of_the_size_asked_for(new, kv, heads, kv_heads, dim)


@pytest.mark.parametrize("new,kv,heads,kv_heads,dim", [
    ([4] * 30, [900 + 100 * i for i in range(30)], 64, 8, 128),
    ([3, 100, 4, 1], [900, 2000, 700, 5000], 64, 8, 64),
    ([8], [3000], 64, 8, 128),                   # 64 rows by 16: few tiles in all
    ([16, 1], [2000, 100], 64, 8, 64),
    ([1000], [1000], 2, 2, 128),
    ([5, 7, 9], [600, 700, 800], 128, 2, 128),   # 64 query heads a key/value head
])
def test_attention_on_both_sides_of_the_limits(new, kv, heads, kv_heads, dim):
    p = _problem(new, kv, heads, kv_heads, dim, 16, seed=25)
    ref, mag = _definition(p)
    bad = (_call(p).double() - ref).abs() > \
        2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * mag
    assert not bool(bad.any()), f"{int(bad.sum())} values off"
