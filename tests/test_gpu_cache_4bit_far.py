"""Attention over the 4-bit cache on tiles of 64 and of 128 rows, where rows of the
cache lie beyond 2^32 bytes, scales beyond 2^28 and queries beyond 2^31 elements: the
same bits as of the same bytes nearby."""

import pytest
import torch

from test_gpu_cache_4bit import DEV, _call, _check, _gpu, _problem  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,kv,heads,kv_heads", [
    ([40, 70], [90, 150], 64, 64),     # tiles of 64 rows
    ([200], [500], 64, 16),            # of 128
])
def test_tiles_of_many_rows_past_32_bits(new, kv, heads, kv_heads):
    page, dim = 64, 128
    small = _problem(new, kv, heads, kv_heads, dim, page, seed=43)
    want = _call(small)
    _check(small, want)
    pages = 2 ** 32 // (kv_heads * page * dim // 2) + 40
    far = [torch.empty((pages, *c.shape[1:]), dtype=torch.uint8, device=DEV).view(c.dtype)
           for c in small["cache"]]
    table = torch.full_like(small["table"], -7)
    at = pages - 1
    for b, m in enumerate(kv):
        for j in range(-(-m // page)):
            for x, y in zip(small["cache"], far):
                y.view(torch.uint8)[at] = x.view(torch.uint8)[int(small["table"][b, j])]
            table[b, j] = at
            at -= 1
    assert at * kv_heads * page * (dim // 2) >= 2 ** 32
    assert torch.equal(_call(dict(small, cache=far, table=table)), want)
    tokens = sum(new)
    stride = 2 ** 31 // (tokens - 1) + 8
    q = torch.empty((tokens - 1) * stride + heads * dim, dtype=torch.bfloat16, device=DEV)
    q = q.as_strided((tokens, heads, dim), (stride, dim, 1))
    q.copy_(small["q"])
    assert torch.equal(_call(dict(small, q=q)), want)
