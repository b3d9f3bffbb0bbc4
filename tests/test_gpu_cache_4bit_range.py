"""Attention over a 4-bit cache whose scales, of another writer, put some values past
bf16's range: those reach the rows and dims that see them, and no others.

Keys of scale 2^-127 weigh alike, one each, so a row is the mean of the values it sees:
their sum, float32, over their number.  Dim 0 has a sum of 2^128 for the rows that see
keys 3 and 30, past float32's range.  Everywhere else sums are exact, and what is left
is one division, 2^-22, and the output's rounding, half a step of bf16."""

import numpy as np
import pytest
import torch

from test_gpu_cache_4bit import DEV, _call, _f64, _gpu, _problem, _stored  # noqa: F401

pytestmark = pytest.mark.gpu

KEYS, LARGE = 50, 20


@pytest.mark.parametrize("new,heads,kv_heads", [(1, 4, 2), (40, 4, 2), (40, 64, 64)])
@pytest.mark.parametrize("dim", [64, 128])
def test_values_past_the_range_are_their_rows_and_dims_own(new, heads, kv_heads, dim):
    p = _problem([new], [KEYS], heads, kv_heads, dim, 16, seed=61)
    p["cache"][2].view(torch.uint8).fill_(0)
    p["cache"][3].view(torch.uint8).fill_(254)          # 2^127
    codes = p["cache"][1].view(torch.uint8)
    codes.zero_()

    def put(key, at, byte):   # two dims of a value row: the even one in the low bits
        codes[int(p["table"][0, key // 16]), :, key % 16, at] = byte

    put(3, 0, 0x93)           # 1.5 and -0.5
    put(30, 0, 0x91)          # 0.5 and -0.5
    put(44, 5, 0x0A)          # -1
    put(LARGE, 17, 0x60)      # dim 35: 4, past the range
    put(LARGE, 20, 0x0F)      # dim 40: -6
    put(49, 20, 0x02)         # and 1 beside it
    v = _stored(p["cache"])[1]
    rows = p["table"][0].numpy()[np.arange(KEYS) // 16], np.arange(KEYS) % 16
    v = np.repeat(v[rows[0], :, rows[1]], heads // kv_heads, axis=1)      # [keys, heads, dim]
    got = _f64(_call(p))
    for i in range(new):
        seen = v[:KEYS - new + i + 1]
        over = (np.abs(seen) >= 2.0 ** 128).any(0)
        assert over.any() == (KEYS - new + i >= LARGE)
        over |= np.abs(np.where(over, 0.0, seen.sum(0))) >= 2.0 ** 128
        assert over[:, 0].all() == (KEYS - new + i >= 30)
        assert not np.isfinite(got[i][over]).any()
        ref = seen.mean(0)[~over]
        assert np.all(np.abs(got[i][~over] - ref) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(ref))
