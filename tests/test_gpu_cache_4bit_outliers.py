"""Attention over the 4-bit cache where one dim's products are far larger than the
others', as channels of real queries and keys are.

Scores are sums in float32.  Every product here is a multiple of 2^-6 and every sum
of them below 2^17, so that float32 holds each partial sum exactly, in any order: a
score has no error, whatever its largest product is.  What is left is the rounding of
the weights and of the output, each half a step of bf16:
2^-8 |o| + (2^-8 + 2^-12) sum_j p_j |v_j|, the last part for the argument of the
exponential: its float32 rounding is 2^-24 of at most 2^9, 2^-15."""

import pytest
import torch

from test_gpu_cache_4bit import DEV, _call, _definition, _gpu, _problem, _randn  # noqa: F401

import tenant_linear_layers_amd as T

pytestmark = pytest.mark.gpu

# new tokens, cached keys, heads, kv_heads: few rows, and more than 192 tiles of 16 rows
# of sequences of more than 32
SHAPES = [([1, 2], [90, 333], 8, 2), ([70, 40], [70, 300], 64, 64), ([200], [500], 64, 16)]


def _outliers(new, kv, heads, kv_heads, dim, of_q, of_k, seed):
    """q in multiples of 1/8 up to 4, k in multiples of 1/8 up to 12, but in one dim,
    where they are of_q and of_k throughout."""
    p = _problem(new, kv, heads, kv_heads, dim, 16, seed=seed)
    p["q"] = ((_randn(tuple(p["q"].shape), seed + 4).float() * 8).round() / 8).clamp(-4, 4)
    at = dim // 2 + 5
    p["q"][..., at] = of_q
    p["q"] = p["q"].bfloat16()
    for b, m in enumerate(kv):
        j = torch.arange(m, device=DEV)
        slots = (p["table"][b].to(DEV)[j // 16] * 16 + j % 16).int()
        k, v = T.kv_read(slots, *p["cache"])
        k[..., at] = of_k
        T.kv_write(k, v, slots, *p["cache"])
        k = T.kv_read(slots, *p["cache"])[0].float()
        assert bool((k[..., at] == of_k).all()) and bool((k * 8 == (k * 8).round()).all())
        k[..., at] = 0
        assert float(k.abs().max()) <= 12
    return p


@pytest.mark.parametrize("of_q,of_k", [(128, 128), (256, 4), (1024, 4), (16384, 4)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,kv,heads,kv_heads", SHAPES)
def test_scores_keep_their_small_products_beside_a_large_one(new, kv, heads, kv_heads, dim, of_q,
                                                             of_k):
    p = _outliers(new, kv, heads, kv_heads, dim, of_q, of_k, seed=sum(kv))
    ref, mag = _definition(p)
    bad = (_call(p).double() - ref).abs() > \
        2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * mag
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} values off"
