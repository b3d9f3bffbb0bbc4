"""The example's decoder layer with several requests in a batch, and over either
cache, on the GPU.

Against float64 the attention's reference reads the values that the cache holds,
so that the roundings left are those of five linears and of what lies between
them: six times the error that helpers.py allows one linear, as for a cache in
bf16.  What the cache holds is compared by itself: one linear's error, half a step
of the norm's output (2^-8) and half a step of the cache's type."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle.layer as OL
import tenant_linear_layers_amd as T
from helpers import REL_FRO_TOL, bits16

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "decoder_layer.py")
LENGTHS, IDS, STEPS = (70, 1, 33), [0, 2, 1], 3


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("decoder_layer_requests", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _f64(t):
    return OL.bf16_values(bits16(t))


def _inputs(seed):
    """(prompts, steps) of the requests."""
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    draw = [torch.randn(n, 512, generator=g, device="cuda:0").bfloat16()
            for n in (*LENGTHS, *[len(LENGTHS)] * STEPS)]
    return draw[:len(LENGTHS)], draw[len(LENGTHS):]


def _serve(example, bits, prompts, steps):
    dev = torch.device("cuda:0")
    layer = example.random_layer(dev, hidden=512, ffn=704, heads=8, kv_heads=2, dim=64)
    cache = example.PagedCache(32, 16, 2, 64, bits, dev)
    return layer, cache, example.serve(layer, cache, prompts, IDS, steps, chunk=32)


@pytest.mark.parametrize("bits", [8, 16])
def test_decoded_tokens_do_not_depend_on_the_other_requests(example, bits):
    """The requests decode in one batch.  Where a request's own inputs stay and
    all others' change, its outputs stay bit for bit."""
    prompts, steps = _inputs(3)
    _, _, first = _serve(example, bits, prompts, steps)
    others, other_steps = _inputs(4)
    for r in range(len(LENGTHS)):
        mixed = [p if i == r else o for i, (p, o) in enumerate(zip(prompts, others))]
        rows = [o.clone() for o in other_steps]
        for row, s in zip(rows, steps):
            row[r] = s[r]
        _, _, got = _serve(example, bits, mixed, rows)
        for i in range(len(LENGTHS)):
            assert torch.equal(got[i], first[i]) == (i == r), (r, i)


@pytest.mark.parametrize("bits", [8, 16])
def test_layer_over_either_cache_matches_float64(example, bits):
    prompts, steps = _inputs(5)
    layer, cache, got = _serve(example, bits, prompts, steps)
    n_heads, hk, d = layer.heads, layer.kv_heads, layer.dim
    rounding = 2.0 ** -4 if bits == 8 else 2.0 ** -8
    for r, p in enumerate(prompts):
        x = _f64(torch.cat([p] + [s[r:r + 1] for s in steps]))
        w = {n: _f64(T.reconstruct(b, *layer.variants[IDS[r]][n], T.ALPHA_PER_ROW))
             for n, b in layer.base.items()}
        n = len(x)
        y, _ = OL.rms_norm(x, _f64(layer.norms["attn"]), 1e-5)
        q, k, v = np.split((y @ w["qkv"].T).reshape(n, -1, d), [n_heads, n_heads + hk], axis=1)
        j = torch.arange(n, device="cuda:0")
        pages = torch.tensor(cache.pages[r], device="cuda:0")
        slots = (pages[j // cache.page] * cache.page + j % cache.page).int()
        held = [_f64(t) for t in T.kv_read(slots, cache.k, cache.v, cache.k_scale, cache.v_scale)]
        for own, ref in zip(held, (k, v)):
            err = np.linalg.norm(own - ref) / np.linalg.norm(ref)
            assert err <= REL_FRO_TOL + 2.0 ** -8 + rounding * 1.02, (r, err)
        o, _ = OL.paged_attention(q, *(h.transpose(1, 0, 2)[None] for h in held),
                                  np.zeros((1, 1), int), [0, n], [n])
        y, h = OL.rms_norm(o.reshape(n, -1) @ w["o"].T, _f64(layer.norms["ffn"]), 1e-5, x)
        gate = y @ w["gate"].T
        ref = gate / (1 + np.exp(-gate)) * (y @ w["up"].T) @ w["down"].T + h
        err = np.linalg.norm(_f64(got[r]) - ref) / np.linalg.norm(ref)
        assert got[r].shape == ref.shape and err <= 6 * REL_FRO_TOL, (r, err)
