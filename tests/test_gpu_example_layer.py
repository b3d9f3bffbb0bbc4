"""The example's decoder layer on the GPU against the same layer in float64.

Tolerance: five linears in a row, each within the relative Frobenius error that
helpers.py allows one of them, and the roundings between them (norms, the
product of gate and up, the stream: 2^-8 of each at most) within a sixth."""

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


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("decoder_layer_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _f64(t):
    return OL.bf16_values(bits16(t))


def _layer64(layer, variant, x):
    """Outputs of one sequence's tokens x [n, hidden] in float64."""
    w = {n: _f64(T.reconstruct(b, *layer.variants[variant][n], T.ALPHA_PER_ROW))
         for n, b in layer.base.items()}
    y, _ = OL.rms_norm(x, _f64(layer.norms["attn"]), 1e-5)
    qkv = y @ w["qkv"].T
    n, d, hk = len(x), layer.dim, layer.kv_heads
    q, k, v = np.split(qkv.reshape(n, -1, d), [layer.heads, layer.heads + hk], axis=1)
    # the oracle's cache: one page of all tokens
    o, _ = OL.paged_attention(q, k.transpose(1, 0, 2)[None], v.transpose(1, 0, 2)[None],
                              np.zeros((1, 1), int), [0, n], [n])
    y, h = OL.rms_norm(o.reshape(n, -1) @ w["o"].T, _f64(layer.norms["ffn"]), 1e-5, x)
    gate = y @ w["gate"].T
    return gate / (1 + np.exp(-gate)) * (y @ w["up"].T) @ w["down"].T + h


def _problem(example, bits):
    dev = torch.device("cuda:0")
    layer = example.random_layer(dev, hidden=512, ffn=704, heads=8, kv_heads=2, dim=64)
    cache = example.PagedCache(32, 16, 2, 64, bits, dev)
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    prompts = [torch.randn(n, 512, generator=g, device=dev).bfloat16() for n in (70, 1, 33)]
    steps = [torch.randn(3, 512, generator=g, device=dev).bfloat16() for _ in range(3)]
    return layer, cache, prompts, [0, 2, 1], steps


def test_layer_matches_float64(example):
    layer, cache, prompts, ids, steps = _problem(example, 16)
    got = example.serve(layer, cache, prompts, ids, steps, chunk=32)
    for r, p in enumerate(prompts):
        ref = _layer64(layer, ids[r], _f64(torch.cat([p] + [s[r:r + 1] for s in steps])))
        err = np.linalg.norm(_f64(got[r]) - ref) / np.linalg.norm(ref)
        assert got[r].shape == ref.shape and err <= 6 * REL_FRO_TOL, (r, err)


@pytest.mark.parametrize("bits", [8, 16])
def test_requests_do_not_touch_each_other_and_pages_are_reused(example, bits):
    """A request served beside others gives the bits that it gives alone, also
    in pages that another has left."""
    layer, cache, prompts, ids, steps = _problem(example, bits)
    first = example.serve(layer, cache, prompts, ids, [])
    for seq in list(cache.pages):
        cache.release(seq)
    cache.free.reverse()
    for r in (2, 0, 1):
        alone = example.serve(layer, cache, [prompts[r]], [ids[r]], [])
        assert torch.equal(alone[0], first[r])
        cache.release(0)
    assert len(cache.free) == 32
