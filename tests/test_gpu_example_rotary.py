"""The example's decoder layer with rotary positions and a norm after attention
(the append, the caches in 16, 8 and 4 bits, the block norm and attention as a
step uses them) on the GPU against float64.

Against float64 the attention's reference reads the values that the cache holds,
so the roundings left are those of five linears (helpers.py) and of what lies
between them, half a step of bf16 each: six times the error allowed one linear.
What the cache holds is compared by itself: one linear's error, half a step of the
norm's output (2^-8) and half a step of the cache's type.  In 4 bits that is 2^-2 of
a value above its scale and of the scale below it; spread evenly over such steps
the errors of normal values, of which half are below the scale at most, have a
norm of 0.16 of theirs."""

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
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("decoder_layer_rotary", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _f64(t):
    return OL.bf16_values(bits16(t))


def _inputs(seed):
    """(prompts, steps) of the requests."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    draw = [torch.randn(n, 512, generator=g, device=DEV).bfloat16()
            for n in (*LENGTHS, *[len(LENGTHS)] * STEPS)]
    return draw[:len(LENGTHS)], draw[len(LENGTHS):]


def _serve(example, bits, prompts, steps, chunk=32):
    layer = example.random_layer(DEV, hidden=512, ffn=704, heads=8, kv_heads=2, dim=64,
                                 positions=100, post=True)
    cache = example.PagedCache(32, 16, 2, 64, bits, DEV)
    return layer, cache, example.serve(layer, cache, prompts, IDS, steps, chunk=chunk)


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_layer_matches_float64(example, bits):
    prompts, steps = _inputs(3)
    layer, cache, got = _serve(example, bits, prompts, steps)
    d, hk, norms = layer.dim, layer.kv_heads, {n: _f64(w) for n, w in layer.norms.items()}
    freq = T.rotary_frequencies(d)[0].numpy()
    for r, p in enumerate(prompts):
        x = _f64(torch.cat([p] + [s[r:r + 1] for s in steps]))
        n = len(x)
        w = {m: _f64(T.reconstruct(b, *layer.variants[IDS[r]][m], T.ALPHA_PER_ROW))
             for m, b in layer.base.items()}
        y, _ = OL.rms_norm(x, norms["attn"], 1e-5)
        q, k, v = np.split((y @ w["qkv"].T).reshape(n, -1, d), [layer.heads, layer.heads + hk], 1)
        angles = np.arange(n)[:, None] * freq
        q, k = OL.rotary(q, angles), OL.rotary(k, angles)
        j = torch.arange(n)
        slots = torch.tensor(cache.pages[r])[j // 16] * 16 + j % 16
        held = T.kv_read(slots.int().to(DEV), cache.k, cache.v, cache.k_scale, cache.v_scale)
        step = {16: 2.0 ** -8, 8: 2.0 ** -4, 4: 2.0 ** -2}[bits]
        for have, want in zip(held, (k, v)):
            err = np.linalg.norm(_f64(have) - want) / np.linalg.norm(want)
            assert err <= REL_FRO_TOL + 2.0 ** -8 + step, (r, err)
        kk, vv = (_f64(t).transpose(1, 0, 2)[None] for t in held)
        o, _ = OL.paged_attention(q, kk, vv, np.zeros((1, 1), int), [0, n], [n])
        y, h = OL.rms_norm_block(o.reshape(n, -1) @ w["o"].T, x, norms["attn_post"], norms["ffn"],
                                 1e-5)
        gate = y @ w["gate"].T
        ref = gate / (1 + np.exp(-gate)) * (y @ w["up"].T) @ w["down"].T + h
        err = np.linalg.norm(_f64(got[r]) - ref) / np.linalg.norm(ref)
        assert got[r].shape == ref.shape and err <= 6 * REL_FRO_TOL, (r, err)


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_requests_do_not_touch_each_other_and_pages_are_reused(example, bits):
    """A request served beside others gives the bits that it gives alone, also
    in pages that another has left."""
    prompts, _ = _inputs(5)
    layer, cache, first = _serve(example, bits, prompts, [])
    for seq in list(cache.pages):
        cache.release(seq)
    cache.free.reverse()
    for r in (2, 0, 1):
        alone = example.serve(layer, cache, [prompts[r]], [IDS[r]], [], chunk=32)
        assert torch.equal(alone[0], first[r])
        cache.release(0)
    assert len(cache.free) == 32


def test_main_runs(example, monkeypatch, capsys):
    for bits in ("4", "8", "16"):
        monkeypatch.setattr("sys.argv", ["decoder_layer.py", "--bits", bits])
        example.main()
        assert "request 2" in capsys.readouterr().out
