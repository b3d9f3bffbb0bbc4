"""The norms around a block on the GPU against float64.

Tolerances: h: float32 steps (a sum of squares whose relative error is below
2^-18, a root, three products and an addition) and a rounding to bf16: 2^-8 |h| +
2^-17 |scale gate u|.  y: the same of h before its rounding, then another sum, root and
two products: 2^-8 |y| + 2^-16 of the row's |scale gate u| and |h| over its root mean
square, times |w|."""

import numpy as np
import pytest
import torch

import oracle.layer as OL
import tenant_linear_layers_amd as T
from helpers import bits16

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-5


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    T.lib()
    yield
    torch.cuda.empty_cache()


def _randn(shape, seed, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _f64(t):
    return OL.bf16_values(bits16(t))


def _inputs(rows, cols, post, gate, seed=0):
    return dict(x=_randn((rows, cols), seed + 1, 1.4), residual=_randn((rows, cols), seed + 2, 3.0),
                post_weight=_randn((cols,), seed + 3, 0.1) + 1.0 if post else None,
                weight=_randn((cols,), seed + 4, 0.1) + 1.0, eps=EPS,
                gate=None if gate is None else
                _randn((cols,) if gate == "cols" else (rows, cols), seed + 5, 0.7))


def _check(a, y, h, scale):
    x, r, w = (_f64(a[n]) for n in ("x", "residual", "weight"))
    p = None if a["post_weight"] is None else _f64(a["post_weight"])
    g = None if a["gate"] is None else _f64(a["gate"])
    yr, hr = OL.rms_norm_block(x, r, p, w, EPS, g, scale)
    part = np.abs(hr - r)
    assert np.all(np.abs(_f64(h) - hr) <= 2.0 ** -8 * np.abs(hr) + 2.0 ** -17 * part)
    rms = np.sqrt(np.mean(hr * hr, -1, keepdims=True) + EPS)
    tol = 2.0 ** -8 * np.abs(yr) + 2.0 ** -16 * (part + np.abs(hr)) / rms * np.abs(w)
    assert np.all(np.abs(_f64(y) - yr) <= tol)


SHAPES = [(1, 1), (3, 7), (2, 33), (4, 511), (9, 512), (3, 520), (5, 1024), (3, 1032), (4, 2048),
          (2, 2049), (3, 4096), (2, 4097), (1, 8192), (2, 8193), (300, 8192), (2, 16384),
          (2, 16385), (1, 30001), (1030, 96)]


@pytest.mark.parametrize("post,gate,scale", [(True, None, 1.0), (True, "rows", 0.5),
                                             (False, "cols", -2.0), (True, "cols", 0.3),
                                             (False, None, 0.0), (False, "rows", 1.0)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rms_norm_block(rows, cols, post, gate, scale):
    a = _inputs(rows, cols, post, gate, rows + cols)
    y, h = T.rms_norm_block(**a, scale=scale)
    assert y.shape == h.shape == (rows, cols)
    _check(a, y, h, scale)


@pytest.mark.parametrize("cols", [1024, 8192, 20000])
def test_without_its_parts_it_is_the_residual_norm(cols):
    """No norm after the block, no gate, scale 1: rms_norm, bit for bit."""
    a = _inputs(5, cols, False, None)
    y, h = T.rms_norm_block(**a)
    y2, h2 = T.rms_norm(a["x"], a["weight"], EPS, a["residual"])
    assert torch.equal(y, y2) and torch.equal(h, h2)


@pytest.mark.parametrize("cols", [1024, 1001, 17000])
def test_strided_rows_leading_dims_and_outputs_given(cols):
    a = _inputs(9, cols, True, "rows", 7)
    want = T.rms_norm_block(**a, scale=0.5)
    wide = _randn((9, 3 * cols + 40), 9)
    b = dict(a)
    for i, n in enumerate(("x", "residual", "gate")):           # odd alignments among them
        wide[:, i * (cols + 7) + 1:][:, :cols] = a[n]
        b[n] = wide[:, i * (cols + 7) + 1:][:, :cols]
    out = [torch.empty_like(a["x"]) for _ in range(2)]
    got = T.rms_norm_block(**b, scale=0.5, y=out[0], h=out[1])
    assert got[0] is out[0] and got[1] is out[1]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c = {n: t.view(3, 3, cols) if n in ("x", "residual", "gate") else t for n, t in a.items()}
    got = T.rms_norm_block(**c, scale=0.5)
    assert got[0].shape == (3, 3, cols)
    assert torch.equal(got[0].view(9, cols), want[0]) and torch.equal(got[1].view(9, cols), want[1])
    # one gate for all rows, as a row and as a view of it
    one = dict(a, gate=a["gate"][0].clone())
    all_rows = dict(a, gate=a["gate"][:1].expand(9, cols))
    for x, z in zip(T.rms_norm_block(**one), T.rms_norm_block(**all_rows)):
        assert torch.equal(x, z)


def test_values_that_are_not_finite_stay_in_their_rows():
    a = _inputs(4, 2048, True, "rows", 11)
    want = T.rms_norm_block(**a)
    a["x"][1, 5], a["gate"][2, 7] = float("nan"), float("inf")
    for got, w in zip(T.rms_norm_block(**a), want):
        assert torch.equal(got[0], w[0]) and torch.equal(got[3], w[3])
        assert not bool(torch.isfinite(got[1]).any())
    y, h = T.rms_norm_block(**a)
    assert not bool(torch.isfinite(h[2, 7])) and bool(torch.isfinite(h[2, :7]).all())


def test_rows_past_32_bits_and_past_a_launch():
    rows, cols = 2 ** 26 + 5, 32                     # 64 threads a row: more than 2^32
    w = _randn((cols,), 2, 0.1) + 1.0
    at = torch.tensor([0, 1, 2 ** 25 - 1, 2 ** 25, 2 ** 25 + 1, rows - 1], device=DEV)
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=DEV)
    x[at] = _randn((len(at), cols), 3, 1.4)
    few = T.rms_norm_block(x[at], x[at], w, w, EPS, x[at])
    for got, want in zip(T.rms_norm_block(x, x, w, w, EPS, x), few):
        assert torch.equal(got[at], want)


def test_in_a_graph_and_on_a_stream():
    a = _inputs(20, 1024, True, "rows", 13)
    s = torch.cuda.Stream()
    want = T.rms_norm_block(**a)
    s.wait_stream(torch.cuda.current_stream())
    got = T.rms_norm_block(**a, stream=s)
    s.synchronize()
    assert all(torch.equal(x, z) for x, z in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = T.rms_norm_block(**a)
    for i in range(3):
        a["x"].copy_(_randn((20, 1024), 30 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, z) for x, z in zip(out, T.rms_norm_block(**a)))


def test_refusals():
    a = _inputs(4, 64, True, "rows")
    for change, kind in ((dict(x=a["x"].float()), TypeError), (dict(residual=a["x"][:3]), ValueError),
                         (dict(weight=a["weight"][:32]), ValueError),
                         (dict(post_weight=a["weight"][:32]), ValueError),
                         (dict(weight=None), TypeError), (dict(residual=None), TypeError),
                         (dict(gate=a["gate"][:, :32]), ValueError),
                         (dict(gate=a["gate"][:2]), ValueError),
                         (dict(gate=a["gate"][0, :32]), ValueError),
                         (dict(gate=a["gate"].float()), TypeError),
                         (dict(scale=float("inf")), ValueError),
                         (dict(scale=float("nan")), ValueError),
                         (dict(y=a["x"][:3]), ValueError), (dict(y=a["x"]), T.BitDeltaError),
                         (dict(h=a["residual"]), T.BitDeltaError)):
        with pytest.raises(kind):
            T.rms_norm_block(**{**a, **change})
    e = _inputs(4, 64, True, "rows")
    none = T.rms_norm_block(e["x"][:0], e["residual"][:0], e["post_weight"], e["weight"], EPS,
                            e["gate"][:0])
    assert none[0].shape == (0, 64)
