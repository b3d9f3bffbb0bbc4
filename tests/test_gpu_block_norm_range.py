"""The norms around a block where a row's sum of squares passes float32's range: the
norm of that row is zeros, as the residual norm's is, and the other rows keep theirs."""

import pytest
import torch

import tenant_linear_layers_amd as T
from test_gpu_block_norm import EPS, _check, _gpu, _inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [512, 2048, 8192, 16384, 20001])
def test_rows_whose_sum_of_squares_passes_the_range(cols):
    a = _inputs(4, cols, True, "rows", cols)
    want = T.rms_norm_block(**a, scale=0.5)
    _check(a, *want, 0.5)
    b = dict(a, x=a["x"].clone(), residual=a["residual"].clone())
    b["x"][1, cols // 2] = 2.0 ** 64            # its square alone is 2^128
    b["residual"][2, cols - 1] = -(2.0 ** 65)
    y, h = T.rms_norm_block(**b, scale=0.5)
    assert torch.equal(h[1], b["residual"][1])
    assert torch.equal(y[1], T.rms_norm(b["residual"][1:2], b["weight"], EPS)[0][0])
    assert bool((y[2] == 0).all()) and torch.equal(h[2, :-1], want[1][2, :-1])
    assert float(h[2, -1]) == -(2.0 ** 65)
    for row in (0, 3):
        assert torch.equal(y[row], want[0][row]) and torch.equal(h[row], want[1][row])
    # one step below the range nothing is lost
    b["x"][1] = 0
    b["x"][1, cols // 2] = 2.0 ** 63
    b["residual"][2] = a["residual"][2]
    _check(b, *T.rms_norm_block(**b, scale=0.5), 0.5)
