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
