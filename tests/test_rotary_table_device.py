"""Where a rotary table is made: on the device that is named, or not at all."""

import pytest
import torch

import tenant_linear_layers_amd as T


@pytest.mark.parametrize("device", ["cpu", torch.device("cpu"), "meta"])
def test_a_table_on_the_host_is_refused(device):
    with pytest.raises(ValueError, match="device"):
        T.rotary_table(T.rotary_frequencies(64)[0], 8, device=device)


@pytest.mark.gpu
def test_a_table_is_where_it_was_asked_for():
    f = T.rotary_frequencies(64)[0]
    want = T.rotary_table(f, 8)
    for device in ("cuda", "cuda:0", torch.device("cuda", 0)):
        for at in (f, f.to("cuda:0")):
            got = T.rotary_table(at, 8, device=device)
            assert got.device == torch.device("cuda:0") and torch.equal(got, want)
    for device in ("cuda:1", "cpu"):
        with pytest.raises(ValueError, match="device"):
            T.rotary_table(f.to("cuda:0"), 8, device=device)
