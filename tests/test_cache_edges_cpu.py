"""Rotary positions and the paged cache's upkeep where a host decision could go wrong,
without a GPU."""
import math

import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea


def without_cuda_names(monkeypatch):
    """The binding as it is on its first call, under a torch without two private names."""
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    for name in ("_torch_module", "_current_device", "_raw_stream"):
        monkeypatch.setattr(ea, name, None)


def test_refusals_and_frequencies_without_torchs_private_names(monkeypatch):
    without_cuda_names(monkeypatch)
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    inv = ea.attn_rope_inv_freq(64, device="cpu")
    assert inv.shape == (32,) and inv[0] == 1.0
    with pytest.raises(ValueError):
        ea.attn_fwd(q, q, q)
    with pytest.raises(ValueError):
        ea.attn_rope(q, None, inv)


class FakeStream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 64 + index


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Two devices' streams stood in for: making the other device's current would launch
    on it, or, with the tensors' device made current again, drop the stream."""
    class Context:
        def __init__(self, *_):
            pass

        __enter__ = __exit__ = lambda self, *_: None

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "device", Context)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    ea._Call(0, FakeStream(0))
    ea._Call(1, FakeStream(1))
    for index in (0, 1):
        with pytest.raises(ValueError):
            ea._Call(index, FakeStream(1 - index))


def test_sizes_past_32_bits_have_no_workspace():
    for rows, pages in ((1 << 32, 12), (4, (1 << 32) + 12), (4, 12 - (1 << 32)), (1 - (1 << 32), 12)):
        assert ea.attn_pages_workspace_size(rows, pages) == 0


@pytest.mark.parametrize("args", [
    dict(base=1e300, scaling="base", factor=1e10),      # the stretched base is infinite
    dict(base=1e-300, scaling="base", factor=1e-200),   # or zero
    dict(base=5e-324, scaling="none"),
    dict(scaling="linear", factor=5e-324),
    dict(scaling="ramp", factor=5e-324, original_length=2048.0)])
def test_frequencies_that_fp64_does_not_hold_are_refused(args):
    with pytest.raises(ea.AttnError) as e:
        ea.attn_rope_inv_freq(128, device="cpu", **args)
    assert e.value.status == ea.ATTN_ERR_INVALID_ARG


def test_frequencies_near_the_ends_of_fp64_are_given():
    for base in (1e-300, 1e300):
        f = ea.attn_rope_inv_freq(64, base, device="cpu").numpy()
        assert np.isfinite(f).all() and (f > 0).all()
        np.testing.assert_allclose(np.log(f), -2 * np.arange(32) / 64 * math.log(base), rtol=1e-13)
