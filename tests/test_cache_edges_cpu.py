"""Rotary positions and the paged cache's upkeep where a host decision could go wrong,
without a GPU."""
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
