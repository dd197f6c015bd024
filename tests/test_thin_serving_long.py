"""The chain of test_thin_serving on prompts that are long enough for their samples to share the
prefix kernel: attended, weighed, cut, forked, decoded."""
import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _thin_ref as ref
from tests import test_thin_serving as serving
from tests._parity import compare, np64
from tests.test_shared_items import shares

pytestmark = pytest.mark.gpu

LAYERS, i32 = serving.LAYERS, serving.i32


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 2, 64), (6, 1, 256)])
def test_long_prompts_cut_forked_and_decoded(Hq, Hkv, d, monkeypatch):
    monkeypatch.setattr(serving, "P", 300)
    monkeypatch.setattr(serving, "W", 100)
    B, counts, keep = 8, [1500, 900] + [0] * 6, [1100, 700] + [0] * 6
    s = serving.Server(B, Hq, Hkv, d)
    s.resize(counts)
    qs, cu = s.append(counts)
    for layer in range(LAYERS):
        o, lse = ea.attn_fwd_paged(qs[layer], s.kp[layer], s.vp[layer], s.pt, i32(cu), s.ln,
                                   max_seqlen_q=1500)
        ea.attn_mass_paged(qs[layer], lse, s.kp[layer], s.pt, i32(cu), s.ln, s.mass[layer],
                           s.pos[layer], max_seqlen_q=1500)
        for b in (0, 1):
            n, q = counts[b], np64(qs[layer][cu[b]:cu[b + 1]].cpu())
            want = np.zeros((Hkv, n))
            for h in range(Hq):
                x = d ** -0.5 * (q[:, h] @ s.k[layer][b][h * Hkv // Hq].T)
                w = np.exp(x - x.max(1, keepdims=True)) * np.tri(n)
                want[h * Hkv // Hq] += (w / w.sum(1, keepdims=True)).sum(0)
            # weights of the kernel's own LSE, which its tests hold to 1e-3; 2e-4 here
            got = s.mass[layer, b, :, :n].double().cpu().numpy()
            assert np.abs(got - want).max() <= 2e-4 * want.max()
    s.resize(s.evict(keep, n_sink=4, recent=16))
    s.fork([0] * 4 + [1] * 2, [2, 3, 4, 5, 6, 7])
    lens = [1100, 700] + [1100] * 4 + [700] * 2
    rows = [0, 2, 3, 4, 5, 1, 6, 7]
    assert shares(5, 1100 // 16, d) and (shares(3, 700 // 16, d) or d == 64)
    for step in range(2):
        lens = [n + 1 for n in lens]
        s.resize(lens)
        qs, _ = s.append([1] * B)
        for layer in range(LAYERS):
            args = qs[layer], s.kp[layer], s.vp[layer], s.pt, s.ln
            before = s.mass[layer].cpu().numpy()
            o1, l1 = ea.attn_decode_paged_shared(*args, i32([0, 5, 8]), i32([1100, 700]), i32(rows))
            o2, l2 = ea.attn_decode_paged_mass(*args, s.mass[layer], s.pos[layer],
                                               i32([n - 1 for n in s.at]))
            ro, rl = np.zeros((B, Hq, d)), np.zeros((B, Hq))
            for b in range(B):
                ro[b], rl[b], w = s.attend(layer, b, np64(qs[layer][b].cpu()))
                for h in range(Hkv):
                    base = before[b, h, :lens[b]].astype(np.float64)
                    base[-1] = 0
                    ref.check_mass(s.mass[layer, b, h, :lens[b]].double().cpu().numpy(), base, w[h])
            compare(o1, l1, ro, rl, f"shared decode, step {step}")
            compare(o2, l2, ro, rl, f"decode with masses, step {step}")
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
