"""attn_mass_paged where a CTA has many units of a key tile: keys held in tensor memory, the rings
of queries and scores past their second turn, runs that end inside a key tile.  Against fp64."""
import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _thin_ref as ref
from tests._parity import np64
from tests.test_mass_parity import Rows, i32

pytestmark = pytest.mark.gpu

SMS, KEYS, ITEM_COST = 152, 256, 3


def plan(lens, nq, Hq, Hkv, d, causal, window, n_sink):
    """Most units of one key tile that a CTA has, by the rule of the split: positions (ITEM_COST
    before a key tile's units) dealt in equal runs."""
    G, tile = Hq // Hkv, 64 if d == 256 else 128
    GP = G if G <= tile else max(x for x in range(1, tile + 1) if G % x == 0)
    TQ = tile // GP
    item = []                                   # key tile of each position, -1 before its units
    for b, (L, Lq) in enumerate(zip(lens, nq)):
        for h in range(Hkv):
            for kt in range(-(-L // KEYS)):
                i, t = np.arange(Lq)[:, None] + L - Lq, np.arange(kt * KEYS, min(L, kt * KEYS + KEYS))
                seen = (t <= i) if causal else np.ones((Lq, len(t)), bool)
                if window:
                    seen = seen & ((t > i - window) | (t < n_sink))
                rows = np.flatnonzero(seen.any(1))
                n = 0 if not len(rows) else (rows[-1] // TQ - rows[0] // TQ + 1) * (G // GP)
                if n:
                    item += [-1] * ITEM_COST + [(b, h, kt)] * n
    T, most = len(item), 0
    for c in range(SMS):
        run = item[T * c // SMS:T * (c + 1) // SMS]
        units = [x for x in run if x != -1]
        for x in set(units):
            most = max(most, units.count(x))
    return most


def weights(r, q, cu, causal, window, n_sink, scale):
    """lse [Hq, T] and the weights [Hkv, n] of every row, one head at a time."""
    lse, w, G = np.full((r.Hq, q.shape[0]), -np.inf), [], r.Hq // r.Hkv
    for b, n in enumerate(r.lens):
        k, _ = r.keys(b)
        Lq = cu[b + 1] - cu[b]
        got = np.zeros((r.Hkv, n))
        seen = np.stack([ref.seen_keys(i, Lq, n, causal, window, n_sink) for i in range(Lq)])
        for h in range(r.Hq):
            x = np.where(seen, scale * (np64(q[cu[b]:cu[b + 1], h]) @ k[:, h // G].T), -np.inf)
            top = x.max(1, keepdims=True)
            z = top[:, 0] + np.log(np.exp(x - top).sum(1))
            lse[h, cu[b]:cu[b + 1]] = z
            got[h // G] += np.exp(x - z[:, None]).sum(0)
        w.append(got)
    return lse, w


CASES = [([1500], [1500], 32, 8, True, 0, 0), ([2100, 1700], [1200, 900], 24, 8, True, 700, 300),
         ([900, 1300], [900, 500], 20, 4, False, 0, 0), ([1500, 40], [1500, 40], 24, 8, True, 0, 0),
         ([1100], [1100], 48, 3, True, 500, 0)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,nq,Hq,Hkv,causal,window,n_sink", CASES)
def test_long_runs(lens, nq, Hq, Hkv, causal, window, n_sink, d):
    assert plan(lens, nq, Hq, Hkv, d, causal, window, n_sink) >= 7  # from four on keys go to tensor memory
    r = Rows(lens, Hq, Hkv, d, seed=Hq + d)
    cu = np.concatenate([[0], np.cumsum(nq)]).tolist()
    q = r.q(cu[-1])
    lse, w = weights(r, q, cu, causal, window, n_sink, d ** -0.5)
    args = (q.cuda(), torch.tensor(lse).float().cuda(), r.k.cuda(), i32(r.table), i32(cu), i32(lens))
    more = dict(max_seqlen_q=max(nq), causal=causal, window=window, n_sink=n_sink)
    out = ea.attn_mass_paged(*args, r.mass.cuda(), **more)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    # A thread adds 16 (d = 256: 8) weights of a unit to each of its four sums, and the sums of
    # some CTAs are added: 2^-24 of the sum for each addition.
    adds = 16 * (-(-sum(nq) * (Hq // Hkv) // 64) + 2) + 4 + SMS
    for b, n in enumerate(lens):
        base = r.mass[b, :, :n].double().numpy().copy()
        base[:, n - nq[b]:] = 0
        got = out[b, :, :n].double().cpu().numpy()
        bound = (ref.WEIGHT + adds * 2.0 ** -24) * w[b] + 2.0 ** -23 * (base + w[b])
        bad = np.abs(got - base - w[b]) > bound + 1e-30
        assert not bad.any(), (b, int(bad.sum()), np.argwhere(bad)[:3].tolist())
        assert torch.equal(out[b, :, n:].cpu(), r.mass[b, :, n:])
    again = ea.attn_mass_paged(*args, r.mass.cuda(), **more)
    torch.cuda.synchronize()
    assert all(torch.equal(again[b, :, :n], out[b, :, :n]) for b, n in enumerate(lens))
