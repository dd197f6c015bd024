"""The operators together, as they are used: a serving loop over one paged cache
(grow, append, attend, fork, cut, compact) and a training step (rotate, attend,
differentiate, rotate back), against the fp64 oracle."""
import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
import oracle
from tests import _cache_ref as ref
from tests._parity import compare, np64

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Server:
    """A paged cache on the GPU; `keys`, `values` hold each row's rotated keys and its
    values as the attention should see them."""

    def __init__(self, B, Hq, Hkv, d, inv, interleaved):
        P, self.W = 80, 12
        self.Hq, self.Hkv, self.d, self.inv, self.inter = Hq, Hkv, d, inv, interleaved
        # two layers share the table; the attention below runs on layer 1
        self.kp = torch.zeros(2, P, 16, Hkv, d, dtype=torch.bfloat16, device="cuda")
        self.vp = torch.zeros_like(self.kp)
        self.pt = torch.full((B, self.W), -1, dtype=torch.int32, device="cuda")
        self.ln, self.refs = i32([0] * B), i32([0] * P)
        self.keys = [torch.zeros(0, Hkv, d, dtype=torch.bfloat16) for _ in range(B)]
        self.values = list(self.keys)
        self.g = torch.Generator().manual_seed(d)

    def resize(self, lens):
        ea.attn_pages_resize(self.pt, self.ln, i32(lens), self.refs, self.kp, self.vp)
        for b, n in enumerate(lens):
            self.keys[b], self.values[b] = self.keys[b][:n], self.values[b][:n]

    def fork(self, src, dst):
        ea.attn_pages_fork(self.pt, self.ln, self.refs, i32(src), i32(dst), self.kp, self.vp)
        for a, b in zip(src, dst):
            self.keys[b], self.values[b] = self.keys[a], self.values[a]

    def tokens(self, T):
        x = torch.randn(T, self.Hq + 2 * self.Hkv, self.d, generator=self.g).bfloat16()
        return x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]

    def append(self, counts):
        """counts[b] new tokens for row b (its length holds them already); returns rotated q."""
        q, k, v = self.tokens(sum(counts))
        cu = np.concatenate([[0], np.cumsum(counts)])
        lens = self.ln.tolist()
        pos = np.concatenate([np.arange(lens[b] - n, lens[b]) for b, n in enumerate(counts)])
        one = all(n == 1 for n in counts)
        for layer in range(2):
            out = ea.attn_append_paged(q.cuda(), k.cuda(), v.cuda(), self.kp[layer],
                                       self.vp[layer], self.pt, self.ln,
                                       None if one else i32(cu), self.inv,
                                       interleaved=self.inter)
        r, size = ref.rotate(np64(q), pos, np64(self.inv.cpu()), 1.0, self.inter)
        ref.check_rotated(out, r, size)
        turned = ea.attn_rope(None, k.cuda(), self.inv, i32(pos), interleaved=self.inter)[1].cpu()
        for b in range(len(counts)):
            self.keys[b] = torch.cat([self.keys[b], turned[cu[b]:cu[b + 1]]])
            self.values[b] = torch.cat([self.values[b], v[cu[b]:cu[b + 1]]])
            assert len(self.keys[b]) == lens[b]
        return out, cu

    def check_decode(self, q, what):
        o, lse = ea.attn_decode_paged(q, self.kp[1], self.vp[1], self.pt, self.ln, num_splits=3)
        torch.cuda.synchronize()
        assert ea.attn_device_status() == ea.ATTN_OK
        n = max(map(len, self.keys))
        pad = lambda x: np.stack([np.pad(np64(t), ((0, n - len(t)), (0, 0), (0, 0)))  # noqa: E731
                                  for t in x])
        ro, rl = oracle.attn_decode(np64(q.cpu()), pad(self.keys), pad(self.values),
                                    self.ln.cpu().numpy(), self.d ** -0.5)
        compare(o, lse, ro, rl, what)
        return o, lse


@pytest.mark.parametrize("Hq,Hkv,d,rot,interleaved", [(8, 2, 128, 128, False),
                                                      (4, 4, 64, 32, True), (4, 1, 256, 64, False)])
def test_serving_loop(Hq, Hkv, d, rot, interleaved):
    B = 6
    s = Server(B, Hq, Hkv, d, ea.attn_rope_inv_freq(rot), interleaved)
    counts = [37, 16, 0, 90, 0, 1]
    s.resize(counts)
    q, cu = s.append(counts)
    o, lse = ea.attn_fwd_paged(q, s.kp[1], s.vp[1], s.pt, i32(cu), s.ln, max_seqlen_q=90)
    for b, n in enumerate(counts):
        if n:
            rows = slice(int(cu[b]), int(cu[b + 1]))
            ro, rl = oracle.attn_fwd(np64(q[rows].cpu())[None], np64(s.keys[b])[None],
                                     np64(s.values[b])[None], d ** -0.5, True)
            compare(o[rows][None], lse[:, rows][None], ro, rl, f"prefill row {b}")
    s.fork([0, 3], [2, 4])                     # continue two prompts twice
    lens = [37, 16, 37, 90, 90, 1]
    for step in range(3):
        lens = [n + 1 for n in lens]
        s.resize(lens)
        q, _ = s.append([1] * B)
        s.check_decode(q, f"decode step {step}")
    assert s.keys[0].shape == s.keys[2].shape and not torch.equal(s.keys[0], s.keys[2])
    lens = [40, 0, 20, 93, 70, 4]              # one row ends, two are cut inside shared pages
    s.resize(lens)
    lens = [41, 0, 21, 94, 74, 5]
    s.resize(lens)
    q, _ = s.append([1, 0, 1, 1, 4, 1])
    last = [int(c) - 1 for c in np.cumsum([1, 0, 1, 1, 4, 1])]
    q1 = q[torch.tensor(last).clamp_min(0)].contiguous()
    before = s.check_decode(q1, "after the cut")
    held = int((s.refs > 0).sum())
    to, live = ea.attn_pages_compact(s.pt, s.ln, s.refs, s.kp, s.vp)
    assert live.item() == held and (to >= held).sum() == 0
    after = s.check_decode(q1, "after the compaction")
    assert all(torch.equal(x, y) for x, y in zip(before, after))
    s.resize([0] * B)
    assert (s.refs == 0).all()


@pytest.mark.parametrize("interleaved,amp", [(False, 1.0), (True, 1.1)])
def test_training_step(interleaved, amp):
    """Gradients of sum(g * attention(rope(q), rope(k), v)).  Tolerance as the backward
    pass's own, 1e-2 in relative L2: its 3e-3 measured, and 2^-9 rms at most for each of
    the three further roundings (rotated q and k, rotated-back gradient)."""
    B, S, Hq, Hkv, d, rot = 2, 200, 4, 2, 128, 64
    g = torch.Generator().manual_seed(4)
    x = torch.randn(B, S, Hq + 2 * Hkv, d, generator=g).bfloat16()
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:].contiguous()
    do = torch.randn(B, S, Hq, d, generator=g).bfloat16()
    pos = torch.randint(0, 300, (B, 1), generator=g, dtype=torch.int32) + \
        torch.arange(S, dtype=torch.int32)
    inv = ea.attn_rope_inv_freq(rot)
    kw = dict(interleaved=interleaved, amplitude=amp)
    xd = x.cuda()
    qr, kr = ea.attn_rope(xd[:, :, :Hq], xd[:, :, Hq:Hq + Hkv], inv, pos.cuda(), **kw)
    o, lse = ea.attn_fwd(qr, kr, v.cuda(), causal=True)
    dqr, dkr, dv = ea.attn_bwd(qr, kr, v.cuda(), o, lse, do.cuda(), causal=True)
    dq, dk = ea.attn_rope_bwd(dqr, dkr, inv, pos.cuda(), **kw)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    iv, p = np64(inv.cpu()), pos.numpy()
    turn = lambda t, sign=1.0: ref.rotate(t, p, iv, amp, interleaved, sign)[0]  # noqa: E731
    Q, K, V, G = np64(q), np64(k), np64(v), np64(do)
    gq, gk, gv = oracle.attn_bwd(turn(Q), turn(K), V, G, d ** -0.5, True)
    for got, want, name in ((dq, turn(gq, -1.0), "dq"), (dk, turn(gk, -1.0), "dk"), (dv, gv, "dv")):
        e = np.linalg.norm(np64(got.cpu()) - want) / np.linalg.norm(want)
        assert e <= 1e-2, (name, e)
    # the reference's own gradient against differences of the loss, in fp64
    loss = lambda a, b: (oracle.attn_fwd(turn(a), turn(b), V, d ** -0.5, True)[0] * G).sum()  # noqa: E731
    rng = np.random.default_rng(0)
    for arr, grad, which in ((Q, turn(gq, -1.0), 0), (K, turn(gk, -1.0), 1)):
        u = rng.standard_normal(arr.shape)
        h = 1e-5
        lo, hi = ((loss(arr - h * u, K), loss(arr + h * u, K)) if which == 0 else
                  (loss(Q, arr - h * u), loss(Q, arr + h * u)))
        want = (grad * u).sum()
        assert abs((hi - lo) / (2 * h) - want) <= 1e-6 * np.linalg.norm(grad) * np.linalg.norm(u)
