"""The operators on shared and thinned caches together, as a server uses them: prompts are
attended, their keys' masses taken, the caches cut to a budget, the rows forked into samples
that decode over their shared prefix and go on collecting masses.  Two layers share the
table; a mirror in fp64 holds what every key head should see."""
import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _thin_ref as ref
from tests._parity import compare, np64

pytestmark = pytest.mark.gpu

LAYERS, P, W = 2, 96, 24


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Server:
    def __init__(self, B, Hq, Hkv, d):
        self.B, self.Hq, self.Hkv, self.d = B, Hq, Hkv, d
        self.g = torch.Generator().manual_seed(d)
        self.kp = torch.zeros(LAYERS, P, 16, Hkv, d, dtype=torch.bfloat16, device="cuda")
        self.vp = torch.zeros_like(self.kp)
        self.pt = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        self.ln, self.refs = i32([0] * B), i32([0] * P)
        self.mass = torch.zeros(LAYERS, B, Hkv, W * 16, device="cuda")
        self.pos = torch.zeros(LAYERS, B, Hkv, W * 16, dtype=torch.int32, device="cuda")
        self.inv = ea.attn_rope_inv_freq(d)
        # keys and values by layer, row and head; the next position of every row
        self.k = [[[np.zeros((0, d)) for _ in range(Hkv)] for _ in range(B)] for _ in range(LAYERS)]
        self.v = [[[np.zeros((0, d)) for _ in range(Hkv)] for _ in range(B)] for _ in range(LAYERS)]
        self.at = [0] * B

    def resize(self, lens):
        ea.attn_pages_resize(self.pt, self.ln, i32(lens) if isinstance(lens, list) else lens,
                             self.refs, self.kp, self.vp)

    def append(self, counts):
        """counts[b] new tokens; returns the rotated queries by layer, and their offsets."""
        T, cu = sum(counts), np.concatenate([[0], np.cumsum(counts)]).tolist()
        pos = np.concatenate([np.arange(self.at[b], self.at[b] + n)
                              for b, n in enumerate(counts)]).astype(np.int32)
        out = []
        for layer in range(LAYERS):
            x = torch.randn(T, self.Hq + 2 * self.Hkv, self.d, generator=self.g).bfloat16().cuda()
            q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]
            # positions are no longer slots once a row was cut: rotated here, stored as they are
            q, k = ea.attn_rope(q, k, self.inv, torch.from_numpy(pos).cuda())
            ea.attn_append_paged(None, k, v, self.kp[layer], self.vp[layer], self.pt, self.ln,
                                 i32(cu))
            out.append(q.contiguous())
            for b, n in enumerate(counts):
                rows = slice(cu[b], cu[b + 1])
                for h in range(self.Hkv):
                    self.k[layer][b][h] = np.concatenate([self.k[layer][b][h],
                                                          np64(k[rows, h].cpu())])
                    self.v[layer][b][h] = np.concatenate([self.v[layer][b][h],
                                                          np64(v[rows, h].cpu())])
        for b, n in enumerate(counts):
            self.at[b] += n
        return out, cu

    def attend(self, layer, b, q, i=0, Lq=1):
        """One query [Hq, d] of row b over what its heads hold -> o, lse, weights by head."""
        G = self.Hq // self.Hkv
        o, lse, w = np.zeros(q.shape), np.zeros(self.Hq), []
        for h in range(self.Hkv):
            k, v = self.k[layer][b][h][:, None], self.v[layer][b][h][:, None]
            r = ref.attend(q[h * G:(h + 1) * G], k, v, self.d ** -0.5,
                           seen=ref.seen_keys(i, Lq, len(k), True, 0, 0))
            o[h * G:(h + 1) * G], lse[h * G:(h + 1) * G] = r[:2]
            w.append(r[2].sum(0))
        return o, lse, w

    def evict(self, keep, **kw):
        before = self.mass.cpu().numpy(), self.pos.cpu().numpy()
        lens = self.ln.tolist()
        new = ea.attn_evict_paged(self.mass, self.pos, self.pt, self.ln, i32(keep), self.kp,
                                  self.vp, self.refs, **kw)
        for b, K in enumerate(new.tolist()):
            if K == lens[b]:
                continue
            for layer in range(LAYERS):
                for h in range(self.Hkv):
                    moves = ref.evict(before[0][layer, b, h], before[1][layer, b, h], lens[b], K,
                                      kw.get("n_sink", 0), kw.get("recent", 0))
                    for x in (self.k, self.v):
                        for s, t in moves:
                            x[layer][b][h][t] = x[layer][b][h][s]
                        x[layer][b][h] = x[layer][b][h][:K]
        return new

    def fork(self, src, dst):
        ea.attn_pages_fork(self.pt, self.ln, self.refs, i32(src), i32(dst), self.kp, self.vp)
        self.mass[:, dst], self.pos[:, dst] = self.mass[:, src], self.pos[:, src]
        for a, b in zip(src, dst):
            for x in (self.k, self.v):
                for layer in range(LAYERS):
                    x[layer][b] = [t.copy() for t in x[layer][a]]
            self.at[b] = self.at[a]


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 4, 64), (3, 1, 256)])
def test_prompt_cut_fork_and_decode(Hq, Hkv, d):
    B = 5
    s = Server(B, Hq, Hkv, d)
    # ---- two prompts, attended and weighed
    counts = [300, 170, 0, 0, 0]
    s.resize(counts)
    qs, cu = s.append(counts)
    for layer in range(LAYERS):
        o, lse = ea.attn_fwd_paged(qs[layer], s.kp[layer], s.vp[layer], s.pt, i32(cu), s.ln,
                                   max_seqlen_q=300)
        ea.attn_mass_paged(qs[layer], lse, s.kp[layer], s.pt, i32(cu), s.ln, s.mass[layer],
                           s.pos[layer], max_seqlen_q=300)
        for b in (0, 1):
            n = counts[b]
            want = np.zeros((Hkv, n))
            for i in range(n):
                want += np.array(s.attend(layer, b, np64(qs[layer][cu[b] + i].cpu()), i, n)[2])
            # weights of the kernel's own LSE, which its tests hold to 1e-3; 2e-4 here
            got = s.mass[layer, b, :, :n].double().cpu().numpy()
            assert np.abs(got - want).max() <= 2e-4 * want.max()
            assert (s.pos[layer, b, :, :n].cpu() == torch.arange(n)).all()
    # ---- cut to a budget, pages given back
    held = int((s.refs > 0).sum())
    new = s.evict([128, 100, 0, 0, 0], n_sink=4, recent=16)
    assert new.tolist() == [128, 100, 0, 0, 0] and s.ln.tolist() == counts
    s.resize(new)
    assert int((s.refs > 0).sum()) == 8 + 7 < held
    pos = s.pos[:, 0, :, :128].cpu()
    assert all(set(range(4)) | set(range(284, 300)) <= set(x.tolist()) for x in pos.view(-1, 128))
    # ---- samples of both, decoding over their shared prefix
    s.fork([0, 0, 1], [2, 3, 4])
    lens = [128, 100, 128, 128, 100]
    groups, members, prefix = i32([0, 3, 5]), i32([0, 2, 3, 1, 4]), i32([128, 100])
    for step in range(3):
        lens = [n + 1 for n in lens]
        s.resize(lens)
        qs, _ = s.append([1] * B)
        for layer in range(LAYERS):
            args = qs[layer], s.kp[layer], s.vp[layer], s.pt, s.ln
            before = s.mass[layer].cpu().numpy()
            o1, l1 = ea.attn_decode_paged_shared(*args, groups, prefix, members)
            o2, l2 = ea.attn_decode_paged_mass(*args, s.mass[layer], s.pos[layer],
                                               i32([n - 1 for n in s.at]), num_splits=2)
            ro, rl = np.zeros((B, Hq, d)), np.zeros((B, Hq))
            for b in range(B):
                ro[b], rl[b], w = s.attend(layer, b, np64(qs[layer][b].cpu()))
                for h in range(Hkv):
                    base = before[b, h, :lens[b]].astype(np.float64)
                    base[-1] = 0
                    ref.check_mass(s.mass[layer, b, h, :lens[b]].double().cpu().numpy(), base, w[h])
                assert (s.pos[layer, b, :, lens[b] - 1] == s.at[b] - 1).all()
            compare(o1, l1, ro, rl, f"shared decode, step {step}")
            compare(o2, l2, ro, rl, f"decode with masses, step {step}")
    # ---- a cut inside pages that others hold too is refused, row by row
    assert ea.attn_device_status() == ea.ATTN_OK
    new = s.evict([64, 200, 131, 60, 103], recent=8)
    assert new.tolist() == [131, 103, 131, 131, 103]
    assert ea.attn_device_status() == ea.ATTN_ERR_BAD_INPUT
    # ---- once a row is alone, it is cut again
    s.resize([131, 103, 0, 0, 0])
    s.resize(s.evict([64, 64, 0, 0, 0], recent=8))
    lens = [65, 65, 0, 0, 0]
    s.resize(lens)
    qs, _ = s.append([1, 1, 0, 0, 0])
    q = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda")
    q[:2] = qs[1]
    for x in (s.k, s.v):
        for b in (2, 3, 4):
            x[1][b] = [t[:0] for t in x[1][b]]
    o, lse = ea.attn_decode_paged_shared(q, s.kp[1], s.vp[1], s.pt, s.ln, i32([0, 1]), i32([40]))
    ro, rl = np.zeros((B, Hq, d)), np.zeros((B, Hq))
    for b in range(B):
        ro[b], rl[b], _ = s.attend(1, b, np64(q[b].cpu()))
    compare(o, lse, ro, rl, "after the second cut")
    s.resize([0] * B)
    assert (s.refs == 0).all() and ea.attn_device_status() == ea.ATTN_OK
