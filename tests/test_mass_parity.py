"""The attention weight that keys accumulate, on the GPU against fp64."""
import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _thin_ref as ref
from tests._parity import compare, np64

pytestmark = pytest.mark.gpu

NAN = float("nan")


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Rows:
    """Rows of given lengths in a paged cache with large junk behind them."""

    def __init__(self, lens, Hq, Hkv, d, slots=None, seed=0, width=None):
        g = torch.Generator().manual_seed(seed)
        self.g, self.lens, self.Hq, self.Hkv, self.d = g, lens, Hq, Hkv, d
        pages = [(max(n, 0) + 15) // 16 for n in lens]
        self.W = width or max(max(pages), 1) + 1
        self.P = sum(pages) + 2
        perm = torch.randperm(self.P, generator=g).tolist()
        self.table = [[-1] * self.W for _ in lens]
        at = 0
        for b, n in enumerate(pages):
            self.table[b][:n] = perm[at:at + n]
            at += n
        self.k = torch.randn(self.P, 16, Hkv, d, generator=g).bfloat16()
        self.v = torch.randn(self.P, 16, Hkv, d, generator=g).bfloat16()
        for b, n in enumerate(lens):
            if n > 0 and n % 16:
                self.k[self.table[b][n // 16], n % 16:] *= 16
        self.slots = slots or self.W * 16
        # entries behind a row's length must not be touched: a bit pattern to tell
        self.mass = torch.rand(len(lens), Hkv, self.slots, generator=g)
        self.pos = torch.randint(0, 9999, self.mass.shape, generator=g, dtype=torch.int32)

    def q(self, n):
        return torch.randn(n, self.Hq, self.d, generator=self.g).bfloat16()

    def keys(self, b):
        n = max(self.lens[b], 0)
        return (ref.gather(x.float().numpy(), self.table[b], n) for x in (self.k, self.v))


def check_decode(r, q, o, lse, out, pos, last, scale, sink=None, mass=None):
    G = r.Hq // r.Hkv
    mass = r.mass if mass is None else mass
    ro, rl = np.zeros(q.shape), np.zeros(q.shape[:2])
    for b, n in enumerate(r.lens):
        k, v = r.keys(b)
        ro[b], rl[b], w = ref.attend(np64(q[b]), k, v, scale, sink)
        n = max(n, 0)
        for h in range(r.Hkv):
            base = mass[b, h, :n].double().numpy().copy()
            if n:
                base[-1] = 0
            ref.check_mass(out[b, h, :n].double().cpu().numpy(), base,
                           w[h * G:(h + 1) * G].sum(0), (b, h))
            assert torch.equal(out[b, h, n:].cpu(), mass[b, h, n:])
            if pos is not None:
                want = r.pos[b, h].clone()
                if n:
                    want[n - 1] = n - 1 if last is None else last[b]
                assert torch.equal(pos[b, h].cpu(), want)
    compare(o, lse, ro, rl, "decode with masses")


@pytest.mark.parametrize("Hq,Hkv,d,splits", [(4, 1, 64, 1), (6, 2, 128, 3), (8, 8, 256, 8),
                                             (34, 2, 64, 64), (40, 1, 256, 5), (132, 1, 128, 2)])
@pytest.mark.parametrize("sink", [False, True])
def test_decode(Hq, Hkv, d, splits, sink):
    lens = [0, 1, 16, 17, 100, 31, 1500]
    r = Rows(lens, Hq, Hkv, d, seed=Hq + d)
    q = r.q(len(lens))
    s = torch.randn(Hq, generator=r.g) * 3 if sink else None
    if sink:
        s[0], s[-1] = -float("inf"), 40.0
    mass, pos, last = r.mass.cuda(), r.pos.cuda(), [b * 1000 for b in range(len(lens))]
    args = q.cuda(), r.k.cuda(), r.v.cuda(), i32(r.table), i32(lens)
    o, lse = ea.attn_decode_paged_mass(*args, mass, pos, i32(last), num_splits=splits,
                                       sink_logit=s.cuda() if sink else None)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    check_decode(r, q, o, lse, mass, pos, last, d ** -0.5, s.double().numpy() if sink else None)
    plain = ea.attn_decode_paged_sink(*args, s.cuda(), num_splits=splits) if sink else \
        ea.attn_decode_paged(*args, num_splits=splits)
    assert torch.equal(o.view(torch.int16), plain[0].view(torch.int16))
    assert torch.equal(lse.view(torch.int32), plain[1].view(torch.int32))


@pytest.mark.parametrize("slots", [112, 113, 119, 500])
def test_decode_slots_scale_and_out_of_place(slots):
    lens = [112, 3, 0]
    r = Rows(lens, 4, 2, 64, slots=slots, seed=slots)
    q = r.q(3)
    mass, out = r.mass.cuda(), r.mass.cuda()
    o, lse = ea.attn_decode_paged_mass(q.cuda(), r.k.cuda(), r.v.cuda(), i32(r.table), i32(lens),
                                       mass, mass_out=out, scale=0.3)
    torch.cuda.synchronize()
    assert torch.equal(mass.cpu(), r.mass)
    check_decode(r, q, o, lse, out, None, None, 0.3)
    # again, over what it left: the same numbers
    again = torch.full_like(out, NAN)
    ea.attn_decode_paged_mass(q.cuda(), r.k.cuda(), r.v.cuda(), i32(r.table), i32(lens),
                              mass, mass_out=again, scale=0.3)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        assert torch.equal(again[b, :, :n], out[b, :, :n])
        assert torch.isnan(again[b, :, n:]).all()
    assert ea.attn_device_status() == ea.ATTN_OK


def test_the_newest_tokens_old_mass_is_not_read():
    r = Rows([33, 17], 4, 2, 128, seed=5)
    r.mass[0, :, 32] = NAN
    r.mass[1, :, 16] = float("inf")
    mass = r.mass.cuda()
    q = r.q(2)
    o, lse = ea.attn_decode_paged_mass(q.cuda(), r.k.cuda(), r.v.cuda(), i32(r.table),
                                       i32(r.lens), mass)
    torch.cuda.synchronize()
    check_decode(r, q, o, lse, mass, None, None, 128 ** -0.5)


def test_decode_lengths_out_of_range():
    r = Rows([20, 20, 20], 2, 2, 64, slots=30, seed=3)
    mass = r.mass.cuda()
    q = r.q(3)
    for bad in (-1, 31, 49, 2 ** 31 - 1, -2 ** 31):
        got = mass.clone()
        ea.attn_decode_paged_mass(q.cuda(), r.k.cuda(), r.v.cuda(), i32([t[:2] + [0] for t in
                                  r.table]), i32([20, bad, 20]), got)
        torch.cuda.synchronize()
        assert ea.attn_device_status() == ea.ATTN_ERR_BAD_INPUT
        assert torch.equal(got[1], mass[1]) and not torch.equal(got[0], mass[0])


def test_decode_captured_on_another_stream():
    lens = [100, 555]
    r = Rows(lens, 8, 2, 128, seed=13)
    q = r.q(2)
    args = q.cuda(), r.k.cuda(), r.v.cuda(), i32(r.table), i32(lens)
    mass, pos = r.mass.cuda(), r.pos.cuda()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    o, lse = ea.attn_decode_paged_mass(*args, mass, pos, stream=other)
    other.synchronize()
    check_decode(r, q, o, lse, mass, pos, None, 128 ** -0.5)
    first = mass.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ea.attn_decode_paged_mass(*args, mass, pos)
    mass.copy_(r.mass.cuda())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(mass, first)
    assert ea.attn_device_status() == ea.ATTN_OK
