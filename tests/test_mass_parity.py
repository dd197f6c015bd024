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


# ------------------------------------------------------------------ blocks of queries

def block_reference(r, q, cu, causal, window, n_sink, scale, sink=None):
    """lse [Hq, T] and per row the weights [Hkv, n] in fp64."""
    lse, w = np.full((r.Hq, q.shape[0]), -np.inf), []
    G = r.Hq // r.Hkv
    for b, n in enumerate(r.lens):
        k, v = r.keys(b)
        got = np.zeros((r.Hkv, len(k)))
        for i in range(cu[b + 1] - cu[b]):
            seen = ref.seen_keys(i, cu[b + 1] - cu[b], len(k), causal, window, n_sink)
            _, z, p = ref.attend(np64(q[cu[b] + i]), k, v, scale, sink, seen)
            lse[:, cu[b] + i] = z
            got += p.reshape(r.Hkv, G, -1).sum(1)
        w.append(got)
    return lse, w


def check_block(r, w, out, new, mass=None):
    mass = r.mass if mass is None else mass
    for b, n in enumerate(r.lens):
        base = mass[b, :, :n].double().numpy().copy()
        base[:, n - new[b]:] = 0
        ref.check_mass(out[b, :, :n].double().cpu().numpy(), base, w[b], b)
        assert torch.equal(out[b, :, n:].cpu(), mass[b, :, n:])


MASKS = [(True, 0, 0), (False, 0, 0), (True, 7, 0), (True, 100, 5), (True, 1, 300)]


@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 64), (8, 2, 128), (6, 2, 64), (4, 1, 256), (5, 1, 256),
                                      (10, 2, 128)])
@pytest.mark.parametrize("causal,window,n_sink", MASKS)
def test_blocks(Hq, Hkv, d, causal, window, n_sink):
    lens = [1, 16, 129, 300, 257, 40, 0, 530]
    nq = [1, 16, 5, 130, 257, 0, 0, 33]
    r = Rows(lens, Hq, Hkv, d, seed=Hq + d + window)
    cu = np.concatenate([[0], np.cumsum(nq)]).tolist()
    q = r.q(cu[-1] + 3)                       # rows behind the last sequence
    q[cu[-1]:] = NAN
    lse, w = block_reference(r, q[:cu[-1]], cu, causal, window, n_sink, d ** -0.5)
    lse = np.concatenate([lse, np.full((Hq, 3), NAN)], 1)
    mass, pos = r.mass.cuda(), r.pos.cuda()
    mass_new = r.mass.clone()
    for b, n in enumerate(lens):
        mass_new[b, :, n - nq[b]:n] = NAN     # of new tokens: not read
    mass = mass_new.cuda()
    out = ea.attn_mass_paged(q.cuda(), torch.tensor(lse).float().cuda(), r.k.cuda(),
                             i32(r.table), i32(cu), i32(lens), mass, pos, max_seqlen_q=257,
                             causal=causal, window=window, n_sink=n_sink)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK and out is mass
    check_block(r, w, out, nq)
    for b, n in enumerate(lens):
        want = r.pos[b].clone()
        want[:, n - nq[b]:n] = torch.arange(n - nq[b], n, dtype=torch.int32)
        assert torch.equal(pos[b].cpu(), want)


def test_lse_of_the_attention_and_more_queries_than_keys():
    """The LSE as attn_fwd_paged returns it: within 1e-3 by its own tests, 1e-4 here, so the
    weights of a query sum to one within that.  Some queries see no key."""
    lens, nq, d = [100, 20, 3], [100, 50, 9], 128
    r = Rows(lens, 4, 2, d, seed=21)
    cu = np.concatenate([[0], np.cumsum(nq)]).tolist()
    q = r.q(cu[-1]).cuda()
    sink = torch.tensor([0.5, -float("inf"), 3.0, 1.0])
    for s in (None, sink):
        o, lse = ea.attn_fwd_paged(q, r.k.cuda(), r.v.cuda(), i32(r.table), i32(cu), i32(lens),
                                   max_seqlen_q=100, sink_logit=None if s is None else s.cuda())
        out = ea.attn_mass_paged(q, lse, r.k.cuda(), i32(r.table), i32(cu), i32(lens),
                                 torch.zeros_like(r.mass).cuda(), max_seqlen_q=100)
        torch.cuda.synchronize()
        _, w = block_reference(r, q.cpu(), cu, True, 0, 0, d ** -0.5,
                               None if s is None else s.double().numpy())
        for b, n in enumerate(lens):
            got = out[b, :, :n].double().cpu().numpy()
            assert np.abs(got - w[b]).max() <= 1e-4 * w[b].max() + 1e-6
            if s is None:
                assert abs(got.sum() - 4 * min(nq[b], n)) <= 1e-4 * 4 * n
    assert ea.attn_device_status() == ea.ATTN_OK


@pytest.mark.parametrize("Hq,Hkv,d", [(130, 1, 64), (134, 1, 64), (70, 1, 256), (67, 1, 256)])
def test_groups_larger_than_a_query_tile(Hq, Hkv, d):
    lens, nq = [33, 300], [3, 2]
    r = Rows(lens, Hq, Hkv, d, seed=Hq)
    cu = [0, 3, 5]
    q = r.q(5)
    lse, w = block_reference(r, q, cu, True, 0, 0, d ** -0.5)
    out = ea.attn_mass_paged(q.cuda(), torch.tensor(lse).float().cuda(), r.k.cuda(),
                             i32(r.table), i32(cu), i32(lens), r.mass.cuda(), max_seqlen_q=3)
    torch.cuda.synchronize()
    check_block(r, w, out, nq)
    assert ea.attn_device_status() == ea.ATTN_OK


@pytest.mark.parametrize("lens,nq,Hkv", [([9000], [32], 2), ([4000, 5, 2500], [2, 5, 600], 1),
                                         ([300] * 40, [1] * 40, 3)])
def test_many_key_tiles(lens, nq, Hkv):
    """Key tiles shared by CTAs, query tiles kept from one key tile to the next; new tokens
    and positions given."""
    d = 64
    r = Rows(lens, 2 * Hkv, Hkv, d, seed=len(lens))
    cu = np.concatenate([[0], np.cumsum(nq)]).tolist()
    q = r.q(cu[-1])
    lse, w = block_reference(r, q, cu, True, 0, 0, d ** -0.5)
    fresh = [min(n, 7 * b + 1) for b, n in enumerate(lens)]
    fresh[0] = lens[0]
    given = list(fresh)
    given[0] = 10 ** 9                        # taken into the row's length
    pos, last = r.pos.cuda(), [3 * n for n in lens]
    args = (q.cuda(), torch.tensor(lse).float().cuda(), r.k.cuda(), i32(r.table), i32(cu),
            i32(lens))
    out = torch.empty_like(r.mass).cuda()
    out.copy_(r.mass)
    got = ea.attn_mass_paged(*args, r.mass.cuda(), pos, i32(last), i32(given),
                             max_seqlen_q=max(nq), mass_out=out)
    torch.cuda.synchronize()
    assert got is out
    check_block(r, w, out, fresh)
    for b, n in enumerate(lens):
        want = r.pos[b].clone()
        want[:, n - fresh[b]:n] = last[b] - torch.arange(fresh[b] - 1, -1, -1, dtype=torch.int32)
        assert torch.equal(pos[b].cpu(), want)
    again = torch.empty_like(out)
    ea.attn_mass_paged(*args, r.mass.cuda(), None, None, i32(given), max_seqlen_q=max(nq),
                       mass_out=again)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        assert torch.equal(again[b, :, :n], out[b, :, :n])
    assert ea.attn_device_status() == ea.ATTN_OK


def test_block_inputs_out_of_range():
    r = Rows([40, 40, 40], 2, 1, 64, slots=45, seed=9)
    q, lse = r.q(12).cuda(), torch.zeros(2, 12).cuda()
    for cu, lens in (([0, 4, 2, 12], [40, 40, 40]), ([-1, 4, 8, 12], [40, 40, 40]),
                     ([0, 4, 8, 13], [40, 40, 40]), ([0, 4, 8, 12], [40, 46, 40]),
                     ([0, 4, 8, 12], [40, -3, 40]), ([0, 2, 10, 12], [40, 40, 40])):
        mass = r.mass.cuda()
        ea.attn_mass_paged(q, lse, r.k.cuda(), i32([t[:3] + [0] for t in r.table]), i32(cu),
                           i32(lens), mass, max_seqlen_q=7)
        torch.cuda.synchronize()
        assert ea.attn_device_status() == ea.ATTN_ERR_BAD_INPUT
        left = [b for b in range(3) if torch.equal(mass[b].cpu(), r.mass[b])]
        assert 0 < len(left) < 3, (cu, lens)
    table = [list(t) for t in r.table]
    table[1][1] = r.P
    ea.attn_mass_paged(q, lse, r.k.cuda(), i32(table), i32([0, 4, 8, 12]), i32([40] * 3),
                       r.mass.cuda(), max_seqlen_q=7)
    assert ea.attn_device_status() == ea.ATTN_ERR_BAD_INPUT


def test_block_captured_on_another_stream_and_empty():
    lens, nq, d = [700, 100], [65, 3], 128
    r = Rows(lens, 8, 2, d, seed=17)
    cu = [0, 65, 68]
    q = r.q(68)
    lse, w = block_reference(r, q, cu, True, 0, 0, d ** -0.5)
    args = (q.cuda(), torch.tensor(lse).float().cuda(), r.k.cuda(), i32(r.table), i32(cu),
            i32(lens))
    mass, out = r.mass.cuda(), r.mass.cuda()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    ea.attn_mass_paged(*args, mass, max_seqlen_q=65, mass_out=out, stream=other)
    other.synchronize()
    check_block(r, w, out, nq)
    first = out.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ea.attn_mass_paged(*args, mass, max_seqlen_q=65, mass_out=out)
    out.copy_(r.mass.cuda())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    # no queries at all: the mass is passed on
    none = ea.attn_mass_paged(q[:0].cuda(), torch.zeros(8, 0).cuda(), r.k.cuda(), i32(r.table),
                              i32([0, 0, 0]), i32(lens), mass, max_seqlen_q=0,
                              mass_out=torch.zeros_like(mass))
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        assert torch.equal(none[b, :, :n], mass[b, :, :n])
    assert ea.attn_device_status() == ea.ATTN_OK


@pytest.mark.parametrize("window,n_sink", [(40, 0), (40, 3), (300, 256), (700, 600), (5000, 1), (1, 4000)])
def test_key_tiles_that_no_query_sees(window, n_sink):
    """Between the sink keys and the windows: at the start, in the middle and at the end of the
    rows, for rows without queries and rows shorter than the window."""
    lens, nq, d = [2900, 700, 1700, 4001, 256, 513], [30, 0, 300, 1, 256, 2], 64
    r = Rows(lens, 4, 2, d, seed=window + n_sink)
    cu = np.concatenate([[0], np.cumsum(nq)]).tolist()
    q = r.q(cu[-1])
    lse, w = block_reference(r, q, cu, True, window, n_sink, d ** -0.5)
    out = ea.attn_mass_paged(q.cuda(), torch.tensor(lse).float().cuda(), r.k.cuda(),
                             i32(r.table), i32(cu), i32(lens), r.mass.cuda(), max_seqlen_q=300,
                             window=window, n_sink=n_sink)
    torch.cuda.synchronize()
    check_block(r, w, out, nq)
    assert ea.attn_device_status() == ea.ATTN_OK
