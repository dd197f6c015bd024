"""attn_evict_paged on the GPU against the rule applied token by token: exactly equal."""
import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _thin_ref as ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Cache:
    """Rows of given lengths on a shuffled pool; every element of the pools is distinct
    enough to tell a wrong move."""

    def __init__(self, lens, layers, Hkv, d, slots=None, seed=0, extra=3):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.lens, self.layers, self.Hkv, self.d = list(lens), layers, Hkv, d
        pages = [(n + 15) // 16 for n in lens]
        self.W = max(max(pages), 1) + 1
        self.P = sum(pages) + extra
        perm = torch.randperm(self.P, generator=g).tolist()
        self.table = [[-1] * self.W for _ in lens]
        at = 0
        for b, n in enumerate(pages):
            self.table[b][:n] = perm[at:at + n]
            at += n
        self.slots = slots or self.W * 16
        shape = (layers, B, Hkv, self.slots)
        self.mass = torch.randn(shape, generator=g).exp() * \
            (torch.rand(shape, generator=g) > 0.2)
        self.positions = torch.randint(0, 5, shape, generator=g, dtype=torch.int32) + \
            7 * torch.arange(self.slots, dtype=torch.int32)
        self.k = torch.randn(layers, self.P, 16, Hkv, d, generator=g).bfloat16()
        self.v = torch.randn(layers, self.P, 16, Hkv, d, generator=g).bfloat16()
        self.refs = [0] * self.P
        for row, n in zip(self.table, pages):
            for p in row[:n]:
                self.refs[p] += 1

    def expect(self, keep, n_sink, recent, skip=()):
        m, p = self.mass.clone().numpy(), self.positions.clone().numpy()
        k, v = self.k.clone(), self.v.clone()
        new = []
        for b, (L, K) in enumerate(zip(self.lens, keep)):
            if b in skip or K >= L or K < 0:
                new.append(L)
                continue
            new.append(K)
            for layer in range(self.layers):
                for h in range(self.Hkv):
                    moves = ref.evict(m[layer, b, h], p[layer, b, h], L, K, n_sink, recent)
                    for s, t in moves:
                        for x in (m, p):
                            x[layer, b, h, t] = x[layer, b, h, s]
                        for x in (k, v):
                            x[layer, self.table[b][t // 16], t % 16, h] = \
                                x[layer, self.table[b][s // 16], s % 16, h]
        return m, p, k, v, new

    def run(self, keep, n_sink=0, recent=0, refs=True, skip=(), layered=True, **kw):
        want = self.expect(keep, n_sink, recent, skip)
        cut = (lambda t: t.cuda()) if layered else (lambda t: t[0].cuda())
        self.dm, self.dp, self.dk, self.dv = map(cut, (self.mass, self.positions, self.k, self.v))
        new = ea.attn_evict_paged(self.dm, self.dp, i32(self.table), i32(self.lens), i32(keep),
                                  self.dk, self.dv, i32(self.refs) if refs else None,
                                  n_sink=n_sink, recent=recent, **kw)
        torch.cuda.synchronize()
        self.check(want, new, layered)

    def check(self, want, new, layered=True):
        m, p, k, v, lens = want
        cut = (lambda t: t) if layered else (lambda t: t[0])
        assert new.tolist() == lens
        bits = lambda t: t.contiguous().view(torch.int32).cpu().numpy()  # noqa: E731
        assert np.array_equal(bits(self.dm), cut(m).view(np.int32))
        assert np.array_equal(self.dp.cpu().numpy(), cut(p))
        assert torch.equal(self.dk.cpu().view(torch.int16), cut(k).view(torch.int16))
        assert torch.equal(self.dv.cpu().view(torch.int16), cut(v).view(torch.int16))


@pytest.mark.parametrize("layers,Hkv,d", [(1, 1, 64), (3, 2, 128), (2, 3, 256)])
@pytest.mark.parametrize("n_sink,recent", [(0, 0), (4, 9), (0, 1000)])
def test_rows_of_all_lengths(layers, Hkv, d, n_sink, recent):
    lens = [0, 1, 1, 15, 16, 17, 33, 100, 257, 600]
    c = Cache(lens, layers, Hkv, d, seed=d + n_sink)
    c.run([0, 0, 1, 7, 3, 16, 40, 64, 128, 599], n_sink, recent)
    assert ea.attn_device_status() == ea.ATTN_OK


@pytest.mark.parametrize("L,K", [(5000, 1), (5000, 2500), (5000, 4999), (70000, 9000),
                                 (41000, 40990)])
def test_long_rows(L, K):
    """Past 40,960 slots the keys no longer fit in shared memory."""
    c = Cache([L, 37], 1, 2, 64, seed=L)
    c.run([K, 20], 4, 50)
    assert ea.attn_device_status() == ea.ATTN_OK


def test_ties_infinities_and_nan():
    c = Cache([300, 300, 300, 300, 300, 300], 1, 1, 64, seed=4)
    c.mass[0, 0] = 1.0
    c.mass[0, 1] = 0.0
    c.mass[0, 1, :, ::2] = -0.0
    c.mass[0, 2, :, 50:250:3] = float("inf")
    c.mass[0, 3, :, 100:] = float("nan")
    c.mass[0, 4, :, ::3] = -float("inf")
    c.mass[0, 4, :, 1::3] *= -1.0
    c.mass[0, 5] = torch.finfo(torch.float32).tiny * torch.rand(c.mass[0, 5].shape) * 1e-3
    c.run([100, 150, 90, 120, 60, 150], 2, 5)
    assert ea.attn_device_status() == ea.ATTN_OK


def test_positions_in_any_order():
    """Rows that were cut before: sinks and recent tokens sit anywhere."""
    c = Cache([200, 513], 2, 2, 128, seed=6)
    g = torch.Generator().manual_seed(1)
    for layer in range(2):
        for b, n in enumerate(c.lens):
            for h in range(2):
                c.positions[layer, b, h, :n] = torch.randperm(n, generator=g).int() * 2 - 3
    c.run([64, 100], 8, 30)
    c = Cache([40], 1, 1, 64, seed=8)
    c.positions[0, 0, 0, :40] = torch.arange(40, dtype=torch.int32) - 2 ** 31
    c.positions[0, 0, 0, 39] = 2 ** 31 - 1
    c.run([9], 0, 2 ** 31 - 1)
    assert ea.attn_device_status() == ea.ATTN_OK


def test_without_layers_and_with_more_slots_than_pages():
    c = Cache([100, 64], 1, 2, 64, slots=333, seed=9)
    c.run([30, 64], 4, 4, refs=False, layered=False)
    assert ea.attn_device_status() == ea.ATTN_OK


def test_rows_left_and_reported():
    lens, keep = [100, 100, 100, 100, 100], [50, -1, 20, 20, 99]
    c = Cache(lens, 2, 1, 64, seed=3)
    c.refs[c.table[0][1]] = 2                   # a page that would be written to
    c.refs[c.table[4][6]] = 2                   # the seventh page: slot 96 on, written to
    c.run(keep, skip=(0, 1, 4))
    assert ea.attn_device_status() == ea.ATTN_ERR_BAD_INPUT
    c = Cache(lens, 2, 1, 64, seed=3)
    c.refs[c.table[0][4]] = 2                   # behind the budget: only read
    c.table[2][6] = c.P
    c.table[3][0] = -1
    c.run([50, 100, 20, 20, 20], skip=(2, 3))
    assert ea.attn_device_status() == ea.ATTN_ERR_BAD_INPUT
    c = Cache([60, 60, 60], 1, 1, 64, slots=61, seed=2)
    c.lens = [-5, 62, 60]
    want = Cache([0, 0, 60], 1, 1, 64, slots=61, seed=2)
    new = ea.attn_evict_paged(*[t.cuda() for t in (c.mass, c.positions)], i32(c.table),
                              i32(c.lens), i32([3, 3, 60]), c.k.cuda(), c.v.cuda())
    torch.cuda.synchronize()
    assert new.tolist() == [-5, 62, 60] and want.lens[2] == 60
    assert ea.attn_device_status() == ea.ATTN_ERR_BAD_INPUT


def test_streams_graphs_and_outputs():
    c = Cache([100, 3000], 2, 2, 128, seed=11)
    want = c.expect([30, 1000], 4, 16)
    c.dm, c.dp, c.dk, c.dv = (t.cuda() for t in (c.mass, c.positions, c.k, c.v))
    args = i32(c.table), i32(c.lens), i32([30, 1000]), c.dk, c.dv
    new = i32([7, 7])
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    out = ea.attn_evict_paged(c.dm, c.dp, *args, new_seqlens=new, n_sink=4, recent=16,
                              stream=other)
    other.synchronize()
    assert out is new
    c.check(want, new)
    c.dm.copy_(c.mass), c.dp.copy_(c.positions), c.dk.copy_(c.k), c.dv.copy_(c.v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ea.attn_evict_paged(c.dm, c.dp, *args, n_sink=4, recent=16)
    graph.replay()
    torch.cuda.synchronize()
    c.check(want, out)
    assert ea.attn_device_status() == ea.ATTN_OK


@pytest.mark.parametrize("L,K", [(3000, 1400), (8000, 3999), (8000, 4001), (33, 32), (64, 31)])
@pytest.mark.parametrize("values", [1, 2, 700])
def test_many_equal_masses(L, K, values):
    """Few distinct masses: more keys at the threshold than are listed, the first by slot."""
    c = Cache([L, L], 1, 2, 64, seed=L + values)
    g = torch.Generator().manual_seed(values)
    c.mass = 0.5 + torch.randint(0, values, c.mass.shape, generator=g).float() / 1024
    c.run([K, min(K, L // 3)], 4, 20)
    assert ea.attn_device_status() == ea.ATTN_OK


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_short_rows(d):
    """Enough rows and heads that each selecting CTA moves its own keys and values."""
    g = np.random.default_rng(d)
    lens = g.integers(1, 120, 180).tolist()
    c = Cache(lens, 1, 2, d, seed=d)
    c.run([int(g.integers(0, n + 2)) for n in lens], 2, 6)
    assert ea.attn_device_status() == ea.ATTN_OK


@pytest.mark.parametrize("width", [340, 2600])
def test_rows_of_all_lengths_in_a_wide_table(width):
    """Short, longer and long rows side by side (selected by kernels of their own), in tables
    wider than any of them."""
    lens = [5000, 30, 4096, 4097, 0, 4700, 33, 1] + ([41100, 40960, 40961, 9000] if width > 340
                                                     else [4500])
    c = Cache(lens, 1, 2, 64, seed=width)
    extra = width - len(c.table[0])
    assert extra > 0
    c.table = [list(t) + [-1] * extra for t in c.table]
    keep = [4000, 10, 4095, 20, 0, 4700, 33, 0] + ([4096, 40900, 100, 4097] if width > 340 else [9])
    c.run(keep, 3, 40)
    assert ea.attn_device_status() == ea.ATTN_OK
