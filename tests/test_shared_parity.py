"""attn_decode_paged_shared on the GPU against fp64: the decode of rows that share leading
pages."""
import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _thin_ref as ref
from tests._parity import assert_masked_rows_zero, compare, np64

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Batch:
    """groups: (prefix length, [row lengths]); rows stand in the table in shuffled order,
    `alone` rows belong to no group.  A row's keys before the whole pages of its prefix are
    the group's."""

    def __init__(self, groups, Hq, Hkv, d, alone=(), seed=0, short=False):
        g = torch.Generator().manual_seed(seed)
        self.groups, self.Hq, self.Hkv, self.d = groups, Hq, Hkv, d
        lens = [n for _, rows in groups for n in rows] + list(alone)
        B = len(lens)
        order = torch.randperm(B, generator=g).tolist()
        self.W = max((n + 15) // 16 for n in lens + [p for p, _ in groups] + [1]) + 1
        P = sum((n + 15) // 16 for n in lens) + sum((p + 15) // 16 for p, _ in groups) + 4
        pages = iter(torch.randperm(P, generator=g).tolist())
        self.P = P
        self.table, self.lens = [[-1] * self.W for _ in range(B)], [0] * B
        self.cu, self.rows = [0], []
        e = 0
        for prefix, rows in groups:
            shared = [next(pages) for _ in range(min(prefix, max(rows, default=0)) // 16)]
            for n in rows:
                b, need = order[e], (n + 15) // 16
                own = [next(pages) for _ in range(max(0, need - len(shared)))]
                self.table[b][:need] = (shared + own)[:need]
                self.lens[b] = n
                self.rows.append(b)
                e += 1
            self.cu.append(len(self.rows))
        for n in alone:
            b, need = order[e], (n + 15) // 16
            self.table[b][:need] = [next(pages) for _ in range(need)]
            self.lens[b] = n
            e += 1
        self.prefix = [p for p, _ in groups]
        self.q = torch.randn(B, Hq, d, generator=g).bfloat16()
        self.k = torch.randn(P, 16, Hkv, d, generator=g).bfloat16()
        self.v = torch.randn(P, 16, Hkv, d, generator=g).bfloat16()
        for b, n in enumerate(self.lens):      # junk behind the last key
            if n % 16:
                self.k[self.table[b][n // 16], n % 16:] *= 16
        self.sink = torch.randn(Hq, generator=g) * 3

    def args(self):
        return (self.q.cuda(), self.k.cuda(), self.v.cuda(), i32(self.table), i32(self.lens))

    def run(self, scale=None, sink=False, rows="list", check=True, status=ea.ATTN_OK, **kw):
        s = self.sink.cuda() if sink else None
        o, lse = ea.attn_decode_paged_shared(
            *self.args(), i32(self.cu), i32(self.prefix),
            i32(self.rows) if rows == "list" else rows, sink_logit=s, scale=scale, **kw)
        torch.cuda.synchronize()
        assert ea.attn_device_status() == status
        if check:
            self.check(o, lse, scale, sink)
        return o, lse

    def check(self, o, lse, scale=None, sink=False):
        ro, rl = np.zeros(self.q.shape), np.zeros(self.q.shape[:2])
        scale = self.d ** -0.5 if scale is None else scale
        for b, n in enumerate(self.lens):
            k, v = (ref.gather(x.float().numpy(), self.table[b], n) for x in (self.k, self.v))
            ro[b], rl[b], _ = ref.attend(np64(self.q[b]), k, v, scale,
                                         self.sink.double().numpy() if sink else None)
        compare(o, lse, ro, rl, "shared decode")
        if not sink:
            assert_masked_rows_zero(o, np.array(self.lens) == 0)


GROUPS = [
    [(64, [70, 65])],                                  # two samples
    [(16, [17, 16, 40, 300]), (200, [201, 250]), (0, [5, 9]), (500, [600])],
    [(1000, [1001 + 3 * i for i in range(17)])],
    [(2047, [2048, 2100, 2047, 2040, 33, 0, 1]), (31, [31, 40, 15])],  # rows that end inside
    [(128, [128] * 3), (130, [144] * 2)],              # nothing or little of their own
]


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 64), (8, 2, 128), (6, 2, 256), (5, 5, 64), (12, 1, 128),
                                      (3, 1, 256)])
@pytest.mark.parametrize("groups", range(len(GROUPS)))
def test_groups(Hq, Hkv, d, groups):
    b = Batch(GROUPS[groups], Hq, Hkv, d, alone=[50, 0, 333], seed=groups + d)
    b.run(sink=groups % 2 == 1)


@pytest.mark.parametrize("n,Hq,Hkv,d", [(31, 4, 1, 128), (32, 4, 1, 128), (33, 4, 1, 128),
                                        (64, 4, 1, 64), (65, 8, 2, 64), (130, 4, 1, 128),
                                        (33, 8, 2, 256), (100, 3, 1, 256), (2, 200, 1, 64),
                                        (3, 140, 1, 256)])
def test_rows_around_a_query_tile(n, Hq, Hkv, d):
    """Items of up to 128 rows keep one tile in both streams, of up to 256 two tiles."""
    b = Batch([(400, [400 + i % 40 for i in range(n)])], Hq, Hkv, d, seed=n)
    b.run()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_prefix_large_scores(d):
    """Scores that grow along the prefix (the running maximum moves often) and a key that
    takes nearly all of a row's weight."""
    b = Batch([(5000, [5000 + 7 * i for i in range(9)])], 8, 2, d, seed=d)
    table = b.table[b.rows[0]]
    for j in range(312):
        b.k[table[j]] *= 0.02 * (j + 1)
    b.run(num_splits=3)
    b.run(scale=1.0)


@pytest.mark.parametrize("splits", [1, 2, 64])
def test_rows_in_order_splits_and_bits(splits):
    b = Batch([(96, [100, 400, 96]), (48, [64, 60])], 8, 4, 128, seed=splits)
    inverse = torch.tensor(b.rows)
    b.q, b.table = b.q[inverse], [b.table[i] for i in b.rows]
    b.lens = [b.lens[i] for i in b.rows]
    o, lse = b.run(rows=None, num_splits=splits)
    for _ in range(3):
        again = b.run(rows=None, num_splits=splits, check=False)
        assert torch.equal(o.view(torch.int16), again[0].view(torch.int16))
        assert torch.equal(lse, again[1])


def test_no_groups_and_no_rows():
    b = Batch([], 4, 2, 64, alone=[100, 3, 0], seed=2)
    o, lse = b.run()
    plain = ea.attn_decode_paged(*b.args(), num_splits=8)
    compare(o, lse, np64(plain[0].float().cpu()), np64(plain[1].cpu()), "no groups")
    args = b.args()
    o, lse = ea.attn_decode_paged_shared(args[0][:0], *args[1:3], args[3][:0], args[4][:0], i32([0]),
                                         i32([]), want_lse=False)
    assert o.shape == (0, 4, 64) and lse is None


def test_bad_groups_are_reported_and_change_nothing():
    def batch():
        return Batch([(64, [70, 65, 64]), (100, [130, 99])], 4, 2, 128, alone=[20], seed=8)

    bad = ea.ATTN_ERR_BAD_INPUT
    for cu in ([0, 6, 5], [-1, 3, 5], [0, 3, 7], [4, 3, 5], [0, 2 ** 31 - 1, 5]):
        b = batch()
        b.cu = cu
        b.run(status=bad)
    for e, row in ((1, -1), (3, 6), (0, 2 ** 31 - 1)):
        b = batch()
        b.rows[e] = row
        b.run(status=bad)
    b = batch()
    b.rows[4] = b.rows[0]                        # in both groups: belongs to the first
    b.run(status=bad)
    b = batch()
    b.rows[2] = b.rows[0]                        # twice in one group
    b.run(status=bad)
    for p in (-5, 10 ** 6):
        b = batch()
        b.prefix[0] = p
        if p < 0:
            b.run(status=bad)
        else:                                    # all pages of the longest row are "shared"
            b.table[b.rows[1]][4] = b.table[b.rows[2]][4] = b.table[b.rows[0]][4]
            b.run(status=bad)
    b = batch()
    b.cu, b.rows = [1, 3, 4], b.rows             # entries before and behind: no group
    b.run()


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 64), (8, 2, 128), (6, 2, 256), (24, 3, 128)])
def test_groups_large_enough_to_share(Hq, Hkv, d):
    """Prefixes on both sides of what sharing is worth, and bad pages in them."""
    b = Batch([(700, [700 + i for i in range(9)]), (16, [17 + i for i in range(40)]),
               (260, [261, 300, 280, 259, 3, 0, 290, 266, 270]), (2100, [2120]), (48, [50, 60])],
              Hq, Hkv, d, alone=[5, 700], seed=d + Hq)
    b.run(sink=True)
    c = Batch([(700, [704] * 40)], Hq, Hkv, d, seed=d)
    for row in c.rows:
        c.table[row][1], c.table[row][7] = -1, c.P
    o, lse = c.run(status=ea.ATTN_ERR_BAD_INPUT, check=False)
    unused = next(p for p in range(c.P) if all(p not in t for t in c.table))
    c.k[unused] = c.v[unused] = 0
    for row in c.rows:
        c.table[row][1] = c.table[row][7] = unused
    c.check(o, lse)


@pytest.mark.parametrize("groups,most", [(40, 1), (100, 2), (70, 7), (600, 1), (33, 20)])
def test_more_groups_than_warps(groups, most):
    rows = [1 + 7 * g % most for g in range(groups)]
    b = Batch([(16 * (g % 5) + 200 * (g % 9 == 8), [16 * (g % 5) + 200 * (g % 9 == 8) + g % 3 + i
                                                    for i in range(n)])
               for g, n in enumerate(rows)], 4, 2, 64, alone=[3, 40], seed=groups)
    b.run()


def test_lengths_and_pages_out_of_range():
    b = Batch([(64, [70, 65, 64])], 4, 2, 128, seed=9)
    b.lens[b.rows[1]] = -7
    o, lse = b.run(status=ea.ATTN_ERR_BAD_INPUT, check=False)
    b.lens[b.rows[1]] = 0
    b.check(o, lse)
    for page in (-1, b.P, 2 ** 31 - 1):
        c = Batch([(64, [70, 65, 64])], 4, 2, 128, seed=9)
        for row in c.rows:
            c.table[row][1] = page
        o, lse = c.run(status=ea.ATTN_ERR_BAD_INPUT, check=False)
        unused = next(p for p in range(c.P) if all(p not in t for t in c.table))
        c.k[unused] = c.v[unused] = 0            # such a page reads zeros
        for row in c.rows:
            c.table[row][1] = unused
        c.check(o, lse)


def test_streams_graphs_outputs_and_shared_workspace():
    b = Batch([(600, [610, 700, 800])], 8, 2, 128, alone=[64], seed=12)
    args = b.args()
    more = i32(b.cu), i32(b.prefix), i32(b.rows)
    need = ea.attn_decode_shared_workspace_size(4, 8, 2, 128, 1, 3, b.W, 2)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(args[0]), torch.empty(4, 8, device="cuda")
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    got = ea.attn_decode_paged_shared(*args, *more, o, lse, num_splits=2, workspace=ws,
                                      stream=other)
    other.synchronize()
    assert got[0] is o and got[1] is lse
    b.check(o, lse)
    first = o.clone(), lse.clone()
    c = Batch([(333, [400] * 5)], 8, 2, 128, seed=13)
    cargs, cmore = c.args(), (i32(c.cu), i32(c.prefix), i32(c.rows))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):              # two calls in one graph, one behind the other
        o1, l1 = ea.attn_decode_paged_shared(*args, *more, num_splits=2)
        o2, l2 = ea.attn_decode_paged_shared(*cargs, *cmore)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, first[0]) and torch.equal(l1, first[1])
    c.check(o2, l2)
    assert ea.attn_device_status() == ea.ATTN_OK


def test_against_the_decode_of_every_row():
    """A larger batch than the reference is quick for: the same cache through
    attn_decode_paged, whose own error is within the same bounds."""
    sizes = [1, 2, 7, 30, 64]
    b = Batch([(300 + 1111 * i, [2000 + 1111 * i + 13 * j for j in range(n)])
               for i, n in enumerate(sizes)], 16, 4, 128, seed=40)
    o, lse = b.run(check=False, sink=True)
    ro, rl = ea.attn_decode_paged_sink(*b.args(), b.sink.cuda())
    # each is within 1e-3 and half a bf16 step of the exact value
    assert (lse - rl).abs().max() <= 2e-5
    assert (o.float() - ro.float()).abs().max() <= 2e-3 + 2 * 2.0 ** -8 * ro.abs().max()
