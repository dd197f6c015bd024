"""attn_decode_paged_shared where groups share: every case here is large enough for the prefix
kernel by the rule of sizes, and says so.  More items than CTAs, many key tiles of an item a
CTA, bad lists beside real work, many groups and rows.  Rows are compared element by element
with fp64, within what the kernel's roundings can make of them."""
import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _thin_ref as ref
from tests._parity import np64
from tests.test_shared_parity import Batch, i32

pytestmark = pytest.mark.gpu

LEAST = 8192        # (rows - 1) * pages * d from which a group shares its prefix
SMS = 152
STEP = 2.0 ** -8    # half a step of bf16, relative


def shares(rows, pages, d):
    return max(rows - 1, 1) * pages * d >= LEAST


def assert_all_share(b):
    """That every group of the batch shares its prefix."""
    for prefix, lens in b.groups:
        assert shares(len(lens), min(prefix, max(lens)) // 16, b.d), (prefix, len(lens))


def check_rows(b, o, lse, rows, scale=None, sink=False):
    """Each element: the weights are rounded to bf16 once (STEP of each), the largest of a key
    tile is left out of the normaliser by as much as it lost (at most STEP of the sum), the
    output is rounded once; scores, exponentials and sums as in ref.WEIGHT."""
    scale = b.d ** -0.5 if scale is None else scale
    o, lse = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for r in rows:
        n = b.lens[r]
        pages = torch.tensor(b.table[r][:(n + 15) // 16], dtype=torch.long)
        k, v = (x[pages].double().numpy().reshape(-1, b.Hkv, b.d)[:n] for x in (b.k, b.v))
        ro, rl, w = ref.attend(np64(b.q[r]), k, v, scale, b.sink.double().numpy() if sink else None)
        G = b.Hq // b.Hkv
        size = np.stack([w[h] @ np.abs(v[:, h // G]) for h in range(b.Hq)])
        bound = STEP * (size + 2 * np.abs(ro)) + 4 * ref.WEIGHT * size + 1e-30
        bad = np.abs(o[r] - ro) > bound
        assert not bad.any(), (r, int(bad.sum()), float((np.abs(o[r] - ro) / bound).max()))
        none = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse[r]), none)
        err = np.abs(lse[r][~none] - rl[~none])
        assert (err <= ref.WEIGHT + 2.0 ** -23 * np.abs(rl[~none])).all(), (r, err.max())


def some(b, n, seed=0):
    g = np.random.default_rng(seed)
    lens = np.array(b.lens)
    rows = set(g.choice(len(lens), min(n, len(lens)), replace=False).tolist())
    return sorted(rows | {int(lens.argmin()), int(lens.argmax())})


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 4, 64), (8, 4, 128), (4, 4, 256)])
def test_more_items_than_ctas(Hq, Hkv, d):
    """50 prompts of 65 pages and more, 3 samples each."""
    b = Batch([(1040 + 3 * (g % 9), [1065 + g + 5 * i for i in range(3)]) for g in range(50)], Hq,
              Hkv, d, seed=d)
    assert_all_share(b)
    assert 50 * Hkv > SMS
    o, lse = b.run(check=False, sink=True)
    check_rows(b, o, lse, some(b, 16), sink=True)
    again = b.run(check=False, sink=True)
    assert torch.equal(o.view(torch.int16), again[0].view(torch.int16))
    assert torch.equal(lse, again[1])


@pytest.mark.parametrize("Hq,Hkv,d,n,rows", [(4, 2, 64, 130000, 3), (34, 1, 128, 110000, 8),
                                             (18, 1, 256, 64000, 8), (6, 2, 256, 64000, 3)])
def test_many_key_tiles_of_an_item(Hq, Hkv, d, n, rows):
    b = Batch([(n, [n + 9 * i for i in range(rows)])], Hq, Hkv, d, seed=rows)
    assert_all_share(b)
    keys, most = (64, 128) if d == 256 else (128, 256)
    items = Hkv * -(-rows * (Hq // Hkv) // most)
    tiles = n // keys
    assert tiles * items / SMS > 10      # key tiles of an item a CTA takes at the least
    o, lse = b.run(check=False)
    check_rows(b, o, lse, some(b, 1))


@pytest.mark.parametrize("splits", [1, 2, 64])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 4, 128), (4, 1, 64), (8, 2, 256)])
def test_rows_in_order_splits_and_bits(splits, Hq, Hkv, d):
    b = Batch([(496, [500, 800, 496, 512, 497, 600]), (980, [1000, 996, 981, 990, 1200])], Hq, Hkv, d,
              seed=splits)
    assert_all_share(b)
    inverse = torch.tensor(b.rows)
    b.q, b.table = b.q[inverse], [b.table[i] for i in b.rows]
    b.lens = [b.lens[i] for i in b.rows]
    o, lse = b.run(rows=None, num_splits=splits, check=False)
    check_rows(b, o, lse, range(len(b.lens)))
    for _ in range(3):
        again = b.run(rows=None, num_splits=splits, check=False)
        assert torch.equal(o.view(torch.int16), again[0].view(torch.int16))
        assert torch.equal(lse, again[1])


def batch(d):
    return Batch([(700, [710, 705, 704, 701, 790, 700]), (1000, [1030, 1009, 1001, 1500])], 4, 2, d,
                 alone=[20], seed=8)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cu", [[0, 11, 10], [-1, 6, 10], [0, 6, 12], [7, 6, 10],
                                [0, 2 ** 31 - 1, 10], [0, 6, -2 ** 31]])
def test_offsets_out_of_range(d, cu):
    b = batch(d)
    assert_all_share(b)
    b.cu = cu
    o, lse = b.run(status=ea.ATTN_ERR_BAD_INPUT, check=False)
    check_rows(b, o, lse, range(len(b.lens)))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("entry,row", [(1, -1), (3, 11), (0, 2 ** 31 - 1), (9, -2 ** 31), (4, "first"),
                                       (8, "first"), (2, "own")])
def test_rows_out_of_range_and_listed_twice(d, entry, row):
    """A row listed again belongs where it stands first; the row that stood there is on its own."""
    b = batch(d)
    assert_all_share(b)
    b.rows[entry] = {"first": b.rows[0], "own": b.rows[1]}.get(row, row)
    o, lse = b.run(status=ea.ATTN_ERR_BAD_INPUT, check=False)
    check_rows(b, o, lse, range(len(b.lens)))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefixes_out_of_range(d):
    b = batch(d)
    b.prefix[0] = -5
    o, lse = b.run(status=ea.ATTN_ERR_BAD_INPUT, check=False)
    check_rows(b, o, lse, range(len(b.lens)))
    c = Batch([(700, [704] * 6), (1000, [1030, 1009, 1001, 1500])], 4, 2, d, seed=9)
    c.prefix[0] = 2 ** 31 - 1              # all whole pages of the longest row: 44, all shared
    for r in c.rows[1:6]:
        c.table[r][43] = c.table[c.rows[0]][43]
    o, lse = c.run(status=ea.ATTN_ERR_BAD_INPUT, check=False)
    check_rows(c, o, lse, range(len(c.lens)))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths_and_pages_out_of_range(d):
    for bad in (-7, -2 ** 31):
        b = batch(d)
        b.lens[b.rows[1]] = bad
        o, lse = b.run(status=ea.ATTN_ERR_BAD_INPUT, check=False)
        b.lens[b.rows[1]] = 0
        check_rows(b, o, lse, range(len(b.lens)))
    for page in (-1, "P", 2 ** 31 - 1):
        c = batch(d)
        for r in c.rows[:6]:
            c.table[r][3] = c.P if page == "P" else page
        o, lse = c.run(status=ea.ATTN_ERR_BAD_INPUT, check=False)
        unused = next(p for p in range(c.P) if all(p not in t for t in c.table))
        c.k[unused] = c.v[unused] = 0      # such a page reads zeros
        for r in c.rows[:6]:
            c.table[r][3] = unused
        check_rows(c, o, lse, range(len(c.lens)))


@pytest.mark.parametrize("groups,most,pages,Hq,Hkv,d", [(40, 1, 33, 4, 1, 256), (100, 2, 130, 4, 2, 64),
                                                        (70, 7, 130, 4, 2, 64), (600, 1, 32, 2, 1, 256),
                                                        (33, 20, 65, 8, 2, 128), (700, 2, 33, 4, 1, 256)])
def test_more_groups_than_warps(groups, most, pages, Hq, Hkv, d):
    """Groups of 1 to `most` rows: as many lanes of the plan each as they have rows."""
    b = Batch([(16 * (pages + g % 3), [16 * (pages + g % 3) + g % 17 + i for i in range(1 + g % most)])
               for g in range(groups)], Hq, Hkv, d, alone=[3, 40], seed=groups)
    assert_all_share(b)
    o, lse = b.run(check=False)
    check_rows(b, o, lse, some(b, 30))


@pytest.mark.parametrize("B,size,pages,Hq,Hkv,d", [(1100, 7, 12, 4, 2, 128), (1050, 1050, 12, 16, 4, 64),
                                                   (5000, 5000, 12, 4, 2, 64), (1024, 512, 20, 4, 2, 128),
                                                   (1025, 205, 9, 4, 1, 256)])
def test_many_rows(B, size, pages, Hq, Hkv, d):
    """The plan of 1,024 threads, the merge with four outputs in flight, lists past the plan's
    shared memory."""
    n = 16 * pages
    b = Batch([(n, [n + (37 * (e0 + i)) % 30 for i in range(min(size, B - e0))])
               for e0 in range(0, B, size)], Hq, Hkv, d, seed=B)
    for _, lens in b.groups[:-1]:
        assert shares(len(lens), pages, d)
    o, lse = b.run(check=False)
    check_rows(b, o, lse, some(b, 40))


@pytest.mark.parametrize("seed", range(30))
def test_random_groups(seed):
    """Groups of any sizes with rows of any lengths: empty ones, some that end inside the prefix,
    some that the prefix does not reach the end of."""
    g = np.random.default_rng(seed)
    d, Hkv = int(g.choice([64, 128, 256])), int(g.choice([1, 2, 3]))
    W = int(g.integers(2, 90))
    groups = []
    for _ in range(int(g.integers(1, 7))):
        prefix = int(g.choice([g.integers(0, 60), g.integers(0, 16 * W + 1), 16 * W]))
        prefix = min(prefix, 16 * W)
        least = int(g.choice([0, 0, prefix]))
        groups.append((prefix, g.integers(least, 16 * W + 1, int(g.choice([1, 2, 8, 17, 40]))).tolist()))
        if g.random() < 0.5:
            groups[-1][1][0] = 0
    for prefix, lens in groups:        # (a page that several rows end in would be scaled by each)
        lens[:] = [n if n >= prefix else n // 16 * 16 for n in lens]
    b = Batch(groups, Hkv * int(g.choice([1, 2, 5, 8])), Hkv, d, alone=[0, 33], seed=seed)
    b.W = max(b.W, W)
    b.table = [t + [-1] * (b.W - len(t)) for t in b.table]
    sink = seed % 3 == 0
    o, lse = b.run(check=False, sink=sink)
    check_rows(b, o, lse, some(b, 30), sink=sink)
