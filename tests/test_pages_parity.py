"""The paged cache's upkeep on the GPU against the host walk of tests/_cache_ref.py:
tables, lengths and counts entry for entry, pages byte for byte."""
import threading

import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _cache_ref as ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class Cache:
    """A cache on the GPU and its host model, kept in step."""

    def __init__(self, B, W, P, layers=1, Hkv=1, d=64, stacked=True, seed=0):
        g = torch.Generator().manual_seed(seed)
        shape = (layers, P, 16, Hkv, d) if stacked else (P, 16, Hkv, d)
        self.kp, self.vp = (torch.randn(shape, generator=g).bfloat16().cuda() for _ in range(2))
        # entries past a row's pages hold junk that nothing may read
        table = (10 ** 9 + torch.arange(B * W)).view(B, W).tolist()
        self.m = ref.Pages(table, [0] * B, [0] * P)
        self.load()

    def load(self):
        """The model's tables onto the GPU."""
        self.pt = i32(self.m.table).view(len(self.m.len), -1)
        self.ln, self.refs = i32(self.m.len), i32(self.m.refs)

    def same(self, before):
        torch.cuda.synchronize()
        status = ea.attn_device_status()
        want = ea.ATTN_ERR_BAD_INPUT if "bad" in self.m.status else \
            ea.ATTN_ERR_NO_PAGES if "pages" in self.m.status else ea.ATTN_OK
        assert status == want, (status, self.m.status)
        assert self.ln.tolist() == self.m.len
        assert self.refs.tolist() == self.m.refs
        assert self.pt.tolist() == self.m.table
        for pool, old in zip((self.kp, self.vp), before):
            page = -4
            if self.m.moves:
                a, b = (torch.tensor(v).cuda() for v in zip(*self.m.moves))
                old.index_copy_(old.dim() + page, b, pool_pages(old, a))
            assert torch.equal(pool, old)

    def resize(self, new, pools=True, **kw):
        before = self.kp.clone(), self.vp.clone()
        self.m.resize(new, share=pools)
        ea.attn_pages_resize(self.pt, self.ln, i32(new), self.refs,
                             *((self.kp, self.vp) if pools else ()), **kw)
        if not pools:
            self.m.moves = []
        self.same(before)

    def fork(self, src, dst, **kw):
        before = self.kp.clone(), self.vp.clone()
        self.m.fork(src, dst)
        ea.attn_pages_fork(self.pt, self.ln, self.refs, i32(src), i32(dst), self.kp, self.vp, **kw)
        self.same(before)

    def compact(self, **kw):
        before = self.kp.clone(), self.vp.clone()
        to, live = self.m.compact()
        got, n = ea.attn_pages_compact(self.pt, self.ln, self.refs, self.kp, self.vp, **kw)
        self.same(before)
        assert got.tolist() == to and n.tolist() == [live]


def pool_pages(pool, index):
    return pool.index_select(pool.dim() - 4, index).clone()


@pytest.mark.parametrize("B,W,P,layers,Hkv,d,stacked", [
    (1, 1, 1, 1, 1, 64, False), (1, 3, 4, 1, 2, 128, False), (5, 4, 31, 2, 1, 64, True),
    (9, 7, 33, 1, 8, 128, True), (64, 6, 260, 3, 1, 64, True), (40, 40, 1100, 1, 1, 64, False),
    (33, 5, 200, 1, 8, 256, False), (700, 3, 2500, 1, 1, 64, False)])
def test_random_steps(B, W, P, layers, Hkv, d, stacked):
    g = np.random.default_rng(B + P)
    c = Cache(B, W, P, layers, Hkv, d, stacked, seed=P)
    for step in range(12):
        kind = step % 4
        if kind in (0, 2):  # rows join, grow, are cut and leave
            new = [n if g.random() < 0.3 else int(g.integers(0, W * 16 + 1)) if g.random() < 0.5
                   else min(n + int(g.integers(0, 3)), W * 16) for n in c.m.len]
            c.resize(new)
        elif kind == 1:
            empty = [b for b in range(B) if c.m.len[b] == 0][:max(1, B // 3)]
            g.shuffle(empty)
            src = [int(g.integers(0, B)) for _ in empty]
            c.fork(src, empty)
        else:
            c.compact()


def test_shared_last_pages_are_copied_before_they_are_written():
    c = Cache(6, 4, 20, layers=2)
    c.resize([40, 0, 0, 5, 0, 0])
    c.fork([0, 0, 3], [1, 2, 4])
    c.resize([40, 20, 20, 5, 5, 0])   # rows 1 and 2 cut inside a page that row 0 holds too
    c.resize([41, 21, 33, 6, 6, 0])   # both grow inside it: each gets a copy
    assert c.m.moves and all(c.m.refs[p] == 1 for p in c.m.table[1][:2][1:])
    c.fork([1], [5])
    c.resize([0, 20, 33, 6, 6, 20])   # and two rows that share it alone: both copy, it is free
    c.fork([], [])
    c.resize([0, 22, 33, 6, 6, 25])


def test_a_cache_that_shares_nothing_needs_no_pools():
    c = Cache(3, 4, 9)
    c.resize([40, 1, 0], pools=False)
    c.resize([41, 17, 16], pools=False)
    c.resize([0, 64, 0], pools=False)


def test_too_few_pages_serve_the_first_rows():
    c = Cache(5, 8, 7, layers=2)
    c.resize([48, 48, 32, 16, 0])        # 3 + 3 pages fit, the third row's two do not
    assert c.m.len == [48, 48, 0, 0, 0]
    c.resize([48, 49, 0, 0, 0])          # the last page
    c.resize([48, 64, 1, 0, 0])
    assert c.m.status == {"pages"}
    c.resize([20, 20, 0, 0, 0])
    c.fork([0, 0, 0, 1], [2, 3, 4, 4])   # three free pages; the last fork finds its row taken
    c = Cache(4, 8, 4)
    c.resize([40, 0, 0, 0])
    c.fork([0, 0, 0], [1, 2, 3])         # one free page: the first is served
    assert c.m.len == [40, 40, 0, 0]
    c.resize([41, 41, 0, 0])
    c.resize([0, 0, 0, 0])
    assert c.m.refs == [0] * 4


def test_bad_device_data_is_reported_and_left():
    c = Cache(4, 4, 12)
    c.resize([40, 0, 64, 5])
    c.resize([-1, 65, 2 ** 31 - 1, -2 ** 31])
    for src, dst in (([0], [0]), ([-1], [1]), ([4], [1]), ([0], [-1]), ([0], [4]), ([0], [2]),
                     ([2 ** 31 - 1], [1]), ([0], [-2 ** 31])):
        c.fork(src, dst)
    c.fork([0, 3, 2], [1, 1, 1])         # the first of three into one row stands
    c.resize([40, 0, 64, 5])
    for bad in (-1, 12, 2 ** 31 - 1, -2 ** 31):
        d = Cache(4, 4, 12)
        d.resize([40, 0, 64, 5])
        keep = d.m.table[0][2]
        d.m.table[0][2] = bad            # the page inside which row 0 would grow
        d.load()
        d.resize([41, 0, 64, 5])
        d.fork([0], [1])
        d.compact()
        d.resize([20, 0, 64, 5])         # given back: nothing to give
        assert d.m.status == {"bad"}
        d.m.table[0][2] = keep
        d.m.table[2][1] = bad
        d.load()
        d.fork([2], [1])                 # a whole page that is none: shared as it stands
        assert d.m.status == {"bad"}
        d.m.len[2] = 1000
        d.load()
        d.compact()
        d.m.len[2] = -5
        d.load()
        d.resize([20, 0, 64, 5])
        d.fork([2], [1])


def test_a_fork_of_a_row_that_another_fork_fills_is_empty():
    c = Cache(4, 4, 12)
    c.resize([33, 0, 0, 0])
    c.fork([0, 1], [1, 2])
    assert c.m.len == [33, 33, 0, 0]


def test_holds_of_the_callers_own_move_with_their_pages():
    c = Cache(2, 4, 10)
    c.resize([64, 33])
    c.m.refs[9] = 2                      # held outside the table
    c.m.refs[1] = 0                      # a page the table names but nothing holds
    c.load()
    c.compact()
    # seven live pages: 9 takes the place of 1
    assert c.m.status == {"bad"} and c.m.refs[1] == 2 and c.m.refs[9] == 0


@pytest.mark.parametrize("P", [262145, (1 << 21) + 7])
def test_large_pools(P):
    """Tables of a pool whose bits fill more than the default shared memory."""
    g = np.random.default_rng(P)
    d, B, W = 64, 16, 64
    kp = torch.zeros(P, 16, 1, d, dtype=torch.bfloat16, device="cuda")
    kp[:, 0, 0, :2] = torch.stack([torch.arange(P) // 128, torch.arange(P) % 128], 1).bfloat16()
    vp = -kp
    m = ref.Pages([[-1] * W for _ in range(B)], [0] * B, (g.random(P) < 0.9).astype(int).tolist())
    pt, ln, refs = i32(m.table), i32(m.len), i32(m.refs)
    new = [int(g.integers(0, W * 16)) for _ in range(B)]
    m.resize(new)
    ea.attn_pages_resize(pt, ln, i32(new), refs, kp, vp)
    m.refs[:P // 2] = [0] * (P // 2)     # the holds outside the table in the lower half end
    for row, n in zip(m.table, m.len):
        for p in row[:ref.pages_of(n)]:
            m.refs[p] = 1
    refs.copy_(i32(m.refs))
    want = kp.clone()
    to, live = m.compact()
    got, n = ea.attn_pages_compact(pt, ln, refs, kp, vp)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    a, b = (torch.tensor(v).cuda() for v in zip(*m.moves))
    want[b] = want[a]
    assert pt.tolist() == m.table and ln.tolist() == m.len and refs.tolist() == m.refs
    assert got.tolist() == to and n.tolist() == [live]
    assert torch.equal(kp, want) and torch.equal(vp, -want)


def test_most_rows():
    B, W = 8192, 2
    c = Cache(B, W, 9000)
    g = np.random.default_rng(0)
    c.resize([int(v) for v in g.integers(0, 20, B)])
    c.resize([0 if i % 3 else n + 1 for i, n in enumerate(c.m.len)])
    empty = [b for b in range(B) if c.m.len[b] == 0]
    full = [b for b in range(B) if c.m.len[b]]
    c.fork([full[i % len(full)] for i in range(len(empty))], empty)
    c.resize([min(n + 1, 32) for n in c.m.len])
    c.compact()


def test_long_rows_and_offsets_past_32_bits():
    """One row of 70,000 pages, two layers of 16 x 8 x 256: pool offsets past 2^32 bytes,
    table work far beyond one pass of the cluster."""
    P, W = 70010, 70001
    kp = torch.zeros(2, P, 16, 8, 256, dtype=torch.bfloat16, device="cuda")
    kp[:, :, 0, 0, 0] = (torch.arange(P) % 251).bfloat16().cuda()
    vp = kp + 1
    pt = torch.full((3, W), -1, dtype=torch.int32, device="cuda")
    ln, refs = i32([0, 0, 0]), torch.zeros(P, dtype=torch.int32, device="cuda")
    n = 70000 * 16 - 3
    ea.attn_pages_resize(pt, ln, i32([n, 0, 0]), refs, kp, vp)
    ea.attn_pages_fork(pt, ln, refs, i32([0]), i32([2]), kp, vp)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    ids = torch.arange(70000, dtype=torch.int32, device="cuda")
    assert torch.equal(pt[0, :70000], ids) and torch.equal(pt[2, :69999], ids[:69999])
    assert pt[2, 69999] == 70000 and (refs[:69999] == 2).all() and (refs[69999:70001] == 1).all()
    assert torch.equal(kp[:, 70000], kp[:, 69999]) and torch.equal(vp[:, 70000], vp[:, 69999])
    ea.attn_pages_resize(pt, ln, i32([0, 0, n]), refs, kp, vp)
    got, live = ea.attn_pages_compact(pt, ln, refs, kp, vp)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    assert live.item() == 70000 and got[69999] == -1 and got[70000] == 69999
    assert torch.equal(pt[2, :70000], ids) and refs.sum() == 70000
    assert torch.equal(kp[:, 69999], kp[:, 70000])


def test_more_table_rows_than_one_resize_takes():
    """A table of 10,000 rows: forked from and compacted; a resize of it is refused."""
    B, P = 10000, 300
    c = Cache(B, 2, P)
    g = np.random.default_rng(4)
    for b in g.choice(B, 100, replace=False):
        n = int(g.integers(1, 33))
        c.m.len[b] = n
        for j in range(ref.pages_of(n)):
            p = int(g.choice([p for p in range(P) if c.m.refs[p] == 0]))
            c.m.table[b][j], c.m.refs[p] = p, 1
    c.load()
    full = [b for b in range(B) if c.m.len[b]]
    c.fork(full[:50], [b for b in range(B) if c.m.len[b] == 0][-50:])
    c.compact()
    with pytest.raises(ea.AttnError) as e:
        ea.attn_pages_resize(c.pt, c.ln, c.ln.clone(), c.refs, c.kp, c.vp)
    assert e.value.status == ea.ATTN_ERR_INVALID_ARG


def test_rows_of_every_length():
    """Rows around the lengths at which a warp, the whole block or several blocks walk
    their entries."""
    lens = [0, 16, 500 * 16, 512 * 16, 513 * 16, 1023 * 16 + 1, 1024 * 16, 1025 * 16 - 7,
            2100 * 16, 1]
    B = 2 * len(lens)
    c = Cache(B, 2200, 2 * sum(map(ref.pages_of, lens)) + 40)
    c.resize(lens + [0] * len(lens))
    c.fork(list(range(len(lens))), list(range(len(lens), B)))
    c.resize([0, 16, 40, 513 * 16, 0, 600 * 16, 0, 0, 1500 * 16, 1] + [n + 3 for n in lens])
    c.compact()
    c.resize([0] * B)
    assert c.m.refs == [0] * len(c.m.refs)


def test_captured_steps_and_own_streams():
    """A captured resize and fork replayed on new lengths, and two caches on two streams
    at once: the tables of the plain calls."""
    def fresh():
        return dict(pt=torch.full((4, 6), -1, dtype=torch.int32, device="cuda"),
                    ln=i32([0] * 4), refs=i32([0] * 30),
                    kp=torch.randn(2, 30, 16, 2, 64, device="cuda").bfloat16(),
                    vp=torch.randn(2, 30, 16, 2, 64, device="cuda").bfloat16())

    def step(s, new, src, dst, **kw):
        ea.attn_pages_resize(s["pt"], s["ln"], new, s["refs"], s["kp"], s["vp"], **kw)
        ea.attn_pages_fork(s["pt"], s["ln"], s["refs"], src, dst, s["kp"], s["vp"], **kw)
        return ea.attn_pages_compact(s["pt"], s["ln"], s["refs"], s["kp"], s["vp"], **kw)

    new, src, dst = i32([40, 0, 0, 7]), i32([0, 3]), i32([1, 2])
    a, b = fresh(), fresh()
    for x in ("kp", "vp"):
        b[x].copy_(a[x])
    warm = fresh()
    step(warm, new, src, dst)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(a, new, src, dst)
    for lens in ([40, 0, 0, 7], [50, 0, 0, 0], [20, 0, 0, 90]):
        new.copy_(i32(lens))
        graph.replay()
        want = step(b, new, src, dst)
        torch.cuda.synchronize()
        assert all(torch.equal(a[x], b[x]) for x in a)
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    assert ea.attn_device_status() == ea.ATTN_OK
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [fresh(), fresh()]
    for x in ("kp", "vp"):
        caches[1][x].copy_(caches[0][x])
    some, none = i32([33, 0, 0, 5]), i32([0] * 4)
    torch.cuda.synchronize()
    for _ in range(20):
        for s, c in zip(streams, caches):
            step(c, some, src, dst, stream=s)
            ea.attn_pages_resize(c["pt"], c["ln"], none, c["refs"], c["kp"], c["vp"], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(caches[0][x], caches[1][x]) for x in caches[0])


def test_two_threads_on_one_stream():
    """Two host threads, each with a cache of its own, launching into one stream: the
    launches of their calls interleave."""
    def run(out, seed):
        try:
            c = Cache(6, 8, 60, layers=2, Hkv=8, d=128, seed=seed)
            lens = [i32(v) for v in ([40, 0, 0, 7, 0, 100], [41, 41, 0, 8, 17, 101],
                                     [3, 0, 20, 0, 17, 0], [0] * 6)]
            src, dst = i32([0, 3]), i32([1, 4])
            for _ in range(60):
                ea.attn_pages_resize(c.pt, c.ln, lens[0], c.refs, c.kp, c.vp)
                ea.attn_pages_fork(c.pt, c.ln, c.refs, src, dst, c.kp, c.vp)
                for n in lens[1:]:
                    ea.attn_pages_resize(c.pt, c.ln, n, c.refs, c.kp, c.vp)
                    ea.attn_pages_compact(c.pt, c.ln, c.refs, c.kp, c.vp)
            out[seed] = c
        except Exception as e:  # a thread's failure is the test's
            out[seed] = e

    alone, both = {}, {}
    for seed in (1, 2):
        run(alone, seed)
    threads = [threading.Thread(target=run, args=(both, seed)) for seed in (1, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    for seed in (1, 2):
        for name in ("pt", "ln", "refs", "kp", "vp"):
            assert torch.equal(getattr(alone[seed], name), getattr(both[seed], name))


def test_workspace_is_the_callers_if_given():
    c = Cache(4, 4, 12)
    ws = torch.full((ea.attn_pages_workspace_size(4, 12) // 4 + 8,), -99, dtype=torch.int32,
                    device="cuda")
    use = ws[:-8]
    c.resize([40, 0, 7, 0], workspace=use)
    c.fork([0, 2], [1, 3], workspace=use)
    c.compact(workspace=use)
    assert (ws[-8:] == -99).all()
    with pytest.raises(ea.AttnError) as e:
        ea.attn_pages_compact(c.pt, c.ln, c.refs, c.kp, c.vp, workspace=ws[:8])
    assert e.value.status == ea.ATTN_ERR_INVALID_ARG


def test_binding_refusals():
    c = Cache(4, 4, 12)
    n = i32([1, 2, 3, 4])
    for bad in (lambda: ea.attn_pages_resize(c.pt, c.ln, n.long(), c.refs, c.kp, c.vp),
                lambda: ea.attn_pages_resize(c.pt, c.ln, n[:3], c.refs, c.kp, c.vp),
                lambda: ea.attn_pages_resize(c.pt, c.ln, n, c.refs, c.kp),
                lambda: ea.attn_pages_resize(c.pt, c.ln, n, c.refs[:11], c.kp, c.vp),
                lambda: ea.attn_pages_resize(c.pt[:, :2], c.ln, n, c.refs, c.kp, c.vp),
                lambda: ea.attn_pages_fork(c.pt, c.ln, c.refs, n, n[:3], c.kp, c.vp),
                lambda: ea.attn_pages_fork(c.pt, c.ln, c.refs, n, n, c.kp, c.vp[:, :6]),
                lambda: ea.attn_pages_compact(c.pt, c.ln.cpu(), c.refs, c.kp, c.vp),
                lambda: ea.attn_pages_compact(c.pt, c.ln, c.refs.cpu(), c.kp, c.vp)):
        with pytest.raises(ValueError):
            bad()
