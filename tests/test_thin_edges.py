"""Calls on shared and thinned caches that a server may make and the parity tests do not:
workspaces of just the size asked for on any 16-byte boundary, two calls at once on two
streams, captured calls replayed on other lengths and groups.  Each is compared bit for bit
with the plain call, whose results the parity tests hold to the reference."""
import pytest
import torch

import exact_attention_08_gb300 as ea

pytestmark = pytest.mark.gpu

GUARD = 1024


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Cache:
    """B rows, each with pages of its own but for the first `shared` ones."""

    def __init__(self, B, Hq, Hkv, d, lens, shared, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.Hq, self.Hkv, self.d, self.shared = B, Hq, Hkv, d, shared
        self.W = max(1, (max(lens) + 15) // 16)
        P = shared + B * self.W
        table = shared + torch.randperm(P - shared, generator=g)[:B * self.W].view(B, self.W)
        table[:, :shared] = torch.arange(min(shared, self.W))
        self.pt, self.ln = table.int().cuda(), i32(lens)
        self.q = torch.randn(B, Hq, d, generator=g).bfloat16().cuda()
        self.k = torch.randn(P, 16, Hkv, d, generator=g).bfloat16().cuda()
        self.v = torch.randn(P, 16, Hkv, d, generator=g).bfloat16().cuda()
        self.slots = 16 * self.W
        self.mass = torch.rand(B, Hkv, self.slots, generator=g).cuda()
        self.pos = torch.arange(self.slots, dtype=torch.int32).repeat(B, Hkv, 1).cuda()

    def paged(self):
        return self.q, self.k, self.v, self.pt, self.ln

    def shared_call(self, **kw):
        return ea.attn_decode_paged_shared(*self.paged(), i32([0, self.B]),
                                           i32([16 * self.shared]), num_splits=2, **kw)

    def decode_call(self, **kw):
        out = torch.zeros_like(self.mass)
        o, lse = ea.attn_decode_paged_mass(*self.paged(), self.mass, mass_out=out, num_splits=3,
                                           **kw)
        return o, lse, out

    def block_call(self, **kw):
        out = torch.zeros_like(self.mass)
        lse = torch.full((self.Hq, self.B), 6.0, device="cuda")
        return (ea.attn_mass_paged(self.q, lse, self.k, self.pt, torch.arange(self.B + 1).int().cuda(),
                                   self.ln, self.mass, max_seqlen_q=1, mass_out=out, **kw),)

    def evict_call(self, **kw):
        m, p, k, v = self.mass.clone(), self.pos.clone(), self.k.clone(), self.v.clone()
        pt = torch.arange(self.B * self.W, dtype=torch.int32, device="cuda").view(self.B, self.W)
        new = ea.attn_evict_paged(m, p, pt, self.ln, self.ln // 2, k, v, n_sink=2, recent=3, **kw)
        keep = (torch.arange(self.slots, device="cuda") < new[:, None])[:, None]
        return m * keep, p * keep, k, v, new

    def sizes(self):
        B, Hq, Hkv, d, W = self.B, self.Hq, self.Hkv, self.d, self.W
        return {"shared_call": ea.attn_decode_shared_workspace_size(B, Hq, Hkv, d, 1, B, W, 2),
                "decode_call": ea.attn_decode_mass_workspace_size(B, Hq, d, W, 3),
                "block_call": ea.attn_mass_workspace_size(B, Hkv, W),
                "evict_call": ea.attn_evict_workspace_size(1, B, Hkv, self.slots, W)}


CALLS = ["shared_call", "decode_call", "block_call", "evict_call"]
SHAPES = [(1, 4, 1, 64, [9], 0), (3, 8, 2, 128, [300, 280, 290], 17),
          (5, 6, 2, 256, [1000, 1, 0, 700, 1000], 40), (70, 32, 8, 128, [400] * 70, 20),
          (300, 5, 5, 64, [33] * 300, 2)]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("offset", [0, 16, 48])
def test_workspace_of_the_size_asked_for(call, shape, offset):
    c = Cache(*SHAPES[shape])
    want = getattr(c, call)()
    n = c.sizes()[call]
    assert n > 0
    whole = torch.full((GUARD + offset + n + GUARD,), 0xa5, dtype=torch.uint8, device="cuda")
    got = getattr(c, call)(workspace=whole[GUARD + offset:GUARD + offset + n])
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (whole[:GUARD + offset] == 0xa5).all() and (whole[GUARD + offset + n:] == 0xa5).all()
    if call != "evict_call" and n > 16:
        with pytest.raises(ea.AttnError):
            getattr(c, call)(workspace=whole[:n - 1])
    with pytest.raises(ea.AttnError):
        getattr(c, call)(workspace=whole[8:8 + n])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_calls_at_once_on_two_streams(d):
    a = Cache(40, 8, 2, d, [900] * 40, 50, seed=1)
    b = Cache(64, 16, 4, d, [30 + 20 * i for i in range(64)], 1, seed=2)
    torch.cuda.synchronize()
    want = {(n, call): getattr(c, call)() for n, c in enumerate((a, b)) for call in CALLS}
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for turn in range(6):
        for i, call in enumerate(CALLS):
            for n, c in enumerate((a, b)):
                other = CALLS[(i + n * (1 + turn)) % len(CALLS)]
                with torch.cuda.stream(streams[n]):
                    got.append(((n, other), getattr(c, other)()))
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    for key, x in got:
        assert all(torch.equal(p, q) for p, q in zip(x, want[key])), key


def test_replays_on_other_lengths_and_groups():
    c = Cache(12, 8, 2, 128, [500] * 12, 20, seed=3)
    cu, prefix, rows = i32([0, 6, 12]), i32([320, 160]), i32(list(range(12)))
    keep, lse_in = i32([100] * 12), torch.full((8, 12), 6.0, device="cuda")
    cu_q = torch.arange(13).int().cuda()
    mass, pos, out = c.mass.clone(), c.pos.clone(), torch.zeros_like(c.mass)
    own = torch.arange(12 * c.W, dtype=torch.int32, device="cuda").view(12, c.W)
    k, v = c.k.clone(), c.v.clone()

    def calls():
        o, lse = ea.attn_decode_paged_shared(*c.paged(), cu, prefix, rows)
        o2, lse2 = ea.attn_decode_paged_mass(*c.paged(), c.mass, mass_out=out)
        ea.attn_mass_paged(c.q, lse_in, c.k, c.pt, cu_q, c.ln, out, max_seqlen_q=1, mass_out=mass)
        new = ea.attn_evict_paged(mass, pos, own, c.ln, keep, k, v)
        return o, lse, o2, lse2, new

    def reset():
        for x in (mass, out):
            x.zero_()
        pos.copy_(c.pos), k.copy_(c.k), v.copy_(c.v)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    changes = [dict(),
               dict(ln=[320 + 15 * i for i in range(12)]),
               dict(ln=[0, 1, 16, 320, 321, 500, 7, 159, 160, 161, 499, 30], prefix=[320, 320]),
               dict(ln=[500] * 12, cu=[0, 12, 12], prefix=[320, 0], rows=[11 - i for i in range(12)]),
               dict(cu=[3, 3, 10], prefix=[48, 311], keep=[0, 500, 499, 1] * 3),
               dict(cu=[0, 0, 0])]
    for change in changes:
        for name, x in change.items():
            {"ln": c.ln, "cu": cu, "prefix": prefix, "rows": rows, "keep": keep}[name].copy_(i32(x))
        reset()
        graph.replay()
        torch.cuda.synchronize()
        a = [x.clone() for x in got] + [out.clone(), k.clone(), v.clone()]
        reset()
        b = list(calls()) + [out, k, v]
        torch.cuda.synchronize()
        assert ea.attn_device_status() == ea.ATTN_OK
        assert all(torch.equal(x, y) for x, y in zip(a, b)), change
        # and against the decode row by row: both within their bounds of the exact values
        ro, rl = ea.attn_decode_paged(*c.paged())
        assert (a[0].float() - ro.float()).abs().max() <= 2e-3 + 2 * 2.0 ** -8 * ro.abs().max()
        seen = c.ln > 0
        assert (a[1] - rl)[seen].abs().max() <= 2e-5


@pytest.mark.parametrize("B,size", [(1100, 1), (1500, 7), (5000, 5000), (1024, 512)])
def test_many_rows(B, size):
    """Groups of `size` rows of a cache whose rows all share 12 pages, against the decode row by
    row: each within its bounds of the exact values."""
    c = Cache(B, 4, 2, 64, [(37 * b) % 300 for b in range(B)], 12, seed=B)
    g = torch.Generator().manual_seed(B)
    rows = torch.randperm(B, generator=g).int().cuda()
    cu = list(range(0, B, size)) + [B]
    o, lse = ea.attn_decode_paged_shared(*c.paged(), i32(cu), i32([192] * (len(cu) - 1)), rows)
    ro, rl = ea.attn_decode_paged(*c.paged(), num_splits=2)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    seen = c.ln > 0
    assert (o.float() - ro.float()).abs().max() <= 2e-3 + 2 * 2.0 ** -8 * ro.abs().max()
    assert (lse - rl)[seen].abs().max() <= 2e-5
    assert torch.isneginf(lse[~seen]).all() and (o[~seen] == 0).all()


def test_pools_past_32_bits():
    """Rows on the last pages of pools of 2.3e9 elements (past 2^31), the same rows on small
    pools: the same bits."""
    c = Cache(6, 16, 8, 128, [300, 290, 17, 0, 256, 299], 15, seed=5)
    P, n = 140000, c.k.shape[0]
    big = [torch.empty(P, 16, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    want = {call: getattr(c, call)() for call in CALLS[:3]}
    for x, pool in zip((c.k, c.v), big):
        pool[P - n:] = x
    small, c.k, c.v, c.pt = (c.k, c.v, c.pt), big[0], big[1], c.pt + (P - n)
    for call in CALLS[:3]:
        got = getattr(c, call)()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[call])), call
    # and the eviction: the first page's rows move on the large pools as on the small ones
    keep, own = c.ln // 3, torch.arange(6 * c.W, dtype=torch.int32, device="cuda").view(6, c.W)
    k, v = small[0].clone(), small[1].clone()
    args = c.mass.clone(), c.pos.clone(), own, c.ln, keep, k, v
    new = ea.attn_evict_paged(*args)
    far = ea.attn_evict_paged(c.mass.clone(), c.pos.clone(), own + (P - n), c.ln, keep, *big)
    torch.cuda.synchronize()
    assert torch.equal(new, far)
    assert torch.equal(big[0][P - n:], k) and torch.equal(big[1][P - n:], v)
    assert ea.attn_device_status() == ea.ATTN_OK


@pytest.mark.parametrize("B,Hq,Hkv,d", [(300, 16, 4, 128), (600, 8, 1, 256), (256, 16, 2, 64),
                                        (257, 16, 2, 64)])
def test_many_rows_and_heads(B, Hq, Hkv, d):
    """4,096 merged (row, head) pairs and more."""
    c = Cache(B, Hq, Hkv, d, [200 + (31 * b) % 150 for b in range(B)], 12, seed=B)
    o, lse = ea.attn_decode_paged_shared(*c.paged(), i32([0, 90, B]), i32([192, 192]))
    ro, rl = ea.attn_decode_paged(*c.paged(), num_splits=2)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    assert (o.float() - ro.float()).abs().max() <= 2e-3 + 2 * 2.0 ** -8 * ro.abs().max()
    assert (lse - rl).abs().max() <= 2e-5
