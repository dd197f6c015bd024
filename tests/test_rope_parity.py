"""Rotary positions and the append to a paged cache against the fp64 formula
(tests/_cache_ref.py states the tolerance)."""
import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _cache_ref as ref

pytestmark = pytest.mark.gpu


def randn(g, *shape):
    return torch.randn(*shape, generator=g).bfloat16()


def np64(t):
    return t.double().cpu().numpy()


def frequencies(rot, base=10000.0):
    return ea.attn_rope_inv_freq(rot, base) if rot else \
        torch.empty(0, dtype=torch.float64, device="cuda")


CASES = [
    # B, S, Hq, Hkv, d, rot, interleaved, amplitude
    (1, 1, 1, 1, 64, 64, False, 1.0),
    (2, 37, 4, 2, 64, 64, True, 1.0),
    (3, 130, 5, 3, 128, 128, False, 1.2),
    (1, 700, 32, 8, 128, 128, False, 1.0),
    (1, 700, 32, 8, 128, 64, True, 1.0),
    (2, 65, 16, 16, 256, 64, False, 0.7),
    (2, 65, 3, 1, 256, 256, True, 1.0),
    (2, 33, 2, 2, 128, 16, False, 1.0),
    (2, 33, 2, 2, 128, 20, False, 1.0),   # pairs that no 16-byte vector holds
    (2, 33, 2, 2, 128, 126, True, 1.3),
    (1, 9, 2, 1, 64, 2, False, 1.0),
    (1, 9, 2, 1, 256, 2, True, 1.0),
    (2, 3, 200, 40, 64, 32, False, 1.0),  # more heads than one pass of a block takes
    (1, 5, 2, 2, 64, 0, False, 1.0),      # nothing rotated: a copy
]


def random_rope(seed):
    g = np.random.default_rng(100 + seed)
    d = int(g.choice([64, 128, 256]))
    rot = int(g.choice([d, d // 2, 16, 2 * int(g.integers(0, d // 2 + 1))]))
    return (int(g.integers(1, 4)), int(g.integers(1, 200)), int(g.integers(1, 50)),
            int(g.integers(1, 20)), d, rot, bool(g.random() < 0.5), float(g.choice([1.0, -0.5, 2])))


CASES += [random_rope(seed) for seed in range(10)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("fn,sign", [(ea.attn_rope, 1.0), (ea.attn_rope_bwd, -1.0)])
def test_rope(case, fn, sign):
    B, S, Hq, Hkv, d, rot, inter, amp = case
    g = torch.Generator().manual_seed(sum(case[:6]))
    q, k = randn(g, B, S, Hq, d), randn(g, B, S, Hkv, d)
    pos = torch.randint(-50, 5000, (B, S), generator=g, dtype=torch.int32)
    inv = frequencies(rot)
    for p in (pos, None):
        used = np.broadcast_to(np.arange(S), (B, S)) if p is None else p.numpy()
        out = fn(q.cuda(), k.cuda(), inv, None if p is None else p.cuda(), interleaved=inter,
                 amplitude=amp)
        for x, y in zip((q, k), out):
            r, size = ref.rotate(np64(x), used, np64(inv), amp, inter, sign)
            ref.check_rotated(y, r, size, what=str(case))
    assert ea.attn_device_status() == ea.ATTN_OK


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    g = torch.Generator().manual_seed(3)
    q = randn(g, 8, 2, 128)
    pos = torch.tensor([0, 1, -1, 10 ** 6, 2 ** 25 - 1, 2 ** 31 - 1, -2 ** 31, 131071],
                       dtype=torch.int32)
    inv = frequencies(128, 1e6)
    y, none = ea.attn_rope(q.cuda(), None, inv, pos.cuda(), interleaved=interleaved)
    assert none is None
    r, size = ref.rotate(np64(q), pos.numpy(), np64(inv), 1.0, interleaved)
    ref.check_rotated(y, r, size, ref.FAR)


@pytest.mark.parametrize("rot", [128, 64, 20])
@pytest.mark.parametrize("interleaved", [False, True])
def test_layouts_and_places(rot, interleaved):
    """Slices of a fused projection, head-major storage, a broadcast gradient, packed rows
    and in place: all the bits of the contiguous call; nothing beside the rows written."""
    g = torch.Generator().manual_seed(5)
    B, S, Hq, Hkv, d = 2, 19, 6, 2, 128
    x = randn(g, B, S, Hq + 2 * Hkv, d).cuda()
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
    pos = torch.randint(0, 900, (B, S), generator=g, dtype=torch.int32).cuda()
    inv = frequencies(rot)
    call = lambda a, b, **kw: ea.attn_rope(a, b, inv, pos, interleaved=interleaved, **kw)  # noqa: E731
    want = call(q.contiguous(), k.contiguous())
    same = lambda got: all(torch.equal(u, w) for u, w in zip(got, want))  # noqa: E731
    assert same(call(q, k))
    assert same(call(q.transpose(1, 2).contiguous().transpose(1, 2), k))
    room = torch.full((B, S + 2, Hq + 3, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[:, 1:-1, 2:2 + Hq, :d]
    assert same(call(q, k, q_out=out))
    keep = torch.ones_like(room, dtype=torch.bool)
    keep[:, 1:-1, 2:2 + Hq, :d] = False
    assert (room[keep] == 7.0).all()
    packed = ea.attn_rope(q.reshape(B * S, Hq, d), k.reshape(B * S, Hkv, d), inv, pos.reshape(-1),
                          interleaved=interleaved)
    assert same([packed[0].view(B, S, Hq, d), packed[1].view(B, S, Hkv, d)])
    xf = x.view(B * S, Hq + 2 * Hkv, d)
    packed = ea.attn_rope(xf[:, :Hq], xf[:, Hq:Hq + Hkv], inv, pos.reshape(-1),
                          interleaved=interleaved)
    assert same([packed[0].view(B, S, Hq, d), packed[1].view(B, S, Hkv, d)])
    alone = call(q, None)[0], call(None, k)[1]
    assert same(alone)
    one = randn(g, 1, 1, 1, d).cuda().expand(B, S, Hq, d)
    assert torch.equal(ea.attn_rope_bwd(one, None, inv, pos, interleaved=interleaved)[0],
                       ea.attn_rope_bwd(one.contiguous(), None, inv, pos,
                                        interleaved=interleaved)[0])
    for part in (x[:1, :, :1].expand(B, S, Hq, d), x[:, :1, :1].expand(B, S, Hq, d),
                 x[:1, :, :Hq].expand(B, S, Hq, d), x[:1, :1, :Hq].expand(B, S, Hq, d),
                 x.transpose(1, 2)[:, :Hq, :1].expand(B, Hq, S, d).transpose(1, 2)):
        got = ea.attn_rope_bwd(part, None, inv, pos, interleaved=interleaved)[0]
        assert torch.equal(got, ea.attn_rope_bwd(part.contiguous(), None, inv, pos,
                                                 interleaved=interleaved)[0])
    y = x.clone()
    qi, ki = y[:, :, :Hq], y[:, :, Hq:Hq + Hkv]
    got = call(qi, ki, q_out=qi, k_out=ki)
    assert got[0] is qi and same(got)
    assert torch.equal(y[:, :, Hq + Hkv:], x[:, :, Hq + Hkv:])


def test_rope_values_that_are_not_finite_stay_in_their_pairs():
    g = torch.Generator().manual_seed(6)
    q = randn(g, 1, 4, 2, 64).cuda()
    inv = frequencies(32)
    clean = ea.attn_rope(q, None, inv)[0]
    q[0, 1, 0, 3], q[0, 2, 1, 40], q[0, 3, 0, 20] = float("nan"), float("inf"), float("-inf")
    got = ea.attn_rope(q, None, inv)[0]
    hit = torch.zeros_like(q, dtype=torch.bool)
    hit[0, 1, 0, [3, 19]] = hit[0, 3, 0, [4, 20]] = True
    hit[0, 2, 1, 40] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert got[0, 1, 0, [3, 19]].isnan().all() and got[0, 2, 1, 40] == float("inf")
    assert not got[0, 3, 0, [4, 20]].isfinite().any()


def test_rope_binding_refusals():
    q = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    inv = frequencies(64)
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for bad in (lambda: ea.attn_rope(q.float(), None, inv), lambda: ea.attn_rope(q, q[:1], inv),
                lambda: ea.attn_rope(q, None, inv.float()),
                lambda: ea.attn_rope(q, None, frequencies(66)),
                lambda: ea.attn_rope(q, None, inv, pos.long()),
                lambda: ea.attn_rope(q, None, inv, pos[:1]),
                lambda: ea.attn_rope(q.transpose(2, 3), None, inv),
                lambda: ea.attn_rope(q, None, inv, q_out=q[:1])):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros(2, 3, 2, 68, dtype=torch.bfloat16, device="cuda")[..., :64]
    for bad in (lambda: ea.attn_rope(odd, None, inv),
                lambda: ea.attn_rope(q, None, inv, q_out=q[:, :1].expand(2, 3, 2, 64)),
                lambda: ea.attn_rope(q.view(-1)[4:260].view(1, 2, 2, 64), None, inv)):
        with pytest.raises(ea.AttnError) as e:
            bad()
        assert e.value.status == ea.ATTN_ERR_INVALID_ARG
    empty = ea.attn_rope(q[:, :0], None, inv)[0]
    assert empty.shape == (2, 0, 2, 64)


# ------------------------------------------------------------------ append

def append_ref(kp, vp, q, k, v, pt, ln, cu, inv, amp, inter):
    """fp64 pools, their error sizes (-1: not written) and q with its."""
    T = k.shape[0]
    kr, ks = np64(kp), np.full(kp.shape, -1.0)
    vr = np64(vp)
    qr, qs = np.full((T, *q.shape[1:]), np.nan), np.full((T, *q.shape[1:]), -1.0)
    P = kp.shape[0]
    for b in range(len(ln)):
        if not 0 <= ln[b] <= pt.shape[1] * 16:
            continue
        for row in range(cu[b], cu[b + 1]):
            t = int(ln[b]) - (cu[b + 1] - row)
            qr[row], qs[row] = ref.rotate(np64(q[row]), np.array(t), inv, amp, inter)
            if t < 0 or not 0 <= pt[b, t // 16] < P:
                continue
            at = int(pt[b, t // 16]), t % 16
            kr[at], ks[at] = ref.rotate(np64(k[row]), np.array(t), inv, amp, inter)
            vr[at] = np64(v[row])
    return kr, ks, vr, qr, qs


APPENDS = [
    # Hq, Hkv, d, rot, interleaved, lengths with the new tokens, new tokens (None: one each)
    (1, 1, 64, 64, False, [1], None),
    (32, 8, 128, 128, False, [1, 16, 17, 100, 0, 31], None),
    (4, 4, 256, 64, True, [5, 33, 64], None),
    (8, 2, 128, 20, False, [5, 33, 64], None),
    (32, 8, 128, 128, False, [70, 3, 0, 16, 200], [70, 2, 0, 16, 33]),
    (4, 1, 64, 32, True, [12, 5], [20, 5]),             # more new tokens than keys
    (2, 2, 128, 0, False, [40, 9], [7, 9]),             # no rotation
    (6, 3, 64, 64, False, list(range(1, 71)), [1 + i % 5 for i in range(70)]),
    (1, 1, 64, 64, False, [0] * 1500 + [3], [0] * 1500 + [3]),
]


def random_append(seed):
    g = np.random.default_rng(seed)
    Hkv = int(g.integers(1, 9))
    d = int(g.choice([64, 128, 256]))
    B = int(g.integers(1, 40))
    new = None if g.random() < 0.4 else [int(v) for v in g.integers(0, 30, B)]
    ln = [int(g.integers(0, 90)) for _ in range(B)]
    rot = int(g.choice([d, d // 2, 16, 2 * int(g.integers(1, d // 2 + 1))]))
    return Hkv * int(g.integers(1, 7)), Hkv, d, rot, bool(g.random() < 0.5), ln, new


APPENDS += [random_append(seed) for seed in range(16)]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: str(c)[:60])
def test_append(case):
    Hq, Hkv, d, rot, inter, ln, new = case
    g = torch.Generator().manual_seed(Hq + d + len(ln))
    B = len(ln)
    cu = np.arange(B + 1) if new is None else np.concatenate([[0], np.cumsum(new)])
    T, tail = int(cu[-1]), 0 if new is None else 3
    width = max(ref.pages_of(max(ln)), 1)
    P = sum(map(ref.pages_of, ln)) + 2
    perm = torch.randperm(P, generator=g).tolist()
    pt = np.full((B, width), -7)
    for b, n in enumerate(ln):
        for j in range(ref.pages_of(n)):
            pt[b, j] = perm.pop()
    x = randn(g, T + tail, Hq + 2 * Hkv, d)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    kp, vp = randn(g, P, 16, Hkv, d), randn(g, P, 16, Hkv, d)
    inv = frequencies(rot)
    kr, ks, vr, qr, qs = append_ref(kp, vp, q, k, v, pt, ln, cu, np64(inv), 1.1, inter)
    xd, kd, vd = x.cuda(), kp.cuda(), vp.cuda()
    out = torch.full((T + tail, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda")
    got = ea.attn_append_paged(
        xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:], kd, vd,
        torch.tensor(pt, dtype=torch.int32).cuda(), torch.tensor(ln, dtype=torch.int32).cuda(),
        None if new is None else torch.tensor(cu, dtype=torch.int32).cuda(),
        inv if rot else None, interleaved=inter, amplitude=1.1, q_out=out)
    assert got is out
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    ref.check_rotated(out[:T], qr[:T], np.maximum(qs[:T], 0), what="q")
    assert (out[T:] == 9.0).all()  # rows behind the last sequence
    ref.check_rotated(kd, kr, np.maximum(ks, 0), what="k pool")
    assert np.array_equal(np64(vd), vr)
    # without q, contiguous k and v, on fresh pools: the same bits
    k2, v2 = kp.cuda(), vp.cuda()
    assert ea.attn_append_paged(
        None, k.contiguous().cuda(), v.contiguous().cuda(), k2, v2,
        torch.tensor(pt, dtype=torch.int32).cuda(), torch.tensor(ln, dtype=torch.int32).cuda(),
        None if new is None else torch.tensor(cu, dtype=torch.int32).cuda(),
        inv if rot else None, interleaved=inter, amplitude=1.1) is None
    assert torch.equal(k2, kd) and torch.equal(v2, vd)


def test_append_in_place():
    g = torch.Generator().manual_seed(8)
    q, k = randn(g, 3, 4, 128).cuda(), randn(g, 3, 2, 128).cuda()
    pools = [torch.zeros(6, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pt = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2)
    ln = torch.tensor([3, 17, 32], dtype=torch.int32, device="cuda")
    inv = frequencies(64)
    want = ea.attn_append_paged(q, k, k, *pools, pt, ln, inv_freq=inv)
    assert ea.attn_append_paged(q, k, k, *pools, pt, ln, inv_freq=inv, q_out=q) is q
    assert torch.equal(q, want)


def test_append_reports_bad_device_data_and_writes_nothing_there():
    g = torch.Generator().manual_seed(9)
    T, P = 6, 5
    k = randn(g, T, 2, 64).cuda()
    q = randn(g, T, 4, 64).cuda()
    inv = frequencies(64)

    def call(pt, ln, cu=None, rows=T):
        pools = [torch.full((P, 16, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
                 for _ in range(2)]
        out = torch.full_like(q[:rows], 9.0)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        ea.attn_append_paged(q[:rows], k[:rows], k[:rows], *pools, i32(pt), i32(ln),
                             None if cu is None else i32(cu), inv, q_out=out)
        torch.cuda.synchronize()
        return ea.attn_device_status(), pools, out

    untouched = lambda pools: all((p == 5.0).all() for p in pools)  # noqa: E731
    ok = [[0], [1], [2], [3], [4], [0]]
    for page in (-1, P, 2 ** 31 - 1, -2 ** 31):
        s, pools, out = call([[page]] * 2, [4, 9], rows=2)
        assert s == ea.ATTN_ERR_BAD_INPUT and untouched(pools) and (out != 9.0).any(-1).all()
    for n in (-1, 17, 2 ** 31 - 1, -2 ** 31):
        s, pools, out = call([[0], [1]], [n, n], rows=2)
        assert s == ea.ATTN_ERR_BAD_INPUT and untouched(pools) and (out == 9.0).all()
    for cu in ([0, 2, 1, 6], [0, 3, 7, 6], [-1, 2, 4, 6], [2 ** 31 - 1, -2 ** 31, 0, 6]):
        s, pools, out = call(ok[:3], [6, 6, 6], cu=cu)
        assert s == ea.ATTN_ERR_BAD_INPUT
    s, pools, out = call(ok[:2], [2, 2], cu=[1, 3, 5])
    assert s == ea.ATTN_OK and (out[[0, 5]] == 9.0).all() and (out[1:5] != 9.0).any(-1).all()


def test_append_into_a_pool_past_32_bits():
    """70,000 pages of 16 x 8 x 256: element offsets past 2^31 in each pool."""
    P, Hkv, d = 70000, 8, 256
    kp = torch.zeros(P, 16, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    g = torch.Generator().manual_seed(10)
    k = randn(g, 3, Hkv, d).cuda()
    pt = torch.tensor([[69999], [66000], [0]], dtype=torch.int32, device="cuda")
    ln = torch.tensor([16, 1, 7], dtype=torch.int32, device="cuda")
    ea.attn_append_paged(None, k, k, kp, vp, pt, ln)
    assert ea.attn_device_status() == ea.ATTN_OK
    for b, (p, n) in enumerate(((69999, 16), (66000, 1), (0, 7))):
        for pool in (kp, vp):
            assert torch.equal(pool[p, n - 1], k[b])
            pool[p, n - 1] = 0
    assert not kp.any() and not vp.any()


def test_captured_and_on_another_stream():
    """One graph of a rotation and an append replayed with new inputs, and calls handed a
    stream of their own: the bits of the plain calls."""
    g = torch.Generator().manual_seed(11)
    q, k = randn(g, 9, 4, 128).cuda(), randn(g, 9, 2, 128).cuda()
    inv = frequencies(128)
    pt = torch.arange(18, dtype=torch.int32, device="cuda").view(9, 2)
    ln = torch.full((9,), 20, dtype=torch.int32, device="cuda")
    make = lambda: [torch.zeros(18, 16, 2, 128, dtype=torch.bfloat16, device="cuda")  # noqa: E731
                    for _ in range(2)]
    pools = make()
    ea.attn_append_paged(q, k, k, *pools, pt, ln, inv_freq=inv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = ea.attn_rope(q, k, inv)
        a = ea.attn_append_paged(q, k, k, *pools, pt, ln, inv_freq=inv)
    for n in (18, 25):
        ln.fill_(n)
        q.copy_(randn(g, 9, 4, 128))
        k.copy_(randn(g, 9, 2, 128))
        for p in pools:
            p.zero_()
        graph.replay()
        want = make()
        assert torch.equal(a, ea.attn_append_paged(q, k, k, *want, pt, ln, inv_freq=inv))
        assert all(torch.equal(x, y) for x, y in zip(pools, want))
        assert all(torch.equal(x, y) for x, y in zip(r, ea.attn_rope(q, k, inv)))
    side = torch.cuda.Stream()
    want = ea.attn_rope(q, k, inv)
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream, 0):
        got = ea.attn_rope(q, k, inv, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
