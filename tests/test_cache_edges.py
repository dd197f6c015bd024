"""Rotary positions and the paged cache's upkeep on the GPU, at the lengths, sizes and
positions where a call could go wrong unnoticed."""
import gc
from fractions import Fraction

import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _cache_ref as ref
from tests.test_cache_edges_cpu import without_cuda_names
from tests.test_pages_parity import Cache, i32

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ fork: stored lengths

@pytest.mark.parametrize("bad", [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 5, -2 ** 31 + 8191,
                                 -2 ** 31 + 8192, -1, 65, 2 ** 31 - 1])
def test_fork_reports_stored_lengths_out_of_range(bad):
    """As a source's length, as a new row's, and as both, by the fork whose number is near
    the length's distance from -2^31 and by others."""
    c = Cache(10, 4, 40, layers=2)
    c.resize([40, 0, 0, 5, 0, 0, 0, 0, 0, 0])
    c.m.len[1] = c.m.len[9] = bad
    c.load()
    for src, dst in (([1], [2]), ([0], [1]), ([1], [9]), ([0, 1, 3], [1, 2, 9]),
                     ([0, 0, 0, 0, 0, 0], [2, 4, 5, 6, 7, 1]), ([1, 0, 0], [4, 1, 4])):
        before = c.m.len[1], c.m.len[9]
        c.fork(src, dst)
        assert "bad" in c.m.status and (c.m.len[1], c.m.len[9]) == before == (bad, bad)
        for b in range(1, 9):
            if b not in (1, 3):
                for p in c.m.table[b][:ref.pages_of(c.m.len[b])]:
                    c.m.refs[p] -= 1
                c.m.len[b] = 0
        c.load()


def test_many_forks_into_few_rows():
    """8,192 forks whose rows repeat: the first of each row stands, whichever block
    holds it, and a row that some fork fills is empty as a source."""
    B = 600
    c = Cache(B, 3, 900)
    g = np.random.default_rng(12)
    c.resize([int(g.integers(1, 49)) if b < 200 else 0 for b in range(B)])
    for _ in range(3):
        c.fork(g.integers(0, B, 8192).tolist(), g.integers(0, B, 8192).tolist())
        c.resize([n if b < 200 else 0 for b, n in enumerate(c.m.len)])


# ------------------------------------------------------------------ memory

def test_a_captured_call_leaves_no_memory_behind():
    """A page call of a size first met in a capture: its graph's memory goes with it."""
    def tables(P):
        return (i32([[0, -1]]), i32([5]), i32([1] + [0] * (P - 1)),
                torch.zeros(P, 16, 1, 64, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(P, 16, 1, 64, dtype=torch.bfloat16, device="cuda"))

    ea.attn_pages_compact(*tables(8))
    args, new = tables(1237), i32([20])
    torch.cuda.synchronize()

    def reserved():
        gc.collect()
        torch.cuda.empty_cache()
        return torch.cuda.memory_reserved()

    before = reserved()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ea.attn_pages_resize(args[0], args[1], new, args[2], *args[3:])
        out = ea.attn_pages_compact(*args)
    graph.replay()
    torch.cuda.synchronize()
    assert out[1].item() == 2 and ea.attn_device_status() == ea.ATTN_OK
    del out, graph
    assert reserved() == before
    ea.attn_pages_compact(*args)         # the same size again, outside it
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK


# ------------------------------------------------------------------ sizes

def test_sizes_past_32_bits_are_refused():
    """Counts, tables and lengths whose sizes a 32-bit int does not hold."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    big = torch.empty((1 << 32) + 12, dtype=torch.int32, device="cuda")
    big[:64] = 0
    pt, ln, new = i32([[-1] * 4] * 2), i32([0, 0]), i32([5, 0])
    refs = i32([0] * 12)
    pools = [torch.zeros(12, 16, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    kv = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    many = kv.expand(big.numel(), 1, 64)
    for call in (lambda: ea.attn_pages_resize(pt, ln, new, big),
                 lambda: ea.attn_pages_resize(big[None], ln[:1], new[:1], refs),
                 lambda: ea.attn_pages_fork(pt, ln, refs, big, big, *pools),
                 lambda: ea.attn_append_paged(None, kv, kv, *pools, big[None], i32([1])),
                 lambda: ea.attn_append_paged(None, many, many, *pools, big[:, None], big)):
        with pytest.raises(ea.AttnError) as e:
            call()
        assert e.value.status == ea.ATTN_ERR_INVALID_ARG
    assert ea.attn_device_status() == ea.ATTN_OK
    assert not any(p.any() for p in pools) and not ln.any() and not refs.any()


# ------------------------------------------------------------------ torch without private names

def test_calls_without_torchs_private_names(monkeypatch):
    g = torch.Generator().manual_seed(2)
    q = torch.randn(2, 5, 3, 64, generator=g).bfloat16().cuda()
    inv = ea.attn_rope_inv_freq(64)
    want = ea.attn_rope(q, None, inv)[0]
    here = torch.cuda.current_device()
    without_cuda_names(monkeypatch)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: here)  # it uses one of the names
    assert torch.equal(ea.attn_rope(q, None, inv)[0], want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = ea.attn_rope(q, None, inv)[0]
    side.synchronize()
    assert torch.equal(got, want)


# ------------------------------------------------------------------ far positions

# pi to 60 digits, for angles in exact arithmetic
TWO_PI = 2 * Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


def exact_angle(p, f):
    """p f less whole turns, to the last bit of fp64."""
    turns = Fraction(f) * p / TWO_PI
    return float((turns - round(turns)) * TWO_PI)


def nearly_cancelling(c, s):
    """bf16 (x, y) with x c - y s as near zero as a search over their mantissas finds."""
    m = 1 + np.arange(128) / 128
    x, y = m[:, None], m[None, :] * 2.0 ** np.round(np.log2(abs(c / s)))
    y = y * np.sign(c * s)
    i, j = np.unravel_index(np.argmin(np.abs(x * c - y * s)), (128, 128))
    return float(x[i, 0]), float(y[0, j])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [128, 20])
def test_angles_of_far_positions(interleaved, rot):
    """Pairs that the turn brings near zero in their first element: what is left is the
    angle's error, no longer under half a step of a large value.  An angle off by the
    documented 1e-6 radians would move that element by sqrt(x^2 + y^2) 1e-6, more than
    the NEAR (|x| + |y|) allowed here for |y| near |x|; the kernel's own angle is
    off by less than 2^-33 of a turn.  The reference's angle is exact, so it
    adds nothing."""
    positions = [1, -1, 131071, 10 ** 6, 2 ** 25 - 1, -2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31]
    inv = ea.attn_rope_inv_freq(rot, 1e4)
    f = inv.cpu().numpy()
    x = np.zeros((len(positions), 1, 128))
    want, size = x.copy(), x.copy()
    for r, p in enumerate(positions):
        for i in range(rot // 2):
            t = exact_angle(p, f[i])
            c, s = np.cos(t), np.sin(t)
            if not 0.02 < abs(s / c) < 50:
                continue
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            u, v = nearly_cancelling(c, s)
            x[r, 0, a], x[r, 0, b] = u, v
            want[r, 0, a], want[r, 0, b] = u * c - v * s, u * s + v * c
            size[r, 0, a] = size[r, 0, b] = abs(u) + abs(v)
    q = torch.tensor(x).bfloat16().cuda()
    assert np.array_equal(q.double().cpu().numpy(), x)
    assert (size > 0).mean() > 0.4 * rot / 128
    y = ea.attn_rope(q, None, inv, i32(positions), interleaved=interleaved)[0]
    ref.check_rotated(y, want, size)
