"""Rotary positions and the paged cache's upkeep on the GPU, at the lengths, sizes and
positions where a call could go wrong unnoticed."""
import gc

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
