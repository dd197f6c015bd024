"""Operators on shared and thinned caches, without a GPU: argument checks that answer before
any CUDA call, workspace sizes, the binding's refusals, and the host reference that the
GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
import oracle
from tests import _thin_ref as ref


def _ptr():
    buf = ctypes.create_string_buffer(4096)
    return buf, (ctypes.cast(buf, ctypes.c_void_p).value + 15) & ~15


def status(name):
    return getattr(ea, "ATTN_" + (name if name == "OK" else "ERR_" + name))


COMMON = [
    (dict(d=96), "UNSUPPORTED"), (dict(page=32), "UNSUPPORTED"), (dict(B=-1), "INVALID_ARG"),
    (dict(Hkv=0), "INVALID_ARG"), (dict(maxp=0), "INVALID_ARG"), (dict(P=0), "INVALID_ARG"),
    (dict(maxp=1 << 27), "INVALID_ARG"), (dict(B=65536), "INVALID_ARG"),
    (dict(ws=None), "INVALID_ARG"), (dict(bytes=16), "INVALID_ARG"), (dict(ws=8), "INVALID_ARG"),
    (dict(pt=None), "INVALID_ARG"), (dict(ln=None), "INVALID_ARG"), (dict(kp=None), "INVALID_ARG"),
    (dict(pt=2), "INVALID_ARG"), (dict(kp=8), "INVALID_ARG"), (dict(B=0), "OK"),
]
HEADS = [
    (dict(Hq=3), "INVALID_ARG"), (dict(Hq=0), "INVALID_ARG"), (dict(scale=0.0), "INVALID_ARG"),
    (dict(scale=math.inf), "INVALID_ARG"), (dict(scale=math.nan), "INVALID_ARG"),
    (dict(q=None), "INVALID_ARG"), (dict(q=4), "INVALID_ARG"),
    (dict(Hq=65536, Hkv=65536), "INVALID_ARG"), (dict(B=65535, Hq=32768), "INVALID_ARG"),
]
DECODE = [(dict(splits=0), "INVALID_ARG"), (dict(splits=65), "INVALID_ARG"),
          (dict(o=None), "INVALID_ARG"), (dict(lse=2), "INVALID_ARG"), (dict(sink=1), "INVALID_ARG")]


def call(fn, order, defaults, change):
    buf, p = _ptr()
    a = {k: p if v is PTR else v for k, v in defaults.items()}
    for k, v in change.items():
        a[k] = p + v if isinstance(v, int) and defaults[k] is PTR else v
    return getattr(ea.lib, fn)(*(a[k] for k in order.split()))


PTR = object()
SIZES = dict(B=2, Hq=4, Hkv=2, d=128, page=16, maxp=4, P=8, splits=2, scale=0.1, sink=None, ws=PTR,
             bytes=1 << 40, stream=None)
SHARED = dict(q=PTR, kp=PTR, vp=PTR, pt=PTR, ln=PTR, cu=PTR, pre=PTR, rows=PTR, o=PTR, lse=PTR,
              groups=1, listed=2, **SIZES)
SHARED_ORDER = ("q kp vp pt ln cu pre rows o lse B Hq Hkv d page maxp P groups listed splits scale "
                "sink ws bytes stream")


@pytest.mark.parametrize("change,want", COMMON + HEADS + DECODE + [
    (dict(groups=-1), "INVALID_ARG"), (dict(listed=-1), "INVALID_ARG"),
    (dict(groups=(1 << 20) + 1), "INVALID_ARG"), (dict(listed=(1 << 20) + 1), "INVALID_ARG"),
    (dict(cu=None), "INVALID_ARG"), (dict(pre=None), "INVALID_ARG"), (dict(rows=2), "INVALID_ARG"),
    (dict(rows=None, listed=3), "INVALID_ARG"), (dict(listed=1 << 20, Hq=2048), "INVALID_ARG")])
def test_shared_arguments(change, want):
    assert call("attn_decode_paged_shared", SHARED_ORDER, SHARED, change) == status(want), \
        ea.attn_last_error()


MASS = dict(q=PTR, kp=PTR, vp=PTR, pt=PTR, ln=PTR, mass=PTR, out=PTR, pos=PTR, last=PTR, o=PTR,
            lse=PTR, slots=64, **SIZES)
MASS_ORDER = ("q kp vp pt ln mass out pos last o lse B Hq Hkv d page maxp P slots splits scale sink "
              "ws bytes stream")


@pytest.mark.parametrize("change,want", COMMON + HEADS + DECODE + [
    (dict(mass=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(mass=2), "INVALID_ARG"),
    (dict(pos=2), "INVALID_ARG"), (dict(last=1), "INVALID_ARG"), (dict(slots=0), "INVALID_ARG")])
def test_decode_mass_arguments(change, want):
    assert call("attn_decode_paged_mass", MASS_ORDER, MASS, change) == status(want), \
        ea.attn_last_error()


BLOCK = dict(q=PTR, lse=PTR, kp=PTR, pt=PTR, cu=PTR, ln=PTR, mass=PTR, out=PTR, pos=PTR, last=PTR,
             new=PTR, sq=4, total=8, slots=64, causal=1, window=0, nsink=0, **SIZES)
BLOCK_ORDER = ("q lse kp pt cu ln mass out pos last new B Hq Hkv sq total d page maxp P slots scale "
               "causal window nsink ws bytes stream")


@pytest.mark.parametrize("change,want", COMMON + HEADS + [
    (dict(mass=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(lse=None), "INVALID_ARG"),
    (dict(cu=None), "INVALID_ARG"), (dict(new=2), "INVALID_ARG"), (dict(slots=0), "INVALID_ARG"),
    (dict(sq=-1), "INVALID_ARG"), (dict(total=-1), "INVALID_ARG"),
    (dict(total=(1 << 29) + 1), "INVALID_ARG"), (dict(sq=(1 << 29) + 1), "INVALID_ARG"),
    (dict(maxp=(1 << 25) + 1), "INVALID_ARG"), (dict(causal=2), "INVALID_ARG"),
    (dict(causal=0, window=4), "INVALID_ARG"), (dict(nsink=2), "INVALID_ARG"),
    (dict(window=4, nsink=-1), "INVALID_ARG")])
def test_mass_arguments(change, want):
    assert call("attn_mass_paged", BLOCK_ORDER, BLOCK, change) == status(want), ea.attn_last_error()


EVICT = dict(mass=PTR, pos=PTR, pt=PTR, ln=PTR, keep=PTR, refs=PTR, new=PTR, kp=PTR, vp=PTR,
             layers=2, slots=64, nsink=0, recent=0, **SIZES)
EVICT_ORDER = ("mass pos pt ln keep refs new kp vp B layers Hkv d slots page maxp P nsink recent ws "
               "bytes stream")


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(layers=0), "INVALID_ARG"), (dict(slots=0), "INVALID_ARG"), (dict(nsink=-1), "INVALID_ARG"),
    (dict(recent=-1), "INVALID_ARG"), (dict(mass=None), "INVALID_ARG"), (dict(pos=None), "INVALID_ARG"),
    (dict(keep=None), "INVALID_ARG"), (dict(new=None), "INVALID_ARG"), (dict(vp=None), "INVALID_ARG"),
    (dict(refs=2), "INVALID_ARG"), (dict(P=(1 << 23) + 1), "INVALID_ARG"),
    (dict(layers=1 << 12, B=1 << 12), "INVALID_ARG")])
def test_evict_arguments(change, want):
    # (the lengths, the budgets and the new lengths are three arrays)
    defaults = dict(EVICT)
    buf, p = _ptr()
    defaults.update(ln=p + 64, keep=p + 128, new=p + 256)
    change = {k: (defaults[k] + v if k in ("ln", "keep", "new") and isinstance(v, int) else v)
              for k, v in change.items()}
    assert call("attn_evict_paged", EVICT_ORDER, defaults, change) == status(want), \
        ea.attn_last_error()


def test_evict_refuses_lengths_over_its_inputs():
    for same in ("ln", "keep"):
        defaults = dict(EVICT)
        buf, p = _ptr()
        defaults.update(ln=p + 64, keep=p + 128, new=p + 256)
        defaults["new"] = defaults[same]
        assert call("attn_evict_paged", EVICT_ORDER, defaults, {}) == ea.ATTN_ERR_INVALID_ARG


def test_workspace_sizes():
    assert ea.attn_decode_mass_workspace_size(2, 4, 128, 3, 2) >= \
        ea.attn_decode_workspace_size(2, 4, 128, 2) + 2 * 4 * 48 * 4
    assert ea.attn_decode_mass_workspace_size(2, 4, 128, 0, 2) == 0
    assert ea.attn_evict_workspace_size(2, 3, 4, 100, 4) == 24 * (32 * 8 + 4)
    assert ea.attn_evict_workspace_size(2, 3, 4, 30, 4) == 24 * (15 * 8 + 4)
    assert ea.attn_mass_workspace_size(2, 4, 0) == ea.attn_mass_workspace_size(-1, 4, 4) == 0
    assert ea.attn_mass_workspace_size(2, 4, 17) > ea.attn_mass_workspace_size(2, 4, 16) > 0
    size = ea.attn_decode_shared_workspace_size
    assert size(2, 4, 2, 128, 1, 2, 10, 2) > ea.attn_decode_workspace_size(2, 4, 128, 2)
    for bad in ((2, 5, 2, 128, 1, 2, 10, 2), (2, 4, 2, 96, 1, 2, 10, 2), (2, 4, 2, 128, -1, 2, 10, 2),
                (2, 4, 2, 128, 1, 2, 10, 65), (1 << 33, 4, 2, 128, 1, 2, 10, 2)):
        assert size(*bad) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    q, pool = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 16, 2, 64,
                                                                       dtype=torch.bfloat16)
    pt, ln = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    mass = torch.zeros(2, 2, 16)
    calls = (lambda q=q: ea.attn_decode_paged_shared(q, pool, pool, pt, ln, ln, ln[:1]),
             lambda q=q: ea.attn_decode_paged_mass(q, pool, pool, pt, ln, mass),
             lambda q=q: ea.attn_mass_paged(q, torch.zeros(4, 2), pool, pt, torch.zeros(3).int(),
                                            ln, mass, max_seqlen_q=1),
             lambda q=mass: ea.attn_evict_paged(q, mass.int(), pt, ln, ln, pool, pool))
    for f in calls:
        with pytest.raises(ValueError):
            f()
        with pytest.raises((TypeError, ValueError)):
            f([1, 2])


def test_reference_against_the_oracle():
    """The reference's attention, masks and gathering against the C oracle."""
    g = np.random.default_rng(3)
    Hq, Hkv, d, L = 4, 2, 64, 37
    pool = g.standard_normal((2, 6, 16, Hkv, d))
    table = [4, 0, 5]
    q = g.standard_normal((1, Hq, d))
    k, v = (ref.gather(p, table, L) for p in pool)
    o, lse = oracle.attn_decode(q, k[None], v[None], np.array([L], np.int32), 0.2)
    ro, rl, w = ref.attend(q[0], k, v, 0.2)
    np.testing.assert_allclose(ro, o[0], atol=1e-12)
    np.testing.assert_allclose(rl, lse[0], atol=1e-12)
    np.testing.assert_allclose(w.sum(1), 1, atol=1e-12)
    Q = g.standard_normal((1, 9, Hq, d))
    o, lse = oracle.attn_fwd(Q, k[None], v[None], 0.2, True)
    for i in range(9):
        ro, rl, _ = ref.attend(Q[0, i], k, v, 0.2, seen=ref.seen_keys(i, 9, L, True, 0, 0))
        np.testing.assert_allclose(ro, o[0, i], atol=1e-12)
        np.testing.assert_allclose(rl, lse[0, :, i], atol=1e-12)


def test_reference_of_the_eviction():
    mass = np.array([5, 1, 4, 4, 0, 9, np.nan, 4], np.float32)
    pos = np.array([0, 10, 2, 3, 4, 5, 6, 7], np.int32)
    assert ref.evict(mass, pos, 8, 4, 0, 0) == [(5, 1)]          # 9, 5 and the first two 4s
    assert ref.evict(mass, pos, 8, 3, 0, 0) == [(5, 1)]          # one 4
    assert ref.evict(mass, pos, 8, 4, 0, 1) == [(5, 3)]          # position 10 is the newest
    assert ref.evict(mass, pos, 8, 2, 1, 4) == []                # 0, 10 and 7: the lowest slots
    assert ref.evict(mass, pos, 8, 8, 0, 0) == []
