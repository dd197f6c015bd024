"""Rotary positions and the paged cache's upkeep, without a GPU: argument
checks that answer before any CUDA call, the frequencies, and the host
reference that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _cache_ref as ref


def _ptr():
    buf = ctypes.create_string_buffer(4096)
    return buf, (ctypes.cast(buf, ctypes.c_void_p).value + 15) & ~15


ROPE = dict(q=0, k=0, qo=0, ko=0, pos=0, inv=0, B=1, S=4, Hq=2, Hkv=2, d=128, rot=128,
            inter=0, amp=1.0, qs=None, ks=None, qos=None, kos=None, stream=None)


@pytest.mark.parametrize("fn", ["attn_rope", "attn_rope_bwd"])
@pytest.mark.parametrize("change,status", [
    (dict(d=96), "UNSUPPORTED"), (dict(rot=130), "INVALID_ARG"), (dict(rot=3), "INVALID_ARG"),
    (dict(rot=-2), "INVALID_ARG"), (dict(inter=2), "INVALID_ARG"),
    (dict(amp=math.inf), "INVALID_ARG"), (dict(amp=math.nan), "INVALID_ARG"),
    (dict(inv=None), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(ko=None), "INVALID_ARG"),
    (dict(B=-1), "INVALID_ARG"), (dict(B=1 << 20, S=1 << 20), "INVALID_ARG"),
    (dict(B=1, S=2 ** 31 - 1), "INVALID_ARG"), (dict(Hq=(1 << 20) + 1), "INVALID_ARG"),
    (dict(q=2), "INVALID_ARG"), (dict(inv=4), "INVALID_ARG"), (dict(pos=1), "INVALID_ARG"),
    (dict(qs=(1024, 260, 128)), "INVALID_ARG"), (dict(ks=(1024, -256, 128)), "INVALID_ARG"),
    (dict(kos=(1024, 0, 128)), "INVALID_ARG"),
    (dict(qo=-256, qs=(1024, 512, 128)), "INVALID_ARG"),  # in place, another stride
    (dict(B=0), "OK"), (dict(S=0), "OK"), (dict(Hq=0, Hkv=0), "OK"),
])
def test_rope_arguments(fn, change, status):
    buf, p = _ptr()
    a = dict(ROPE, q=p, k=p + 128, qo=p + 256, ko=p + 384, pos=p, inv=p)
    for key, v in change.items():
        if key in ("q", "qo", "inv", "pos") and isinstance(v, int):
            v = a[key] + v
        elif key in ("qs", "ks", "qos", "kos"):
            v = (ctypes.c_longlong * 3)(*v)
        a[key] = v
    assert getattr(ea.lib, fn)(*a.values()) == getattr(ea, "ATTN_" + (
        status if status == "OK" else "ERR_" + status))


APPEND = dict(q=0, k=0, v=0, qo=0, kp=0, vp=0, pt=0, cu=None, ln=0, inv=0, B=2, Hq=4, Hkv=2,
              T=2, d=128, rot=128, inter=0, amp=1.0, page=16, maxp=4, P=8, qs=None, ks=None,
              vs=None, qos=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(d=32), "UNSUPPORTED"), (dict(page=32), "UNSUPPORTED"), (dict(T=3), "INVALID_ARG"),
    (dict(Hkv=0), "INVALID_ARG"), (dict(P=0), "INVALID_ARG"), (dict(maxp=1 << 27), "INVALID_ARG"),
    (dict(rot=129), "INVALID_ARG"), (dict(inv=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"),
    (dict(qo=None), "INVALID_ARG"), (dict(pt=None), "INVALID_ARG"), (dict(ln=None), "INVALID_ARG"),
    (dict(vs=(250, 128)), "INVALID_ARG"), (dict(qos=(0, 128)), "INVALID_ARG"),
    (dict(B=0, T=0), "OK"), (dict(B=2 ** 31 - 1, T=2 ** 31 - 1), "INVALID_ARG"),
    (dict(B=2 ** 31 - 1, T=4, cu=16), "INVALID_ARG"),
])
def test_append_arguments(change, status):
    buf, p = _ptr()
    a = dict(APPEND)
    for key in ("q", "k", "v", "qo", "kp", "vp", "pt", "ln", "inv"):
        a[key] = p
    a["qo"] = p + 1024
    for key, v in change.items():
        a[key] = (ctypes.c_longlong * 2)(*v) if key in ("qs", "ks", "vs", "qos") else v
    assert ea.lib.attn_append_paged(*a.values()) == getattr(ea, "ATTN_" + (
        status if status == "OK" else "ERR_" + status))


def _pages_args(which):
    buf, p = _ptr()
    tail = dict(kp=p, vp=p, B=4, layers=2, Hkv=2, d=64, page=16, maxp=4, P=8, ws=p,
                bytes=2048, stream=None)
    if which == "resize":
        return buf, dict(dict(pt=p, ln=p, new=p, refs=p), **tail)
    if which == "fork":
        return buf, dict(dict(pt=p, ln=p, refs=p, src=p, dst=p, n=2), **tail)
    return buf, dict(dict(pt=p, ln=p, refs=p, idx=p, live=p), **tail)


@pytest.mark.parametrize("which", ["resize", "fork", "compact"])
@pytest.mark.parametrize("change,status", [
    (dict(page=8), "UNSUPPORTED"), (dict(d=80), "UNSUPPORTED"), (dict(layers=0), "INVALID_ARG"),
    (dict(P=0), "INVALID_ARG"), (dict(P=(1 << 23) + 1), "INVALID_ARG"),
    (dict(maxp=0), "INVALID_ARG"), (dict(refs=None), "INVALID_ARG"), (dict(pt=None), "INVALID_ARG"),
    (dict(bytes=16), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"), (dict(kp=None), "INVALID_ARG"),
    (dict(B=-1), "INVALID_ARG"), (dict(B=(1 << 20) + 1, bytes=1 << 30), "INVALID_ARG"),
])
def test_pages_arguments(which, change, status):
    buf, a = _pages_args(which)
    a.update(change)
    rc = getattr(ea.lib, "attn_pages_" + which)(*a.values())
    assert rc == getattr(ea, "ATTN_ERR_" + status), ea.attn_last_error()


def test_pages_row_limits_and_empty_calls():
    buf, a = _pages_args("resize")
    assert ea.lib.attn_pages_resize(*dict(a, B=8193, bytes=1 << 30).values()) == \
        ea.ATTN_ERR_INVALID_ARG
    assert ea.lib.attn_pages_resize(*dict(a, B=0).values()) == ea.ATTN_OK
    assert ea.lib.attn_pages_resize(*dict(a, new=None).values()) == ea.ATTN_ERR_INVALID_ARG
    buf, a = _pages_args("fork")
    assert ea.lib.attn_pages_fork(*dict(a, n=0).values()) == ea.ATTN_OK
    assert ea.lib.attn_pages_fork(*dict(a, n=-1).values()) == ea.ATTN_ERR_INVALID_ARG
    assert ea.lib.attn_pages_fork(*dict(a, n=8193, bytes=1 << 30).values()) == \
        ea.ATTN_ERR_INVALID_ARG
    assert ea.lib.attn_pages_fork(*dict(a, src=None).values()) == ea.ATTN_ERR_INVALID_ARG
    buf, a = _pages_args("compact")
    assert ea.lib.attn_pages_compact(*dict(a, idx=None).values()) == ea.ATTN_ERR_INVALID_ARG
    assert ea.attn_pages_workspace_size(0, 0) == 0
    assert ea.attn_pages_workspace_size(8193, 4) == 0
    assert ea.attn_pages_workspace_size(3, 5) > 4 * (2 * 5 + 2 * 3)
    assert ea.attn_status_string(ea.ATTN_ERR_NO_PAGES) != "unknown status"


def test_binding_refuses_host_tensors_and_wrong_types():
    q, inv = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        ea.attn_rope(q, None, inv)
    with pytest.raises(ValueError):
        ea.attn_rope(None, None, inv)
    with pytest.raises(ValueError):
        ea.attn_append_paged(None, q, q, q[None], q[None], torch.zeros(4, 1, dtype=torch.int32),
                             torch.ones(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        ea.attn_pages_compact(torch.zeros(1, 1, dtype=torch.int32),
                              torch.zeros(1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
                              q, q)


def test_frequencies():
    r = 64
    i = np.arange(r // 2)
    f = 500.0 ** (-2.0 * i / r)
    get = lambda **k: ea.attn_rope_inv_freq(r, 500.0, device="cpu", **k).numpy()  # noqa: E731
    np.testing.assert_allclose(get(), f, rtol=1e-14)
    np.testing.assert_allclose(get(scaling="linear", factor=4.0), f / 4, rtol=1e-14)
    g = get(scaling="base", factor=4.0)
    assert g[0] == 1.0
    np.testing.assert_allclose(g[-1], f[-1] / 4, rtol=1e-12)
    g = get(scaling="ramp", factor=8.0, original_length=2048.0, ramp=(1.0, 32.0))
    turns = 2048 * f / (2 * math.pi)
    np.testing.assert_allclose(g[turns > 32], f[turns > 32], rtol=1e-14)
    np.testing.assert_allclose(g[turns < 1], f[turns < 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((g[mid] < f[mid]) & (g[mid] > f[mid] / 8)).all()
    for bad in (dict(scaling="linear", factor=0.0), dict(scaling="ramp", factor=2.0),
                dict(scaling="ramp", factor=2.0, original_length=10.0, ramp=(2.0, 2.0)),
                dict(scaling="base", factor=-1.0)):
        with pytest.raises(ea.AttnError):
            get(**bad)
    with pytest.raises(ea.AttnError):
        ea.attn_rope_inv_freq(7, device="cpu")
    with pytest.raises(ValueError):
        ea.attn_rope_inv_freq(8, scaling="other", device="cpu")


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation(interleaved):
    """The reference keeps lengths, depends on position differences alone in q.k, and its
    transpose is the turn by the negated position (central differences)."""
    g = np.random.default_rng(0)
    inv = 100.0 ** (-np.arange(4) / 4)
    q, k = g.standard_normal((2, 3, 1, 12))
    rot = lambda x, p: ref.rotate(x, p, inv, 1.25, interleaved)[0]  # noqa: E731
    p = np.array([5, 900, -3])
    np.testing.assert_allclose((rot(q, p)[..., :8] ** 2).sum(-1),
                               1.25 ** 2 * (q[..., :8] ** 2).sum(-1))
    np.testing.assert_allclose((rot(q, p) * rot(k, p + 7)).sum(-1),
                               (rot(q, p + 50) * rot(k, p + 57)).sum(-1))
    grad = ref.rotate(k, p, inv, 1.25, interleaved, -1.0)[0]
    h = 0.5  # the turn is linear: any step is exact
    for j in range(12):
        e = np.zeros(12)
        e[j] = h
        d = ((rot(q + e, p) - rot(q - e, p)) * k).sum(-1) / (2 * h)
        np.testing.assert_allclose(d, grad[..., j], atol=1e-12)


def test_reference_pages_keep_the_counts():
    """After any calls every count is the number of table entries that hold the page."""
    g = np.random.default_rng(1)
    B, W, P = 7, 6, 30
    m = ref.Pages([[-1] * W for _ in range(B)], [0] * B, [0] * P)
    for step in range(200):
        kind = int(g.integers(0, 4))
        if kind < 2:
            m.resize([int(g.integers(0, W * 16 + 1)) if g.random() < 0.4 else n for n in m.len])
        elif kind == 2:
            m.fork(g.integers(0, B, 3).tolist(), g.integers(0, B, 3).tolist())
        else:
            m.compact()
        count = [0] * P
        for row, n in zip(m.table, m.len):
            for p in row[:ref.pages_of(n)]:
                count[p] += 1
        assert count == m.refs
        for row, n in zip(m.table, m.len):
            assert len(set(row[:ref.pages_of(n)])) == ref.pages_of(n)
