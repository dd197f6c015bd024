"""Plain references for the operators on shared and thinned caches, in fp64 numpy: one row
and one head at a time, nothing shared with the library."""
import numpy as np

PAGE = 16

# How far a weight exp(x - LSE), x = scale q.k, may be off, relative to itself.  The scores
# are fp32 sums of exact products of bf16 values: at most d / 16 + 4 roundings of 2^-23
# each of the partial sums, which sum |q_i k_i| scale bounds (below 14 for the values here,
# normal ones and d = 256): 14 * 20 * 2^-23 = 3.4e-5.  The exponent's argument in base 2,
# below 64, and the LSE's are rounded to 2^-24 of themselves (8e-6 together) and 2^x is
# good to 2^-22 in each of a row's terms and its sum (1e-6).
WEIGHT = 5e-5
# the mass's own additions: one rounding a head and query tile, 2^-24 of the sum each
SUM = 2.0 ** -20


def gather(pool, table, n):
    """[n, Hkv, d] fp64 of one row's first n slots."""
    p = np.asarray(pool, np.float64)
    if n == 0:
        return np.zeros((0,) + p.shape[2:])
    return np.concatenate([p[j] for j in table[:(n + PAGE - 1) // PAGE]])[:n]


def attend(q, k, v, scale, sink=None, seen=None):
    """q [Hq, d] over k, v [n, Hkv, d] -> o [Hq, d], lse [Hq], weights [Hq, n]."""
    Hq, G = q.shape[0], q.shape[0] // k.shape[1]
    o, lse, w = np.zeros(q.shape), np.zeros(Hq), np.zeros((Hq, len(k)))
    for h in range(Hq):
        x = scale * (k[:, h // G] @ q[h])
        if seen is not None:
            x = np.where(seen, x, -np.inf)
        terms = x if sink is None else np.append(x, sink[h])
        top = terms.max() if terms.size else -np.inf
        if top == -np.inf:
            lse[h] = -np.inf
            continue
        lse[h] = top + np.log(np.exp(terms - top).sum())
        w[h] = np.exp(x - lse[h])
        o[h] = w[h] @ v[:, h // G]
    return o, lse, w


def seen_keys(i, Lq, Lk, causal, window, n_sink):
    """Which keys query i of Lq sees."""
    t = np.arange(Lk)
    at = i + Lk - Lq
    ok = np.ones(Lk, bool)
    if causal:
        ok &= t <= at
        if window > 0:
            ok &= (t > at - window) | (t < n_sink)
    return ok


def check_mass(got, base, w, what=""):
    """got = base + w within the weights' error and the sums' roundings."""
    err = np.abs(got - (base + w))
    bad = err > WEIGHT * w + SUM * np.abs(base + w) + 1e-30
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), err.max())


def evict(mass, positions, L, K, n_sink, recent):
    """Moves (from, to) of one row, layer and head."""
    m, p = np.asarray(mass[:L], np.float64), np.asarray(positions[:L], np.int64)
    held = p < n_sink
    if recent > 0:
        held |= p > p.max() - recent
    lowest = np.isnan(m)
    rank = np.lexsort((np.arange(L), np.where(held | lowest, 0, -m), lowest & ~held, ~held))
    stay = np.zeros(L, bool)
    stay[rank[:K]] = True
    return list(zip(np.flatnonzero(stay[K:]) + K, np.flatnonzero(~stay[:K])))
