"""Plain references for rotary positions and the paged cache's upkeep.

rotate() is the formula in fp64 on numpy arrays; Pages walks over host lists
one row at a time.  Neither shares code with the library.
"""
import numpy as np

PAGE = 16

# A rotated element before its rounding to bf16: the angle as half turns in
# fp32 (2^-25 of at most pi: 9.4e-8), sincospif within 2 ulp of values up to 1
# (2 * 2^-24: 1.2e-7), the amplitude's product (2^-24) and the two products
# and their sum (2 * 2^-24) each relative to |x| + |y|.  Together below 6e-7
# of amplitude * (|x| + |y|) while the angle's 64-bit error, |p| * 2^-52, is
# below 1e-8 (|p| < 2^25); at the ends of int32 that error and the one of the
# reference's own p * f are 5e-7 and 2.4e-7 more.
NEAR, FAR = 6e-7, 1.5e-6
HALF_STEP = 2.0 ** -8  # bf16


def rotate(x, pos, inv, amplitude=1.0, interleaved=False, sign=1.0):
    """x [..., H, d] fp64, pos [...] integers, inv [r / 2] -> (turned, |x| + |y| per element)."""
    x = np.asarray(x, np.float64)
    r = 2 * len(inv)
    ang = np.asarray(pos, np.float64)[..., None, None] * np.asarray(inv, np.float64)
    c, s = np.cos(ang) * amplitude, sign * np.sin(ang) * amplitude
    out, size = x.copy(), np.zeros_like(x)
    i = np.arange(r // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., a] * s + x[..., b] * c
    size[..., a] = size[..., b] = abs(amplitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, size


def check_rotated(got, ref, size, slack=NEAR, what=""):
    """|got - ref| within half a bf16 step of the value and the fp32 error before it;
    elements that were not turned (size 0) are equal."""
    g = got.double().cpu().numpy()
    e = slack * size
    bad = np.abs(g - ref) > e + HALF_STEP * (np.abs(ref) + e) * (size > 0)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist())


def pages_of(n):
    return (n + PAGE - 1) // PAGE


class Pages:
    """Table, lengths and counts as host lists; `moves` collects (from, to) page copies of
    the last call, `status` the names of what the call reports."""

    def __init__(self, table, lengths, refs):
        self.table = [list(r) for r in table]
        self.len = list(lengths)
        self.refs = list(refs)
        self.moves, self.status = [], set()

    def _free(self):
        return [p for p, c in enumerate(self.refs) if c <= 0]

    def _page(self, p):
        return 0 <= p < len(self.refs)

    def resize(self, new, share=True):
        self.moves, self.status = [], set()
        most = len(self.table[0]) * PAGE if self.table else 0
        ok = [0 <= a <= most and 0 <= n <= most for a, n in zip(self.len, new)]
        for b, n in enumerate(new):
            if not ok[b]:
                self.status.add("bad")
                continue
            for j in range(pages_of(n), pages_of(self.len[b])):
                if self._page(self.table[b][j]):
                    self.refs[self.table[b][j]] -= 1
                else:
                    self.status.add("bad")
        free, held = self._free(), list(self.refs)
        room, asked = len(free), 0
        for b, n in enumerate(new):
            if not ok[b]:
                continue
            old, split = self.len[b], False
            need = max(0, pages_of(n) - pages_of(old))
            if share and n > old and old % PAGE:
                last = self.table[b][old // PAGE]
                if not self._page(last):
                    self.status.add("bad")
                    continue
                split = held[last] > 1
            need += split
            asked += need
            if need and asked > room:
                self.status.add("pages")
                continue
            at = asked - need
            if split:
                self.moves.append((last, free[at]))
                self.table[b][old // PAGE] = free[at]
                self.refs[free[at]] = 1
                self.refs[last] -= 1
                at += 1
            for j in range(pages_of(old), pages_of(n)):
                self.table[b][j] = free[at]
                self.refs[free[at]] = 1
                at += 1
            self.len[b] = n

    def fork(self, src, dst):
        self.moves, self.status = [], set()
        before, free = list(self.len), self._free()
        room, asked, taken = len(free), 0, set()
        B, most = len(self.len), len(self.table[0]) * PAGE
        for a, b in zip(src, dst):
            if not (0 <= a < B and 0 <= b < B) or a == b:
                self.status.add("bad")
                continue
            n = before[a]
            if not 0 <= n <= most or before[b] != 0 or \
                    (n % PAGE and not self._page(self.table[a][n // PAGE])):
                self.status.add("bad")
                continue
            if b in taken:
                self.status.add("bad")
                continue
            taken.add(b)
            if n % PAGE:
                asked += 1
                if asked > room:
                    self.status.add("pages")
                    continue
                p = free[asked - 1]
                self.moves.append((self.table[a][n // PAGE], p))
                self.table[b][n // PAGE] = p
                self.refs[p] = 1
            for j in range(n // PAGE):
                p = self.table[b][j] = self.table[a][j]
                if self._page(p):
                    self.refs[p] += 1
                else:
                    self.status.add("bad")
            self.len[b] = n

    def compact(self):
        self.moves, self.status = [], set()
        live = [p for p, c in enumerate(self.refs) if c > 0]
        L = len(live)
        holes = iter([p for p in range(L) if self.refs[p] <= 0])
        to = [p if c > 0 else -1 for p, c in enumerate(self.refs)]
        for p in live:
            if p >= L:
                to[p] = next(holes)
                self.moves.append((p, to[p]))
                self.refs[to[p]], self.refs[p] = self.refs[p], 0
        for b, n in enumerate(self.len):
            if not 0 <= n <= len(self.table[b]) * PAGE:
                self.status.add("bad")
                continue
            for j in range(pages_of(n)):
                p = self.table[b][j]
                if self._page(p) and to[p] >= 0:
                    self.table[b][j] = to[p]
                else:
                    self.status.add("bad")
        return to, L
