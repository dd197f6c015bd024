"""What the rotary-position and paged-cache operators are timed on.

Every case is one call that a program around the attention kernels makes:

  rope, rope_bwd   queries and keys of a training step rotated by their positions,
                   and the gradients rotated back;
  append           new tokens of a serving step: queries and keys rotated, keys and
                   values written to their slots of the paged cache;
  fork             rows of the page table that start as copies of other rows (several
                   samples of one prompt): whole pages shared, the last one copied;
  resize           pages given back by rows that finished or were cut, and handed to
                   rows that grow, with a copy of a shared last page before it is written;
  compact          the live pages moved to the front of the pool.

`own` chooses between the plain form (elementary torch operations) and the library.
Both take the same state and leave the same buffers behind.
"""
import math

import torch

own = False

PAGE = 16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest attention call: one head, 128 rows; the launch is all of it
        dict(name="rope-tiny", op="rope", B=1, S=128, Hq=1, Hkv=1, d=64, rot=64,
             interleaved=False, fused=False, far=0, factor=1.0),
        # a GQA training step: q and k are slices of one projection's output
        dict(name="rope-gqa-4096", op="rope", B=2, S=4096, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, fused=True, far=0, factor=1.0),
        # gradients of wide heads that rotate a quarter of their width, odd length
        dict(name="rope-bwd-part-2047", op="rope_bwd", B=4, S=2047, Hq=16, Hkv=16, d=256, rot=64,
             interleaved=True, fused=False, far=0, factor=1.0),
        # gradients of one long sequence whose positions are stretched 8 times
        dict(name="rope-bwd-long-8192", op="rope_bwd", B=1, S=8192, Hq=16, Hkv=16, d=128, rot=128,
             interleaved=False, fused=False, far=120000, factor=8.0),
        # one new token for each of 64 requests
        dict(name="append-decode-64", op="append", B=64, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, lo=1024, hi=8192, new=1, factor=1.0),
        # chunked prefill: 512 new tokens for each of 8 requests
        dict(name="append-chunk-8x512", op="append", B=8, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, lo=2048, hi=8192, new=512, factor=1.0),
        # four samples of one prompt
        dict(name="fork-1-to-4", op="fork", B=16, n=4, parents=1, Hkv=8, d=128, layers=1,
             lo=200, hi=1000),
        # 64 running requests, each continued twice, all layers of the cache
        dict(name="fork-64-layers-4", op="fork", B=128, n=64, parents=64, Hkv=8, d=128, layers=4,
             lo=256, hi=2048),
        # a decode step: every row grows by one token
        dict(name="resize-step-64", op="resize", B=64, Hkv=8, d=128, layers=1, lo=1024, hi=8192,
             shared=0.0, leave=0.0, join=0.0, copies=False),
        # a busy step: rows leave, rows join, shared pages are copied before they are written
        dict(name="resize-mixed-256", op="resize", B=256, Hkv=8, d=128, layers=4, lo=64, hi=512,
             shared=0.4, leave=0.2, join=0.2, copies=True),
        # a small pool, half of it free
        dict(name="compact-512", op="compact", P=512, B=8, Hkv=8, d=64, layers=1, live=0.5),
        # a pool of a quarter million tokens, 60 % of it live
        dict(name="compact-16384", op="compact", P=16384, B=128, Hkv=8, d=128, layers=1,
             live=0.6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "fork", "resize", "compact"])
    d = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    if op in ("rope", "rope_bwd"):
        Hq = Hkv * rng.choice([1, 2, 4])
        B = _log(rng, 1, 4)
        S = _log(rng, 1, min(8192, (32 << 20) // (B * (Hq + Hkv) * d)))
        return dict(op=op, B=B, S=S, Hq=Hq, Hkv=Hkv, d=d, rot=rng.choice([d, d // 2, d // 4, 16]),
                    interleaved=rng.random() < 0.5, fused=rng.random() < 0.5,
                    far=rng.choice([0, 5000, 1000000]), factor=rng.choice([1.0, 4.0, 32.0]))
    if op == "append":
        new = rng.choice([1, 1, _log(rng, 2, 512)])
        B = _log(rng, 1, 64 if new < 33 else 8)
        lo = _log(rng, 1, 2048)
        return dict(op=op, B=B, Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv, d=d,
                    rot=rng.choice([d, d // 2, 32]), interleaved=rng.random() < 0.5, lo=lo,
                    hi=lo + _log(rng, 1, 2048), new=new, factor=rng.choice([1.0, 4.0]))
    if op == "fork":
        parents = _log(rng, 1, 64)
        n = parents if rng.random() < 0.5 else _log(rng, 1, 64)
        lo = _log(rng, 16, 512)
        return dict(op=op, B=parents + n, n=n, parents=parents, Hkv=Hkv, d=d,
                    layers=rng.choice([1, 2, 4]), lo=lo, hi=lo + _log(rng, 1, 1024))
    if op == "resize":
        lo = _log(rng, 1, 128)
        return dict(op=op, B=_log(rng, 1, 256), Hkv=Hkv, d=rng.choice([64, 128]),
                    layers=rng.choice([1, 2, 4]), lo=lo, hi=lo + _log(rng, 1, 384),
                    shared=rng.choice([0.0, 0.3]), leave=round(rng.uniform(0, 0.5), 2),
                    join=round(rng.uniform(0, 0.5), 2), copies=True)
    P, live = _log(rng, 16, 8192), round(rng.uniform(0.1, 0.95), 2)
    return dict(op=op, P=P, B=_log(rng, 1, max(1, min(64, int(P * live)))), Hkv=Hkv,
                d=rng.choice([64, 128]), layers=rng.choice([1, 2]), live=live)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).bfloat16()


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _frequencies(rot, factor):
    """Radians per position of each rotated pair, float64.  factor > 1: waves longer
    than the trained length (4096) are stretched, shorter than 1/32 of it kept,
    blended in between; with it comes the amplitude."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor == 1.0:
        return f.cuda(), 1.0
    keep = ((4096.0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
    return (f * (keep + (1 - keep) / factor)).cuda(), 0.1 * math.log(factor) + 1.0


def _table(g, counts, P, width):
    """A page table [B, width] whose rows hold `counts` pages, drawn from a shuffled pool of P."""
    B = counts.numel()
    perm = torch.randperm(P, generator=g, device="cuda").int()
    start = counts.cumsum(0) - counts
    cols = torch.arange(width, device="cuda")
    at = (start[:, None] + cols).clamp_max(P - 1)
    return torch.where(cols < counts[:, None], perm[at], torch.full((), -1, dtype=torch.int32,
                                                                    device="cuda"))


def _book(pt, ln, refs):
    """Page table, lengths and reference counts in one buffer, as a scheduler keeps them."""
    return torch.cat([pt.reshape(-1), ln, refs]).int(), pt.shape[0], pt.shape[1]


def _pools(g, layers, P, Hkv, d):
    out = []
    for _ in range(2):
        x = torch.empty(layers, P, PAGE, Hkv, d, device="cuda", dtype=torch.bfloat16)
        x.normal_(generator=g)
        out.append(x)
    return out


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("rope", "rope_bwd"):
        B, S, Hq, Hkv, d = (case[n] for n in ("B", "S", "Hq", "Hkv", "d"))
        if case["fused"]:
            x = _randn(g, B, S, Hq + 2 * Hkv, d)
            q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
        else:
            q, k = _randn(g, B, S, Hq, d), _randn(g, B, S, Hkv, d)
        inv, amp = _frequencies(case["rot"], case["factor"])
        pos = torch.arange(S, device="cuda", dtype=torch.int32) + _ints(g, 0, case["far"], B, 1)
        return dict(case=case, q=q, k=k, inv=inv, amp=amp, pos=pos)
    if op == "append":
        B, Hq, Hkv, d, new = (case[n] for n in ("B", "Hq", "Hkv", "d", "new"))
        ln = _ints(g, case["lo"], case["hi"], B)
        if new == 1:
            T, cu = B, None
        else:  # ragged chunks: every fourth is the shorter end of a prompt
            sizes = [new - (7 * b % new if b % 4 == 3 else 0) for b in range(B)]
            cnt = torch.tensor(sizes, dtype=torch.int32, device="cuda")
            ln = torch.maximum(ln, cnt)
            cu = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"),
                            cnt.cumsum(0).int()])
            T = sum(sizes)
        counts = (ln + PAGE - 1) // PAGE
        width = (max(case["hi"], new) + PAGE - 1) // PAGE
        P = B * width + 8
        kp, vp = _pools(g, 1, P, Hkv, d)
        x = _randn(g, T, Hq + 2 * Hkv, d)
        inv, amp = _frequencies(case["rot"], case["factor"])
        return dict(case=case, q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], inv=inv,
                    amp=amp, cu=cu, ln=ln, kp=kp[0], vp=vp[0],
                    pt=_table(g, counts, P, width))
    layers, Hkv, d, B = case["layers"], case["Hkv"], case["d"], case["B"]
    if op == "fork":
        n, parents = case["n"], case["parents"]
        order = torch.randperm(B, generator=g, device="cuda").int()
        src = order[torch.arange(n, device="cuda") % parents]
        dst = order[parents:parents + n].contiguous()
        ln = torch.zeros(B, dtype=torch.int32, device="cuda")
        ln[order[:parents].long()] = _ints(g, case["lo"], case["hi"], parents)
        counts = (ln + PAGE - 1) // PAGE
        width = (case["hi"] + PAGE - 1) // PAGE + 4
        P = parents * width + 2 * n
    elif op == "resize":
        ln = _ints(g, case["lo"], case["hi"], B)
        u = torch.rand(B, generator=g, device="cuda")
        ln = torch.where(u < case["join"], 0, ln).int()
        # a row that shares every page of the one before it
        twin = (torch.rand(B, generator=g, device="cuda") < case["shared"]) & \
               (torch.arange(B, device="cuda") % 2 == 1)
        ln = torch.where(twin, ln.roll(1), ln)
        grown = torch.where(ln == 0, _ints(g, case["lo"], case["hi"], B), ln + 1)
        gone = (torch.rand(B, generator=g, device="cuda") < case["leave"]) & (ln > 0)
        new = torch.where(gone, torch.where(_ints(g, 0, 3, B) == 0, ln // 2, 0), grown).int()
        counts = torch.where(twin, 0, (ln + PAGE - 1) // PAGE)
        width = (case["hi"] + PAGE) // PAGE + 2
        P = 2 * B * width
    else:  # compact
        P = case["P"]
        mean = max(1, int(P * case["live"]) // B)
        swing = _ints(g, 0, mean, (B + 1) // 2)  # what one row of a pair has more, the other less
        counts = mean + torch.stack([swing, -swing], 1).reshape(-1)[:B]
        if B % 2:
            counts[-1] = mean
        ln = (counts * PAGE - _ints(g, 0, PAGE - 1, B)).clamp_min(0)
        width = 2 * mean + 2
    pt = _table(g, counts, P, width)
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[pt[pt >= 0].long()] = 1
    if op == "resize":
        pt = torch.where(twin[:, None], pt.roll(1, 0), pt)
        refs.index_add_(0, pt.clamp_min(0).reshape(-1).long(),
                        ((pt >= 0) & twin[:, None]).int().reshape(-1))
    kp, vp = _pools(g, layers, P, Hkv, d)
    book, rows, width = _book(pt, ln, refs)
    s = dict(case=case, book=book, rows=rows, width=width, kp=kp, vp=vp)
    if op == "fork":
        s.update(src=src, dst=dst)
    if op == "resize":
        s.update(new=new)
    return s


# ------------------------------------------------------------------ one pass

def _rotate(x, pos, inv, amp, interleaved, sign=1.0):
    """x [..., H, d] by pos [...]; angles in 64 bits, products in 32."""
    r = 2 * inv.numel()
    ang = pos.double()[..., None, None] * inv
    c, s = (ang.cos() * amp).float(), (ang.sin() * (sign * amp)).float()
    y = x.float()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    u, w = a * c - b * s, a * s + b * c
    rot = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([rot, y[..., r:]], -1).bfloat16()


def _plain_append(s):
    ln, pt = s["ln"].long(), s["pt"]
    T = s["q"].shape[0]
    rows = torch.arange(T, device=pt.device)
    if s["cu"] is None:
        seq, pos = rows, ln - 1
    else:
        cu = s["cu"].long()
        seq = torch.searchsorted(cu[1:], rows, right=True)
        pos = ln[seq] - (cu[seq + 1] - rows)
    inter = s["case"]["interleaved"]
    page, slot = pt[seq, pos // PAGE].long(), pos % PAGE
    s["kp"][page, slot] = _rotate(s["k"], pos, s["inv"], s["amp"], inter)
    s["vp"][page, slot] = s["v"]
    return _rotate(s["q"], pos, s["inv"], s["amp"], inter)


def _lowest_free(refs):
    return torch.argsort((refs > 0).to(torch.int8), stable=True)


def _plain_fork(s, pt, ln, refs):
    src, dst = s["src"].long(), s["dst"].long()
    size = ln[src]
    full, part = size // PAGE, size % PAGE != 0
    cols = torch.arange(pt.shape[1], device=pt.device)
    fresh = _lowest_free(refs)[(part.cumsum(0) - 1).clamp_min(0)]
    parent = pt[src]
    keep = cols < full[:, None]
    child = torch.where(keep, parent, pt[dst])
    child = torch.where(part[:, None] & (cols == full[:, None]), fresh[:, None].int(), child)
    refs.index_add_(0, torch.where(keep, parent, 0).reshape(-1).long(), keep.int().reshape(-1))
    refs.index_add_(0, fresh, part.int())
    pt[dst] = child
    ln[dst] = size
    # a row that ends on a page boundary copies nothing: its first page onto itself
    old = parent.gather(1, full.clamp_max(pt.shape[1] - 1)[:, None].long())[:, 0].long()
    a = torch.where(part, old, parent[:, 0].long())
    b = torch.where(part, fresh, parent[:, 0].long())
    for pool in (s["kp"], s["vp"]):
        pool[:, b] = pool[:, a]


def _plain_resize(s, pt, ln, refs):
    new = s["new"]
    cols = torch.arange(pt.shape[1], device=pt.device)
    had, want = (ln + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    drop = (cols >= want[:, None]) & (cols < had[:, None])
    refs.index_add_(0, torch.where(drop, pt, 0).reshape(-1).long(), -drop.int().reshape(-1))
    last = (ln // PAGE).clamp_max(pt.shape[1] - 1)[:, None].long()
    old = pt.gather(1, last)[:, 0]
    grows = (new > ln) & (ln % PAGE != 0)
    split = grows & (refs[torch.where(grows, old, 0).long()] > 1)
    need = (want - had).clamp_min(0) + split.int()
    begin = need.cumsum(0) - need
    ok = (need == 0) | (begin + need <= (refs <= 0).sum())
    split = split & ok
    free = _lowest_free(refs).int()
    at = begin[:, None] + split.int()[:, None] + (cols - had[:, None])
    add = ok[:, None] & (cols >= had[:, None]) & (cols < want[:, None])
    table = torch.where(add, free[at.clamp(0, refs.numel() - 1)], pt)
    mine = free[begin.clamp_max(refs.numel() - 1)]
    table = torch.where(split[:, None] & (cols == last), mine[:, None], table)
    refs.index_add_(0, torch.where(add, table, 0).reshape(-1).long(), add.int().reshape(-1))
    refs.index_add_(0, torch.where(split, mine, 0).long(), split.int())
    refs.index_add_(0, torch.where(split, old, 0).long(), -split.int())
    pt.copy_(table)
    ln.copy_(torch.where(ok, new, ln))
    if s["case"]["copies"]:
        i = split.nonzero()[:, 0]
        a, b = old[i].long(), mine[i].long()
        for pool in (s["kp"], s["vp"]):
            pool[:, b] = pool[:, a]


def _plain_compact(s, pt, ln, refs):
    P = refs.numel()
    idx = torch.arange(P, device=refs.device)
    live = refs > 0
    count = live.sum(dtype=torch.int32).reshape(1)
    movers = (live & (idx >= count)).nonzero()[:, 0]
    holes = (~live & (idx < count)).nonzero()[:, 0]
    to = torch.where(live, idx, -1).int()
    to[movers] = holes.int()
    cols = torch.arange(pt.shape[1], device=pt.device)
    used = cols < ((ln + PAGE - 1) // PAGE)[:, None]
    pt.copy_(torch.where(used, to[torch.where(used, pt, 0).long()], pt))
    refs[holes] = refs[movers]
    refs[movers] = 0
    for pool in (s["kp"], s["vp"]):
        pool[:, holes] = pool[:, movers]
    return to, count


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import exact_attention_08_gb300 as ea
    if op in ("rope", "rope_bwd"):
        inter = s["case"]["interleaved"]
        if own:
            f = ea.attn_rope if op == "rope" else ea.attn_rope_bwd
            return f(s["q"], s["k"], s["inv"], s["pos"], interleaved=inter, amplitude=s["amp"])
        sign = 1.0 if op == "rope" else -1.0
        return tuple(_rotate(x, s["pos"], s["inv"], s["amp"], inter, sign)
                     for x in (s["q"], s["k"]))
    if op == "append":
        if own:
            q = ea.attn_append_paged(s["q"], s["k"], s["v"], s["kp"], s["vp"], s["pt"], s["ln"],
                                     s["cu"], s["inv"], interleaved=s["case"]["interleaved"],
                                     amplitude=s["amp"])
        else:
            q = _plain_append(s)
        return dict(q=q, k_pages=s["kp"], v_pages=s["vp"])
    # the scheduler's tables as they stood before the step
    book, n = s["book"].clone(), s["rows"] * s["width"]
    pt = book[:n].view(s["rows"], s["width"])
    ln, refs = book[n:n + s["rows"]], book[n + s["rows"]:]
    more = {}
    if op == "fork":
        if own:
            ea.attn_pages_fork(pt, ln, refs, s["src"], s["dst"], s["kp"], s["vp"])
        else:
            _plain_fork(s, pt, ln, refs)
    elif op == "resize":
        if own:
            pools = (s["kp"], s["vp"]) if s["case"]["copies"] else ()
            ea.attn_pages_resize(pt, ln, s["new"], refs, *pools)
        else:
            _plain_resize(s, pt, ln, refs)
    else:
        if own:
            to, count = ea.attn_pages_compact(pt, ln, refs, s["kp"], s["vp"])
        else:
            to, count = _plain_compact(s, pt, ln, refs)
        more = dict(new_index=to, num_live=count)
    return dict(page_table=pt, seqlens=ln, refs=refs, k_pages=s["kp"], v_pages=s["vp"], **more)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("rope", "rope_bwd"):
        rows = case["B"] * case["S"]
        heads = case["Hq"] + case["Hkv"]
        return dict(bytes=rows * (heads * case["d"] * 4 + 4), flops=rows * heads * case["rot"] * 3)
    if op == "append":
        rows = case["B"] * min(case["new"], case["hi"])
        heads = case["Hq"] + 2 * case["Hkv"]
        return dict(bytes=rows * (heads * case["d"] * 4 + 4) + case["B"] * 8,
                    flops=rows * (case["Hq"] + case["Hkv"]) * case["rot"] * 3)
    page = 2 * case["layers"] * PAGE * case["Hkv"] * case["d"] * 2 * 2  # K and V, read and written
    if op == "fork":
        shared = case["n"] * (case["lo"] + case["hi"]) // (2 * PAGE)
        return dict(bytes=case["n"] * (page + 24) + shared * 16, flops=0)
    if op == "resize":
        B, mean = case["B"], (case["lo"] + case["hi"]) / (2 * PAGE)
        moved = B * (case["leave"] + case["join"]) * mean + B / PAGE
        twins = B * case["shared"] / 2 * (1 - case["leave"]) if case["copies"] else 0
        return dict(bytes=B * 12 + moved * 12 + twins * page, flops=0)
    live = int(case["P"] * case["live"])
    moved = live * (1 - case["live"])
    return dict(bytes=case["P"] * 12 + live * 8 + moved * page, flops=0)


# ------------------------------------------------------------------ from the definition, in 64 bits

def _exact_rotation(x, pos, inv, amp, interleaved, sign):
    r = 2 * inv.numel()
    y = x.double().clone()
    turn = torch.polar(torch.full_like(inv, amp).expand(*pos.shape, -1),
                       sign * pos.double().unsqueeze(-1) * inv).unsqueeze(-2)
    re, im = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2),
                                                                   slice(r // 2, r))
    z = torch.complex(y[..., re], y[..., im]) * turn
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_pages(case, s):
    """The tables by walking over them on the host, and the pages' moves as (from, to)."""
    n, B, W = s["rows"] * s["width"], s["rows"], s["width"]
    book = s["book"].tolist()
    pt = [book[b * W:(b + 1) * W] for b in range(B)]
    ln, refs = book[n:n + B], book[n + B:]
    moves, more = [], {}
    if case["op"] == "fork":
        before = list(refs)
        free = iter([p for p, c in enumerate(before) if c <= 0])
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            whole, rest = divmod(ln[a], PAGE)
            for j in range(whole):
                pt[b][j] = pt[a][j]
                refs[pt[a][j]] += 1
            if rest:
                p = next(free)
                moves.append((pt[a][whole], p))
                pt[b][whole] = p
                refs[p] = 1
            ln[b] = ln[a]
    elif case["op"] == "resize":
        new = s["new"].tolist()
        up = lambda x: (x + PAGE - 1) // PAGE  # noqa: E731
        for b in range(B):
            for j in range(up(new[b]), up(ln[b])):
                refs[pt[b][j]] -= 1
        free = iter([p for p, c in enumerate(refs) if c <= 0])
        room, asked, then = sum(c <= 0 for c in refs), 0, list(refs)
        for b in range(B):
            old = pt[b][ln[b] // PAGE] if new[b] > ln[b] and ln[b] % PAGE else None
            split = old is not None and then[old] > 1
            need = max(0, up(new[b]) - up(ln[b])) + int(split)
            asked += need
            if need and asked > room:
                continue
            if split:
                p = next(free)
                moves.append((old, p))
                pt[b][ln[b] // PAGE] = p
                refs[p] += 1
                refs[old] -= 1
            for j in range(up(ln[b]), up(new[b])):
                pt[b][j] = next(free)
                refs[pt[b][j]] += 1
            ln[b] = new[b]
        moves = moves if case["copies"] else []
    else:
        live = [p for p, c in enumerate(refs) if c > 0]
        gaps = iter([p for p in range(len(live)) if refs[p] <= 0])
        to = [p if c > 0 else -1 for p, c in enumerate(refs)]
        for p in live:
            if p >= len(live):
                to[p] = next(gaps)
                moves.append((p, to[p]))
                refs[to[p]], refs[p] = refs[p], 0
        for b in range(B):
            for j in range((ln[b] + PAGE - 1) // PAGE):
                pt[b][j] = to[pt[b][j]]
        more = dict(new_index=torch.tensor(to, dtype=torch.int32),
                    num_live=torch.tensor([len(live)], dtype=torch.int32))
    out = dict(page_table=torch.tensor(pt, dtype=torch.int32),
               seqlens=torch.tensor(ln, dtype=torch.int32),
               refs=torch.tensor(refs, dtype=torch.int32), **more)
    for name, pool in (("k_pages", s["kp"]), ("v_pages", s["vp"])):
        x = pool.double()
        if moves:
            a, b = (torch.tensor(v, device=x.device) for v in zip(*moves))
            for layer in range(x.shape[0]):
                x[layer].index_copy_(0, b, pool[layer].index_select(0, a).double())
        out[name] = x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rope", "rope_bwd"):
        sign = 1.0 if op == "rope" else -1.0
        return tuple(_exact_rotation(x, s["pos"], s["inv"], s["amp"], case["interleaved"], sign)
                     for x in (s["q"], s["k"]))
    if op != "append":
        return _exact_pages(case, s)
    ln, pt = s["ln"].tolist(), s["pt"].tolist()
    cu = list(range(case["B"] + 1)) if s["cu"] is None else s["cu"].tolist()
    where, pos = [], []
    for b in range(case["B"]):
        for i in range(cu[b + 1] - cu[b]):
            p = ln[b] - (cu[b + 1] - cu[b]) + i
            pos.append(p)
            where.append(pt[b][p // PAGE] * PAGE + p % PAGE)
    where = torch.tensor(where, device="cuda")
    pos = torch.tensor(pos, device="cuda")
    q, k = (_exact_rotation(x, pos, s["inv"], s["amp"], case["interleaved"], 1.0)
            for x in (s["q"], s["k"]))
    out = dict(q=q)
    for name, pool, x in (("k_pages", s["kp"], k), ("v_pages", s["vp"], s["v"].double())):
        y = pool.double()
        y.view(-1, *y.shape[2:]).index_copy_(0, where, x)
        out[name] = y
    return out
