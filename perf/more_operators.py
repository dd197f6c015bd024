"""What the operators on shared and thinned caches are timed on.

Every case is one call that a serving program makes of a paged cache:

  shared   a decode step of rows that share the pages of a prompt: the prompt's
           keys are attended once for all of them;
  decode   a decode step that also adds each key's attention weight to its mass;
  prompt   the mass that the keys get from a block of prompt queries, after their
           attention;
  evict    rows cut to their budget: the keys of the largest mass stay, and those
           behind the budget move into the slots of the evicted ones.

`own` chooses between the plain form (elementary torch operations) and the library.
Both take the same state.
"""
import math

import numpy
import torch

own = False

PAGE = 16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # two samples of a short prompt, one key head: the launches are all of it
        dict(name="shared-tiny", op="shared", groups=1, per=2, spread=0, Hq=4, Hkv=1, d=64,
             plo=131, phi=131, slo=1, shi=20, sink=False),
        # 64 samples of one long prompt, GQA
        dict(name="shared-64-of-8192", op="shared", groups=1, per=64, spread=0, Hq=32, Hkv=8,
             d=128, plo=8192, phi=8192, slo=1, shi=512, sink=False),
        # a mixed batch: 16 prompts with 1 to 7 samples each, a logit sink per head
        dict(name="shared-16-prompts", op="shared", groups=16, per=4, spread=3, Hq=32, Hkv=8,
             d=128, plo=1024, phi=4096, slo=16, shi=700, sink=True),
        # a system prompt of 64 thousand tokens under 48 chats, wide heads
        dict(name="shared-48-of-65519", op="shared", groups=1, per=48, spread=0, Hq=16, Hkv=4,
             d=256, plo=65519, phi=65519, slo=33, shi=2000, sink=False),
        # one request, one key head
        dict(name="decode-tiny", op="decode", B=1, Hq=4, Hkv=1, d=64, lo=100, hi=100),
        # 64 requests, GQA
        dict(name="decode-64", op="decode", B=64, Hq=32, Hkv=8, d=128, lo=1024, hi=8192),
        # every query head with its own keys, few long requests of odd lengths
        dict(name="decode-mha-7", op="decode", B=7, Hq=16, Hkv=16, d=64, lo=4001, hi=16001),
        # one whole prompt, causal
        dict(name="prompt-8192", op="prompt", B=1, Hq=32, Hkv=8, d=128, lo=8192, hi=8192,
             qlo=8192, qhi=8192, causal=True, window=0),
        # ragged chunks of 8 prompts in a sliding window, wide heads
        dict(name="prompt-chunks-8", op="prompt", B=8, Hq=8, Hkv=2, d=256, lo=1000, hi=5000,
             qlo=100, qhi=512, causal=True, window=1024),
        # the last 32 queries of 8 long prompts judge all their keys
        dict(name="prompt-observe-32", op="prompt", B=8, Hq=32, Hkv=8, d=128, lo=8000, hi=32000,
             qlo=32, qhi=32, causal=True, window=0),
        # rows that have grown 64 tokens past their budget
        dict(name="evict-step-64", op="evict", layers=1, B=64, Hkv=8, d=128, klo=1024, khi=1024,
             over=64, sink=4, recent=128),
        # prompts cut to an eighth, all layers of the cache
        dict(name="evict-prompt-8192", op="evict", layers=8, B=8, Hkv=8, d=128, klo=900, khi=1100,
             over=7168, sink=4, recent=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "decode", "prompt", "evict"])
    d = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8] if Hkv <= 4 else [1, 2, 3, 4])
    if op == "shared":
        groups = _log(rng, 1, 16)
        per = _log(rng, 1, 64 // groups)
        plo = _log(rng, 17, 8192 // groups)
        slo = _log(rng, 1, 64)
        return dict(op=op, groups=groups, per=per, spread=rng.randint(0, per - 1), Hq=Hq, Hkv=Hkv,
                    d=d, plo=plo, phi=plo + _log(rng, 1, 1 + 16384 // groups), slo=slo,
                    shi=slo + _log(rng, 1, 1024), sink=rng.random() < 0.3)
    if op == "decode":
        B = _log(rng, 1, min(64, 65536 // (Hkv * d)))
        lo = _log(rng, 1, 4096)
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, lo=lo, hi=lo + _log(rng, 1, 4096))
    if op == "prompt":
        B = _log(rng, 1, 8)
        lo = _log(rng, 1, 8192 // B)
        hi = lo + _log(rng, 1, max(1, 8192 // B))
        most = max(1, min(lo, (1 << 37) // (B * Hq * d * hi)))
        q = _log(rng, 1, most)
        causal = rng.random() < 0.8
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, lo=lo, hi=hi, qlo=q,
                    qhi=min(most, q + _log(rng, 1, 512)), causal=causal,
                    window=_log(rng, 1, 2048) if causal and rng.random() < 0.3 else 0)
    layers = rng.choice([1, 1, 2, 4])
    B = _log(rng, 1, min(64, 65536 // (Hkv * d)) // layers)
    klo = _log(rng, 16, 1024)
    return dict(op=op, layers=layers, B=B, Hkv=Hkv, d=d, klo=klo, khi=klo + _log(rng, 1, 256),
                over=_log(rng, 1, 4096), sink=rng.choice([0, 4]),
                recent=rng.choice([0, min(klo // 2, 64)]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).bfloat16()


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pools(g, *shape):
    out = []
    for _ in range(2):
        x = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
        x.normal_(generator=g)
        out.append(x)
    return out


def _table(g, counts, P, width):
    """A page table [B, width] whose rows hold `counts` pages, drawn from a shuffled pool of P."""
    perm = torch.randperm(P, generator=g, device="cuda").int()
    start = counts.cumsum(0) - counts
    cols = torch.arange(width, device="cuda")
    at = (start[:, None] + cols).clamp_max(P - 1)
    return torch.where(cols < counts[:, None], perm[at], -1).int().contiguous()


def _group_sizes(case):
    """Samples of each prompt: `per`, more and fewer by turns."""
    s = case["spread"]
    return [case["per"] + (s if g % 2 else -s) * (1 + g % 3) // 3 for g in range(case["groups"])]


def _prepare_shared(case, g):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    sizes = _group_sizes(case)
    n, R = len(sizes), sum(sizes)
    cu = _i32([sum(sizes[:i]) for i in range(n + 1)])
    gid = torch.repeat_interleave(torch.arange(n, device="cuda"), _i32(sizes).long(),
                                  output_size=R)
    rows = torch.randperm(R, generator=g, device="cuda").int()  # rows of the table, group by group
    prompt = _ints(g, case["plo"], case["phi"], n)
    own_len = _ints(g, case["slo"], case["shi"], R)             # tokens a row has of its own
    whole = prompt // PAGE                                      # pages that a fork shares
    length = prompt[gid] + own_len                              # in the order of `rows`
    width = (case["phi"] + case["shi"] + PAGE - 1) // PAGE
    mine = (length + PAGE - 1) // PAGE - whole[gid]
    P = int(n * (case["phi"] // PAGE) + R * ((case["shi"] + 2 * PAGE) // PAGE)) + 8
    both = _table(g, torch.cat([whole, mine.int()]), P, width)
    cols = torch.arange(width, device="cuda")
    at = cols - whole[gid][:, None]
    table = torch.where(at < 0, both[:n][gid], both[n:].gather(1, at.clamp_min(0)))
    pt, ln = torch.empty_like(table), torch.empty_like(length)
    pt[rows.long()], ln[rows.long()] = table, length
    kp, vp = _pools(g, P, PAGE, Hkv, d)
    sink = torch.rand(Hq, generator=g, device="cuda") * 8 if case["sink"] else None
    return dict(case=case, q=_randn(g, R, Hq, d), kp=kp, vp=vp, pt=pt.int().contiguous(),
                ln=ln.int(), cu=cu, prompt=prompt, rows=rows, sink=sink,
                most=max(sizes), prefix_pages=case["phi"] // PAGE,
                own_pages=(case["shi"] + 2 * PAGE - 1) // PAGE)


def _prepare_decode(case, g):
    B, Hq, Hkv, d = (case[n] for n in ("B", "Hq", "Hkv", "d"))
    ln = _ints(g, case["lo"], case["hi"], B)
    counts = (ln + PAGE - 1) // PAGE
    width = (case["hi"] + PAGE - 1) // PAGE
    P = B * width + 8
    kp, vp = _pools(g, P, PAGE, Hkv, d)
    mass = torch.rand(B, Hkv, width * PAGE, generator=g, device="cuda")
    # the newest token of a row whose cache was thinned before
    last = ln - 1 + _ints(g, 0, 5000, B)
    return dict(case=case, q=_randn(g, B, Hq, d), kp=kp, vp=vp, pt=_table(g, counts, P, width),
                ln=ln, mass=mass, out=mass.clone(), last=last,
                positions=torch.zeros(B, Hkv, width * PAGE, dtype=torch.int32, device="cuda"))


def _seen(case, i, t, Lq, Lk):
    """May query i of Lq see key t of Lk?  Queries end where the keys end."""
    ok = (t < Lk) & (i < Lq)
    if case["causal"]:
        at = i + (Lk - Lq)
        ok = ok & (t <= at)
        if case["window"] > 0:
            ok = ok & (t > at - case["window"])
    return ok


def _prepare_prompt(case, g):
    B, Hq, Hkv, d = (case[n] for n in ("B", "Hq", "Hkv", "d"))
    ln = _ints(g, case["lo"], case["hi"], B)
    nq = _ints(g, case["qlo"], case["qhi"], B)
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), nq.cumsum(0).int()])
    T = int(cu[-1])
    counts = (ln + PAGE - 1) // PAGE
    width = (case["hi"] + PAGE - 1) // PAGE
    P = B * width + 8
    kp = _pools(g, P, PAGE, Hkv, d)[0]
    q = _randn(g, T, Hq, d)
    pt = _table(g, counts, P, width)
    lse = torch.empty(Hq, T, device="cuda")  # what the attention of these queries returned
    for b in range(B):
        a, e, L = int(cu[b]), int(cu[b + 1]), int(ln[b])
        keys = kp[pt[b, :(L + PAGE - 1) // PAGE].long()].flatten(0, 1)[:L].float()
        ok = _seen(case, torch.arange(e - a, device="cuda")[:, None],
                   torch.arange(L, device="cuda"), e - a, L)
        for h in range(Hq):
            s = (q[a:e, h].float() @ keys[:, h // (Hq // Hkv)].T) * d ** -0.5
            lse[h, a:e] = s.masked_fill_(~ok, -math.inf).logsumexp(1)
    mass = torch.rand(B, Hkv, width * PAGE, generator=g, device="cuda")
    return dict(case=case, q=q, lse=lse, kp=kp, pt=pt, cu=cu, ln=ln, mass=mass, out=mass.clone(),
                positions=torch.zeros(B, Hkv, width * PAGE, dtype=torch.int32, device="cuda"))


def _prepare_evict(case, g):
    layers, B, Hkv, d = (case[n] for n in ("layers", "B", "Hkv", "d"))
    keep = _ints(g, case["klo"], case["khi"], B)
    ln = keep + case["over"]
    counts = (ln + PAGE - 1) // PAGE
    width = (case["khi"] + case["over"] + PAGE - 1) // PAGE
    P = B * width + 8
    kp, vp = _pools(g, layers, P, PAGE, Hkv, d)
    pt = _table(g, counts, P, width)
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[pt[pt >= 0].long()] = 1
    shape = (layers, B, Hkv, width * PAGE)
    # masses of a softmax are spread over many orders; keys that a window hid have none
    mass = (1.5 * torch.randn(shape, generator=g, device="cuda")).exp()
    mass = mass * (torch.rand(shape, generator=g, device="cuda") > 0.1)
    # slots before the budget were filled by an earlier cut, in no order; the rest follow
    slot = torch.arange(width * PAGE, device="cuda")
    mixed = torch.rand(shape, generator=g, device="cuda").masked_fill_(
        slot >= keep[:, None, None], 2.0).argsort(-1)
    positions = torch.where(slot < keep[:, None, None], mixed * 2, slot + keep[:, None, None])
    return dict(case=case, kp=kp, vp=vp, pt=pt, ln=ln, keep=keep, refs=refs, mass=mass,
                positions=positions.int())


def prepare(case, seed):
    make = dict(shared=_prepare_shared, decode=_prepare_decode, prompt=_prepare_prompt,
                evict=_prepare_evict)[case["op"]]
    return make(case, _gen(seed))


# ------------------------------------------------------------------ one pass

def _gather(pool, table):
    """[n, slots, Hkv, d] in fp32: the pages of a table, one behind the other."""
    return pool[table.clamp_min(0).long()].flatten(1, 2).float()


def _plain_shared(s):
    q, pt, ln = s["q"].float(), s["pt"], s["ln"]
    R, Hq, d = q.shape
    Hkv = s["kp"].shape[2]
    cu, rows = s["cu"].long(), s["rows"].long()
    entry = torch.arange(R, device=q.device)
    gid = torch.searchsorted(cu[1:], entry, right=True)
    nth = entry - cu[gid]
    whole = s["prompt"] // PAGE
    n = whole.numel()
    qr = q[rows].view(R, Hkv, Hq // Hkv, d) * d ** -0.5
    qg = torch.zeros(n, s["most"], *qr.shape[1:], device=q.device)
    qg[gid, nth] = qr
    first = pt[rows[cu[:-1]]][:, :s["prefix_pages"]]
    kg, vg = _gather(s["kp"], first), _gather(s["vp"], first)
    a = torch.einsum("nmhgd,nlhd->nmhgl", qg, kg)[gid, nth]
    cols = whole[gid][:, None] + torch.arange(s["own_pages"], device=q.device)
    mine = pt[rows].gather(1, cols.clamp_max(pt.shape[1] - 1).long())
    km, vm = _gather(s["kp"], mine), _gather(s["vp"], mine)
    b = torch.einsum("rhgd,rlhd->rhgl", qr, km)
    at = torch.arange(a.shape[-1], device=q.device)
    a = a.masked_fill(~(at < (whole * PAGE)[gid][:, None])[:, None, None], -math.inf)
    at = (whole * PAGE)[gid][:, None] + torch.arange(b.shape[-1], device=q.device)
    b = b.masked_fill(~(at < ln[rows][:, None])[:, None, None], -math.inf)
    x = torch.cat([a, b], -1)
    if s["sink"] is not None:
        x = torch.cat([x, s["sink"].view(1, Hkv, -1, 1).expand(R, -1, -1, 1)], -1)
    top = x.amax(-1, keepdim=True)
    e = (x - top).exp()
    total = e.sum(-1, keepdim=True)
    p = e / total
    na = a.shape[-1]
    pg = torch.zeros(*qg.shape[:-1], na, device=q.device)
    pg[gid, nth] = p[..., :na]
    og = torch.einsum("nmhgl,nlhd->nmhgd", pg, vg)[gid, nth]
    og = og + torch.einsum("rhgl,rlhd->rhgd", p[..., na:na + b.shape[-1]], vm)
    o, lse = torch.empty_like(s["q"]), torch.empty(R, Hq, device=q.device)
    o[rows] = og.view(R, Hq, d).bfloat16()
    lse[rows] = (top + total.log()).view(R, Hq)
    return o, lse


def _plain_decode(s):
    q, ln = s["q"].float(), s["ln"]
    B, Hq, d = q.shape
    k, v = _gather(s["kp"], s["pt"]), _gather(s["vp"], s["pt"])
    Hkv = k.shape[2]
    x = torch.einsum("bhgd,blhd->bhgl", q.view(B, Hkv, -1, d) * d ** -0.5, k)
    t = torch.arange(k.shape[1], device=q.device)
    x = x.masked_fill(~(t < ln[:, None])[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    e = (x - top).exp()
    total = e.sum(-1, keepdim=True)
    p = e / total
    o = torch.einsum("bhgl,blhd->bhgd", p, v).reshape(B, Hq, d).bfloat16()
    w = p.sum(2)
    newest = (t == ln[:, None] - 1)[:, None]
    out = torch.where(newest, w, s["mass"] + w)
    s["out"].copy_(torch.where((t < ln[:, None])[:, None], out, s["out"]))
    s["positions"].copy_(torch.where(newest, s["last"][:, None, None], s["positions"]))
    return o, (top + total.log()).view(B, Hq)


def _plain_prompt(s):
    case, cu, ln = s["case"], s["cu"].long(), s["ln"]
    T, Hq, d = s["q"].shape
    k = _gather(s["kp"], s["pt"])
    B, M, Hkv = k.shape[:3]
    row = torch.arange(T, device=k.device)
    seq = torch.searchsorted(cu[1:], row, right=True)
    i = row - cu[seq]
    nq = cu[1:] - cu[:-1]
    most = case["qhi"]
    q = torch.zeros(B, most, Hkv, Hq // Hkv, d, device=k.device)
    q[seq, i] = s["q"].float().view(T, Hkv, -1, d) * d ** -0.5
    lse = torch.zeros(B, most, Hkv, Hq // Hkv, device=k.device)
    lse[seq, i] = s["lse"].T.reshape(T, Hkv, -1)
    x = torch.einsum("bihgd,blhd->bhgil", q, k)
    x = (x - lse.permute(0, 2, 3, 1)[..., None]).exp()
    t = torch.arange(M, device=k.device)
    ok = _seen(case, torch.arange(most, device=k.device)[:, None], t,
               nq[:, None, None], ln[:, None, None])
    w = torch.where(ok[:, None, None], x, 0.0).sum((2, 3))
    valid = (t < ln[:, None])[:, None]
    new = valid & (t >= ln[:, None] - nq[:, None])[:, None]
    out = torch.where(new, w, s["mass"] + w)
    s["out"].copy_(torch.where(valid, out, s["out"]))
    s["positions"].copy_(torch.where(new, t.int(), s["positions"]))


def _plain_evict(s, mass, positions):
    case, ln, keep = s["case"], s["ln"][:, None, None], s["keep"][:, None, None]
    slot = torch.arange(mass.shape[-1], device=mass.device)
    valid = slot < ln
    newest = positions.masked_fill(~valid, -1).amax(-1, keepdim=True)
    held = (positions < case["sink"]) | (positions > newest - case["recent"])
    key = mass.masked_fill(held, math.inf).masked_fill(~valid, -1.0)
    order = key.sort(stable=True, dim=-1, descending=True).indices
    stays = torch.zeros_like(valid.expand_as(mass)).scatter_(-1, order, (slot < keep).expand_as(mass))
    src = (stays & (slot >= keep)).nonzero(as_tuple=True)
    dst = (~stays & (slot < keep)).nonzero(as_tuple=True)
    mass[dst], positions[dst] = mass[src], positions[src]
    a, b = (s["pt"][x[1], x[3] // PAGE].long() for x in (src, dst))
    for pool in (s["kp"], s["vp"]):
        pool[dst[0], b, dst[3] % PAGE, dst[2]] = pool[src[0], a, src[3] % PAGE, src[2]]
    return s["keep"].clone()


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import exact_attention_08_gb300 as ea
    if op == "shared":
        if own:
            o, lse = ea.attn_decode_paged_shared(s["q"], s["kp"], s["vp"], s["pt"], s["ln"],
                                                 s["cu"], s["prompt"], s["rows"],
                                                 sink_logit=s["sink"])
        else:
            o, lse = _plain_shared(s)
        return dict(o=o, lse=lse)
    if op == "decode":
        if own:
            o, lse = ea.attn_decode_paged_mass(s["q"], s["kp"], s["vp"], s["pt"], s["ln"],
                                               s["mass"], s["positions"], s["last"],
                                               mass_out=s["out"])
        else:
            o, lse = _plain_decode(s)
        return dict(o=o, lse=lse, mass=s["out"], positions=s["positions"])
    if op == "prompt":
        if own:
            ea.attn_mass_paged(s["q"], s["lse"], s["kp"], s["pt"], s["cu"], s["ln"], s["mass"],
                               s["positions"], max_seqlen_q=s["case"]["qhi"],
                               causal=s["case"]["causal"], window=s["case"]["window"],
                               mass_out=s["out"])
        else:
            _plain_prompt(s)
        return dict(mass=s["out"], positions=s["positions"])
    # masses and positions as they stood before the cut
    mass, positions = s["mass"].clone(), s["positions"].clone()
    if own:
        new = ea.attn_evict_paged(mass, positions, s["pt"], s["ln"], s["keep"], s["kp"], s["vp"],
                                  s["refs"], n_sink=s["case"]["sink"],
                                  recent=s["case"]["recent"])
    else:
        new = _plain_evict(s, mass, positions)
    return dict(mass=mass, positions=positions, seqlens=new, k_pages=s["kp"], v_pages=s["vp"])


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, Hkv, d = case["op"], case["Hkv"], case["d"]
    token = Hkv * d * 4  # K and V of one token
    if op == "shared":
        sizes = _group_sizes(case)
        R, prompt = sum(sizes), (case["plo"] + case["phi"]) / 2
        mine = (case["slo"] + case["shi"]) / 2
        return dict(bytes=(len(sizes) * prompt + R * mine) * token + R * case["Hq"] * (d * 4 + 4),
                    flops=R * (prompt + mine) * case["Hq"] * d * 4)
    if op == "decode":
        keys = case["B"] * (case["lo"] + case["hi"]) / 2
        return dict(bytes=keys * (token + Hkv * 8) + case["B"] * case["Hq"] * (d * 4 + 4),
                    flops=keys * case["Hq"] * d * 4)
    if op == "prompt":
        keys, nq = (case["lo"] + case["hi"]) / 2, (case["qlo"] + case["qhi"]) / 2
        pairs = nq * (keys - nq / 2 if case["causal"] else keys)
        if case["window"]:
            pairs = nq * min(case["window"], keys)
        return dict(bytes=case["B"] * (keys * (token / 2 + Hkv * 8) + nq * case["Hq"] * (d * 2 + 4)),
                    flops=case["B"] * pairs * case["Hq"] * d * 2)
    keep = (case["klo"] + case["khi"]) / 2
    each = case["layers"] * case["B"] * Hkv
    moved = keep * case["over"] / (keep + case["over"])
    return dict(bytes=each * ((keep + case["over"]) * 8 + moved * (d * 8 + 16)), flops=0)


# ------------------------------------------------------------------ from the definition, in 64 bits

def _row_keys(pool, pt, b, L):
    return pool[pt[b, :(L + PAGE - 1) // PAGE].long()].flatten(0, 1)[:L].double()


def _exact_row(q, keys, values, sink):
    """One query [Hq, d] over its keys [L, Hkv, d]: output, log-sum-exp and weights, in fp64."""
    Hq, d = q.shape
    G = Hq // keys.shape[1]
    o, lse, w = [], [], []
    for h in range(keys.shape[1]):
        x = q[h * G:(h + 1) * G].double() @ keys[:, h].T / math.sqrt(d)
        if sink is not None:
            x = torch.cat([x, sink[h * G:(h + 1) * G, None].double()], 1)
        z = x.logsumexp(1)
        p = (x - z[:, None]).exp()[:, :keys.shape[0]]
        o.append(p @ values[:, h])
        lse.append(z)
        w.append(p.sum(0))
    return torch.cat(o), torch.cat(lse), torch.stack(w)


def _exact_prompt(case, s):
    out, positions = s["out"].double(), s["positions"].clone()
    G, d = case["Hq"] // case["Hkv"], case["d"]
    for b in range(case["B"]):
        a, e, L = int(s["cu"][b]), int(s["cu"][b + 1]), int(s["ln"][b])
        n = e - a
        keys = _row_keys(s["kp"], s["pt"], b, L)
        t = torch.arange(L, device="cuda")
        at = torch.arange(L - n, L, device="cuda")[:, None]
        hidden = torch.zeros(n, L, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= t > at
            if case["window"]:
                hidden |= at - t >= case["window"]
        base = torch.cat([s["mass"][b, :, :L - n].double(),
                          torch.zeros(case["Hkv"], n, dtype=torch.float64, device="cuda")], 1)
        for h in range(case["Hq"]):
            x = s["q"][a:e, h].double() @ keys[:, h // G].T / math.sqrt(d)
            x -= s["lse"][h, a:e, None].double()
            base[h // G] += x.exp_().masked_fill_(hidden, 0).sum(0)
        out[b, :, :L] = base
        positions[b, :, L - n:L] = t[L - n:].int()
    return dict(mass=out, positions=positions)


def _exact_evict(case, s):
    mass, positions = s["mass"].cpu().numpy().copy(), s["positions"].cpu().numpy().copy()
    pt = s["pt"].tolist()
    moves = []
    for layer in range(case["layers"]):
        for b in range(case["B"]):
            L, K = int(s["ln"][b]), int(s["keep"][b])
            for h in range(case["Hkv"]):
                m, p = mass[layer, b, h], positions[layer, b, h]
                newest = p[:L].max()
                held = (p[:L] < case["sink"]) | (p[:L] > newest - case["recent"])
                # protected tokens first, then by mass, equal ones by slot
                rank = numpy.lexsort((numpy.arange(L), numpy.where(held, 0, -m[:L]), ~held))
                stay = set(rank[:K].tolist())
                holes = [t for t in range(K) if t not in stay]
                movers = sorted(t for t in stay if t >= K)
                for a, c in zip(movers, holes):
                    m[c], p[c] = m[a], p[a]
                    moves.append((layer, pt[b][a // PAGE] * PAGE + a % PAGE,
                                  pt[b][c // PAGE] * PAGE + c % PAGE, h))
    out = dict(mass=torch.from_numpy(mass).double(), positions=torch.from_numpy(positions),
               seqlens=s["keep"].clone())
    layer, a, c, h = torch.tensor(moves, device="cuda").T
    for name, pool in (("k_pages", s["kp"]), ("v_pages", s["vp"])):
        x = pool.double()
        flat = x.view(case["layers"], -1, case["Hkv"], case["d"])
        flat[layer, c, h] = flat[layer, a, h]
        out[name] = x
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "evict":
        return _exact_evict(case, s)
    if op == "prompt":
        return _exact_prompt(case, s)
    rows, Hq = s["ln"].numel(), case["Hq"]
    o = torch.empty(rows, Hq, case["d"], dtype=torch.float64, device="cuda")
    lse = torch.empty(rows, Hq, dtype=torch.float64, device="cuda")
    more = {}
    if op == "decode":
        more = dict(mass=s["out"].double(), positions=s["positions"].clone())
    for b in range(rows):
        L = int(s["ln"][b])
        o[b], lse[b], w = _exact_row(s["q"][b], _row_keys(s["kp"], s["pt"], b, L),
                                     _row_keys(s["vp"], s["pt"], b, L), s.get("sink"))
        if op == "decode":
            w[:, :L - 1] += s["mass"][b, :, :L - 1].double()
            more["mass"][b, :, :L] = w
            more["positions"][b, :, L - 1] = s["last"][b]
    return dict(o=o, lse=lse, **more)
