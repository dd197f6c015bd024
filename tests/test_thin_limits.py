"""Calls on shared and thinned caches at the ends of what they accept."""
import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _thin_ref as ref
from tests._parity import compare, np64
from tests.test_mass_parity import Rows
from tests.test_shared_parity import Batch, i32

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("listed", [0, 3])
def test_no_groups_and_no_lists(d, listed):
    """n_groups = 0: neither offsets nor prefixes nor rows are read, whatever n_rows is."""
    b = Batch([], 4, 2, d, alone=[100, 3, 0], seed=2)
    q, k, v, pt, ln = b.args()
    o, lse = torch.empty_like(q), torch.empty(3, 4, device="cuda")
    n = ea.attn_decode_shared_workspace_size(3, 4, 2, d, 0, listed, b.W, 2)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    rc = ea.lib.attn_decode_paged_shared(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), pt.data_ptr(), ln.data_ptr(), None, None, None,
        o.data_ptr(), lse.data_ptr(), 3, 4, 2, d, 16, b.W, b.P, 0, listed, 2, d ** -0.5, None,
        ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == ea.ATTN_OK and ea.attn_device_status() == ea.ATTN_OK
    b.check(o, lse)


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("d,prefix,lens", [
    (64, 700, [710, 100, 700, 0, 730, 650, 16, 5, 709]),    # a few rows end inside the prefix
    (128, 700, [690, 710, 670, 200, 30, 699, 660, 400, 688]),   # all but one do
    (256, 300, [290, 310, 260, 300, 17, 299, 270, 400, 288, 1]),
])
def test_values_behind_a_rows_end_stay_out_of_it(d, prefix, lens, value):
    """Keys and values of a shared prefix that are not finite: rows that end before them are
    what they are without them."""
    b = Batch([(prefix, lens)], 8, 2, d, seed=d)
    table = b.table[b.rows[int(np.argmax(lens))]]
    at = prefix // 16 * 16 - 5             # a token of the prefix's last whole pages
    b.v[table[at // 16], at % 16] = value
    b.k[table[at // 16], at % 16, :, ::3] = value
    o, lse = b.run(check=False)
    before = [r for r, n in zip(b.rows, lens) if n <= at // 16 * 16]  # no page of theirs holds it
    assert len(before) >= 4
    want = Batch([(prefix, lens)], 8, 2, d, seed=d)
    ro, rl = np.zeros((len(before), 8, d)), np.zeros((len(before), 8))
    for i, r in enumerate(before):
        k, v = (ref.gather(x.float().numpy(), want.table[r], want.lens[r]) for x in (want.k, want.v))
        ro[i], rl[i], _ = ref.attend(np64(want.q[r]), k, v, d ** -0.5)
    compare(o[before], lse[before], ro, rl, "rows before a value that is not finite")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [
    [900] * 3 + [480, 496, 512] * 3,                 # many rows end inside: their whole pages
    [900 + i for i in range(9)] + [480, 16, 0],      # few do: the longest rows' pages
    [900, 48, 32, 48, 0, 16]])                       # hardly anything to share
def test_rows_of_unequal_lengths(d, lens):
    """Rows that end inside their group's prefix, on both sides of what sharing fewer pages saves;
    a value that is not finite shows in the rows that see it, and in no other."""
    b = Batch([(896, lens)], 8, 2, d, seed=len(lens))
    o, lse = b.run()
    for _ in range(2):
        again = b.run(check=False)
        assert torch.equal(o.view(torch.int16), again[0].view(torch.int16))
        assert torch.equal(lse, again[1])
    table = b.table[b.rows[0]]
    b.v[table[55], 3] = NAN
    o, _ = b.run(check=False)
    for r, n in zip(b.rows, lens):
        assert torch.isfinite(o[r]).all() == (n <= 55 * 16)


def test_queries_past_2_to_the_24():
    """2^24 queries and more of 65 heads on one key head (a query tile is one token then), of
    which the last few see keys: 140 GB, of which only those few are read."""
    Lq, L, H, d = (1 << 24) + 300, 300, 65, 64
    torch.cuda.empty_cache()
    r = Rows([L], H, 1, d, seed=1)
    few = r.q(L)
    q = torch.empty(Lq, H, d, dtype=torch.bfloat16, device="cuda")
    q[-L:] = few.cuda()
    lse = torch.full((H, Lq), 7.0, device="cuda")
    args = r.k.cuda(), i32(r.table)
    got = ea.attn_mass_paged(q, lse, *args, i32([0, Lq]), i32([L]),
                             torch.zeros_like(r.mass).cuda(), max_seqlen_q=Lq)
    want = ea.attn_mass_paged(few.cuda(), lse[:, :L].contiguous(), *args, i32([0, L]), i32([L]),
                              torch.zeros_like(r.mass).cuda(), max_seqlen_q=L)
    torch.cuda.synchronize()
    del q, lse
    torch.cuda.empty_cache()
    assert ea.attn_device_status() == ea.ATTN_OK
    a, b = (x[0, 0, :L].double().cpu().numpy() for x in (want, got))
    # the plain block against the formula, then the same sums in another order
    k, _ = r.keys(0)
    w = np.zeros((1, L))
    for i in range(L):
        x = d ** -0.5 * (k[:i + 1, 0] @ np64(few[i]).T)
        w[0, :i + 1] += np.exp(x - 7.0).sum(1)
    # (a thread adds 16 weights of each of 300 query tiles to one of its four sums)
    for x in (a, b):
        assert (np.abs(x - w[0]) <= (ref.WEIGHT + 4810 * 2.0 ** -24) * w[0]).all()


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 64), (8, 2, 128), (16, 2, 256)])
def test_scores_of_minus_infinity_leave_no_weight(Hq, Hkv, d):
    """A row whose scores are all -inf attends to nothing, O = 0 and LSE = -inf: its keys get no
    weight from that step."""
    lens = [40, 17, 300, 1]
    r = Rows(lens, Hq, Hkv, d, seed=d)
    for b in (1, 2, 3):
        for page in r.table[b][:(lens[b] + 15) // 16]:
            r.k[page] = -INF
    q = r.q(4).abs() + 0.5
    args = q.cuda(), r.k.cuda(), r.v.cuda(), i32(r.table), i32(lens)
    for splits in (1, 5):
        mass = r.mass.cuda()
        o, lse = ea.attn_decode_paged_mass(*args, mass, num_splits=splits)
        torch.cuda.synchronize()
        assert ea.attn_device_status() == ea.ATTN_OK
        k, v = r.keys(0)
        ro, rl, w = ref.attend(np64(q[0]), k, v, d ** -0.5)
        compare(o[:1], lse[:1], ro[None], rl[None])
        assert (o[1:] == 0).all() and torch.isneginf(lse[1:]).all()
        for b, n in enumerate(lens):
            want = r.mass[b].clone()
            want[:, n - 1] = 0
            if b == 0:
                base = want[:, :n].double().numpy()
                ref.check_mass(mass[b, :, :n].double().cpu().numpy(), base,
                               w.reshape(Hkv, Hq // Hkv, n).sum(1))
            else:
                assert torch.equal(mass[b].cpu(), want), b


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 1, 64), (8, 2, 128), (16, 2, 256)])
def test_queries_without_a_key_have_no_weight(Hq, Hkv, d):
    """LSE = -inf is a query that attended to nothing, whatever its scores: as if it were not
    there."""
    lens, nq = [300, 40], [50, 7]
    r = Rows(lens, Hq, Hkv, d, seed=d)
    q = r.q(57)
    cu = i32([0, 50, 57])
    lse = torch.full((Hq, 57), 6.0)
    out = {}
    for drop in (-INF, INF):             # a weight exp(s - inf) is none in any case
        z = lse.clone()
        z[:, 3:20], z[1, 55] = drop, drop
        out[drop] = ea.attn_mass_paged(q.cuda(), z.cuda(), r.k.cuda(), i32(r.table), cu, i32(lens),
                                       torch.zeros_like(r.mass).cuda(), max_seqlen_q=50)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_OK
    for b, n in enumerate(lens):
        assert torch.isfinite(out[INF][b, :, :n]).all()
        assert torch.equal(out[-INF][b, :, :n], out[INF][b, :, :n])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("prefix,shortest", [(22, 82), (16, 500), (170, 333), (15, 400)])
def test_an_empty_row_among_rows_longer_than_the_prefix(d, prefix, shortest):
    """No more pages are shared than the prefix has, whatever the rows that are not empty hold."""
    b = Batch([(prefix, [shortest + 7 * i for i in range(40)] + [0])], 4, 2, d, seed=prefix)
    b.run()
