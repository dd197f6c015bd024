"""What calls on thinned caches leave as it was: rows with bad input, bit for bit and no other,
and everything where the workspace is too small."""
import numpy as np
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests import _thin_ref as ref
from tests._parity import np64
from tests.test_evict_parity import Cache
from tests.test_mass_parity import Rows, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[-5, 62, 60], [60, -1, 62], [2 ** 31 - 1, 60, -2 ** 31], [81, 60, 61]])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_evict_leaves_rows_of_bad_lengths(lens, d):
    c = Cache([60, 60, 60], 2, 2, d, slots=61, seed=2)
    bad = [not 0 <= n <= 61 for n in lens]
    c.lens = [0 if x else n for x, n in zip(bad, lens)]
    keep = [20, 31, 60]
    m, p, k, v, new = c.expect(keep, 2, 3)
    c.dm, c.dp, c.dk, c.dv = (t.cuda() for t in (c.mass, c.positions, c.k, c.v))
    got = ea.attn_evict_paged(c.dm, c.dp, i32(c.table), i32(lens), i32(keep), c.dk, c.dv,
                              i32(c.refs), n_sink=2, recent=3)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_ERR_BAD_INPUT
    c.check((m, p, k, v, [n if x else w for x, n, w in zip(bad, lens, new)]), got)
    for i in range(3):
        if bad[i]:
            assert torch.equal(c.dm[:, i].cpu(), c.mass[:, i])
            assert torch.equal(c.dp[:, i].cpu(), c.positions[:, i])


@pytest.mark.parametrize("cu,lens,left", [
    ([0, 4, 2, 12], [40, 40, 40], [1, 2]),      # its queries decrease; the next has 10 of 7 at most
    ([-1, 4, 8, 12], [40, 40, 40], [0]), ([0, 4, 8, 13], [40, 40, 40], [2]),
    ([0, 4, 8, 12], [40, 46, 40], [1]), ([0, 4, 8, 12], [40, -3, 40], [1]),
    ([0, 2, 10, 12], [40, 40, 40], [1]), ([0, 4, 8, 12], [2 ** 31 - 1, 40, -2 ** 31], [0, 2])])
def test_masses_of_bad_sequences_are_left_and_no_others(cu, lens, left):
    d = 64
    r = Rows([40, 40, 40], 2, 1, d, slots=45, seed=9)
    q, lse = r.q(13), torch.full((2, 13), 4.0)
    mass, pos = r.mass.cuda(), r.pos.cuda()
    ea.attn_mass_paged(q[:12].cuda(), lse[:, :12].contiguous().cuda(), r.k.cuda(),
                       i32([t[:3] + [0] for t in r.table]), i32(cu), i32(lens), mass, pos,
                       max_seqlen_q=7)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_ERR_BAD_INPUT
    for b in range(3):
        if b in left:
            assert torch.equal(mass[b].cpu(), r.mass[b]) and torch.equal(pos[b].cpu(), r.pos[b])
            continue
        Lq, k = cu[b + 1] - cu[b], next(r.keys(b))[:, 0]
        w = 0
        for i in range(Lq):
            x = d ** -0.5 * (np64(q[cu[b] + i]) @ k.T)
            w = w + (np.exp(x - 4.0) * (np.arange(40) <= i + 40 - Lq)).sum(0)
        base = r.mass[b, 0, :40].double().numpy().copy()
        base[40 - Lq:] = 0
        ref.check_mass(mass[b, 0, :40].double().cpu().numpy(), base, w, b)
        want = r.pos[b].clone()
        want[:, 40 - Lq:40] = torch.arange(40 - Lq, 40, dtype=torch.int32)
        assert torch.equal(pos[b].cpu(), want)
        assert torch.equal(mass[b, :, 40:].cpu(), r.mass[b, :, 40:])


@pytest.mark.parametrize("bad", [-1, 31, 49, 2 ** 31 - 1, -2 ** 31])
def test_masses_of_a_step_of_bad_rows_are_left_and_no_others(bad):
    """Slots for 30 tokens, pages for 48."""
    r = Rows([20, 20, 20], 2, 2, 64, slots=30, seed=3)
    mass, pos, q = r.mass.cuda(), r.pos.cuda(), r.q(3)
    ea.attn_decode_paged_mass(q.cuda(), r.k.cuda(), r.v.cuda(), i32([t[:2] + [0] for t in r.table]),
                              i32([20, bad, 20]), mass, pos)
    torch.cuda.synchronize()
    assert ea.attn_device_status() == ea.ATTN_ERR_BAD_INPUT
    assert torch.equal(mass[1].cpu(), r.mass[1]) and torch.equal(pos[1].cpu(), r.pos[1])
    for b in (0, 2):
        k, v = r.keys(b)
        _, _, w = ref.attend(np64(q[b]), k, v, 64 ** -0.5)
        base = r.mass[b, :, :20].double().numpy().copy()
        base[:, 19] = 0
        ref.check_mass(mass[b, :, :20].double().cpu().numpy(), base, w)
        assert torch.equal(mass[b, :, 20:].cpu(), r.mass[b, :, 20:])
        assert (pos[b, :, 19] == 19).all()


def test_evict_refuses_a_workspace_that_is_too_small():
    c = Cache([100, 70], 1, 2, 64, seed=5)
    n = ea.attn_evict_workspace_size(1, 2, 2, c.slots, c.W)
    c.dm, c.dp, c.dk, c.dv = (t.cuda() for t in (c.mass, c.positions, c.k, c.v))
    args = c.dm, c.dp, i32(c.table), i32(c.lens), i32([30, 40]), c.dk, c.dv
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for short in (1, 8, n - 16):
        with pytest.raises(ea.AttnError):
            ea.attn_evict_paged(*args, workspace=ws[:n - short])
    torch.cuda.synchronize()
    assert torch.equal(c.dm.cpu(), c.mass) and torch.equal(c.dk.cpu(), c.k)
    new = ea.attn_evict_paged(*args, workspace=ws)
    torch.cuda.synchronize()
    c.check(c.expect([30, 40], 0, 0), new)
    assert ea.attn_device_status() == ea.ATTN_OK
