"""Calls on shared and thinned caches at the ends of what they accept."""
import pytest
import torch

import exact_attention_08_gb300 as ea
from tests.test_shared_parity import Batch

pytestmark = pytest.mark.gpu


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
