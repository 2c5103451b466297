"""Block-scaled decode over page tables that hold more pages than the lengths use (pages allocated ahead, padded batches):
the spare pages may hold anything, and a request of length 0 with pages is empty."""
import pytest
import torch

import decode_context_paged_gb300 as dcp
from test_gpu_block_scales import Case, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["page", "token"])
@pytest.mark.parametrize("T,H,N,block", [(1, 64, 4, 16), (3, 24, 2, 1), (2, 80, 3, 64)])
def test_spare_pages(cuda_device, layout, T, H, N, block):
    pages_for = [1000, 20000, 640, 64, 5000, 129]
    lens = [77, 9001, 0, 0, T, 128]
    c = Case(pages_for, T, H, N, block, layout, cuda_device, seed=81)
    c.lens, c.seq = lens, torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    used = torch.zeros(c.scales.shape[:2] + (64,), dtype=torch.bool)
    for b in range(len(lens)):
        d, s, r, _ = c.rows(b)
        used[d, s, r] = True
    c.pool.view(torch.uint8)[~used.to(cuda_device)] = 0x7F
    groups = used.view(used.shape[:2] + (64 // block, block)).any(-1).to(cuda_device)
    c.scales = torch.where(groups, c.scales, float("nan"))
    o, lse, op, lp = dcp.decode_attn_merged(*c.args(), **c.kw())
    assert int(c.err.item()) == 0
    for b in range(len(lens)):
        close(o[b], lse[b], c.reference(b), f"request {b}")
        for r in range(N):
            close(op[r, b], lp[r, b], c.reference(b, r), f"request {b} rank {r}")
