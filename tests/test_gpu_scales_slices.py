"""reshard_scales where the ranks' scales are slices of one tensor, so that a rank starts at any multiple of 4 bytes."""
import pytest
import torch

import decode_context_paged_gb300 as dcp
from test_gpu_scales_reshard import case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lead", [0, 1, 2])
@pytest.mark.parametrize("layers,n_cp,n_dcp", [(1, 1, 2), (1, 3, 5), (5, 3, 3), (8, 4, 4)])
@pytest.mark.parametrize("block", [64, 32, 16, 1])
def test_slices_of_one_tensor(cuda_device, block, layers, n_cp, n_dcp, lead):
    """Odd page and slot counts; `lead` values in front of the first rank's."""
    lens = [101 * 64 - 5, 1, 1000]  # 101 + 1 + 16 pages, and three more in the pools: 121
    c = case(lens, layers, n_cp, n_dcp, block, cuda_device, seed=block + lead)
    shapes = [x.shape for x in c["src"]], [x.shape for x in c["dst"]]
    src = torch.cat([torch.zeros(lead, device=cuda_device)] + [x.flatten() for x in c["src"]])
    dst = torch.cat([torch.full((lead,), 9.0, device=cuda_device)] + [x.flatten() for x in c["dst"]])

    def ranks(flat, shapes):
        out, at = [], lead
        for s in shapes:
            out.append(flat[at:at + s.numel()].view(s))
            at += s.numel()
        return out

    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    dcp.reshard_scales(c["ptr"], c["at"], c["vp"], layers, ranks(src, shapes[0]), ranks(dst, shapes[1]), dev_error=err)
    assert int(err.item()) == 0
    assert torch.equal(torch.stack([x.cpu() for x in ranks(dst, shapes[1])]), c["want"])
    assert (dst[:lead] == 9.0).all()
