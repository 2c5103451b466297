"""append_kv's query rows where q_out lies beside q_rope or its strides interleave: the bits of a call into its own tensor."""
import pytest
import torch

from test_gpu_append import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,tok,head,q_at,o_at", [
    (3, 576, 192, 0, 64),      # slices of one [n][heads][192] tensor
    (3, 576, 192, 128, 64),
    (3, 192, 128, 0, 1 << 16),  # neither tokens nor heads outermost
    (5, 64, 70 * 64, 0, 1 << 16),  # heads outermost
    (1, 128, 64, 0, 64),
])
def test_layouts_that_do_not_meet(cuda_device, heads, tok, head, q_at, o_at):
    c = Case([300, 65], [69, 1], 4, "e4m3", 16, "page", heads=heads, seed=29)
    _, opt = c.call(cuda_device)
    want = opt["q_out"]
    flat = torch.full((1 << 17,), 3.0, dtype=torch.bfloat16, device=cuda_device)
    view = lambda start: flat.as_strided((70, heads, 64), (tok, head, 1), start)  # noqa: E731
    view(q_at).copy_(c.q.to(cuda_device)[..., 128:])
    before = flat.clone()
    d, opt = c.call(cuda_device, q_rope=view(q_at), q_out=view(o_at))
    assert int(opt["dev_error"].item()) == 0
    assert torch.equal(view(o_at), want)
    view(o_at).copy_(before.as_strided((70, heads, 64), (tok, head, 1), o_at))
    assert torch.equal(flat, before)
