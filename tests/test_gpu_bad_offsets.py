"""append_kv and prefill_attn report every request whose offsets or length do not fit, wherever the offsets lead, and the
requests that fit get the results that they have without it."""
import pytest
import torch

import decode_context_paged_gb300 as dcp
from test_gpu_append import Case
from test_gpu_prefill import SCALE, make

pytestmark = pytest.mark.gpu


def appended(c, dev, new_ptr, lens=None):
    d, opt = c.call(dev, new_ptr=torch.tensor(new_ptr, device=dev),
                    **(dict(seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev)) if lens else {}))
    return d, opt, int(opt["dev_error"].item())


@pytest.mark.parametrize("layout", ["page", "token"])
@pytest.mark.parametrize("new_ptr", [[1000, 1005], [1 << 40, (1 << 40) + 2], [21, 22], [-5, 20], [15, 5], [0, 21]])
def test_append_of_one_request(cuda_device, new_ptr, layout):
    c = Case([20], [20], 2, "e4m3", 16, layout, heads=3, seed=71)
    d, opt, err = appended(c, cuda_device, new_ptr)
    assert err == dcp.DEVERR_OUT_OF_RANGE
    c.check(d, opt, requests=[])  # nothing is written, queries included


@pytest.mark.parametrize("block", [1, 32, 64])
def test_append_of_many_requests(cuda_device, block):
    """140 requests; the last, and one in the middle, do not fit; requests without new tokens may hold any length."""
    new = [3] * 140
    c = Case([10] * 140, new, 2, "e4m3", block, "page", heads=1, seed=72)
    d, opt, err = appended(c, cuda_device, c.new_ptr[:-1] + [9999])
    assert err == dcp.DEVERR_OUT_OF_RANGE
    c.check(d, opt, requests=range(139))
    lens = list(c.lens)
    lens[77] = 2
    d, opt, err = appended(c, cuda_device, c.new_ptr, lens)
    assert err == dcp.DEVERR_OUT_OF_RANGE
    c.check(d, opt, requests=[b for b in range(140) if b != 77])
    c = Case([10] * 140, new[:100] + [0] * 40, 2, "e4m3", block, "page", heads=1, seed=73)
    d, opt, err = appended(c, cuda_device, c.new_ptr, c.lens[:100] + [-1] * 40)
    assert err == 0
    c.check(d, opt)


def test_decreasing_offsets_of_an_append(cuda_device):
    c = Case([20, 20, 20], [5, 5, 10], 2, "e4m3", 16, "page", seed=74)
    for ptr in ([0, 900, 5, 20], [0, 5, 4, 20], [900, 0, 5, 20]):
        assert appended(c, cuda_device, ptr)[2] == dcp.DEVERR_OUT_OF_RANGE


@pytest.mark.parametrize("H", [1, 5])
@pytest.mark.parametrize("name,offsets", [
    ("q_ptr", [-5, 100]), ("q_ptr", [-5000, 100]), ("q_ptr", [2000, 2100]), ("q_ptr", [1 << 40, 1 << 41]), ("q_ptr", [90, 10]),
    ("q_ptr", [0, 101]), ("k_ptr", [0, 5000]), ("k_ptr", [-1, 100]), ("k_ptr", [300, 400]), ("k_ptr", [50, 20])])
def test_prompt_of_one_request(cuda_device, name, offsets, H):
    a = make([100], [100], H, cuda_device, seed=75)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    dcp.prefill_attn(**{**a, name: torch.tensor(offsets, device=cuda_device)}, softmax_scale=SCALE, dev_error=err)
    assert int(err.item()) == dcp.DEVERR_OUT_OF_RANGE


@pytest.mark.parametrize("B", [40, 140])  # offsets kept in shared memory, and not
def test_prompts_of_many_requests(cuda_device, B):
    a = make([30] * B, [40] * B, 3, cuda_device, seed=76)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    ref, rlse = dcp.prefill_attn(**a, softmax_scale=SCALE, dev_error=err)
    assert int(err.item()) == 0
    for name, at, value, fit in (("q_ptr", B, 30 * B + 1, slice(0, 30 * (B - 1))), ("k_ptr", B, 40 * B + 7, slice(0, 30 * (B - 1))),
                                 ("q_ptr", 0, -400, slice(30, None)), ("k_ptr", 0, -1, slice(30, None))):
        bad = a[name].clone()
        bad[at] = value
        err.zero_()
        out, lse = dcp.prefill_attn(**{**a, name: bad}, softmax_scale=SCALE, dev_error=err)
        assert int(err.item()) == dcp.DEVERR_OUT_OF_RANGE
        assert torch.equal(out[fit], ref[fit]) and torch.equal(lse[fit], rlse[fit])
