"""append_kv's block scales at the ends of their range: what the appender writes is what the attention reads."""
import math

import pytest
import torch

import decode_context_paged_gb300 as dcp
from test_gpu_append import INV_FREQ

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [1, 16, 64])
def test_scales_stay_in_the_range_the_attention_reads(cuda_device, block):
    dev, n = cuda_device, 64
    x = torch.ones(n, 576, dtype=torch.bfloat16)
    x[:, 512:] = 0
    x[3, 7], x[20, 9], x[40, 100], x[50, 1] = 2.0 ** 56, -2.0 ** 57, 2.0 ** 100, -3e38  # 448 * 2^48 = 2^56.8
    x = x.to(dev)
    pool = torch.zeros(1, 64, 576, device=dev).to(torch.float8_e4m3fn)
    scales = torch.zeros(1, 64 // block, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    err = torch.zeros(1, **i32)
    seq, ptr, vp = torch.tensor([n], **i32), torch.tensor([0, 1], device=dev), torch.zeros(1, **i32)
    dcp.append_kv(x[:, :512], x[:, 512:], torch.tensor([0, n], device=dev), seq, ptr, vp, [pool], INV_FREQ.to(dev),
                  kv_scales=[scales], dev_error=err)
    amax = x.double().abs().view(64 // block, -1).amax(1)
    want = torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(-40, 48))
    assert torch.equal(scales[0].double(), want)
    size = want.repeat_interleave(block)[:, None]
    held = (x.double() / size).clamp(-448, 448).to(torch.float8_e4m3fn).double() * size
    assert torch.equal(pool[0].double() * size, held)
    # a query that sees the position only through a rope element of 0: the mean of the values as held
    q = torch.zeros(1, 1, 16, 576, dtype=torch.bfloat16, device=dev)
    o, lse, _, _ = dcp.decode_attn_merged(q, seq, ptr, vp, [pool], 1 / math.sqrt(192.0), kv_scales=[scales], dev_error=err)
    assert int(err.item()) == 0
    # equal weights 1/64: in two 8-bit terms they are off by at most 2^-7 where the scale is near the largest, below
    # 2^-22 of it they are lost with the rest of their column
    ref = held[:, :512].mean(0)
    tol = 2.0 ** -7 * held[:, :512].abs().mean(0) + 2.0 ** -22 * size.max() * held[:, :512].abs().div(size).sum(0) / n
    assert ((o[0, 0].double() - ref).abs() <= tol + 1e-6 * ref.abs()).all()
    assert ((lse[0, 0].double() - math.log(n)).abs() <= 1e-4).all()
