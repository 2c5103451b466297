"""A NaN or +inf score makes its row NaN, O and LSE, through every split of the keys and every merge; it never makes the
keys around it disappear, and it changes no other row.  (A row without keys stays O = 0, LSE = -inf.)"""
import math

import pytest
import torch

import decode_context_paged_gb300 as dcp
from test_gpu_block_scales import Case
from test_gpu_prefill import SCALE, make

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def all_nan(o, lse):
    return bool(torch.isnan(o).all() and torch.isnan(lse).all())


@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,k_lens,key", [
    ([200], [200], 77),         # one range of keys
    ([300, 40], [300, 90], 0),
    ([60], [5000], 1300),       # the keys are split over the SMs, the NaN in one range of them
    ([60], [5000], 4990),
])
def test_prompts(cuda_device, q_lens, k_lens, key, causal, dtype, value):
    a = {k: v.clone() for k, v in make(q_lens, k_lens, 3, cuda_device, seed=51).items()}
    a["q"][..., 5] = 1.0
    kw = dict(softmax_scale=SCALE, causal=causal, out_dtype=dtype)
    ref, rlse = dcp.prefill_attn(**a, **kw)
    a["k_nope"][key, 1, 5] = value
    out, lse = dcp.prefill_attn(**a, **kw)
    hit = torch.zeros(sum(q_lens), dtype=torch.bool, device=cuda_device)  # rows of request 0 that see the key
    hit[:q_lens[0]] = torch.arange(q_lens[0], device=cuda_device) + k_lens[0] - q_lens[0] >= key if causal else True
    assert hit.any()
    assert all_nan(out[hit, 1], lse[hit, 1])
    assert torch.equal(out[~hit, 1], ref[~hit, 1]) and torch.equal(lse[~hit, 1], rlse[~hit, 1])
    for h in (0, 2):
        assert torch.equal(out[:, h], ref[:, h]) and torch.equal(lse[:, h], rlse[:, h])
    # ... and on through the merge of two key ranges
    if dtype is torch.float32:
        o, z = dcp.lse_merge(torch.stack([ref, out]), torch.stack([rlse, lse]))
        assert all_nan(o[hit, 1], z[hit, 1]) and torch.isfinite(o[~hit, 1]).all()


def test_prompt_query_and_a_row_of_nothing_but_nan(cuda_device):
    a = {k: v.clone() for k, v in make([130, 5], [130, 0], 2, cuda_device, seed=52).items()}
    ref, rlse = dcp.prefill_attn(**a, softmax_scale=SCALE)
    a["q"][0, 0, 3] = NAN      # its one visible key
    a["q"][128, 1, 191] = INF  # in the second tile
    out, lse = dcp.prefill_attn(**a, softmax_scale=SCALE)
    assert all_nan(out[0, 0], lse[0, 0]) and all_nan(out[128, 1], lse[128, 1])
    rest = torch.ones(135, 2, dtype=torch.bool, device=cuda_device)
    rest[0, 0] = rest[128, 1] = False
    assert torch.equal(out[rest], ref[rest]) and torch.equal(lse[rest], rlse[rest])
    assert (out[130:] == 0).all() and torch.isneginf(lse[130:]).all()  # a request without keys


@pytest.mark.parametrize("v_dim", [128, 256, 512])
@pytest.mark.parametrize("n,at", [(2, 0), (2, 1), (5, 4), (40, 33)])
def test_lse_merge(cuda_device, n, at, v_dim):
    """Beside empty parts only, beside finite ones, and one among rows without."""
    g = torch.Generator(device=cuda_device).manual_seed(n + at)
    o = torch.randn(n, 6, v_dim, generator=g, device=cuda_device)
    lse = torch.randn(n, 6, generator=g, device=cuda_device)
    lse[:, 1], o[:, 1] = -INF, 0.0
    lse[:, 4], o[:, 4] = -INF, 0.0
    ref, rlse = dcp.lse_merge(o, lse)
    for row in (1, 3):
        o[at, row], lse[at, row] = NAN, NAN
    got, z = dcp.lse_merge(o, lse)
    assert all_nan(got[[1, 3]], z[[1, 3]])
    rest = [0, 2, 4, 5]
    assert torch.equal(got[rest], ref[rest]) and torch.equal(z[rest], rlse[rest])
    assert (got[4] == 0).all() and torch.isneginf(z[4])


def decode(c, form, pools=None, **kw):
    """A merged call over pools of the form: block scales, one scale or BF16."""
    opt = dict(layout=c.layout, dev_error=c.err, **kw)
    if form == "blocks":
        opt["kv_scales"] = list(c.scales)
    else:
        opt["kv_scale"] = 2.0 ** -7 if form == "one" else 1.0
    return dcp.decode_attn_merged(c.q, c.seq, c.ptr, c.vp, list(c.pool if pools is None else pools), c.scale, **opt)


@pytest.mark.parametrize("form", ["blocks", "one", "bf16"])
@pytest.mark.parametrize("lens,T,H,N,layout,pos", [
    ([30, 500], 1, 16, 4, "page", 7),          # the request's keys are all on one rank: the others' parts are empty
    ([700, 64], 2, 48, 3, "page", 130),
    ([70000, 900], 1, 64, 2, "page", 40000),   # one of many pieces of a rank's keys
    ([2000, 70], 1, 80, 4, "token", 1001),
])
def test_decode_key(cuda_device, lens, T, H, N, layout, pos, form):
    c = Case(lens, T, H, N, 16, layout, cuda_device, seed=53)
    pools = c.pool.clone() if form != "bf16" else (c.pool.float() * 2.0 ** -7).to(torch.bfloat16)
    ref = decode(c, form, pools)
    d, s, r, _ = c.rows(0)
    d = int(d[pos])
    if form == "bf16":
        pools[d, int(s[pos]), int(r[pos]), 555] = NAN
    else:
        pools.view(torch.uint8)[d, int(s[pos]), int(r[pos]), 555] = 0x7F
    for o_dtype in (torch.float32, torch.bfloat16):
        o, lse, op, lp = decode(c, form, pools, o_dtype=o_dtype)
        assert int(c.err.item()) == 0
        assert all_nan(o[0], lse[0]) and all_nan(op[d, 0], lp[d, 0])
        assert torch.equal(o[1], ref[0][1].to(o_dtype)) and torch.equal(lse[1], ref[1][1])
        others = [x for x in range(N) if x != d]
        assert torch.equal(op[others], ref[2][others]) and torch.equal(lp[others], ref[3][others])
        m, z = dcp.lse_merge(op, lp)
        assert all_nan(m[0], z[0]) and torch.equal(m[1], ref[0][1]) and torch.equal(z[1], ref[1][1])


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("form", ["blocks", "one", "bf16"])
def test_decode_query(cuda_device, form, value):
    """A NaN or an infinity in one query row makes that row NaN, no other (an empty request's rows stay empty)."""
    c = Case([700, 0, 300], 2, 48, 3, 16, "page", cuda_device, seed=54)
    pools = c.pool if form != "bf16" else (c.pool.float() * 2.0 ** -7).to(torch.bfloat16)
    ref = decode(c, form, pools)
    for at in ((0, 1, 5), (1, 0, 0), (2, 0, 47)):
        c.q[at][100] = value
    o, lse, _, _ = decode(c, form, pools)
    rest = torch.ones(3, 2, 48, dtype=torch.bool, device=cuda_device)
    for at in ((0, 1, 5), (2, 0, 47)):
        rest[at] = False
        assert all_nan(o[at], lse[at])
    assert torch.equal(o[rest], ref[0][rest]) and torch.equal(lse[rest], ref[1][rest])
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_an_appended_nan_reaches_the_answer(cuda_device):
    """append_kv keeps a NaN element; the attention over that request is NaN, over another request finite."""
    dev = cuda_device
    n, lens = 2, [130, 70]
    c = Case(lens, 1, 16, n, 16, "page", dev, seed=55)
    c.seq += 1
    g = torch.Generator(device=dev).manual_seed(1)
    row = torch.randn(2, 576, generator=g, device=dev).to(torch.bfloat16)
    row[0, 17] = NAN
    scales, pools = list(c.scales), list(c.pool)
    inv = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device=dev) / 64)
    dcp.append_kv(row[:, :512], row[:, 512:], torch.tensor([0, 1, 2], device=dev), c.seq, c.ptr, c.vp, pools, inv,
                  kv_scales=scales, dev_error=c.err)
    o, lse, _, _ = dcp.decode_attn_merged(c.q, c.seq, c.ptr, c.vp, pools, 1 / math.sqrt(192.0), kv_scales=scales, dev_error=c.err)
    assert int(c.err.item()) == 0
    assert all_nan(o[0], lse[0]) and torch.isfinite(o[1]).all() and torch.isfinite(lse[1]).all()
