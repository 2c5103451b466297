"""CPU checks of the binding: calls that must be refused before anything is allocated or launched.  (The tensors are on the
CPU: a check that comes too late shows as another error.)"""
import os
import subprocess
import sys
import types

import pytest
import torch

import decode_context_paged_gb300 as dcp


@pytest.fixture(scope="module", autouse=True)
def built():
    from decode_context_paged_gb300 import _build
    _build.build()


def attention(B=2, T=1, H=4, N=2, slots=3, dtype=torch.bfloat16):
    return dict(q=torch.zeros(B, T, H, 576, dtype=torch.bfloat16), seq_lens=torch.ones(B, dtype=torch.int32),
                req_page_ptr=torch.arange(B + 1), dst_vpages=torch.zeros(B, dtype=torch.int32),
                kv_pools=[torch.zeros(slots, 64, 576, dtype=dtype) for _ in range(N)], softmax_scale=0.1)


SCALED = dict(kv_scales=[torch.ones(3, 4) for _ in range(2)])


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("call", [dcp.partial_decode_attn, dcp.decode_attn_merged], ids=lambda f: f.__name__)
def test_a_planned_run_needs_the_workspace_of_its_plan(call, scaled):
    """Without it the call would run whatever plan a new allocation happens to hold."""
    a = attention(dtype=torch.float8_e4m3fn if scaled else torch.bfloat16)
    with pytest.raises(ValueError, match="planned run needs the workspace"):
        call(**a, **(SCALED if scaled else {}), planned=True)


@pytest.mark.parametrize("short,what", [(dict(seq_lens=torch.ones(1, dtype=torch.int32)), "seq_lens holds 1"),
                                        (dict(req_page_ptr=torch.arange(2)), "req_page_ptr holds 2")])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("call", [dcp.partial_decode_attn, dcp.decode_attn_merged, dcp.partial_decode_attn_static],
                         ids=lambda f: f.__name__)
def test_lengths_and_offsets_of_every_request(call, scaled, short, what):
    """The number of requests is q's: a shorter seq_lens or req_page_ptr would be read past its end."""
    if scaled and call is dcp.partial_decode_attn_static:
        pytest.skip("takes no block scales")
    a = attention(dtype=torch.float8_e4m3fn if scaled else torch.bfloat16)
    with pytest.raises(ValueError, match=what):
        call(**{**a, **short}, **(SCALED if scaled else {}))


def test_a_plan_needs_offsets_of_every_request():
    a = attention()
    with pytest.raises(ValueError, match="req_page_ptr holds 2"):
        dcp.attn_plan((2, 1, 4), torch.arange(2), a["dst_vpages"], a["kv_pools"], torch.zeros(1 << 20, dtype=torch.uint8))


def test_a_helper_of_another_torch_or_python_is_not_used():
    """It reads torch's objects by the layouts it was compiled with; the binding goes without it then."""
    if dcp._views is None:
        pytest.skip("the C++ helper was not built here")
    have = dict(open=dcp._views.open, built_for_torch=dcp._views.built_for_torch, built_for_python=dcp._views.built_for_python)
    assert dcp._usable(types.SimpleNamespace(**have))
    for change in (dict(built_for_torch="1.0.0"), dict(built_for_python=0x030b)):
        assert not dcp._usable(types.SimpleNamespace(**{**have, **change}))
    assert not dcp._usable(types.SimpleNamespace(open=have["open"]))  # of an earlier source


NO_STORAGE = """
import sys
import torch
from torch._subclasses import FakeTensorMode
import decode_context_paged_gb300 as dcp
if dcp._views is None:
    print("no helper")
    sys.exit(0)
with FakeTensorMode(allow_non_fake_inputs=True):
    x = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda")
questions = dict(ptr=lambda t: dcp._ptr(t, "t", torch.bfloat16, 0), ptrs=lambda t: dcp._ptrs([t], "t", t, torch.bfloat16, 0),
                 rows=lambda t: dcp._rows(t, "t", 64, 2, 2, 0))
def ask(t):
    try:
        questions[sys.argv[1]](t)
    except RuntimeError as e:
        print("raised", e)
    return t
torch.vmap(ask)(x)
"""


@pytest.mark.parametrize("question", ["ptr", "ptrs", "rows"])
def test_a_tensor_without_storage_raises(question):
    """Inside torch.vmap a tensor has no pointer: a Python error, not the end of the process."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", NO_STORAGE, question], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-500:]
    if "no helper" in r.stdout:
        pytest.skip("the C++ helper was not built here")
    assert "raised" in r.stdout, r.stdout
