"""append_kv refuses query rows that share memory, on the host (CPU: nothing is launched in the refused calls)."""
import ctypes
import itertools

import pytest

from test_abi_cache_ops import APPEND, INVALID, P, lib  # noqa: F401


def at(elements):
    return ctypes.c_void_p(P.value + 2 * elements)


def meet(n, tok, heads, head, apart):
    """The definition: two different rows (or a row shifted against itself) within 64 elements of one another."""
    rows = [(t, h) for t in range(n) for h in range(heads)]
    return any(abs(apart + (b[0] - a[0]) * tok + (b[1] - a[1]) * head) < 64 for a, b in itertools.product(rows, rows)
               if apart or a != b)


SHAPES = [  # new tokens, token stride, heads, head stride; True: rows of q_out overlap
    (4, 64, 2, 64, True), (4, 128, 3, 64, True), (4, 192, 4, 128, True), (4, 96, 2, 64, True), (3, 640, 8, 100, True),
    (64, 64, 65, 64 * 63, True), (1 << 20, 64, 2, 64 << 19, True), (1, 2, 3, 64, False), (4, 128, 2, 64, False),
    (4, 192, 3, 128, False), (5, 64, 7, 320, False), (4, 576 * 8, 8, 576, False)]


@pytest.mark.parametrize("n,tok,heads,head,overlap", SHAPES)
def test_rows_of_q_out(lib, n, tok, heads, head, overlap):  # noqa: F811
    if n <= 64:
        assert meet(n, tok if n > 1 else 0, heads, head, 0) == overlap
    if not overlap:
        return  # (a call that is taken goes on to the GPU: tested there)
    args = {**APPEND, "num_new": n, "num_heads": heads, "q_out_token_stride": tok, "q_out_head_stride": head,
            "q_rope": at(1 << 41), "q_token_stride": 64 * heads}
    assert lib.dcp_append_kv(*args.values()) == INVALID


@pytest.mark.parametrize("apart", [32, -62, 64, -64, 128, 64 * 7 + 2])
def test_q_out_shifted_over_q_rope(lib, apart):  # noqa: F811
    n, heads = 4, 2
    assert meet(n, 128, heads, 64, apart)
    args = {**APPEND, "num_new": n, "num_heads": heads, "q_rope": at(1 << 20), "q_out": at((1 << 20) + apart)}
    assert lib.dcp_append_kv(*args.values()) == INVALID


@pytest.mark.parametrize("change", [dict(q_token_stride=256), dict(q_head_stride=128), dict(q_token_stride=0)])
def test_in_place_with_other_strides(lib, change):  # noqa: F811
    assert lib.dcp_append_kv(*{**APPEND, **change}.values()) == INVALID
