"""Refusals of attn_page_plan_granted through the C ABI (nothing is launched)."""
import ctypes

import pytest

from exact_tiled_attention_gqa_b200 import _native
from exact_tiled_attention_gqa_b200.build import build

A, ODD, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002), None
PLAN = dict(sl=A, new=A, bt=A, free=A, nf=A, slots=A, ol=A, onf=A, st=A, granted=A, B=4, L=8, ps=64, mp=16, cap=100, n_pages=100)


@pytest.mark.parametrize("bad,code", [
    (dict(granted=ODD), -1), (dict(sl=NULL), -1), (dict(new=ODD), -1), (dict(st=NULL), -1), (dict(st=NULL, granted=NULL), -1),
    (dict(B=-1), -1), (dict(L=1 << 30), -2), (dict(cap=1 << 30), -2),
])
def test_page_plan_granted_rejects(bad, code):
    build()
    assert _native.lib().attn_page_plan_granted(*{**PLAN, **bad}.values(), None) == code
    assert _native.lib().attn_last_error() != b""
