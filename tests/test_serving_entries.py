"""Refusals of attn_page_plan_granted through the C ABI (nothing is launched), and the
file of the C++ binding."""
import ctypes
import os
import sys

import pytest
import torch

from exact_tiled_attention_gqa_b200 import _native
from exact_tiled_attention_gqa_b200 import build as build_module
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


def test_binding_is_of_this_torch_and_python(monkeypatch):
    """A module built against another torch, its C++ ABI or another Python has another name: it is never loaded or
    taken for up to date."""
    path = build_module.calls_path()
    assert path == build_module.CALLS_PATH == build_module.build_calls() and os.path.exists(path)
    assert torch.__version__ in path and f"cpython-{sys.version_info[0]}{sys.version_info[1]}" in path
    others = []
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "1.0.0+other")
        others.append(build_module.calls_path())
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
        others.append(build_module.calls_path())
    with monkeypatch.context() as m:
        m.setattr(build_module.sysconfig, "get_config_var", lambda name: "cpython-39-x86_64-linux-gnu")
        others.append(build_module.calls_path())
    assert len({path, *others}) == 4
    for other in others:
        monkeypatch.setattr(_native, "_calls", None)
        monkeypatch.setattr(_native, "CALLS_PATH", other)
        with pytest.raises(RuntimeError, match="this Python and torch, is missing"):
            _native.calls()
