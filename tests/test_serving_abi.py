"""Refusals of the serving-step calls through the C ABI: argument checks fail before
anything reaches a GPU (these calls never launch work), and the tree mask packing."""
import ctypes

import pytest
import torch

import exact_tiled_attention_gqa_b200 as attn
from exact_tiled_attention_gqa_b200 import _native
from exact_tiled_attention_gqa_b200.build import build, build_calls

# an aligned fake address, only ever passed together with an invalid argument
A = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10002)
HALF = ctypes.c_void_p(0x10008)
NULL = None


@pytest.fixture(scope="module")
def lib():
    build()
    build_calls()
    return _native.lib()


def _call(fn, defaults, kw):
    assert set(kw) <= {n for n, _ in defaults}
    return fn(*[kw.get(n, d) for n, d in defaults], None)


TREE = (("q", A), ("k", A), ("v", A), ("sl", A), ("mask", A), ("per_seq", 1), ("lens", NULL), ("out", A), ("lse", NULL), ("B", 2),
        ("Hq", 8), ("Hkv", 2), ("T", 5), ("Lmax", 640), ("D", 128), ("scale", 0.1), ("ws", A), ("wsb", 1 << 30))


@pytest.mark.parametrize("bad,code", [
    (dict(q=NULL), -1), (dict(k=NULL), -1), (dict(out=NULL), -1), (dict(sl=NULL), -1), (dict(mask=NULL), -1),
    (dict(mask=ODD), -1), (dict(lens=ODD), -1), (dict(lse=ODD), -1), (dict(v=HALF), -1), (dict(T=0), -1), (dict(T=-1), -1),
    (dict(Lmax=0), -1), (dict(B=-1), -1), (dict(Hq=7), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(T=1025), -2), (dict(D=96), -2), (dict(D=512), -2), (dict(ws=NULL), -3), (dict(wsb=64), -3), (dict(ws=ctypes.c_void_p(0x10010)), -1),
    (dict(B=1 << 20, Hq=1024, Hkv=1024, T=1024), -2),
])
def test_decode_tree_rejects(lib, bad, code):
    assert _call(lib.attn_decode_tree, TREE, bad) == code
    assert lib.attn_last_error() != b""


def test_decode_tree_empty_batch_and_workspace(lib):
    assert _call(lib.attn_decode_tree, TREE, dict(B=0)) == 0
    assert _call(lib.attn_decode_tree, TREE, dict(B=0, q=NULL, k=NULL, v=NULL, out=NULL, sl=NULL, mask=NULL, ws=NULL)) == 0
    f = lib.attn_decode_tree_workspace_size
    assert f(0, 8, 2, 5, 640, 128) == 0 and f(2, 7, 2, 5, 640, 128) == 0 and f(2, 8, 2, 0, 640, 128) == 0
    assert f(2, 8, 2, 1025, 640, 128) == 0 and f(2, 8, 2, 5, 0, 128) == 0 and f(2, 8, 2, 5, 640, 96) == 0
    w = f(2, 8, 2, 5, 640, 128)
    assert w % 256 == 0 and w >= 2 * 8 * 5 * (128 + 1) * 4
    g = lib.attn_decode_tree_paged_workspace_size
    assert g(2, 8, 2, 5, 128, 5, 128) == w and g(2, 8, 2, 5, 96, 5, 128) == 0 and g(2, 8, 2, 5, 128, 0, 128) == 0
    assert g(2, 8, 2, 5, 1 << 20, 1 << 12, 128) == 0


TREE_PAGED = (("q", A), ("k", A), ("v", A), ("bt", A), ("sl", A), ("mask", A), ("per_seq", 1), ("lens", NULL), ("out", A), ("lse", NULL),
              ("B", 2), ("Hq", 8), ("Hkv", 2), ("T", 5), ("n_pages", 16), ("ps", 128), ("mp", 8), ("D", 128), ("scale", 0.1), ("ws", A),
              ("wsb", 1 << 30))


@pytest.mark.parametrize("bad,code", [
    (dict(ps=96), -1), (dict(ps=0), -1), (dict(ps=-64), -1), (dict(n_pages=0), -1), (dict(mp=0), -1), (dict(bt=NULL), -1), (dict(bt=ODD), -1),
    (dict(mp=1 << 25), -2), (dict(n_pages=1 << 30, Hq=4, Hkv=4), -2), (dict(T=0), -1), (dict(ws=NULL), -3), (dict(T=2000), -2),
])
def test_decode_tree_paged_rejects(lib, bad, code):
    assert _call(lib.attn_decode_tree_paged, TREE_PAGED, bad) == code


PLAN = (("sl", A), ("new", A), ("bt", A), ("free", A), ("nf", A), ("slots", A), ("ol", A), ("onf", A), ("st", A), ("B", 4), ("L", 8),
        ("ps", 64), ("mp", 16), ("cap", 100), ("n_pages", 100))


@pytest.mark.parametrize("bad,code", [
    (dict(sl=NULL), -1), (dict(new=NULL), -1), (dict(bt=NULL), -1), (dict(free=NULL), -1), (dict(nf=NULL), -1), (dict(slots=NULL), -1),
    (dict(ol=NULL), -1), (dict(onf=NULL), -1), (dict(st=NULL), -1), (dict(sl=ODD), -1), (dict(slots=ODD), -1), (dict(B=-1), -1),
    (dict(L=-1), -1), (dict(ps=0), -1), (dict(mp=0), -1), (dict(n_pages=0), -1), (dict(cap=-1), -1),
    (dict(n_pages=1 << 26), -2), (dict(mp=1 << 26), -2), (dict(B=1 << 20, mp=1 << 12), -2), (dict(cap=1 << 30), -2),
])
def test_page_plan_rejects(lib, bad, code):
    assert _call(lib.attn_page_plan, PLAN, bad) == code


RELEASE = (("sl", A), ("keep", A), ("bt", A), ("free", A), ("nf", A), ("onf", A), ("B", 4), ("ps", 64), ("mp", 16), ("cap", 100),
           ("n_pages", 100))


@pytest.mark.parametrize("bad,code", [
    (dict(sl=NULL), -1), (dict(keep=NULL), -1), (dict(bt=NULL), -1), (dict(free=NULL), -1), (dict(nf=NULL), -1), (dict(onf=NULL), -1),
    (dict(free=ODD), -1), (dict(B=-1), -1), (dict(ps=0), -1), (dict(mp=0), -1), (dict(n_pages=0), -1), (dict(cap=1 << 30), -2),
])
def test_page_release_rejects(lib, bad, code):
    assert _call(lib.attn_page_release, RELEASE, bad) == code


ROPE = (("q", A), ("k", A), ("v", A), ("qs", 1024), ("ks", 256), ("vs", 256), ("pos", A), ("inv", A), ("slots", A), ("out", A), ("kc", A),
        ("vc", A), ("ksc", NULL), ("vsc", NULL), ("fmt", 0), ("B", 2), ("L", 3), ("Hq", 8), ("Hkv", 2), ("D", 128), ("rot", 128),
        ("n", 4), ("rows", 64), ("axes", 2), ("sec", (32, 32)), ("cycle", 0), ("adj", 0))


def _rope(lib, **kw):
    args = {n: kw.get(n, d) for n, d in ROPE}
    assert set(kw) <= set(args)
    if args["sec"] is not None:
        args["sec"] = (ctypes.c_int * len(args["sec"]))(*args["sec"])
    return lib.attn_rope_append(*args.values(), None)


@pytest.mark.parametrize("bad,code", [
    (dict(q=NULL), -1), (dict(k=NULL), -1), (dict(v=NULL), -1), (dict(pos=NULL), -1), (dict(inv=NULL), -1), (dict(slots=NULL), -1),
    (dict(out=NULL), -1), (dict(kc=NULL), -1), (dict(vc=NULL), -1), (dict(q=HALF), -1), (dict(kc=HALF), -1), (dict(slots=ODD), -1),
    (dict(qs=1016), -1), (dict(qs=1028), -1), (dict(ks=248), -1), (dict(vs=260), -1), (dict(B=-1), -1), (dict(L=-1), -1), (dict(Hq=0), -1),
    (dict(Hkv=0), -1), (dict(rows=0), -1), (dict(n=-1), -1), (dict(fmt=3), -1), (dict(fmt=-1), -1), (dict(fmt=1), -1),
    (dict(fmt=2, ksc=A), -1), (dict(D=96), -2), (dict(D=512), -2), (dict(fmt=1, D=256, rot=64, ksc=A, vsc=A), -2),
    (dict(rot=24), -1), (dict(rot=144), -1), (dict(rot=-16), -1), (dict(axes=0), -1), (dict(axes=5, sec=(16, 16, 16, 8, 8)), -1),
    (dict(sec=NULL), -1), (dict(sec=(32, 31)), -1), (dict(sec=(65, -1)), -1), (dict(sec=(0, 64), cycle=1), -1),
    (dict(n=1 << 26), -2), (dict(B=1 << 17, L=1 << 15), -2),
])
def test_rope_append_rejects(lib, bad, code):
    assert _rope(lib, **bad) == code
    assert lib.attn_last_error() != b""


def test_rope_append_without_tokens_is_noop(lib):
    assert _rope(lib, B=0) == 0 and _rope(lib, L=0, q=NULL, k=NULL, v=NULL, out=NULL, slots=NULL) == 0


COMMIT = (("k", A), ("v", A), ("bt", NULL), ("sl", A), ("lens", NULL), ("acc", A), ("n", A), ("ol", A), ("B", 4), ("Hkv", 2), ("T", 8),
          ("A", 3), ("D", 128), ("outer", 4), ("rows", 64), ("mp", 0))


@pytest.mark.parametrize("bad,code", [
    (dict(k=NULL), -1), (dict(v=NULL), -1), (dict(sl=NULL), -1), (dict(acc=NULL), -1), (dict(n=NULL), -1), (dict(ol=NULL), -1),
    (dict(k=HALF), -1), (dict(acc=ODD), -1), (dict(bt=ODD, mp=4), -1), (dict(lens=ODD), -1), (dict(B=-1), -1), (dict(Hkv=0), -1),
    (dict(T=0), -1), (dict(A=-1), -1), (dict(rows=0), -1), (dict(outer=3), -1), (dict(bt=A, mp=0), -1), (dict(bt=A, mp=4, outer=0), -1),
    (dict(D=96), -2), (dict(T=1025), -2), (dict(bt=A, mp=1 << 26), -2),
])
def test_tree_commit_rejects(lib, bad, code):
    assert _call(lib.attn_tree_commit, COMMIT, bad) == code


def test_tree_commit_empty_batch_is_noop(lib):
    assert _call(lib.attn_tree_commit, COMMIT, dict(B=0, k=NULL, v=NULL, sl=NULL, acc=NULL, n=NULL, ol=NULL, outer=0)) == 0


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 100])
def test_pack_tree_mask(T):
    g = torch.Generator().manual_seed(T)
    allowed = torch.rand(3, T, T, generator=g) < 0.5
    words = attn.pack_tree_mask(allowed)
    assert words.dtype == torch.int32 and words.shape == (3, T, (T + 31) // 32)
    back = (words.unsqueeze(-1) >> torch.arange(32)) & 1
    back = back.flatten(-2)
    assert torch.equal(back[..., :T].bool(), allowed) and not back[..., T:].any()
    assert torch.equal(attn.pack_tree_mask(allowed[1]), words[1])


@pytest.mark.parametrize("bad", [torch.ones(3, 4, dtype=torch.bool), torch.ones(4, 4), torch.ones(4, dtype=torch.bool), None])
def test_pack_tree_mask_rejects(bad):
    with pytest.raises(ValueError):
        attn.pack_tree_mask(bad)


def test_host_tensors_are_refused(lib):
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        attn.page_plan(z(2), z(2), z(2, 4), z(8), z(1), L=1, page_size=64, n_pages=8)
    with pytest.raises(ValueError, match="CUDA"):
        attn.page_release(z(2), z(2), z(2, 4), z(8), z(1), page_size=64, n_pages=8)
    with pytest.raises(ValueError, match="CUDA"):
        attn.rope_append(bf(1, 1, 4, 64), bf(1, 1, 2, 64), bf(1, 1, 2, 64), z(1, 1), z(32, dt=torch.float32), z(1, 1), bf(1, 2, 64, 64),
                         bf(1, 2, 64, 64))
    with pytest.raises(ValueError, match="CUDA"):
        attn.decode_tree(bf(1, 4, 3, 64), bf(1, 2, 64, 64), bf(1, 2, 64, 64), z(1), z(1, 3, 1))
    with pytest.raises(ValueError, match="CUDA"):
        attn.tree_commit(bf(1, 2, 64, 64), bf(1, 2, 64, 64), z(1), z(1, 2), z(1), T=3)


def test_missing_binding_raises(monkeypatch, tmp_path):
    monkeypatch.setattr(_native, "_calls", None)
    monkeypatch.setattr(_native, "CALLS_PATH", str(tmp_path / "absent.so"))
    with pytest.raises(RuntimeError, match="missing"):
        _native.calls()


def test_binding_reaches_the_loaded_library(lib):
    """The C++ binding is handed the functions of the library ctypes loaded, and raises AttnError with its words."""
    calls = _native.calls()
    assert _native.calls() is calls and all(hasattr(lib, name) for name in _native.BOUND)
    cpu = torch.zeros(1, dtype=torch.int32)
    for bad in (None, 3, "x"):
        with pytest.raises(TypeError):
            calls.page_release(cpu, bad, cpu, cpu, cpu, 64, 8, None)


def test_sizes_are_refused_with_words(lib):
    """(Numbers in the binding's messages: a module with a C++ library of its own would crash on them.)"""
    z = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16)
    for kw, words in ((dict(L=-1), "L=-1"), (dict(page_size=1 << 31), "page_size=2147483648"), (dict(n_pages=-7), "n_pages=-7")):
        with pytest.raises(ValueError, match=words):
            attn.page_plan(z(2), z(2), z(2, 4), z(8), z(1), **{**dict(L=1, page_size=64, n_pages=8), **kw})
    with pytest.raises(ValueError, match="page_size=-64"):
        attn.page_release(z(2), z(2), z(2, 4), z(8), z(1), page_size=-64, n_pages=8)
    with pytest.raises(ValueError, match="T=-2"):
        attn.tree_commit(bf, bf, z(1), z(1, 2), z(1), T=-2)


def test_sizes_past_32_bit_indexes_are_refused(lib):
    """Rows of a step are counted in steps of up to 1024 past L, and a commit's 16-byte
    columns as 2 * Hkv * D / 8, both in 32 bits."""
    for L in (1 << 30, 2**31 - 1024, 2**31 - 1):
        assert _call(lib.attn_page_plan, PLAN, dict(L=L)) == -2
        assert b"too large" in lib.attn_last_error()
    for Hkv in (1 << 24, 1 << 26, 2**31 - 1):
        assert _call(lib.attn_tree_commit, COMMIT, dict(Hkv=Hkv, D=256)) == -2
        assert b"heads" in lib.attn_last_error()
