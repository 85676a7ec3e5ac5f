"""The serving-step calls over the whole of their documented range: trees of up to 1024
nodes, more query blocks than the GPU holds CTAs, pairs of more partials than one round of
the combine takes, and caches of other page sizes."""
import math

import pytest
import torch

import exact_tiled_attention_gqa_b200 as attn
import serving_ref as ref
import test_serving_step_gpu as step
from test_serving_step_gpu import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.device_error(reset=True)
    yield
    assert attn.device_error(reset=True) == 0


def _reference(q, masks, rows, sizes, scale):
    """ref.tree for many nodes: whole heads at a time, in 64 bits, with its tolerance."""
    B, Hq, T, D = q.shape
    out, tol = (torch.zeros(B, Hq, T, D, dtype=torch.float64) for _ in range(2))
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    for b, (k, v) in enumerate(rows):
        n, size = k.shape[1], sizes[b]
        j = torch.arange(n)[None] - (n - size)                        # tree column of a row
        see = (j < 0) | masks[b % len(masks)].gather(1, j.clamp(0, T - 1).expand(T, n))
        see[size:] = False
        some = see.any(1)
        for h in range(Hq):
            g = h // (Hq // k.shape[0])
            s = (torch.nan_to_num(q[b, h]).double() @ k[g].double().T * scale).masked_fill(~see, -math.inf)
            l = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(some, l, 0.0)[:, None])
            lse[b, h] = torch.where(some, l, -math.inf)
            out[b, h] = p @ v[g].double()
            a = p @ v[g].double().abs()
            tol[b, h] = 2 ** -8 * (a + 2 * out[b, h].abs()) + 4e-4 * (a + out[b, h].abs()) + 1e-30
    return out, lse, tol


def _check(Hq, Hkv, T, D, lens, sizes, kind, page=64, shared=False):
    q, masks, rows = step._tree_case(lens, sizes, Hq, Hkv, T, D, kind, T + D + sum(lens), shared_mask=shared)
    want = _reference(q, masks, rows, sizes, 1 / math.sqrt(D))
    words, sl, tl = attn.pack_tree_mask(masks[0] if shared else masks).cuda(), i32(lens), i32(sizes)
    kp, vp, table = (t.cuda() for t in step._paged(rows, page, T))
    out, lse = attn.decode_tree_paged(q.cuda(), kp, vp, table, sl, words, tree_lens=tl)
    assert attn.device_error(reset=True) == 0
    ref.check_tree(out, lse, want, f"paged D{D} T{T}")
    kc, vc = (t.cuda() for t in step._contiguous(rows, max(lens) + 1))
    out, lse = attn.decode_tree(q.cuda(), kc, vc, sl, words, tree_lens=tl)
    assert attn.device_error(reset=True) == 0
    ref.check_tree(out, lse, want, f"contiguous D{D} T{T}")


def test_reference_is_the_plain_form():
    """The head-at-a-time reference here against the row-by-row one, masks of every kind."""
    for kind, lens, sizes in (("tree", [40, 9], [9, 5]), ("any", [12, 3], [9, 9])):
        q, masks, rows = step._tree_case(lens, [9, 9], 4, 2, 9, 64, kind, 1)
        a = step._reference(q, masks, rows, lens, sizes, 0.125)
        b = _reference(q, masks, rows, sizes, 0.125)
        for x, y in zip(a, b):
            assert torch.equal(x.isinf(), y.isinf()) and (torch.nan_to_num(x) - torch.nan_to_num(y)).abs().max() < 1e-12


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,T,lens,sizes,kind", [
    (4, 2, 257, [1300, 257, 300], [257, 200, 257], "tree"),
    (2, 1, 512, [513, 40], [512, 512], "linear"),               # the second holds fewer rows than its tree has nodes
    (3, 3, 1024, [1024, 1500], [1024, 1000], "tree"),           # a tree over 17 tiles, 32 mask words
    (2, 1, 1024, [1100, 1024], [1024, 33], "any"),              # every third node sees nothing of the tree
])
def test_tree_of_many_nodes(D, Hq, Hkv, T, lens, sizes, kind):
    _check(Hq, Hkv, T, D, lens, sizes, kind)


@pytest.mark.parametrize("D,G", [(64, 40), (128, 40), (256, 20)])
def test_more_query_blocks_than_ctas(D, G):
    """320 (D = 256: 160) blocks of 128 query rows for 296 (148) CTAs at once: one range, every pair whole in it."""
    assert G * 1024 // 128 > (148 if D == 256 else 296)
    _check(G, 1, 1024, D, [1030, 0, 90], [1024, 0, 90], "tree", shared=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,T", [(1, 1, 1), (2, 1, 2), (4, 1, 1), (31, 1, 1), (8, 1, 8), (4, 2, 40)])
def test_many_partials_of_a_pair(D, Hq, Hkv, T):
    """One sequence of 12000 rows, few query rows: a pair's partials fill more than one round of either combine."""
    _check(Hq, Hkv, T, D, [12000], [T], "tree", page=128)


@pytest.mark.parametrize("fmt,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("e4m3", 64), ("e4m3", 128), ("q8_0", 64), ("q8_0", 128)])
@pytest.mark.parametrize("tokens", [(3, 19), (1, 4800)])        # a token and several tokens a CTA
def test_rope_page_sizes(fmt, D, tokens):
    """A slot's row does not depend on the page size: caches of pages of 1 to all rows hold the same rows, bit for bit."""
    (B, L), Hq, Hkv = tokens, 4, 2
    q, k, v, pos, inv, _, sections, _ = step._rope_case(B, L, Hq, Hkv, D, D, 1, 0, 0, fmt, D)
    total = 960 * -(-B * L // 800)
    g = torch.Generator().manual_seed(D)
    slots = torch.randperm(total, generator=g)[:B * L].int().view(B, L)
    slots[torch.rand(B, L, generator=g) < 0.1] = -1
    args = [step._on_gpu(q), step._on_gpu(k), step._on_gpu(v), pos.cuda(), inv.cuda(), slots.cuda()]
    kind = dict(bf16=torch.bfloat16, e4m3=torch.float8_e4m3fn, q8_0=torch.int8)[fmt]
    held = {}
    for page in (64, 1, 15, 192, 320, total):
        shape = (total // page, Hkv, page, D)
        caches = [torch.full(shape, 3.0, device="cuda").to(kind) for _ in range(2)]
        scales = [None, None]
        if fmt == "e4m3":
            scales = [torch.tensor([0.02, 0.013], device="cuda") for _ in range(2)]
        elif fmt == "q8_0":
            scales = [torch.full((*shape[:3], D // 32), 5.0, dtype=torch.float16, device="cuda") for _ in range(2)]
        out = attn.rope_append(*args, *caches, sections=sections, k_scale=scales[0], v_scale=scales[1])
        assert attn.device_error(reset=True) == 0
        by_slot = [t.view(torch.uint8).transpose(1, 2).flatten(0, 1) for t in caches + (scales if fmt == "q8_0" else [])]
        held[page] = [out, *by_slot]
        assert all(torch.equal(a, b) for a, b in zip(held[64], held[page])), page
