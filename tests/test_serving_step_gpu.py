"""GPU parity of the serving-step calls (page_plan, page_release, rope_append,
decode_tree, decode_tree_paged, tree_commit) against plain 64-bit forms, through
the Python binding: sizes from one token up, odd and ragged ones, every cache
format and head dim, masks that leave rows empty, NaN wherever nothing may be
read, strided inputs, inputs the host cannot check, and the calls together as a
serving step makes them, eager and captured into CUDA graphs."""
import math
import os
import random
import subprocess
import sys

import pytest
import torch

import exact_tiled_attention_gqa_b200 as attn
from exact_tiled_attention_gqa_b200 import _native, build
import serving_ref as ref

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.device_error(reset=True)
    yield
    assert attn.device_error(reset=True) == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bf16(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------

def _plan_inputs(B, L, page, max_pages, seed, spare):
    r = random.Random(seed)
    cap = max_pages * page
    lens = [r.choice([0, 1, page - 1, page, page + 1, r.randrange(0, cap + 1), cap]) for _ in range(B)]
    lens = [min(x, cap) for x in lens]
    new = [r.choice([0, min(1, L), L, r.randrange(0, L + 1)]) for _ in range(B)]
    used = [-(-x // page) for x in lens]
    n_pages = sum(used) + spare
    order = list(range(n_pages))
    r.shuffle(order)
    table = [[-7] * max_pages for _ in range(B)]
    for b in range(B):
        for c in range(used[b]):
            table[b][c] = order.pop()
    free = order + [-9] * 5
    return lens, new, table, free, spare, max(1, n_pages)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,L,page,max_pages,spare", [
    (1, 1, 64, 1, 0), (1, 1, 64, 3, 1), (3, 5, 64, 4, 2), (64, 1, 64, 9, 7), (33, 100, 1, 130, 900), (200, 700, 128, 12, 500),
    (1024, 9, 64, 3, 300), (1025, 3, 64, 2, 100), (2500, 2, 256, 2, 1000), (4, 0, 64, 4, 3), (0, 4, 64, 2, 3),
    (5, 3000, 64, 60, 150), (1, 9000, 128, 80, 100), (130, 63, 64, 5, 200),
])
def test_page_plan(B, L, page, max_pages, spare, in_place):
    lens, new, table, free, n_free, n_pages = _plan_inputs(B, L, page, max_pages, B + L + page, spare)
    want = ref.plan(lens, new, table, free, n_free, L, page)
    sl, nf = i32(lens), i32([n_free])
    bt = i32(table) if B else torch.zeros(0, max_pages, dtype=torch.int32, device="cuda")
    extra = dict(out_seqlens=sl, out_n_free=nf) if in_place else {}
    free_t = i32(free)
    got = attn.page_plan(sl, i32(new), bt, free_t, nf, L=L, page_size=page, n_pages=n_pages, **extra)
    assert attn.device_error(reset=True) == 0
    assert free_t.tolist() == free
    assert [bt.tolist(), got[0].tolist(), got[1].tolist(), got[2].item(), got[3].tolist()] == [
        want[0], want[1], want[2], want[3], want[4]]


@pytest.mark.parametrize("B,page,max_pages", [(1, 64, 1), (5, 64, 7), (1000, 64, 5), (1030, 128, 3), (0, 64, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_release(B, page, max_pages, in_place):
    lens, _, table, free, n_free, n_pages = _plan_inputs(B, 1, page, max_pages, B + page, 6)
    r = random.Random(B)
    keep = [r.choice([0, x, r.randrange(0, x + 1)]) for x in lens]
    free = free[:n_free] + [-9] * (n_pages - n_free)
    want_free, want_n = ref.release(lens, keep, table, free, n_free, page)
    free_t, nf = i32(free), i32([n_free])
    bt = i32(table) if B else torch.zeros(0, max_pages, dtype=torch.int32, device="cuda")
    got = attn.page_release(i32(lens), i32(keep), bt, free_t, nf, page_size=page, n_pages=n_pages,
                            out_n_free=nf if in_place else None)
    assert attn.device_error(reset=True) == 0
    assert got.item() == want_n and free_t.tolist() == want_free
    assert bt.tolist() == table


def test_pages_bad_inputs_are_flagged_and_harmless():
    bt, free, nf = i32([[3, -1], [4, -1], [5, -1], [6, -1]]), i32([0, 1, 2, 7]), i32([3])
    args = dict(L=4, page_size=64, n_pages=8)
    # a negative length, one past the table, a new length past L: refused; the sound request is served
    out = attn.page_plan(i32([-1, 129, 64, 64]), i32([1, 0, 5, 1]), bt, free, nf, **args)
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_SEQLEN
    assert out[3].tolist() == [1, 1, 1, 0] and out[2].item() == 2 and bt[3].tolist() == [6, 2]
    assert out[0].tolist() == [[-1] * 4] * 3 + [[2 * 64, -1, -1, -1]] and out[1].tolist() == [-1, 129, 64, 65]
    # an n_free outside the stack is clamped
    for bad, left in ((-3, 0), (99, 4)):
        out = attn.page_plan(i32([1]), i32([1]), i32([[3]]), free, i32([bad]), **args)
        assert attn.device_error(reset=True) == _native.ATTN_DEVERR_PAGE and out[2].item() == left
    # a page outside the pool: no slot
    out = attn.page_plan(i32([1]), i32([2]), i32([[8]]), free, nf, **args)
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_PAGE and out[0].tolist() == [[-1] * 4]
    # release: keep past the length; a stack without room
    assert attn.page_release(i32([64]), i32([65]), i32([[3]]), free.clone(), nf, page_size=64, n_pages=8).item() == 3
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_SEQLEN
    small = free.clone()
    assert attn.page_release(i32([128]), i32([0]), i32([[5, 6]]), small, nf, page_size=64, n_pages=8).item() == 4
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_PAGE and small.tolist() == [0, 1, 2, 5]


# ---------------------------------------------------------------------------
# rotary append
# ---------------------------------------------------------------------------

def _rope_case(B, L, Hq, Hkv, D, rot, axes, cycle, adjacent, fmt, seed, page=64, far=40000, strided=True):
    g = torch.Generator().manual_seed(seed)
    if strided:
        qkv = bf16(g, B, L, (Hq + 2 * Hkv) * D + 8)
        q = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
        k = qkv[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
        v = qkv[..., (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].unflatten(-1, (Hkv, D))
    else:
        q, k, v = bf16(g, B, L, Hq, D), bf16(g, B, L, Hkv, D), bf16(g, B, L, Hkv, D)
    n = rot // 2
    sections = [n - n // axes * (axes - 1)] + [n // axes] * (axes - 1)
    pos = torch.randint(-5, far, (axes, B, L), generator=g, dtype=torch.int32)
    inv = (1e6 ** (-torch.arange(n) / max(1, n))).float()
    n_pages = -(-B * L // page) + 2
    slots = torch.randperm(n_pages * page, generator=g)[:B * L].int().view(B, L)
    slots[torch.rand(B, L, generator=g) < 0.2] = -1
    return q, k, v, pos, inv, slots, sections, n_pages


def _on_gpu(t):
    """The tensor on the GPU with its strides (a part of one projection stays one)."""
    if t._base is None:
        return t.cuda()
    return t._base.cuda().as_strided(t.shape, t.stride(), t.storage_offset())


@pytest.mark.parametrize("B,L,Hq,Hkv,D,rot,axes,cycle,adjacent,fmt", [
    (1, 1, 1, 1, 64, 64, 1, 0, 0, "bf16"), (3, 7, 4, 2, 128, 128, 1, 0, 0, "bf16"), (2, 33, 8, 1, 128, 64, 2, 0, 1, "bf16"),
    (1, 50, 3, 3, 256, 256, 3, 1, 0, "bf16"), (2, 9, 40, 8, 256, 48, 4, 1, 1, "bf16"), (5, 1, 32, 8, 128, 128, 3, 1, 0, "bf16"),
    (2, 17, 6, 2, 64, 0, 1, 0, 0, "bf16"), (1, 4, 2, 2, 128, 16, 4, 0, 0, "bf16"),
    (1, 1, 1, 1, 64, 64, 1, 0, 0, "e4m3"), (2, 31, 16, 4, 128, 96, 2, 0, 1, "e4m3"), (3, 5, 7, 7, 64, 32, 3, 1, 0, "e4m3"),
    (1, 1, 1, 1, 64, 64, 1, 0, 0, "q8_0"), (2, 31, 16, 4, 128, 96, 2, 0, 1, "q8_0"), (3, 5, 7, 7, 64, 48, 3, 1, 0, "q8_0"),
    (4, 16, 12, 3, 128, 128, 4, 0, 0, "q8_0"), (1, 300, 33, 17, 64, 64, 1, 0, 1, "q8_0"),
    # many tokens: several a CTA, the last one with fewer
    (1, 4737, 2, 1, 64, 64, 2, 1, 0, "bf16"), (3, 1603, 3, 2, 128, 96, 1, 0, 1, "e4m3"), (2, 2503, 1, 3, 128, 128, 3, 0, 0, "q8_0"),
    (1, 5001, 1, 1, 256, 64, 4, 0, 1, "bf16"),
])
@pytest.mark.parametrize("strided", [True, False])
def test_rope_append(B, L, Hq, Hkv, D, rot, axes, cycle, adjacent, fmt, strided):
    page = 64
    q, k, v, pos, inv, slots, sections, n_pages = _rope_case(B, L, Hq, Hkv, D, rot, axes, cycle, adjacent, fmt, B * L + D + rot, page,
                                                             strided=strided)
    g = torch.Generator().manual_seed(1)
    shape = (n_pages, Hkv, page, D)
    scales = [None, None]
    if fmt == "bf16":
        caches = [torch.full(shape, NAN, dtype=torch.bfloat16) for _ in range(2)]
    elif fmt == "e4m3":
        caches = [torch.full(shape, NAN).to(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.rand(Hkv, generator=g) * 0.02 + 0.004 for _ in range(2)]     # some values pass 448 scales
    else:
        caches = [torch.full(shape, 77, dtype=torch.int8) for _ in range(2)]
        scales = [torch.full((n_pages, Hkv, page, D // 32), NAN, dtype=torch.float16) for _ in range(2)]
    gc, gs = [c.cuda() for c in caches], [None if s is None else s.cuda() for s in scales]
    out = attn.rope_append(_on_gpu(q), _on_gpu(k), _on_gpu(v), pos.cuda(), inv.cuda(), slots.cuda(), *gc, sections=sections,
                           axis_order="cycle" if cycle else "blocks", pairs="adjacent" if adjacent else "half", k_scale=gs[0],
                           v_scale=gs[1])
    assert attn.device_error(reset=True) == 0
    # fp32 angle and arithmetic: the angle to 2.2e-7 rad (its float's half step at one half turn, 2^-24 pi, and its
    # fixed point), sin and cos to a few 2^-24, three roundings: 1e-6 (|a| + |b|) in all
    y, size = ref.rope(q, pos, inv, sections, cycle, adjacent)
    err = (out.double().cpu().transpose(1, 2) - y).abs()
    assert (err <= 2 ** -8 * y.abs() + 1e-6 * size + 1e-30).all(), err.max()
    assert torch.equal(out.cpu().transpose(1, 2)[..., rot:], q[..., rot:])
    ky, ksize = ref.rope(k, pos, inv, sections, cycle, adjacent)
    kept = slots >= 0
    slot = slots[kept].long()
    for i, (x, size) in enumerate(((ky, ksize), (v.double(), v.double().abs()))):
        x, size = x[kept], 1e-6 * size[kept]
        got = gc[i].cpu()
        rows = got[slot // page, :, slot % page]
        if fmt == "bf16":
            assert ((rows.double() - x).abs() <= 2 ** -8 * x.abs() + size + 1e-30).all()
            if i == 1:
                assert torch.equal(rows, v[kept])
        elif fmt == "e4m3":
            z = (x / scales[i].double()[:, None]).clamp(-448, 448)
            # to nearest: half a step of 2^-3 relative, or of the subnormal step 2^-9
            tol = (2 ** -4 * z.abs()).clamp(min=2 ** -10) + size / scales[i].double()[:, None] * 1.1
            assert ((rows.double() - z).abs() <= tol).all()
        else:
            d = gs[i].cpu()[slot // page, :, slot % page].double()
            blocks = x.unflatten(-1, (-1, 32))
            top = blocks.abs().amax(-1)
            # the scale: max / 127 rounded to fp16 (half a step 2^-11, subnormal half step 2^-25), of a max off by `size`
            slack = size.unflatten(-1, (-1, 32)).amax(-1)
            assert ((d - top / 127).abs() <= 2 ** -11 * top / 127 + 2 ** -25 + slack).all()
            # codes to nearest of the stored scale; the largest may clamp at 127 (127 2^-11 of a scale)
            err = (rows.double().unflatten(-1, (-1, 32)) * d[..., None] - blocks).abs()
            assert (err <= (0.5 + 127 * 2 ** -11) * d[..., None] + 1.1 * slack[..., None]).all()
            left = torch.ones(n_pages * page, dtype=torch.bool)
            left[slot] = False
            assert gs[i].cpu().transpose(1, 2).flatten(0, 1)[left].isnan().all()
        left = torch.ones(n_pages * page, dtype=torch.bool)
        left[slot] = False
        old, new = (c.view(torch.int8).transpose(1, 2).flatten(0, 1)[left] for c in (caches[i], got))
        assert torch.equal(old, new)          # rows no token has are left as they were


@pytest.mark.parametrize("fmt", ["e4m3", "q8_0"])
def test_stored_codes_are_the_quotients_to_nearest(fmt):
    """V's codes, which no rotation precedes, are those of the division itself, to the last one: every bf16 value of
    64K bit patterns but NaN over scales with ties among the quotients, and scales at the ends of float32."""
    D, Hkv = 128, 8
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    bits = torch.where(bits.isnan(), torch.zeros_like(bits), bits)
    g = torch.Generator().manual_seed(0)
    if fmt == "q8_0":
        bits = torch.where(bits.isinf() | (bits.abs() > 8e6), torch.ones_like(bits), bits)
        bits = bits[torch.randperm(1 << 16, generator=g)] * torch.exp2(torch.randint(-30, 3, (1 << 11, 1), generator=g).float()).to(
            torch.bfloat16).expand(-1, 32).reshape(-1)
        bits = torch.where(bits.abs() > 8e6, torch.ones_like(bits), bits)
    L = (1 << 16) // D
    v = bits.view(1, L, 1, D).expand(1, L, Hkv, D).contiguous()
    slots = torch.arange(L).int().view(1, L)
    n_pages = -(-L // 64)
    inv, pos = torch.zeros(0), torch.zeros(1, L, dtype=torch.int32)
    args = [t.cuda() for t in (v, v, v, pos, inv, slots)]
    if fmt == "e4m3":
        scale = torch.tensor([1.0, 0.75, 0.1, 3.0, 1e-3, 1.7e-38, 3e38, 2.0 ** -40])
        kc, vc = (torch.zeros(n_pages, Hkv, 64, D, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
        attn.rope_append(*args, kc, vc, k_scale=scale.cuda(), v_scale=scale.cuda())
        want = (v.float() / scale[None, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        for c in (kc, vc):
            got = c.cpu().transpose(1, 2).flatten(0, 1)[:L]
            assert torch.equal(got.view(torch.int8), want[0].view(torch.int8))
    else:
        kc, vc = (torch.zeros(n_pages, Hkv, 64, D, dtype=torch.int8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros(n_pages, Hkv, 64, D // 32, dtype=torch.float16, device="cuda") for _ in range(2))
        attn.rope_append(*args, kc, vc, k_scale=ks, v_scale=vs)
        x = v[0].float().unflatten(-1, (-1, 32))
        d = (x.abs().amax(-1) / 127).half()
        want = torch.where(d[..., None] > 0, (x / d[..., None].float()).round().clamp(-127, 127), torch.zeros_like(x)).to(torch.int8)
        for c, sc in ((kc, ks), (vc, vs)):
            assert torch.equal(sc.cpu().transpose(1, 2).flatten(0, 1)[:L], d)
            assert torch.equal(c.cpu().transpose(1, 2).flatten(0, 1)[:L], want.flatten(-2))
    assert attn.device_error(reset=True) == 0


def test_rope_far_positions_and_special_values():
    """Angles at the ends of int32 hold to 3e-6 rad (2^31 2^-52 f turns more than near ones); infinities and NaN come
    through; a contiguous cache is a pool of B slabs; a slot past the cache is flagged and not written."""
    D, n = 128, 64
    g = torch.Generator().manual_seed(3)
    q, k, v = bf16(g, 1, 6, 2, D), bf16(g, 1, 6, 1, D), bf16(g, 1, 6, 1, D)
    pos = torch.tensor([[[2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, -1, 0, 1]]], dtype=torch.int32)
    inv = (1e4 ** (-torch.arange(n) / n)).float()
    slots = torch.tensor([[5, 0, 63, 64, -2 ** 31, 2 ** 31 - 1]], dtype=torch.int32)
    kc, vc = (torch.full((1, 1, 64, D), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = attn.rope_append(q.cuda(), k.cuda(), v.cuda(), pos.cuda(), inv.cuda(), slots.cuda(), kc, vc)
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_PAGE
    y, size = ref.rope(q, pos, inv, [n], 0, 0)
    err = (out.double().cpu().transpose(1, 2) - y).abs()
    assert (err <= 2 ** -8 * y.abs() + 3e-6 * size).all()
    assert torch.equal(vc[0, 0, [5, 0, 63]].cpu(), v[0, :3, 0]) and vc[0, 0].isnan().all(-1).sum() == 61
    # NaN and infinity in one pair reach that pair alone; a NaN frequency its pair in every token
    q[0, 1, 0, 3], q[0, 2, 1, 70] = NAN, math.inf
    inv[9] = NAN
    out = attn.rope_append(q.cuda(), k.cuda(), v.cuda(), pos.cuda(), inv.cuda(), (slots * 0 - 1).cuda(), kc, vc).cpu()
    assert attn.device_error(reset=True) == 0
    bad = ~torch.isfinite(out[0].transpose(0, 1))
    want = torch.zeros(6, 2, D, dtype=torch.bool)
    want[..., [9, 9 + n]] = True
    want[1, 0, [3, 3 + n]] = True
    want[2, 1, [6, 6 + n]] = True
    assert torch.equal(bad, want)


def test_q8_0_special_values():
    """A block of zeros has scale 0 and codes 0; a NaN makes its block NaN and no other; an infinity saturates."""
    D = 64
    x = torch.zeros(1, 4, 1, D, dtype=torch.bfloat16)
    x[0, 1, 0, 5] = NAN
    x[0, 2, 0, 40], x[0, 2, 0, 41] = math.inf, -1.0
    x[0, 3, 0, :] = 1e-30
    codes = [torch.full((1, 1, 64, D), 9, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.full((1, 1, 64, 2), 9, dtype=torch.float16, device="cuda") for _ in range(2)]
    attn.rope_append(x.cuda(), x.cuda(), x.cuda(), i32([[0, 0, 0, 0]]), torch.ones(32, device="cuda"), i32([[0, 1, 2, 3]]), *codes,
                     k_scale=scales[0], v_scale=scales[1])
    assert attn.device_error(reset=True) == 0
    held = codes[1].float().unflatten(-1, (2, 32)) * scales[1].float().unsqueeze(-1)
    held = held[0, 0, :4].cpu()
    assert (held[0] == 0).all() and held[1, 0].isnan().all() and (held[1, 1] == 0).all()
    assert (held[2, 0] == 0).all() and held[2, 1, 8] == 65504 * 127.0 and (held[3] == 0).all()


def test_rope_refusals():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    inv = torch.ones(64, device="cuda")
    q, k, c = bf(2, 3, 4, 128), bf(2, 3, 2, 128), bf(4, 2, 64, 128)
    ok = dict(q=q, k=k, v=k, positions=z(1, 2, 3), inv_freq=inv, slots=z(2, 3) - 1, k_cache=c, v_cache=c.clone())
    attn.rope_append(**ok)
    bad = [dict(k=bf(2, 3, 2, 64)), dict(v=bf(2, 3, 1, 128)), dict(q=bf(2, 3, 128, 4).transpose(2, 3)), dict(q=bf(3, 2, 4, 128).transpose(0, 1)),
           dict(positions=z(1, 2, 4)), dict(slots=z(3, 2)), dict(k_cache=bf(4, 1, 64, 128)), dict(v_cache=bf(5, 2, 64, 128)),
           dict(k_scale=torch.ones(2, device="cuda")), dict(sections=[32, 32]), dict(axis_order="rows"), dict(pairs="both"),
           dict(positions=z(2, 2, 3)), dict(out=bf(2, 3, 4, 128)), dict(sections=[-1])]
    for kw in bad:
        with pytest.raises(ValueError):
            attn.rope_append(**{**ok, **kw})
    for kw in (dict(sections=[63]), dict(positions=z(2, 2, 3), sections=[32, 31]), dict(positions=z(2, 2, 3), sections=[1, 63], axis_order="cycle"),
               dict(inv_freq=torch.ones(4, device="cuda")), dict(positions=z(5, 2, 3), sections=[64, 0, 0, 0, 0])):
        with pytest.raises(attn.AttnError):
            attn.rope_append(**{**ok, **kw})
    for kw in (dict(k_cache=c.float(), v_cache=c.float()), dict(positions=z(1, 2, 3).long()), dict(inv_freq=inv.double())):
        with pytest.raises(TypeError):
            attn.rope_append(**{**ok, **kw})


# ---------------------------------------------------------------------------
# tree attention
# ---------------------------------------------------------------------------

def _random_mask(r, T, kind):
    m = torch.zeros(T, T, dtype=torch.bool)
    if kind == "tree":
        for i in range(T):
            if i:
                m[i] = m[r.randrange(max(0, i - 4), i)]
            m[i, i] = True
    elif kind == "linear":
        m = torch.ones(T, T, dtype=torch.bool).tril()
    elif kind == "any":                      # not a tree at all: any bits, some rows empty
        m = torch.tensor([[r.random() < 0.4 for _ in range(T)] for _ in range(T)]).view(T, T)
        m[::3] = False
    return m


def _tree_case(lens, sizes, Hq, Hkv, T, D, kind, seed, shared_mask=False):
    """CPU inputs with NaN in every row behind a sequence; rows as [B][Hkv,n,D]."""
    g, r = torch.Generator().manual_seed(seed), random.Random(seed)
    B = len(lens)
    q = bf16(g, B, Hq, T, D)
    masks = torch.stack([_random_mask(r, T, kind) for _ in range(1 if shared_mask else B)])
    rows = [(bf16(g, Hkv, n, D), bf16(g, Hkv, n, D)) for n in lens]
    for b, size in enumerate(sizes):         # what is behind a tree must not matter
        q[b, :, size:] = NAN
    return q, masks, rows


def _contiguous(rows, Lmax):
    kc, vc = (torch.full((len(rows), rows[0][0].shape[0], Lmax, rows[0][0].shape[2]), NAN, dtype=torch.bfloat16) for _ in range(2))
    for b, (k, v) in enumerate(rows):
        kc[b, :, :k.shape[1]], vc[b, :, :k.shape[1]] = k, v
    return kc, vc


def _paged(rows, page, seed):
    g = torch.Generator().manual_seed(seed)
    used = [-(-k.shape[1] // page) for k, _ in rows]
    n_pages = sum(used) + 2
    order = torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((len(rows), max(1, max(used)) + 1), -1, dtype=torch.int32)
    kp, vp = (torch.full((n_pages, rows[0][0].shape[0], page, rows[0][0].shape[2]), NAN, dtype=torch.bfloat16) for _ in range(2))
    for b, (k, v) in enumerate(rows):
        for c in range(used[b]):
            pg = table[b, c] = order.pop()
            m = min(page, k.shape[1] - c * page)
            kp[pg, :, :m], vp[pg, :, :m] = k[:, c * page:c * page + m], v[:, c * page:c * page + m]
    return kp, vp, table


def _reference(q, masks, rows, lens, sizes, scale):
    refs = [ref.tree(q[b], *rows[b], ref.tree_sees(lens[b], sizes[b], q.shape[2], masks[b % len(masks)]), scale) for b in range(len(lens))]
    return [torch.stack([x[i] for x in refs]) for i in range(3)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,T,lens,sizes,kind", [
    (1, 1, 1, [1], [1], "tree"),
    (4, 2, 1, [200, 1, 0, 64], [1, 1, 0, 0], "tree"),
    (8, 2, 8, [500, 8, 71, 129], [8, 8, 7, 1], "tree"),
    (4, 4, 16, [64, 65, 16, 80], [16, 16, 16, 16], "linear"),
    (6, 2, 33, [700, 33, 96, 40], [33, 20, 32, 33], "tree"),
    (16, 2, 63, [300, 63], [63, 31], "tree"),          # 504 query rows a KV head: four blocks, the last short
    (3, 1, 64, [64, 130, 1000], [64, 64, 64], "any"),
    (2, 1, 65, [1100, 66], [65, 65], "any"),
    (5, 1, 130, [200, 130], [130, 77], "tree"),        # a tree over three tiles
    (8, 1, 16, [5, 3, 0], [16, 16, 16], "tree"),       # fewer rows than nodes: the first nodes have none
])
def test_tree_against_plain(D, Hq, Hkv, T, lens, sizes, kind):
    q, masks, rows = _tree_case(lens, sizes, Hq, Hkv, T, D, kind, T + D + Hq)
    scale = 1 / math.sqrt(D)
    want = _reference(q, masks, rows, lens, sizes, scale)
    words, sl, tl = attn.pack_tree_mask(masks).cuda(), i32(lens), i32(sizes)
    Lmax = max(lens) + 3
    kc, vc = (t.cuda() for t in _contiguous(rows, Lmax))
    out, lse = attn.decode_tree(q.cuda(), kc, vc, sl, words, tree_lens=tl)
    assert attn.device_error(reset=True) == 0
    ref.check_tree(out, lse, want, f"contiguous D{D} T{T}")
    for page in (64, 192):
        kp, vp, table = (t.cuda() for t in _paged(rows, page, T + page))
        po, pl = attn.decode_tree_paged(q.cuda(), kp, vp, table, sl, words, tree_lens=tl)
        assert attn.device_error(reset=True) == 0
        ref.check_tree(po, pl, want, f"page {page} D{D} T{T}")
    # the same answer, bit for bit, every time
    again, lagain = attn.decode_tree(q.cuda(), kc, vc, sl, words, tree_lens=tl)
    assert torch.equal(again, out) and torch.equal(lagain, lse)


@pytest.mark.parametrize("D,B,Hq,Hkv,T,top", [(64, 150, 8, 8, 3, 200), (128, 120, 16, 8, 5, 300), (256, 100, 8, 8, 2, 260), (128, 40, 40, 8, 30, 150),
                                             (64, 300, 4, 4, 1, 140)])
def test_tree_many_short_sequences(D, B, Hq, Hkv, T, top):
    """More (sequence, KV head) pairs than CTAs: a CTA takes several, whole or in part, some sequences are empty."""
    r = random.Random(B)
    lens = [r.choice([0, 1, 63, 64, 65, r.randrange(0, top)]) for _ in range(B)]
    sizes = [min(n, r.randrange(0, T + 1)) for n in lens]
    q, masks, rows = _tree_case(lens, sizes, Hq, Hkv, T, D, "tree", B)
    want = _reference(q, masks, rows, lens, sizes, 1 / math.sqrt(D))
    words, sl, tl = attn.pack_tree_mask(masks).cuda(), i32(lens), i32(sizes)
    kp, vp, table = (t.cuda() for t in _paged(rows, 64, B))
    out, lse = attn.decode_tree_paged(q.cuda(), kp, vp, table, sl, words, tree_lens=tl)
    assert attn.device_error(reset=True) == 0
    ref.check_tree(out, lse, want, f"B{B} D{D}")
    kc, vc = (t.cuda() for t in _contiguous(rows, max(lens)))
    out, lse = attn.decode_tree(q.cuda(), kc, vc, sl, words, tree_lens=tl)
    ref.check_tree(out, lse, want, f"B{B} D{D} contiguous")


def test_tree_defaults_shared_mask_results_and_scale():
    """tree_lens None is T for all; a [T,W] mask serves every sequence; out, lse and workspace are the caller's."""
    Hq, Hkv, T, D, lens = 8, 4, 20, 128, [300, 20, 77]
    q, masks, rows = _tree_case(lens, [T] * 3, Hq, Hkv, T, D, "tree", 5, shared_mask=True)
    want = _reference(q, masks, rows, lens, [T] * 3, 0.25)
    kc, vc = (t.cuda() for t in _contiguous(rows, 300))
    out, lse = torch.empty_like(q, device="cuda"), torch.empty(3, Hq, T, device="cuda")
    ws = torch.full((attn.decode_tree_workspace_size(3, Hq, Hkv, T, 300, D),), 255, dtype=torch.uint8, device="cuda")   # NaN bytes
    o, l = attn.decode_tree(q.cuda(), kc, vc, i32(lens), attn.pack_tree_mask(masks[0]).cuda(), scale=0.25, out=out, lse=lse, workspace=ws)
    assert o is out and l is lse
    # scores four times the usual: so is their fp32 error, within the tolerances' slack (lse: 1.6e-3 > 4e-4), so lse goes by parts
    assert ((out.double().cpu() - want[0]).abs() <= want[2] * 1.0 + 1.2e-3 * want[2] * 2 ** 8).all()
    assert (lse.double().cpu() - want[1]).abs().max() <= 4 * ref.LSE_TOL
    o2, l2 = attn.decode_tree(q.cuda(), kc, vc, i32(lens), attn.pack_tree_mask(masks[0]).cuda(), scale=0.25, want_lse=False)
    assert l2 is None and torch.equal(o2, out)


def test_linear_tree_is_decode_mq():
    """A chain's mask gives decode_mq's attention (both against the plain form's tolerance)."""
    Hq, Hkv, T, D, lens = 16, 4, 7, 128, [900, 7, 64, 3]
    q, masks, rows = _tree_case(lens, [T] * 4, Hq, Hkv, T, D, "linear", 6, shared_mask=True)
    kc, vc = (t.cuda() for t in _contiguous(rows, 900))
    want = _reference(q, masks, rows, lens, [T] * 4, 1 / math.sqrt(D))
    ref.check_tree(*attn.decode_tree(q.cuda(), kc, vc, i32(lens), attn.pack_tree_mask(masks[0]).cuda()), want, "tree")
    ref.check_tree(*attn.decode_mq(q.cuda(), kc, vc, i32(lens)), want, "mq")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("paged", [False, True])
def test_tree_rows_with_nan_and_infinity_reach_only_their_nodes(D, paged):
    """NaN and infinities in K or V of a tree row reach the nodes that see it, in their columns, and no other."""
    Hq, Hkv, T, n = 8, 2, 40, 171                       # the tree lies over two tiles
    q, masks, rows = _tree_case([n, 90], [T, T], Hq, Hkv, T, D, "tree", 9)
    k, v = rows[0]
    c = n - T
    clean = _reference(q, masks, rows, [n, 90], [T, T], 1 / math.sqrt(D))
    v[0, c + 5, 3], v[0, c + 30, 7], v[1, c + 12, 0] = NAN, math.inf, -math.inf
    k[1, c + 20, 1] = NAN
    if paged:
        kp, vp, table = (t.cuda() for t in _paged(rows, 64, 3))
        out, lse = attn.decode_tree_paged(q.cuda(), kp, vp, table, i32([n, 90]), attn.pack_tree_mask(masks).cuda())
    else:
        kc, vc = (t.cuda() for t in _contiguous(rows, n))
        out, lse = attn.decode_tree(q.cuda(), kc, vc, i32([n, 90]), attn.pack_tree_mask(masks).cuda())
    assert attn.device_error(reset=True) == 0
    out, lse = out.cpu(), lse.cpu()
    m, G = masks[0], Hq // Hkv
    lost = torch.zeros(2, Hq, T, D, dtype=torch.bool)
    for h in range(Hq):
        for i in range(T):
            g = h // G
            if g == 0 and m[i, 5]:
                assert out[0, h, i, 3].isnan()
                lost[0, h, i, 3] = True
            if g == 0 and m[i, 30]:
                assert out[0, h, i, 7] == math.inf
                lost[0, h, i, 7] = True
            if g == 1 and m[i, 20]:
                assert out[0, h, i].isnan().all() and lse[0, h, i].isnan()
                lost[0, h, i] = True
            elif g == 1 and m[i, 12]:
                assert out[0, h, i, 0] == -math.inf
                lost[0, h, i, 0] = True
    err = (out.double() - clean[0]).abs()
    assert (err[~lost] <= clean[2][~lost]).all()
    ok = ~lost.all(-1)
    assert (lse.double() - clean[1]).abs()[ok].max() <= ref.LSE_TOL


def test_tree_bad_device_inputs_are_flagged():
    """Lengths and pages the host cannot check: clamped or replaced, flagged, never read out of bounds."""
    q, masks, rows = _tree_case([100, 60], [5, 5], 4, 2, 5, 64, "tree", 1)
    words = attn.pack_tree_mask(masks).cuda()
    q = torch.nan_to_num(q).cuda()
    kc, vc = (t.cuda() for t in _contiguous(rows, 100))
    want, _ = attn.decode_tree(q, kc, vc, i32([100, 60]), words, tree_lens=i32([5, 0]))
    got, _ = attn.decode_tree(q, kc, vc, i32([101, 60]), words, tree_lens=i32([5, 0]))
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_SEQLEN and torch.equal(got, want)
    got, _ = attn.decode_tree(q, kc, vc, i32([100, 60]), words, tree_lens=i32([6, -1]))
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_INDEX and torch.equal(got, want)
    kp, vp, table = (t.cuda() for t in _paged(rows, 64, 1))
    table[0, 1] = 10_000
    attn.decode_tree_paged(q, kp, vp, table, i32([100, 60]), words)
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_PAGE


def test_tree_refusals():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    q, c, sl, m = bf(2, 4, 5, 64), bf(2, 2, 100, 64), i32([100, 60]), torch.zeros(2, 5, 1, dtype=torch.int32, device="cuda")
    for bad in (m[:1].contiguous(), m[:, :4].contiguous(), torch.zeros(2, 5, 2, dtype=torch.int32, device="cuda"), m[0, 0]):
        with pytest.raises(ValueError):
            attn.decode_tree(q, c, c, sl, bad)
    with pytest.raises(TypeError):
        attn.decode_tree(q, c, c, sl, m.long())
    with pytest.raises(ValueError):
        attn.decode_tree(q, c, c, sl, m, tree_lens=i32([5]))
    with pytest.raises(ValueError):
        attn.decode_tree(q, c, c, sl, m, out=bf(2, 4, 4, 64))
    with pytest.raises(ValueError):
        attn.decode_tree(q, bf(2, 2, 100, 128), bf(2, 2, 100, 128), sl, m)
    with pytest.raises(attn.AttnError, match="workspace"):
        attn.decode_tree(q, c, c, sl, m, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(attn.AttnError, match="nodes"):
        attn.decode_tree(bf(1, 2, 1025, 64), bf(1, 2, 64, 64), bf(1, 2, 64, 64), i32([64]),
                         torch.zeros(1025, 33, dtype=torch.int32, device="cuda"))
    with pytest.raises(attn.AttnError, match="page_size"):
        attn.decode_tree_paged(q, bf(4, 2, 96, 64), bf(4, 2, 96, 64), i32([[0, 1], [2, 3]]), sl, m)


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("D,Hkv,T,A,page,ragged", [
    (64, 1, 1, 1, 0, False), (128, 8, 16, 5, 0, False), (128, 2, 64, 17, 64, True), (256, 3, 40, 40, 128, True), (64, 4, 130, 9, 64, True),
    (128, 1, 8, 0, 64, False),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_tree_commit(D, Hkv, T, A, page, ragged, in_place):
    r = random.Random(T + A)
    g = torch.Generator().manual_seed(T)
    B = 7
    sizes = [T if not ragged else r.randrange(1, T + 1) for _ in range(B)]
    sizes[0] = T
    lens = [s + r.choice([0, 1, 63, r.randrange(0, 300)]) for s in sizes]
    paths = []
    for s in sizes:
        n = r.choice([0, min(A, s), r.randrange(0, min(A, s) + 1)])
        paths.append(sorted(r.sample(range(s), n)))
    rows = [(bf16(g, Hkv, n, D), bf16(g, Hkv, n, D)) for n in lens]
    if page:
        kc, vc, table = _paged(rows, page, 2)
    else:
        (kc, vc), table = _contiguous(rows, max(lens) + 2), None
    kc, vc = torch.nan_to_num(kc, 7.0).cuda(), torch.nan_to_num(vc, 7.0).cuda()
    want = [kc.cpu().clone(), vc.cpu().clone()]
    for b, path in enumerate(paths):
        for w, x in zip(want, rows[b]):
            for j, node in enumerate(path):
                to, frm = lens[b] - sizes[b] + j, lens[b] - sizes[b] + node
                if page:
                    w[table[b, to // page], :, to % page] = x[:, frm]
                else:
                    w[b, :, to] = x[:, frm]
    sl = i32(lens)
    acc = torch.tensor([p + [-5] * (A - len(p)) for p in paths], dtype=torch.int32, device="cuda").view(B, A)
    out = attn.tree_commit(kc, vc, sl, acc, i32([len(p) for p in paths]), T=T, block_table=None if table is None else table.cuda(),
                           tree_lens=i32(sizes) if ragged else None, out_seqlens=sl if in_place else None)
    assert attn.device_error(reset=True) == 0
    assert out.tolist() == [n - s + len(p) for n, s, p in zip(lens, sizes, paths)]
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


def test_tree_commit_bad_paths_move_nothing():
    D, T = 64, 6
    c = torch.randn(9, 1, 64, D, device="cuda").to(torch.bfloat16)
    was = c.clone()
    lens = [10, 10, 10, 10, 5, 10, 65, -1, 10]
    acc = [[0, 2, 1], [0, 0, 1], [-1, 2, 3], [1, 2, 6], [1, 2, 3], [1, 2, 3], [1, 2, 3], [1, 2, 3], [3, 4, 5]]
    n = [3, 3, 3, 3, 3, 4, 3, 3, -1]
    out = attn.tree_commit(c, c.clone(), i32(lens), i32(acc), i32(n), T=T)
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_INDEX | _native.ATTN_DEVERR_SEQLEN
    assert out.tolist() == lens and torch.equal(c, was)
    # a page outside the pool: its rows stay
    attn.tree_commit(c, c.clone(), i32([70]), i32([[1]]), i32([1]), T=T, block_table=i32([[0, 99]]))
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_PAGE and torch.equal(c, was)


def test_commit_refusals():
    c = torch.zeros(2, 1, 64, 64, dtype=torch.bfloat16, device="cuda")
    sl, acc, n = i32([10, 10]), i32([[0], [0]]), i32([1, 1])
    for kw in (dict(seqlens=i32([10])), dict(accept=i32([[0]])), dict(n_accept=i32([1])), dict(v_cache=c[:1].contiguous()),
               dict(block_table=i32([[0]])), dict(tree_lens=i32([1])), dict(out_seqlens=i32([0])), dict(T=-1), dict(T=1 << 31)):
        with pytest.raises(ValueError):
            attn.tree_commit(**{**dict(k_cache=c, v_cache=c.clone(), seqlens=sl, accept=acc, n_accept=n, T=4), **kw})
    with pytest.raises(attn.AttnError):
        attn.tree_commit(c, c.clone(), sl, acc, n, T=0)


def test_empty_batches():
    """No requests, no tokens: every call returns its empty results and touches nothing."""
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    out, lse = attn.decode_tree(bf(0, 4, 3, 64), bf(0, 2, 9, 64), bf(0, 2, 9, 64), z(0), z(0, 3, 1))
    assert out.shape == (0, 4, 3, 64) and lse.shape == (0, 4, 3)
    out, lse = attn.decode_tree_paged(bf(0, 4, 3, 64), bf(2, 2, 64, 64), bf(2, 2, 64, 64), z(0, 3), z(0), z(3, 1))
    assert out.shape == (0, 4, 3, 64)
    pool = torch.ones(2, 2, 64, 64, dtype=torch.bfloat16, device="cuda")
    for B, L in ((0, 5), (5, 0)):
        q = attn.rope_append(bf(B, L, 4, 64), bf(B, L, 2, 64), bf(B, L, 2, 64), z(B, L), torch.ones(32, device="cuda"), z(B, L), pool, pool.clone())
        assert q.shape == (B, 4, L, 64)
    assert attn.tree_commit(pool, pool.clone(), z(0), z(0, 2), z(0), T=4, block_table=z(0, 2)).shape == (0,)
    assert (pool == 1).all() and attn.device_error(reset=True) == 0


def test_every_sequence_empty():
    """Lengths of zero everywhere: nothing is read, every row is 0 and -inf."""
    B, Hq, Hkv, T, D = 5, 12, 2, 30, 128
    q = torch.full((B, Hq, T, D), NAN, dtype=torch.bfloat16, device="cuda")
    c = torch.full((B, Hkv, 70, D), NAN, dtype=torch.bfloat16, device="cuda")
    out, lse = attn.decode_tree(q, c, c, i32([0] * B), torch.full((T, 1), -1, dtype=torch.int32, device="cuda"))
    assert attn.device_error(reset=True) == 0 and (out == 0).all() and (lse == -math.inf).all()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

class _Server:
    """The state of a serving loop: a pool of pages, request lengths, a free list, all on the GPU."""

    def __init__(self, B, Hq, Hkv, D, T, A, prompt, page=64, max_pages=8, seed=0):
        self.B, self.Hq, self.Hkv, self.D, self.T, self.A, self.page = B, Hq, Hkv, D, T, A, page
        self.n_pages = B * max_pages
        g = torch.Generator().manual_seed(seed)
        shape = (self.n_pages, Hkv, page, D)
        self.k, self.v = (torch.full(shape, NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(self.n_pages, generator=g).int().cuda()
        self.n_free, self.lens = i32([self.n_pages]), i32([0] * B)
        self.inv = (1e4 ** (-torch.arange(D // 2) / (D // 2))).float().cuda()
        self.new = i32(prompt)
        self.L = max(prompt)
        # buffers of the step
        self.qkv = torch.zeros(B, T, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device="cuda")
        self.depth = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        self.sizes, self.mask = i32([T] * B), torch.zeros(B, T, -(-T // 32), dtype=torch.int32, device="cuda")
        self.accept, self.n_accept = torch.zeros(B, A, dtype=torch.int32, device="cuda"), i32([0] * B)
        self.full, self.status = i32([0] * B), i32([0] * B)

    def split(self, qkv):
        q, k, v = qkv.split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], -1)
        return (x.unflatten(-1, (-1, self.D)) for x in (q, k, v))

    def prompt(self, qkv):
        slots, *_ = attn.page_plan(self.lens, self.new, self.table, self.free, self.n_free, L=self.L, page_size=self.page,
                                   n_pages=self.n_pages, out_seqlens=self.lens, out_n_free=self.n_free)
        pos = torch.arange(self.L, dtype=torch.int32, device="cuda").expand(self.B, -1).contiguous()
        return attn.rope_append(*self.split(qkv), pos, self.inv, slots, self.k, self.v)

    def verify(self, stream=None):
        """One step: pages for the drafted nodes, their rows, their attention, the accepted path, pages back."""
        pos = self.lens[:, None] + self.depth
        slots, *_ = attn.page_plan(self.lens, self.sizes, self.table, self.free, self.n_free, L=self.T, page_size=self.page,
                                   n_pages=self.n_pages, out_seqlens=self.full, out_n_free=self.n_free, status=self.status)
        q = attn.rope_append(*self.split(self.qkv), pos, self.inv, slots, self.k, self.v)
        out, lse = attn.decode_tree_paged(q, self.k, self.v, self.table, self.full, self.mask, tree_lens=self.sizes)
        attn.tree_commit(self.k, self.v, self.full, self.accept, self.n_accept, T=self.T, block_table=self.table, tree_lens=self.sizes,
                         out_seqlens=self.lens)
        attn.page_release(self.full, self.lens, self.table, self.free, self.n_free, page_size=self.page, n_pages=self.n_pages,
                          out_n_free=self.n_free)
        return out, lse


def _drafts(r, g, s):
    """A step's random trees and accepted paths (root to a node), as CPU tensors."""
    sizes = [r.randrange(1, s.T + 1) for _ in range(s.B)]
    mask, depth = torch.zeros(s.B, s.T, s.T, dtype=torch.bool), torch.zeros(s.B, s.T, dtype=torch.int32)
    accept, n_accept = torch.full((s.B, s.A), -1, dtype=torch.int32), []
    for b in range(s.B):
        for i in range(s.T):
            if i:
                up = r.randrange(max(0, i - 3), i)
                mask[b, i], depth[b, i] = mask[b, up], depth[b, up] + 1
            mask[b, i, i] = True
        path = mask[b, r.randrange(sizes[b])].nonzero().flatten().tolist()[:s.A]
        accept[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
        n_accept.append(len(path))
    return sizes, mask, depth, accept, torch.tensor(n_accept, dtype=torch.int32), bf16(g, *s.qkv.shape)


def _load(s, drafts):
    sizes, mask, depth, accept, n_accept, qkv = drafts
    s.sizes.copy_(torch.tensor(sizes))
    s.mask.copy_(attn.pack_tree_mask(mask))
    s.depth.copy_(depth), s.accept.copy_(accept), s.n_accept.copy_(n_accept), s.qkv.copy_(qkv)


PROMPT = [70, 1, 64, 0, 129]


def test_serving_loop_against_plain():
    """Prompts, then four verify steps; every step's attention is the plain attention over the rows that a list per
    request holds, and after the last step decode_paged reads the same rows."""
    r, g = random.Random(4), torch.Generator().manual_seed(4)
    s = _Server(5, 8, 2, 64, 12, 4, PROMPT)
    qkv = bf16(g, 5, s.L, (s.Hq + 2 * s.Hkv) * s.D)
    s.prompt(qkv.cuda())

    def turned(x, pos):     # as the library rounds it: once, to bf16
        return ref.rope(x, pos, s.inv.cpu(), [s.D // 2], 0, 0)[0].to(torch.bfloat16)

    def rows_of(x, pos):    # -> K, V rows [B, L, Hkv, D]
        q, k, v = s.split(x)
        return turned(q, pos), turned(k, pos), v

    pos = torch.arange(s.L).int().expand(1, 5, -1)
    _, k, v = rows_of(qkv, pos)
    held = [(k[b, :n].transpose(0, 1), v[b, :n].transpose(0, 1)) for b, n in enumerate(PROMPT)]
    # K held here may differ from the library's by one bf16 rounding at a tie of the fp32 value: half a step more on K
    for _ in range(4):
        drafts = _drafts(r, g, s)
        _load(s, drafts)
        out, lse = s.verify()
        assert attn.device_error(reset=True) == 0 and s.status.sum() == 0
        sizes, mask, depth, accept, n_accept, x = drafts
        lens = [h[0].shape[1] for h in held]
        q, k, v = rows_of(x, (torch.tensor(lens)[:, None] + depth).int()[None])
        rows = [tuple(torch.cat((h, y[b, :sizes[b]].transpose(0, 1)), 1) for h, y in zip(held[b], (k, v))) for b in range(5)]
        want = _reference(q.transpose(1, 2), mask, rows, [a.shape[1] for a, _ in rows], sizes, 1 / math.sqrt(s.D))
        # a few of q and K round the other way: scores move by up to 2^-7 |q k| scale where they do, rarely; allow for
        # one such element in each score, 2^-7 * 4 * 4 / 8 = 1.6e-2 at most, as a relative error of the weights
        slack = 2 * 1.6e-2 * (want[2] / 2 ** -8)
        o, l = out.double().cpu(), lse.double().cpu()
        assert torch.equal(l > -math.inf, want[1] > -math.inf)
        assert ((o - want[0]).abs() <= want[2] + slack).all()
        seen = want[1] > -math.inf
        assert (l - want[1])[seen].abs().max() <= ref.LSE_TOL + 1.6e-2
        held = []
        for b in range(5):
            ids = list(range(lens[b])) + [lens[b] + i for i in accept[b, :n_accept[b]].tolist()]
            held.append(tuple(x[:, ids] for x in rows[b]))
        assert s.lens.tolist() == [h[0].shape[1] for h in held]
        # pages: every page is free or in a table, once
        used = [-(-n // s.page) for n in s.lens.tolist()]
        pages = s.free[:s.n_free.item()].tolist() + [p for b, u in enumerate(used) for p in s.table[b, :u].tolist()]
        assert sorted(pages) == list(range(s.n_pages))
    for b in range(5):      # the rows themselves
        for c, h in zip((s.k, s.v), held[b]):
            n = h.shape[1]
            got = c[s.table[b, :-(-n // s.page)].long()].transpose(0, 1).flatten(1, 2)[:, :n].cpu()
            assert ((got.double() - h.double()).abs() <= 2 ** -7 * h.double().abs() + 1e-6).all()
    q = bf16(g, 5, s.Hq, 1, s.D)
    got = attn.decode_paged(q.cuda(), s.k, s.v, s.table, s.lens)
    tree = attn.decode_tree_paged(q.cuda(), s.k, s.v, s.table, s.lens, torch.ones(1, 1, dtype=torch.int32, device="cuda"))
    assert (got[0].float() - tree[0].float()).abs().max() <= 2 ** -7 * got[0].float().abs().max()


def test_serving_step_captured():
    """The whole step in a CUDA graph, replayed with new drafts in its buffers, is the eager step bit for bit."""
    eager, graph = (_Server(5, 8, 2, 128, 12, 4, PROMPT, seed=1) for _ in range(2))
    g = torch.Generator().manual_seed(8)
    qkv = bf16(g, 5, eager.L, (eager.Hq + 2 * eager.Hkv) * eager.D).cuda()
    for s in (eager, graph):
        s.prompt(qkv)
    r = random.Random(8)
    drafts = [_drafts(r, g, eager) for _ in range(4)]
    for s in (eager, graph):
        _load(s, drafts[0])
    want, got = [eager.verify()], [graph.verify()]
    torch.cuda.synchronize()
    rec = torch.cuda.CUDAGraph()
    saved = [t.clone() for t in (graph.lens, graph.n_free, graph.table, graph.free, graph.k, graph.v)]
    with torch.cuda.graph(rec):
        captured = graph.verify()
    for t, old in zip((graph.lens, graph.n_free, graph.table, graph.free, graph.k, graph.v), saved):
        assert torch.equal(t.view(torch.uint8), old.view(torch.uint8))        # capturing ran nothing
    for d in drafts[1:]:
        for s in (eager, graph):
            _load(s, d)
        want.append(eager.verify())
        rec.replay()
        got.append(tuple(x.clone() for x in captured))
    torch.cuda.synchronize()
    assert attn.device_error(reset=True) == 0
    assert all(torch.equal(a, b) for w, x in zip(want, got) for a, b in zip(w, x))
    for a, b in zip((eager.lens, eager.n_free, eager.table, eager.k, eager.v), (graph.lens, graph.n_free, graph.table, graph.k, graph.v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    del rec


def test_calls_on_another_stream():
    """stream= launches there, and the results the call makes belong to it: they are right while the current stream
    is busy, and two calls at once on two streams do not disturb each other."""
    Hq, Hkv, T, D, n = 16, 4, 16, 128, 3000
    q, masks, rows = _tree_case([n, n], [T, T], Hq, Hkv, T, D, "tree", 2)
    kc, vc = (t.cuda() for t in _contiguous(rows, n))
    qc, words, sl = q.cuda(), attn.pack_tree_mask(masks).cuda(), i32([n, n])
    want, lse = attn.decode_tree(qc, kc, vc, sl, words)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for i in range(20):
        torch.empty(1 << 22, device="cuda").fill_(NAN)        # freed at once: the current stream's memory, still being written
        outs += [attn.decode_tree(qc, kc, vc, sl, words, stream=st) for st in (sa, sb)]
    torch.cuda.synchronize()
    assert attn.device_error(reset=True) == 0
    assert all(torch.equal(o, want) and torch.equal(l, lse) for o, l in outs)
    x = torch.randn(2, 8, 4, D, device="cuda").to(torch.bfloat16)
    args = (x, x, x, torch.arange(16, device="cuda").int().view(1, 2, 8).contiguous(), torch.ones(D // 2, device="cuda"),
            torch.arange(16, device="cuda").int().view(2, 8))
    pools = [torch.zeros(1, 4, 64, D, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    a = attn.rope_append(*args, *pools[:2])
    b = attn.rope_append(*args, *pools[2:], stream=sa)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


def test_long_cache_offsets():
    """Rows past 2^31 elements of one cache: 1.1 million rows of 8 heads of 256, two sequences."""
    B, Hkv, D, T, n = 2, 8, 256, 3, 560_000
    if torch.cuda.mem_get_info()[0] < 20e9:
        pytest.skip("needs 20 GB")
    kc, vc = (torch.zeros(B, Hkv, n, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(0)
    q = bf16(g, B, Hkv, T, D)
    tail = [(bf16(g, Hkv, 70, D), bf16(g, Hkv, 70, D)) for _ in range(B)]
    mask = _random_mask(random.Random(1), T, "tree")
    for b, (k, v) in enumerate(tail):
        kc[b, :, -70:], vc[b, :, -70:] = 8 * k, v             # the zeros weigh little against these
    out, lse = attn.decode_tree(q.cuda(), kc, vc, i32([n, n]), attn.pack_tree_mask(mask).cuda(), scale=1.0)
    # plain: n - 70 zero scores with zero values, and the last rows
    see = torch.ones(T, 70, dtype=torch.bool)
    see[:, -T:] = mask
    for b in range(B):
        s = (q[b].double() @ (8 * tail[b][0]).to(torch.bfloat16).double().transpose(1, 2)).masked_fill(~see, -math.inf)
        m = s.amax(-1, keepdim=True).clamp(min=0)
        w = torch.exp(s - m)
        total = w.sum(-1, keepdim=True) + (n - 70) * torch.exp(-m)
        want = (w @ tail[b][1].double()) / total
        a = (w @ tail[b][1].double().abs()) / total
        # scores up to about 8 * 16 * 5 = 640 with |q k| sums of 8 * 256 * 0.64 = 1300: fp32 error 258 * 6e-8 * 1300 = 2e-2
        assert ((out[b].double().cpu() - want).abs() <= (2 ** -7 + 4e-2) * (a + want.abs()) + 1e-30).all()
        assert (lse[b].double().cpu() - (m + total.log())[..., 0]).abs().max() <= 4e-2
    # the same rows through rope_append and tree_commit
    x = bf16(g, 1, 2, Hkv, D)
    slots = i32([[2 * n - 1, n + 5]])
    attn.rope_append(x.cuda(), x.cuda(), x.cuda(), i32([[0, 0]]), torch.ones(D // 2, device="cuda"), slots, kc, vc)
    assert torch.equal(vc[1, :, n - 1].cpu(), x[0, 0]) and torch.equal(kc[1, :, 5].cpu(), x[0, 1])
    row = vc[1, :, n - 1].clone()
    assert attn.tree_commit(kc, vc, i32([n, n]), i32([[1], [2]]), i32([0, 1]), T=3).tolist() == [n - 3, n - 2]
    assert torch.equal(vc[1, :, n - 3], row)
    assert attn.device_error(reset=True) == 0


def test_debug_bounds_build():
    """The tree kernel's unit mapping, ring positions, coordinates and output indices, checked by the kernel itself."""
    build.build(debug_bounds=True)
    res = subprocess.run([sys.executable, os.path.join(HERE, "serving_bounds_cases.py")], env=dict(os.environ, ATTN_GQA_DEBUG_BOUNDS="1"),
                         capture_output=True, text=True, timeout=900)
    assert res.returncode == 0 and "serving bounds cases passed" in res.stdout, res.stdout[-3000:] + res.stderr[-3000:]
