"""Cases, inputs and plain forms of the serving-step operators around the paged KV cache.

One step of a serving loop that verifies drafted token trees makes these calls, in this order:

  page_plan / page_release   block tables and slot maps from request lengths, pages from a free list
  rope_append                rotary positions (one or several axes) of the new tokens' q and k, k and v
                             written to their cache slots (bf16, E4M3 or q8_0 caches)
  decode_tree[_paged]        attention of every tree's drafted tokens over the cache
  tree_commit                the accepted path's rows moved together, the lengths set

``own`` false: elementary torch operations in 32 bits (64 for angles).  ``own`` true: the
framework's calls.  ``exact``: the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a 64-request batch: every request gets one row, few a new page
        _plan("plan_decode_b64", B=64, L=1, page=64, max_pages=512, lo=1024, hi=32768, short=False),
        # prompts of very different lengths admitted at once; the free list runs out before the last
        _plan("plan_prompts_b512", B=512, L=4096, page=64, max_pages=128, lo=0, hi=4000, short=True),
        # a few requests of a batch end and give their pages back
        _release("release_b64", B=64, page=64, max_pages=512, hi=4096),
        # the largest batch shrinks after long prompts
        _release("release_b512", B=512, page=64, max_pages=256, hi=16384),
        # one token for each request of a batch into a bf16 paged cache: the latency of every decode step
        _rope("rope_decode_b64", B=64, L=1, Hq=32, Hkv=8, D=128, rot=128, axes=1, order="blocks", pairs="half", fmt="bf16", page=64,
              far=32768),
        # a long image-and-text prompt into an E4M3 cache: three position axes taken in turn
        _rope("rope_prompt_8192_e4m3", B=1, L=8192, Hq=32, Hkv=8, D=128, rot=128, axes=3, order="cycle", pairs="half",
              fmt="e4m3", page=64, far=131072),
        # ragged chunks into a q8_0 cache, half of each head rotated, neighbouring elements paired
        _rope("rope_q8_ragged", B=8, L=1000, Hq=16, Hkv=2, D=128, rot=64, axes=2, order="blocks", pairs="adjacent",
              fmt="q8_0", page=128, far=1000003),
        # a single user's small tree on a short context, head dim 64: latency
        _tree("tree_b1_t8_d64", B=1, Hq=32, Hkv=8, T=8, D=64, lo=500, hi=500, page=64, ragged=False),
        # the serving batch: 64 requests of 1K to 32K rows, 16 drafted tokens each, paged
        _tree("tree_b64_t16_paged", B=64, Hq=32, Hkv=8, T=16, D=128, lo=1024, hi=32768, page=64, ragged=True),
        # large trees of uneven size, eight query heads a KV head, contiguous caches of head dim 256
        _tree("tree_b8_t63_d256", B=8, Hq=32, Hkv=4, T=63, D=256, lo=3000, hi=16000, page=0, ragged=True),
        # accepted paths of a small batch, contiguous cache
        _commit("commit_b8", B=8, Hkv=8, D=128, T=16, A=5, page=0, rows=512),
        # accepted paths of the serving batch, paged cache
        _commit("commit_b64_paged", B=64, Hkv=8, D=128, T=64, A=9, page=64, rows=320),
    ]


def _plan(name, **kw):
    return {"op": "plan", "name": name, **kw}


def _release(name, **kw):
    return {"op": "release", "name": name, **kw}


def _rope(name, **kw):
    return {"op": "rope", "name": name, **kw}


def _tree(name, **kw):
    return {"op": "tree", "name": name, **kw}


def _commit(name, **kw):
    return {"op": "commit", "name": name, **kw}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "release", "rope", "rope", "tree", "tree", "commit"])
    if op in ("plan", "release"):
        B = _log_int(rng, 1, 512)
        page = rng.choice([64, 128, 256])
        if op == "plan":
            L = _log_int(rng, 1, 4096)
            lo = rng.randrange(0, 3000)
            hi = lo + rng.randrange(0, 5000)
            case = _plan(None, B=B, L=L, page=page, max_pages=-(-(hi + L) // page) + rng.randrange(0, 9), lo=lo, hi=hi,
                         short=rng.random() < 0.5)
        else:
            hi = _log_int(rng, 1, 16384)
            case = _release(None, B=B, page=page, max_pages=-(-hi // page), hi=hi)
    elif op == "rope":
        D = rng.choice([64, 128, 128, 256])
        fmt = rng.choice(["bf16", "e4m3", "q8_0"]) if D < 256 else "bf16"
        tokens = _log_int(rng, 1, 8192)
        B = min(tokens, _log_int(rng, 1, 64))
        Hkv = rng.choice([1, 2, 4, 8])
        axes = rng.choice([1, 1, 2, 3, 4])
        case = _rope(None, B=B, L=max(1, tokens // B), Hq=Hkv * rng.choice([1, 2, 3, 4]), Hkv=Hkv, D=D,
                     rot=D if rng.random() < 0.6 else 16 * rng.randrange(1, D // 16 + 1), axes=axes,
                     order=rng.choice(["blocks", "cycle"]), pairs=rng.choice(["half", "adjacent"]), fmt=fmt,
                     page=rng.choice([64, 128]), far=rng.choice([4096, 32768, 1000003]))
    elif op == "tree":
        D = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 8])
        T = _log_int(rng, 1, 128)
        B = _log_int(rng, 1, 32)
        hi = _log_int(rng, T + 1, 16000)
        while B > 1 and B * Hkv * G * T * hi * D > 8 * 32 * 63 * 9500 * 64:   # no more than the largest listed tree
            B //= 2
        case = _tree(None, B=B, Hq=Hkv * G, Hkv=Hkv, T=T, D=D, lo=max(T, hi // rng.choice([1, 2, 16])), hi=hi,
                     page=rng.choice([0, 64, 128]), ragged=rng.random() < 0.5)
    else:
        T = _log_int(rng, 2, 128)
        case = _commit(None, B=_log_int(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 256]), T=T,
                       A=rng.randrange(1, min(T, 16) + 1), page=rng.choice([0, 64, 128]), rows=T + rng.randrange(1, 256))
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng(seed)
    return {"plan": _prepare_plan, "release": _prepare_release, "rope": _prepare_rope, "tree": _prepare_tree,
            "commit": _prepare_commit}[case["op"]](case, g, r)


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _spread(case, r, lo, hi):
    """B lengths spread evenly over [lo, hi], in an order of the seed (their sum is the case's)."""
    n = case["B"]
    x = np.round(np.linspace(lo, hi, n)).astype(np.int64) if n > 1 else np.array([(lo + hi) // 2])
    return r.permutation(x)


def _tables(lens, page, max_pages, r, spare=0, n_pages=None):
    """Block tables of pages in random order, -1 past each request's last page, and the pages left over."""
    used = -(-lens // page)
    n_pages = n_pages or int(used.sum()) + spare
    order = r.permutation(n_pages)
    table = np.full((len(lens), max_pages), -1, dtype=np.int64)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    return table, order[at:], n_pages


def _prepare_plan(case, g, r):
    lens = _spread(case, r, case["lo"], case["hi"])
    new = r.permutation(_spread(case, r, 0 if case["L"] > 1 else 1, case["L"]))
    page = case["page"]
    need = int((-(-(lens + new) // page) + (-lens // page)).sum())
    spare = need - need // 8 if case["short"] else need + 7   # short: the last requests find no page
    table, free, n_pages = _tables(lens, page, case["max_pages"], r, spare)
    cap = max(1, n_pages)
    stack = np.full(cap, -1, dtype=np.int64)
    stack[:len(free)] = free
    return {"case": case, "seqlens": _i32(lens), "new_lens": _i32(new), "table": _i32(table), "free": _i32(stack),
            "n_free": _i32([len(free)]), "n_pages": max(1, n_pages)}


def _prepare_release(case, g, r):
    lens = _spread(case, r, 0, case["hi"])
    keep = np.minimum(lens, r.integers(0, case["hi"] + 1, case["B"]))
    keep[r.random(case["B"]) < 0.3] = 0                       # finished requests give up every page
    table, free, n_pages = _tables(lens, case["page"], case["max_pages"], r, 16)
    stack = np.full(n_pages, -1, dtype=np.int64)
    stack[:len(free)] = free
    return {"case": case, "seqlens": _i32(lens), "keep": _i32(keep), "table": _i32(table), "free": _i32(stack),
            "n_free": _i32([len(free)]), "n_pages": n_pages}


def _sections(case):
    n, a = case["rot"] // 2, case["axes"]
    rest = n // a
    return [n - rest * (a - 1)] + [rest] * (a - 1)


def _axis_of_pair(case):
    n, a, sec = case["rot"] // 2, case["axes"], _sections(case)
    if case["order"] == "blocks":
        return np.repeat(np.arange(a), sec)
    axis = np.zeros(n, dtype=np.int64)
    for k in range(1, a):
        axis[k:k + a * sec[k]:a] = k
    return axis


def _prepare_rope(case, g, r):
    B, L, Hq, Hkv, D, page = (case[k] for k in ("B", "L", "Hq", "Hkv", "D", "page"))
    qkv = _bf16(g, B, L, (Hq + 2 * Hkv) * D)                  # one projection's output
    new = _spread(case, r, max(1, L // 3), L)                 # ragged: the rest of a request's L tokens is padding
    old = r.integers(0, 200, B)
    # a pool of the same size for every seed
    table, _, n_pages = _tables(old + new, page, -(-(199 + L) // page), r, n_pages=int((-(-(199 + new) // page)).sum()) + 3)
    j = np.arange(L)[None, :]
    row = old[:, None] + j
    ok = j < new[:, None]
    slots = np.where(ok, table[np.arange(B)[:, None], np.minimum(row // page, table.shape[1] - 1)] * page + row % page, -1)
    start = r.integers(0, max(1, case["far"] - L), (case["axes"], B, 1))
    step = np.stack([j // (1 << k) for k in range(case["axes"])])
    inv = (1e6 ** (-np.arange(case["rot"] // 2) / (case["rot"] // 2))).astype(np.float32)
    st = {"case": case, "q": qkv[..., :Hq * D].view(B, L, Hq, D), "k": qkv[..., Hq * D:(Hq + Hkv) * D].view(B, L, Hkv, D),
          "v": qkv[..., (Hq + Hkv) * D:].view(B, L, Hkv, D), "positions": _i32(start + step), "inv_freq": torch.as_tensor(inv, device=DEV),
          "axis": torch.as_tensor(_axis_of_pair(case), device=DEV), "slots": _i32(slots),
          "tokens": torch.as_tensor(np.flatnonzero(slots.reshape(-1) >= 0), device=DEV), "sections": _sections(case),
          "n_pages": n_pages, "k_scale": None, "v_scale": None}
    shape = (n_pages, Hkv, page, D)
    if case["fmt"] == "bf16":
        st["k_cache"], st["v_cache"] = _bf16(g, *shape), _bf16(g, *shape)
    elif case["fmt"] == "e4m3":
        st["k_cache"], st["v_cache"] = (_bf16(g, *shape).to(torch.float8_e4m3fn) for _ in range(2))
        st["k_scale"], st["v_scale"] = (torch.rand(Hkv, generator=g, device=DEV) * 0.03 + 0.01 for _ in range(2))
    else:
        st["k_cache"], st["v_cache"] = (torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8) for _ in range(2))
        st["k_scale"], st["v_scale"] = ((torch.rand(n_pages, Hkv, page, D // 32, generator=g, device=DEV) * 0.03).half() for _ in range(2))
    return st


def _trees(B, T, sizes, r):
    """Random trees, a node's parent before it: allowed[b, i, j] = node j is node i or above it."""
    see = np.zeros((B, T, T), dtype=bool)
    for i in range(T):
        if i:
            up = np.maximum(0, i - 1 - r.integers(0, 1 + i // 2, B))
            see[:, i] = see[np.arange(B), up]
        see[:, i, i] = True
    live = np.arange(T)[None] < sizes[:, None]
    return see & live[:, :, None] & live[:, None, :]


def _pack(see):
    B, T, _ = see.shape
    W = -(-T // 32)
    bits = np.zeros((B, T, W * 32), dtype=np.uint64)
    bits[..., :T] = see
    words = (bits.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return words.view(np.int32)


def _prepare_tree(case, g, r):
    B, Hq, Hkv, T, D, page = (case[k] for k in ("B", "Hq", "Hkv", "T", "D", "page"))
    lens = _spread(case, r, case["lo"], case["hi"])
    sizes = r.permutation(_spread(case, r, max(1, T // 2), T)) if case["ragged"] else np.full(B, T)
    sizes = np.minimum(sizes, lens)
    see = _trees(B, T, sizes, r)
    st = {"case": case, "q": _bf16(g, B, Hq, T, D), "seqlens": _i32(lens), "mask": _i32(_pack(see)),
          "tree_lens": _i32(sizes) if case["ragged"] else None, "sizes": torch.as_tensor(sizes, device=DEV),
          "see": torch.as_tensor(see, device=DEV), "longest": int(lens.max()), "table": None}
    if page:
        table, _, n_pages = _tables(lens, page, -(-int(lens.max()) // page), r, 3)
        st["table"] = _i32(table)
        shape = (n_pages, Hkv, page, D)
    else:
        shape = (B, Hkv, int(lens.max()), D)
    st["k_cache"], st["v_cache"] = _bf16(g, *shape), _bf16(g, *shape)
    return st


def _prepare_commit(case, g, r):
    B, Hkv, D, T, A, page = (case[k] for k in ("B", "Hkv", "D", "T", "A", "page"))
    lens = r.integers(T, case["rows"] + 1, B)
    # increasing paths whose moved rows come from at or past A, so a second pass moves the same rows
    accept = np.full((B, A), -1, dtype=np.int64)
    n = r.integers(1, A + 1, B)
    for b in range(B):
        stay = int(r.integers(0, n[b] + 1)) if T - A >= 1 else int(n[b])
        stay = max(stay, int(n[b]) - (T - A))
        accept[b, :stay] = np.arange(stay)
        accept[b, stay:n[b]] = A + np.sort(r.choice(T - A, int(n[b]) - stay, replace=False)) if n[b] > stay else []
    st = {"case": case, "seqlens": _i32(lens), "accept": _i32(accept), "n_accept": _i32(n), "table": None}
    if page:
        table, _, n_pages = _tables(lens, page, -(-case["rows"] // page), r, n_pages=B * -(-case["rows"] // page) + 3)
        st["table"] = _i32(table)
        shape = (n_pages, Hkv, page, D)
    else:
        shape = (B, Hkv, case["rows"], D)
    st["k_cache"], st["v_cache"] = _bf16(g, *shape), _bf16(g, *shape)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        import exact_tiled_attention_gqa_b200 as attn
        if op == "plan":
            slots, lens, n_free, status = attn.page_plan(st["seqlens"], st["new_lens"], st["table"], st["free"], st["n_free"],
                                                         L=st["case"]["L"], page_size=st["case"]["page"], n_pages=st["n_pages"])
            return slots, lens, n_free, status, st["table"]
        if op == "release":
            n_free = attn.page_release(st["seqlens"], st["keep"], st["table"], st["free"], st["n_free"],
                                       page_size=st["case"]["page"], n_pages=st["n_pages"])
            return n_free, st["free"]
        if op == "rope":
            q = attn.rope_append(st["q"], st["k"], st["v"], st["positions"], st["inv_freq"], st["slots"], st["k_cache"], st["v_cache"],
                                 sections=st["sections"], axis_order=st["case"]["order"], pairs=st["case"]["pairs"],
                                 k_scale=st["k_scale"], v_scale=st["v_scale"])
            return (q, *_held(st))
        if op == "tree":
            if st["table"] is None:
                return attn.decode_tree(st["q"], st["k_cache"], st["v_cache"], st["seqlens"], st["mask"], tree_lens=st["tree_lens"])
            return attn.decode_tree_paged(st["q"], st["k_cache"], st["v_cache"], st["table"], st["seqlens"], st["mask"],
                                          tree_lens=st["tree_lens"])
        lens = attn.tree_commit(st["k_cache"], st["v_cache"], st["seqlens"], st["accept"], st["n_accept"], T=st["case"]["T"],
                                block_table=st["table"])
        return lens, st["k_cache"], st["v_cache"]
    return {"plan": _plain_plan, "release": _plain_release, "rope": _plain_rope, "tree": _plain_tree, "commit": _plain_commit}[op](st)


def _held(st):
    """The caches as the values they hold (8-bit: E4M3 values of the shared head scale; q8_0 code x scale)."""
    if st["case"]["fmt"] != "q8_0":
        return st["k_cache"], st["v_cache"]
    return tuple(st[c].unflatten(-1, (-1, 32)) * st[s].unsqueeze(-1) for c, s in (("k_cache", "k_scale"), ("v_cache", "v_scale")))


def _up(x, page):
    return (x + page - 1) // page


def _plain_plan(st):
    case, page, table = st["case"], st["case"]["page"], st["table"]
    old, new = st["seqlens"].long(), st["new_lens"].long()
    used, total = _up(old, page), _up(old + new, page)
    fits = total <= table.shape[1]                       # a request the table has no room for asks for nothing
    need = (total - used) * fits
    last = torch.cumsum(need, 0)
    served = ((need == 0) | (last <= st["n_free"].long())) & fits
    first = last - need
    # new page k of the step is popped from the top of the stack
    col = torch.arange(table.shape[1], device=DEV)[None]
    pick = (st["n_free"].long() - 1 - (first[:, None] + col - used[:, None])).clamp(0, st["free"].numel() - 1)
    fresh = served[:, None] & (col >= used[:, None]) & (col < total[:, None])
    table.copy_(torch.where(fresh, st["free"][pick], table))
    j = torch.arange(case["L"], device=DEV)[None]
    row = old[:, None] + j
    at = table.long().gather(1, (row // page).clamp(max=table.shape[1] - 1))
    slots = torch.where(served[:, None] & (j < new[:, None]), at * page + row % page, -1).int()
    lens = torch.where(served, old + new, old).int()
    n_free = (st["n_free"].long() - (need * served).sum()).int()
    return slots, lens, n_free, (~served).int(), table


def _plain_release(st):
    page, table, free = st["case"]["page"], st["table"], st["free"]
    kept, used = _up(st["keep"].long(), page), _up(st["seqlens"].long(), page)
    gone = used - kept
    last = torch.cumsum(gone, 0)
    col = torch.arange(table.shape[1], device=DEV)[None]
    out = (col >= kept[:, None]) & (col < used[:, None])
    at = st["n_free"].long() + (last - gone)[:, None] + col - kept[:, None]
    # entries that stay go to a place behind the stack
    wide = torch.cat((free, free[:1]))
    wide[torch.where(out, at, free.numel()).reshape(-1)] = table.reshape(-1)
    free.copy_(wide[:-1])
    return (st["n_free"] + gone.sum()).int(), free


def _turned(x, case, cos, sin):
    """x [B,L,H,D] float32 with its first `rot` elements rotated."""
    n, rot = case["rot"] // 2, case["rot"]
    if case["pairs"] == "half":
        a, b = x[..., :n], x[..., n:rot]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., rot:]), -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., rot:]), -1)


def _plain_rope(st):
    case, page = st["case"], st["case"]["page"]
    B, L, Hkv, D = case["B"], case["L"], case["Hkv"], case["D"]
    angle = st["positions"][st["axis"]].permute(1, 2, 0).double() * st["inv_freq"].double()   # [B,L,rot/2]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    q = _turned(st["q"].float(), case, cos, sin).to(torch.bfloat16).transpose(1, 2).contiguous()
    k = _turned(st["k"].float(), case, cos, sin)
    slot = st["slots"].reshape(-1).long()[st["tokens"]]
    where = (slot // page, slice(None), slot % page)
    for x, c, s in ((k, "k_cache", "k_scale"), (st["v"].float(), "v_cache", "v_scale")):
        x = x.reshape(B * L, Hkv, D)[st["tokens"]]
        if case["fmt"] == "bf16":
            st[c][where] = x.to(torch.bfloat16)
        elif case["fmt"] == "e4m3":
            st[c].view(torch.int8)[where] = (x / st[s][None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.int8)
        else:
            x = x.unflatten(-1, (-1, 32))
            d = (x.abs().amax(-1) / 127).half()
            code = torch.where(d[..., None] > 0, (x / d[..., None].float()).round().clamp(-127, 127), 0)
            st[c][where] = code.flatten(-2).to(torch.int8)
            st[s][where] = d
    return (q, *_held(st))


def _rows_of(st, cache, n):
    """Rows 0 .. n-1 of every request, [B,Hkv,n,D]."""
    if st["table"] is None:
        return cache[:, :, :n]
    page = st["case"]["page"]
    pages = cache[st["table"][:, :-(-n // page)].long().clamp(min=0)]       # [B,pages,Hkv,page,D]
    return pages.transpose(1, 2).flatten(2, 3)[:, :, :n]


def _visible(st, n):
    """[B,T,n]: which cache rows each drafted token sees."""
    T = st["case"]["T"]
    ctx = st["seqlens"].long() - st["sizes"]
    node = torch.arange(n, device=DEV)[None] - ctx[:, None]                 # [B,n]
    in_tree = st["see"].gather(2, node.clamp(0, T - 1)[:, None].expand(-1, T, -1))
    live = torch.arange(T, device=DEV)[None] < st["sizes"][:, None]
    return live[:, :, None] & ((node < 0)[:, None] | ((node < st["sizes"][:, None])[:, None] & in_tree))


def _plain_tree(st):
    case, n = st["case"], st["longest"]
    B, Hq, Hkv, T, D = (case[k] for k in ("B", "Hq", "Hkv", "T", "D"))
    q = st["q"].float().view(B, Hkv, Hq // Hkv * T, D) * (1 / math.sqrt(D))
    s = (q @ _rows_of(st, st["k_cache"], n).float().transpose(2, 3)).view(B, Hkv, Hq // Hkv, T, n)
    s.masked_fill_(~_visible(st, n)[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = s.sum(-1, keepdim=True)
    v = _rows_of(st, st["v_cache"], n).float()
    o = (s.view(B, Hkv, -1, n) @ v).view(B, Hkv, Hq // Hkv, T, D) / total.clamp(min=1e-37)
    return o.to(torch.bfloat16).view(B, Hq, T, D), (top + total.log()).view(B, Hq, T)


def _plain_commit(st):
    case = st["case"]
    B, T, A, page = case["B"], case["T"], case["A"], case["page"]
    ctx = (st["seqlens"] - T).long()[:, None]
    j = torch.arange(A, device=DEV)[None].expand(B, A)
    take = j < st["n_accept"][:, None]
    to = ctx + j
    frm = torch.where(take, ctx + st["accept"], to)      # what is not taken stays where it is
    b = torch.arange(B, device=DEV)[:, None].expand(B, A)

    def place(row):
        if st["table"] is None:
            return b, row
        return st["table"].long().gather(1, row // page), row % page

    (pf, rf), (pt, rt) = place(frm), place(to)
    for c in ("k_cache", "v_cache"):
        st[c][pt, :, rt] = st[c][pf, :, rf]
    return (ctx[:, 0] + st["n_accept"]).int(), st["k_cache"], st["v_cache"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _lens_sum(case, lo, hi):
    return int(np.round(np.linspace(lo, hi, case["B"])).sum()) if case["B"] > 1 else (lo + hi) // 2


def work(case):
    B = case["B"]
    if case["op"] == "plan":
        # lengths in and out, the new pages (free list to table), the slot map
        pages = _lens_sum(case, 0 if case["L"] > 1 else 1, case["L"]) // case["page"]
        return {"bytes": 4 * (4 * B + 2 * pages + B * case["L"] + 2), "flops": 0}
    if case["op"] == "release":
        pages = _lens_sum(case, 0, case["hi"]) // case["page"] // 2
        return {"bytes": 4 * (2 * B + 2 * pages + 2), "flops": 0}
    if case["op"] == "rope":
        L, Hq, Hkv, D = (case[k] for k in ("L", "Hq", "Hkv", "D"))
        held = _lens_sum(case, max(1, L // 3), L)
        row = {"bf16": 2 * D, "e4m3": D, "q8_0": D + D // 16}[case["fmt"]]
        return {"bytes": B * L * (Hq * D * 4 + 4 * case["axes"] + 4) + held * 2 * Hkv * (2 * D + row),
                "flops": 3 * case["rot"] * (B * L * Hq + held * Hkv)}
    if case["op"] == "tree":
        Hq, Hkv, T, D = (case[k] for k in ("Hq", "Hkv", "T", "D"))
        rows = _lens_sum(case, case["lo"], case["hi"])
        sizes = _lens_sum(case, max(1, T // 2), T) if case["ragged"] else B * T
        return {"bytes": 4 * rows * Hkv * D + B * Hq * T * (4 * D + 4) + B * T * 4 * -(-T // 32),
                "flops": int(4 * Hq * D * rows * sizes / B)}
    A, Hkv, D = case["A"], case["Hkv"], case["D"]
    return {"bytes": int(B * (A + 1) / 2 * Hkv * D * 2 * 2 * 2) // 2 + 4 * B * (A + 3), "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("plan", "release"):
        return None       # whole numbers
    st = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "commit": _exact_commit}[case["op"]](st)


def _exact_commit(st):
    case, page = st["case"], st["case"]["page"]
    ctx, n = (st["seqlens"] - case["T"]).tolist(), st["n_accept"].tolist()
    out = []
    for c in ("k_cache", "v_cache"):
        was, now = st[c].double(), st[c].double()
        for b, path in enumerate(st["accept"].tolist()):
            for j in range(n[b]):
                at = [(b, x) if not page else (int(st["table"][b, x // page]), x % page) for x in (ctx[b] + j, ctx[b] + path[j])]
                now[at[0][0], :, at[0][1]] = was[at[1][0], :, at[1][1]]
        out.append(now)
    return None, *out


def _exact_rope(st):
    case, page = st["case"], st["case"]["page"]
    B, L, D, rot = case["B"], case["L"], case["D"], case["rot"]
    n = rot // 2
    pos, inv = st["positions"].double(), st["inv_freq"].double()
    # the rotation as complex numbers, pair by pair
    turn = torch.stack([torch.polar(torch.ones_like(pos[0]), pos[a] * f) for a, f in zip(st["axis"].tolist(), inv.tolist())], -1)

    def rotated(x):
        x = x.double()
        lo = torch.arange(n, device=DEV) if case["pairs"] == "half" else 2 * torch.arange(n, device=DEV)
        hi = lo + (n if case["pairs"] == "half" else 1)
        z = torch.complex(x[..., lo], x[..., hi]) * turn[:, :, None]
        y = x.clone()
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    q = rotated(st["q"]).permute(0, 2, 1, 3).contiguous()
    out = [q]
    for x, c, s in ((rotated(st["k"]), "k_cache", "k_scale"), (st["v"].double(), "v_cache", "v_scale")):
        held = st[c].float().double()
        if case["fmt"] == "q8_0":
            held = held.unflatten(-1, (-1, 32)) * st[s].double().unsqueeze(-1)
        for t in st["tokens"].tolist() if B * L <= 512 else []:
            slot = int(st["slots"].view(-1)[t])
            held[slot // page, :, slot % page] = _stored(x[t // L, t % L], st, s)
        if B * L > 512:
            slot = st["slots"].view(-1)[st["tokens"]].long()
            rows = x.flatten(0, 1)[st["tokens"]]
            held.transpose(1, 2)[slot // page, slot % page] = _stored(rows, st, s)
        out.append(held)
    return tuple(out)


def _stored(x, st, s):
    """What a cache row should stand for, unrounded: x itself, in the unit its format is returned in."""
    fmt = st["case"]["fmt"]
    if fmt == "e4m3":
        return (x / st[s].double()[:, None]).clamp(-448, 448)
    return x.unflatten(-1, (-1, 32)) if fmt == "q8_0" else x


def _exact_tree(st):
    case = st["case"]
    B, Hq, Hkv, T, D, page = (case[k] for k in ("B", "Hq", "Hkv", "T", "D", "page"))
    if sum(st["seqlens"].tolist()) * Hq * T * D > 1e12:
        return None
    out = torch.zeros(B, Hq, T, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(B):
        n, size = int(st["seqlens"][b]), int(st["sizes"][b])
        if st["table"] is None:
            K, V = st["k_cache"][b, :, :n], st["v_cache"][b, :, :n]
        else:
            ids = st["table"][b, :-(-n // page)].long()
            K, V = (st[c][ids].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :n] for c in ("k_cache", "v_cache"))
        seen = torch.ones(size, n, dtype=torch.bool, device=DEV)
        seen[:, n - size:] = st["see"][b, :size, :size]
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            s = torch.einsum("gtd,nd->gtn", st["q"][b, heads, :size].double(), K[h].double()) / math.sqrt(D)
            s = s.masked_fill(~seen, -math.inf)
            lse[b, heads, :size] = torch.logsumexp(s, -1)
            out[b, heads, :size] = torch.einsum("gtn,nd->gtd", torch.softmax(s, -1), V[h].double())
    return out, lse
