"""Serving steps whose free list runs out: a refused request keeps its rows, its length and
its pages through page_plan, decode_tree_paged, tree_commit and page_release, eager and in
a CUDA graph, and is served once pages come back."""
import math
import random

import pytest
import torch

import exact_tiled_attention_gqa_b200 as attn
import serving_ref as ref
import test_serving_step_gpu as step
from test_serving_step_gpu import bf16, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.device_error(reset=True)
    yield
    assert attn.device_error(reset=True) == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,L,page,max_pages,spare", [
    (1, 1, 64, 1, 0), (5, 12, 64, 4, 2), (64, 1, 64, 9, 7), (200, 700, 128, 12, 500), (1025, 3, 64, 2, 100), (2500, 9, 256, 2, 400),
    (0, 4, 64, 2, 3),
])
def test_granted_rows(B, L, page, max_pages, spare, in_place):
    """granted is new_lens of the served requests and 0 of the refused, also where it is new_lens itself."""
    lens, new, table, free, n_free, n_pages = step._plan_inputs(B, L, page, max_pages, B + L, spare)
    want = ref.plan(lens, new, table, free, n_free, L, page)
    bt = i32(table) if B else torch.zeros(0, max_pages, dtype=torch.int32, device="cuda")
    sl, nf, nl = i32(lens), i32([n_free]), i32(new)
    granted = nl if in_place else torch.full((B,), -7, dtype=torch.int32, device="cuda")
    extra = dict(out_seqlens=sl, out_n_free=nf) if in_place else {}
    got = attn.page_plan(sl, nl, bt, i32(free), nf, L=L, page_size=page, n_pages=n_pages, granted=granted, **extra)
    assert attn.device_error(reset=True) == 0
    assert [bt.tolist(), got[0].tolist(), got[1].tolist(), got[2].item(), got[3].tolist()] == list(want)
    assert granted.tolist() == [0 if st else n for n, st in zip(new, want[4])]


def test_granted_refusals():
    args = (i32([1, 2]), i32([1, 1]), i32([[0], [1]]), i32([2, 3]), i32([2]))
    for bad in (i32([0]), i32([[0, 0]]), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            attn.page_plan(*args, L=1, page_size=64, n_pages=4, granted=bad)
    with pytest.raises(TypeError):
        attn.page_plan(*args, L=1, page_size=64, n_pages=4, granted=torch.zeros(2, device="cuda"))


class _Server(step._Server):
    """The loop of a server that may run out of pages: trees have the rows page_plan granted."""

    def __init__(self, pages, **kw):
        super().__init__(5, 8, 2, 64, 12, 4, PROMPT, **kw)
        self.n_free.fill_(pages)
        self.granted = i32([0] * self.B)

    def verify(self):
        pos = self.lens[:, None] + self.depth
        slots, *_ = attn.page_plan(self.lens, self.sizes, self.table, self.free, self.n_free, L=self.T, page_size=self.page,
                                   n_pages=self.n_pages, out_seqlens=self.full, out_n_free=self.n_free, status=self.status,
                                   granted=self.granted)
        q = attn.rope_append(*self.split(self.qkv), pos, self.inv, slots, self.k, self.v)
        out, lse = attn.decode_tree_paged(q, self.k, self.v, self.table, self.full, self.mask, tree_lens=self.granted)
        attn.tree_commit(self.k, self.v, self.full, self.accept, self.n_accept, T=self.T, block_table=self.table,
                         tree_lens=self.granted, out_seqlens=self.lens)
        attn.page_release(self.full, self.lens, self.table, self.free, self.n_free, page_size=self.page, n_pages=self.n_pages,
                          out_n_free=self.n_free)
        return out, lse

    def finish(self, b):
        """Request b ends: its pages come back."""
        keep = self.lens.clone()
        keep[b] = 0
        attn.page_release(self.lens, keep, self.table, self.free, self.n_free, page_size=self.page, n_pages=self.n_pages,
                          out_n_free=self.n_free)
        self.lens.copy_(keep)


PROMPT = [70, 1, 64, 128, 129]      # 9 pages of 64 rows; requests 2 and 3 need one for their next row
PAGES = 10                          # request 2 gets the last one, 3 is refused until 4 ends


def _rows(s, b, n):
    """The first n rows of request b, K and V, [Hkv, n, D]."""
    ids = s.table[b, :-(-n // s.page)].long()
    return [c[ids].transpose(0, 1).flatten(1, 2)[:, :n].cpu() for c in (s.k, s.v)]


def test_refused_request_keeps_its_rows():
    r, g = random.Random(11), torch.Generator().manual_seed(11)
    s = _Server(PAGES, seed=3)
    qkv = bf16(g, 5, s.L, (s.Hq + 2 * s.Hkv) * s.D)
    s.prompt(qkv.cuda())
    assert s.lens.tolist() == PROMPT and s.n_free.item() == 1
    refused_in = []
    for n_step in range(4):
        if n_step == 2:
            s.finish(4)
        drafts = step._drafts(r, g, s)
        step._load(s, drafts)
        sizes, mask, depth, accept, n_accept, _ = drafts
        assert (n_accept > 0).all()                      # the refused ones have a path too: it must not be taken
        lens, table = s.lens.tolist(), s.table.tolist()
        before = [_rows(s, b, lens[b]) for b in range(5)]
        want = ref.plan(lens, sizes, table, s.free.tolist(), s.n_free.item(), s.T, s.page)
        out, lse = s.verify()
        assert attn.device_error(reset=True) == 0
        assert s.status.tolist() == want[4] and s.granted.tolist() == [0 if st else n for n, st in zip(sizes, want[4])]
        after = s.lens.tolist()
        for b, st in enumerate(want[4]):
            if st:
                refused_in.append((n_step, b))
                assert after[b] == lens[b] and (out[b] == 0).all() and (lse[b] == -math.inf).all()
                assert s.table[b].tolist() == table[b]
            else:
                assert after[b] == lens[b] + n_accept[b]
            kept = _rows(s, b, lens[b])                  # what was committed stays, bit for bit
            assert all(torch.equal(x, y) for x, y in zip(before[b], kept))
        # every page is free or in a table, once
        used = [-(-n // s.page) for n in after]
        pages = s.free[:s.n_free.item()].tolist() + [p for b, u in enumerate(used) for p in s.table[b, :u].tolist()]
        assert len(set(pages)) == len(pages) == PAGES
        # the served requests' attention: rows as the caches held them, drafted ones from the plain rotation
        x = drafts[5]
        pos = (torch.tensor(lens)[:, None] + depth).int()[None]
        q, k, v = s.split(x)
        q, k = (ref.rope(t, pos, s.inv.cpu(), [s.D // 2], 0, 0)[0].to(torch.bfloat16) for t in (q, k))
        rows = [tuple(torch.cat((h, y[b, :s.granted[b]].transpose(0, 1)), 1) for h, y in zip(before[b], (k, v))) for b in range(5)]
        o, l, tol = step._reference(q.transpose(1, 2), mask, rows, [a.shape[1] for a, _ in rows], s.granted.tolist(), 1 / math.sqrt(s.D))
        # a few of q and K may round the other way: scores move by at most 2^-7 * 4 * 4 / 8 = 1.6e-2 (one such element a score)
        seen = l > -math.inf
        assert torch.equal(lse.cpu() > -math.inf, seen)
        assert ((out.double().cpu() - o).abs() <= tol + 2 * 1.6e-2 * tol * 2 ** 8).all()
        assert (lse.double().cpu() - l)[seen].abs().max() <= ref.LSE_TOL + 1.6e-2
    assert refused_in == [(0, 3), (1, 3)]                # refused while pages were short, served after


def test_refused_request_captured():
    """The same steps from a CUDA graph are the eager ones bit for bit."""
    eager, graph, warm = (_Server(PAGES, seed=3) for _ in range(3))
    r, g = random.Random(12), torch.Generator().manual_seed(12)
    qkv = bf16(g, 5, eager.L, (eager.Hq + 2 * eager.Hkv) * eager.D).cuda()
    drafts = [step._drafts(r, g, eager) for _ in range(4)]
    for s in (eager, graph, warm):
        s.prompt(qkv)
        step._load(s, drafts[0])
    warm.verify()
    rec = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(rec):
        captured = graph.verify()
    refused = []
    for i, d in enumerate(drafts):
        for s in (eager, graph):
            if i == 2:
                s.finish(4)
            step._load(s, d)
        want = eager.verify()
        rec.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, captured))
        refused.append(eager.status.tolist())
        for a, b in zip((eager.lens, eager.n_free, eager.table, eager.status, eager.k, eager.v),
                        (graph.lens, graph.n_free, graph.table, graph.status, graph.k, graph.v)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert attn.device_error(reset=True) == 0
    assert [x[3] for x in refused] == [1, 1, 0, 0]
    del rec


def test_commit_without_a_tree():
    """tree_lens 0: the path and its length are not read, nothing moves, the length stays, nothing is flagged."""
    c = torch.randn(4, 2, 64, 64, device="cuda").to(torch.bfloat16)
    was = c.clone()
    lens = [0, 1, 20, 64]
    out = attn.tree_commit(c, c.clone(), i32(lens), i32([[1, 2], [-1, 0], [1, 1], [5, 3]]), i32([2, -3, 1, 99]), T=4,
                           tree_lens=i32([0] * 4))
    assert attn.device_error(reset=True) == 0
    assert out.tolist() == lens and torch.equal(c, was)
