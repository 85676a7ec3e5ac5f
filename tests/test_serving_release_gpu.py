"""page_release with entries outside the pool: they are flagged and left out, so that
page_plan never hands them out, whichever kernel form the sizes take."""
import random

import pytest
import torch

import exact_tiled_attention_gqa_b200 as attn
from exact_tiled_attention_gqa_b200 import _native
import serving_ref as ref
from test_serving_step_gpu import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    attn.device_error(reset=True)
    yield
    assert attn.device_error(reset=True) == 0


# tables of up to 4096 entries run on one CTA, larger ones on a cluster; past 1024 requests in chunks
@pytest.mark.parametrize("B,max_pages,n_bad", [(1, 1, 1), (1, 40, 3), (7, 9, 5), (1100, 3, 1), (1, 5000, 4), (60, 100, 1), (600, 8, 40),
                                               (1500, 4, 7), (2100, 3, 2000), (600, 8, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_bad_pages_stay_off_the_stack(B, max_pages, n_bad, in_place):
    page, r = 64, random.Random(B + n_bad)
    lens = [r.choice([0, max_pages * page, r.randrange(0, max_pages * page + 1)]) for _ in range(B)]
    lens[r.randrange(B)] = max_pages * page
    keep = [r.choice([0, n, r.randrange(0, n + 1)]) for n in lens]
    keep[max(range(B), key=lambda b: lens[b])] = 0
    used = [-(-n // page) for n in lens]
    n_free = 3
    n_pages = sum(used) + n_free
    order = list(range(n_pages))
    r.shuffle(order)
    table = [[-7] * max_pages for _ in range(B)]
    for b in range(B):
        for c in range(used[b]):
            table[b][c] = order.pop()
    gone = [(b, c) for b in range(B) for c in range(-(-keep[b] // page), used[b])]
    for b, c in r.sample(gone, min(n_bad, len(gone))):
        table[b][c] = r.choice([-1, n_pages, -2 ** 31, 2 ** 31 - 1])
    want = order + [table[b][c] for b, c in gone if 0 <= table[b][c] < n_pages]
    # room for exactly the good pages: the bad ones must not push any out
    free, nf = i32(order + [-9] * (len(want) - n_free)), i32([n_free])
    bt = i32(table)
    got = attn.page_release(i32(lens), i32(keep), bt, free, nf, page_size=page, n_pages=n_pages, out_n_free=nf if in_place else None)
    assert attn.device_error(reset=True) == (_native.ATTN_DEVERR_PAGE if n_bad else 0)
    assert got.item() == len(want) and free.tolist() == want
    assert bt.tolist() == table
    # and a plan that takes them all gets pages of the pool only
    n = len(want)
    out = attn.page_plan(i32([0]), i32([n * page]), i32([[-1] * n]), free, got, L=n * page, page_size=page, n_pages=n_pages)
    assert attn.device_error(reset=True) == 0 and out[3].item() == 0 and out[2].item() == 0 and out[0].min() >= 0


def test_bad_lengths_and_bad_pages_together():
    """A pair of lengths that cannot be releases nothing beside a bad page; good pages past the capacity are dropped."""
    page, table = 64, [[0, 1], [2, 99], [3, 4], [5, 6]]
    free = i32([7, -9, -9, -9])
    got = attn.page_release(i32([128, 128, 64, 128]), i32([129, 0, -1, 64]), i32(table), free, i32([1]), page_size=page, n_pages=8)
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_PAGE | _native.ATTN_DEVERR_SEQLEN
    assert got.item() == 3 and free[:3].tolist() == [7, 2, 6]
    free = i32([7, -9])
    got = attn.page_release(i32([128] * 2), i32([0] * 2), i32([[99, 1], [2, 3]]), free, i32([1]), page_size=page, n_pages=8)
    assert attn.device_error(reset=True) == _native.ATTN_DEVERR_PAGE
    assert got.item() == 2 and free.tolist() == [7, 1]
