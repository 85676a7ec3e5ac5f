"""tree_commit in a model of several layers: one call a layer, all with the lengths that
still hold the tree's rows."""
import random

import pytest
import torch

import exact_tiled_attention_gqa_b200 as attn
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


@pytest.mark.parametrize("paged", [False, True])
def test_commit_of_several_layers(paged):
    """Every layer's commit takes the lengths that still hold the tree's rows; out_seqlens is another tensor, and all
    layers write the same lengths to it."""
    layers, B, Hkv, T, D, r = 3, 4, 2, 12, 64, random.Random(5)
    g = torch.Generator().manual_seed(5)
    lens = [12, 40, 70, 130]
    paths = [sorted(r.sample(range(T), n)) for n in (0, 1, 5, 12)]
    paths[2] = [1, 4, 5, 9, 11]
    full, out = i32(lens), i32([0] * B)
    acc = i32([p + [-1] * (T - len(p)) for p in paths])
    table = None
    for _ in range(layers):
        rows = [(bf16(g, Hkv, n, D), bf16(g, Hkv, n, D)) for n in lens]
        if paged:
            kc, vc, table = step._paged(rows, 64, 1)
        else:
            kc, vc = step._contiguous(rows, 130)
        caches = [torch.nan_to_num(c, 3.0).cuda() for c in (kc, vc)]
        got = attn.tree_commit(*caches, full, acc, i32([len(p) for p in paths]), T=T, block_table=None if table is None else table.cuda(),
                               out_seqlens=out)
        assert got is out and out.tolist() == [n - T + len(p) for n, p in zip(lens, paths)] and full.tolist() == lens
        for b, path in enumerate(paths):
            ids = list(range(lens[b] - T)) + [lens[b] - T + j for j in path]
            for cache, x in zip(caches, rows[b]):
                n = len(ids)
                mine = cache[table[b, :-(-n // 64)].long().cuda()].transpose(0, 1).flatten(1, 2)[:, :n] if paged else cache[b, :, :n]
                assert torch.equal(mine.cpu(), x[:, ids])
    assert attn.device_error(reset=True) == 0
