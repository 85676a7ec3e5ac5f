"""Tree attention on the bounds-checking build of the library (ATTN_GQA_DEBUG_BOUNDS=1 in
the environment): results against the plain form, device error word clear."""
import math
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]

import exact_tiled_attention_gqa_b200 as attn  # noqa: E402
from exact_tiled_attention_gqa_b200 import _native  # noqa: E402
import serving_ref as ref  # noqa: E402
import test_serving_step_gpu as cases  # noqa: E402


def main():
    assert _native.LIB_PATH.endswith("_debug_bounds.so"), _native.LIB_PATH
    attn.device_error(reset=True)
    for D in (64, 128, 256):
        for Hq, Hkv, T, lens, sizes in ((4, 2, 1, [200, 1, 0], [1, 1, 0]), (16, 2, 63, [1300, 63], [63, 31]), (5, 1, 130, [200, 700], [130, 77]),
                                        (8, 1, 16, [5, 2100], [16, 16])):
            q, masks, rows = cases._tree_case(lens, sizes, Hq, Hkv, T, D, "tree", T)
            want = cases._reference(q, masks, rows, lens, sizes, 1 / math.sqrt(D))
            words, sl, tl = attn.pack_tree_mask(masks).cuda(), cases.i32(lens), cases.i32(sizes)
            kc, vc = (t.cuda() for t in cases._contiguous(rows, max(lens)))
            kp, vp, table = (t.cuda() for t in cases._paged(rows, 64, T))
            for got in (attn.decode_tree(q.cuda(), kc, vc, sl, words, tree_lens=tl),
                        attn.decode_tree_paged(q.cuda(), kp, vp, table, sl, words, tree_lens=tl)):
                assert attn.device_error(reset=True) == 0
                ref.check_tree(*got, want, f"D{D} T{T}")
    print("serving bounds cases passed")


if __name__ == "__main__":
    main()
