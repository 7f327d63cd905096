"""Tree attention at both edges of every arrangement of its waves (1 to 8 groups of rows, with
and without a split of a tile's tokens), with contexts inside one tile, over a tile's end and in
joined parts; and trees and chains as long as they are accepted.  Against float64; tolerances as
in test_gpu_attention."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import require_gpu, say
from test_gpu_attention import check, problem

pytestmark = pytest.mark.gpu

# rows of a kv head = nodes * group: (nodes, group)
ROWS = [(1, 1), (15, 1), (4, 4), (17, 1), (31, 1), (8, 4), (33, 1), (47, 1), (6, 8), (7, 7), (63, 1),
        (16, 4), (65, 1), (127, 1), (32, 4), (43, 3), (51, 5), (64, 4), (257, 1), (75, 4), (171, 3)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,group", ROWS, ids=lambda v: str(v))
def test_rows_of_every_arrangement(kind, D, T, group):
    svd = require_gpu()
    rows, tile = T * group, 8192 // D
    say("rows", rows, "D", D, kind)
    for lo, hi in ((3, 9), (tile - 2, tile), (4 * tile + 5, 5 * tile)):
        p = problem(2, T, 2 * group, 2, D, 16, kind, lo, hi, T % 2 == 0, seed=rows + hi)
        parts = svd.svd_tree_attention_workspace_bytes(2, T, 2 * group, 2, D,
                                                       p["tab"].shape[1] * 16) > 256
        assert parts or hi < 4 * tile
        check(svd, p)


def far_tree(B, T, seed, width):
    """Trees in which a node's parent is any earlier node, the paths at most `width` long."""
    g = np.random.default_rng(seed)
    on = np.zeros((B, T, T), bool)
    for b in range(B):
        depth = np.zeros(T, int)
        for t in range(T):
            if t:
                par = g.integers(0, t)
                while depth[par] >= width:
                    par = g.integers(0, par)
                depth[t] = depth[par] + 1
                on[b, t] = on[b, par]
            on[b, t, t] = True
    return on


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,Hq,D,ctx", [(130, 2, 128, 500), (161, 3, 64, 0), (700, 2, 64, 77),
                                        (1025, 1, 128, 30), (4096, 1, 64, 41)],
                         ids=lambda v: str(v))
def test_long_chains(kind, T, Hq, D, ctx):
    svd = require_gpu()
    say("chain", T, Hq, D, ctx, kind)
    p = problem(1, T, Hq, 1, D, 64, kind, ctx, ctx, False, seed=T)
    check(svd, p)
    # the same rows from the ancestors' bits of the chain
    got = svd.tree_attention(p["q"], p["c"], torch.from_numpy(p["tab"]).cuda(),
                             torch.from_numpy(p["ctx"]).cuda())["out"]
    p["anc"] = R.pack(np.tril(np.ones((1, T, T), bool)))
    bits = svd.tree_attention(p["q"], p["c"], torch.from_numpy(p["tab"]).cuda(),
                              torch.from_numpy(p["ctx"]).cuda(),
                              anc=torch.from_numpy(p["anc"]).cuda())["out"]
    assert torch.equal(got, bits)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,ctx", [(2, 200, 2, 1, 64, 100), (1, 577, 4, 2, 128, 9),
                                              (1, 2047, 1, 1, 128, 0), (1, 4096, 2, 1, 64, 63)],
                         ids=lambda v: str(v))
def test_long_trees(kind, B, T, Hq, Hkv, D, ctx):
    # nodes far behind their ancestors: every word of the bits counts
    svd = require_gpu()
    say("tree", B, T, Hq, Hkv, D, ctx, kind)
    p = problem(B, T, Hq, Hkv, D, 32, kind, ctx, ctx, False, seed=T)
    on = far_tree(B, T, T, 12)
    on[0, T // 3] = False  # and one row that sees the context only, or nothing
    p["anc"] = R.pack(on)
    got, lse = check(svd, p)
    if ctx == 0:
        assert (got[0, T // 3] == 0).all() and np.isneginf(lse[0, T // 3]).all()
