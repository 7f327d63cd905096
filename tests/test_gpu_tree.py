"""The draft tree on the GPU against a dictionary of prefixes, exactly."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import host, require_gpu, say

pytestmark = pytest.mark.gpu


def drafts(B, K, G, fan, seed, vocab=1000):
    g = np.random.default_rng(seed)
    cand = g.integers(0, vocab, (B, 1, G, fan))
    pick = g.integers(0, fan, (B, K, G, 1))
    return np.take_along_axis(np.broadcast_to(cand, (B, K, G, fan)), pick, 3)[..., 0].astype(np.int32)


def check(d, T=None, root=None):
    svd = require_gpu()
    T_ = 1 + d.shape[1] * d.shape[2] if T is None else T
    r = None if root is None else torch.from_numpy(root).cuda()
    got = host(svd.draft_tree(torch.from_numpy(d).cuda(), root=r, n_max=T))
    want = R.draft_tree(d, root, T_)
    for n in want:
        assert np.array_equal(got[n], want[n]), n
    return want


@pytest.mark.parametrize("B,K,G,fan", [
    (1, 1, 1, 1), (3, 1, 8, 2), (2, 8, 16, 2), (5, 16, 32, 2), (2, 64, 5, 3), (1, 64, 63, 2),
    (1, 2, 4000, 1), (4, 7, 33, 1), (2, 3, 65, 4), (9, 5, 1, 2), (1, 40, 100, 2)],
    ids=lambda v: str(v))
def test_trees(B, K, G, fan):
    d = drafts(B, K, G, fan, 7 * B + K + G)
    say("tree", B, K, G, fan)
    T = min(1 + K * G, 4096)
    root = np.arange(B, dtype=np.int32) + 3
    w = check(d, T, root)
    say("nodes", w["n_nodes"].tolist()[:8])


def test_identical_and_disjoint_drafts():
    one = drafts(1, 1, 20, 1, 5)
    check(np.repeat(one, 12, 1))
    d = np.arange(6 * 9, dtype=np.int32).reshape(1, 6, 9)
    assert check(d)["n_nodes"][0] == 55
    # a later draft can equal, extend or shorten an earlier one
    d = np.array([[[1, 2, 3, -1], [1, 2, 3, 4], [1, 2, -1, -1], [1, 2, 3, 4], [-1, 9, 9, 9],
                   [2147483647, 0, 0, 0]]], np.int32)
    check(d)


def test_negative_tokens_end_a_draft():
    g = np.random.default_rng(8)
    d = drafts(16, 6, 12, 2, 9)
    for b in range(16):
        for k in range(6):
            d[b, k, g.integers(0, 13):] = -g.integers(1, 5)
    check(d)
    check(np.full((2, 3, 4), -1, np.int32))


def test_too_many_nodes_is_a_data_error():
    d = drafts(8, 4, 6, 3, 10)
    n = R.draft_tree(d, None, 25)["n_nodes"]
    T = int(np.median(n))
    w = check(d, T)
    assert (w["n_nodes"] < 0).any() and (w["n_nodes"] > 0).any()
    check(d, 1)


def test_full_tree_of_the_largest_size():
    g = np.random.default_rng(11)
    d = g.integers(0, 100, (1, 64, 63)).astype(np.int32)
    d[:, :, 0] = np.arange(64)
    w = check(d, 4096)
    assert w["n_nodes"][0] == 4033
