"""What the calls around a verification step ask of each other."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_the_root_counts_once():
    # tokens 3 (prompt), 4 (generated) and 5 (the last committed one, the root)
    svd = require_gpu()
    z = torch.zeros(1, 2, 8, device="cuda")
    one = torch.ones(1, device="cuda")
    kw = dict(hist_len=i32([2]), prompt_len=i32([1]), frequency=one)
    got = svd.adjust_logits(z, i32([[3, 4]]), tokens=i32([[5, 6]]), **kw)[0].tolist()
    assert got == [[0, 0, 0, 0, -1, -1, 0, 0], [0, 0, 0, 0, -1, -1, -1, 0]]
    # in the history as well it counts twice
    kw["hist_len"] = i32([3])
    got = svd.adjust_logits(z, i32([[3, 4, 5]]), tokens=i32([[5, 6]]), **kw)[0].tolist()
    assert got[0][5] == -2
    # a root that is the prompt's last token: in the history, as prompt, and no token of its node
    kw["prompt_len"], kw["hist_len"] = i32([2]), i32([2])
    got = svd.adjust_logits(z, i32([[3, 5]]), tokens=i32([[-1, 6]]), repetition=2 * one,
                            out=torch.empty_like(z), **kw)
    assert got[0].tolist() == [[0] * 8, [0, 0, 0, 0, 0, 0, -1, 0]]
    got = svd.adjust_logits(z + 1, i32([[3, 5]]), tokens=i32([[-1, 6]]), repetition=2 * one, **kw)
    assert got[0].tolist() == [[1, 1, 1, .5, 1, .5, 1, 1], [1, 1, 1, .5, 1, .5, -.5, 1]]


def test_a_draft_that_ends_early_is_not_verified():
    svd = require_gpu()
    B, K, G, V = 3, 2, 4, 500
    g = np.random.default_rng(2)
    d = g.integers(0, V, (B, K, G)).astype(np.int32)
    d[1, 1, 2] = -1
    drafts = torch.from_numpy(d).cuda()
    tree = svd.draft_tree(drafts)
    assert tree["n_nodes"].tolist() == R.draft_tree(d, None, 1 + K * G)["n_nodes"].tolist()
    torch.manual_seed(0)
    p = torch.randn(B * (1 + K * G), V, device="cuda")
    q = torch.randn(B * G, V, device="cuda")
    qx = (torch.arange(B * G, dtype=torch.int32, device="cuda").view(B, 1, G).expand(B, K, G)
          .contiguous())
    r = svd.select_and_verify_rows(p, tree["p_index"], q, qx, drafts)
    assert [x >= 0 for x in r["selected"].tolist()] == [True, False, True]
    assert r["accept_len"][1] == -1 and r["next_token"][1] == -1
