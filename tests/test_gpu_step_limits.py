"""The operators around a verification step at the ends of their documented ranges."""
import math

import pytest
import torch

from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_masks_of_the_largest_vocabulary():
    # 2^31 - 1 tokens: a mask row has 2^26 words, and the second row of the table applies
    svd = require_gpu()
    V = 2 ** 31 - 1
    W = (V + 31) // 32
    z = torch.zeros((1, 1, V), dtype=torch.bfloat16, device="cuda")
    allow = torch.empty((2, W), dtype=torch.int32, device="cuda")
    allow[0] = 0
    allow[1] = -1
    off = (0, 5, 4095, 4096, 2 ** 30 + 7, V - 9, V - 1)
    for v in off:
        w = int(allow[1, v // 32]) & 0xFFFFFFFF & ~(1 << (v % 32))
        allow[1, v // 32] = w - (1 << 32) if w >= 1 << 31 else w
    say("mask words", W)
    svd.adjust_logits(z, allow=allow, allow_index=i32(1).view(1, 1), out=z)
    row = z.view(-1)
    for v in off:
        assert row[v] == -float("inf"), v
        row[v] = 0
    for part in row.split(1 << 28):
        assert not part.any()


def test_attention_over_the_longest_sequence():
    # 2^31 - 16 positions, all of them in one page of 16: rounded up to whole tiles the length
    # passes 32 bits.  Keys of zero give every token weight 1, so the output is the mean of the
    # page's values and the log-sum log(n).  The sums are whole multiples of 16 below 2^28 in
    # every part, so exact; joining the parts rounds at most 64 + 16 times.  The means are
    # bf16 values, which an error of 80 * 2^-24 does not leave
    svd = require_gpu()
    D, page = 64, 16
    mp = 2 ** 31 // page - 1
    n = mp * page
    assert n + 8192 // D - 1 >= 2 ** 31
    c = svd.kv_cache(3, 1, page, D)
    c["v"][1] = (torch.arange(D, device="cuda") % 3).float()
    c["v"][1, 0, ::2] += 1
    c["v"][2] = float("nan")
    tab = torch.ones((1, mp), dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, 1, D, device="cuda").to(torch.bfloat16)
    say("positions", n)
    r = svd.tree_attention(q, c, tab, i32(n - 1), want_lse=True)
    assert torch.equal(r["out"].float().view(-1), c["v"][1].float().mean((0, 1)))
    want = math.log(n)
    assert abs(float(r["lse"]) - want) <= 2.0 ** -24 * (80 + 4 * want)
