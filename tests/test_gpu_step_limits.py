"""The operators around a verification step at the ends of their documented ranges."""
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
