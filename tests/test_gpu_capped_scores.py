"""How far a capped score is off: rows that attend to one token alone, whose lse is the score."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

N = 8192


@pytest.mark.parametrize("cap", [0.5, 30.0, 16384.0])
@pytest.mark.parametrize("sloped", [False, True])
def test_capped_scores_are_off_by_2_21_of_the_cap(cap, sloped):
    svd = require_gpu()
    g = np.random.default_rng(3)
    # q = (1, 0, ..), k = (x, 0, ..): the score is x, a bf16 value
    x = np.concatenate([g.uniform(-9, 9, N // 2), g.choice([-1, 1], N - N // 2) *
                        2.0 ** g.uniform(-30, 2, N - N // 2)]) * cap
    k = torch.zeros(N, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    k[:, 0, 0, 0] = torch.from_numpy(x).to(torch.bfloat16).cuda()
    cache = {"k": k, "v": torch.ones_like(k), "k_scale": None, "v_scale": None}
    q = torch.zeros(N, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    table = torch.arange(N, dtype=torch.int32, device="cuda").view(N, 1)
    kw = dict(slopes=torch.ones(1, device="cuda")) if sloped else {}  # at distance 0
    r = svd.prefix_attention(q, cache, table, torch.zeros(N, dtype=torch.int32, device="cuda"),
                             scale=1.0, cap=cap, want_lse=True, **kw)
    z = k[:, 0, 0, 0].double().cpu().numpy()
    want = cap * np.tanh(z / cap)
    off = np.abs(r["lse"].double().cpu().numpy().ravel() - want)
    say("cap", cap, "off by 2^%.2f of it" % np.log2(off.max() / cap))
    # the logarithm's base is changed by a rounded factor and a rounded product
    assert (off <= cap * 2.0 ** -21 + np.abs(want) * 2.0 ** -23).all()
    assert (r["out"] == 1).all()
