"""Logit adjustments with n_rows: the rows below it are those of a call on all rows, bit for
bit (every node comes after its parent, so nodes behind n_rows are on no path below it); and
trees as large as they are accepted."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu, say
from test_gpu_adjust import DT, check, dev, problem
from test_gpu_attention_shapes import far_tree
import step_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [
    # B, T, V, H, bias, mask, tree
    (3, 1, 1000, 50, 0, False, True), (4, 4, 1003, 200, 20, True, False),
    (5, 9, 8192, 64, 0, True, True), (3, 33, 4099, 100, 6, True, True),
    (2, 300, 515, 30, 8, True, True), (9, 17, 20001, 300, 0, False, False)],
    ids=lambda c: "B%d_T%d_V%d_H%d_b%d_%s_%s" % c)
def test_rows_below_n_rows(dtype, case):
    svd = require_gpu()
    B, T, V, H, bias, mask, tree = case
    p = problem(B, T, V, H, seed=sum(case[:5]), bias=bias, mask=mask, tree=tree)
    d = {n: dev(x) for n, x in p.items()}
    torch.manual_seed(V)
    z = (torch.randn(B, T, V, device="cuda") * 4).to(DT[dtype])
    want = svd.adjust_logits(z, **d)
    it = torch.int16 if dtype == "bf16" else torch.int32
    rng = np.random.default_rng(T)
    for n in (np.full(B, T), np.zeros(B), np.ones(B), rng.integers(0, T + 1, B)):
        n = n.astype(np.int32)
        part, place = torch.full_like(z, 7.0), z.clone()
        svd.adjust_logits(z, out=part, n_rows=dev(n), **d)
        svd.adjust_logits(place, out=place, n_rows=dev(n), **d)
        for b in range(B):
            k = int(n[b])
            for got, rest in ((part[b], torch.full_like(z[b], 7.0)), (place[b], z[b])):
                assert torch.equal(got[:k].view(it), want[b, :k].view(it))
                assert torch.equal(got[k:].view(it), rest[k:].view(it))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,pool", [(257, 5000, 40), (1000, 1003, 500), (4096, 777, 777)],
                         ids=lambda v: str(v))
def test_large_trees(dtype, T, V, pool):
    svd = require_gpu()
    say("adjust", dtype, T, V)
    p = problem(1, T, V, 90, seed=T, bias=5, mask=T < 1000, pool=pool)
    p["anc"] = R.pack(far_tree(1, T, T, 9))
    torch.manual_seed(T)
    check(svd, (torch.randn(1, T, V, device="cuda") * 4).to(DT[dtype]), p)
