"""Filtered rows of prefixes with temperatures of their own, verified in the ways that the header
names: one call per temperature, or logits that were divided first.  Acceptances against the
filtered laws in float64, decisions against the uniforms."""
import numpy as np
import pytest
import torch

import serve_ref as S
from gpu_util import require_gpu, say
from hash_ref import uniform_bits
from parity_harness import ALPHA_TOL

pytestmark = pytest.mark.gpu

B, G, V = 6, 5, 501
TEMPS = np.array([0.5, 1.0, 1.7, 0.0, 0.5, 1.0], np.float32)
TOP_K = np.array([0, 40, 0, 9, 20, 0], np.int32)
TOP_P = np.array([0.9, 1.0, 0.7, 1.0, 0.95, 0.8], np.float32)
SEED, BASE = 5, 100


def laws(z, t, b):
    """float64 laws of rows [n,V] that prefix b's settings keep, at temperature t."""
    out = np.zeros(z.shape)
    for i, row in enumerate(z):
        keep = S.kept(row, float(t), int(TOP_K[b]), float(TOP_P[b]))
        w = np.where(keep, np.exp((row - row.max()) / (float(t) or 1.0)), 0.0)
        out[i] = w / w.sum()
    return out


def problem(dtype):
    svd = require_gpu()
    torch.manual_seed(8)
    p = (torch.randn(B, G + 1, V, device="cuda") * 3).to(dtype)
    q = (p[:, :G].float() + torch.randn(B, G, V, device="cuda")).to(dtype)
    return svd, p, q


def dev(x):
    return torch.from_numpy(x).cuda()


def check(b, t, p, q, draft, got):
    zp, zq = p[b].double().cpu().numpy(), q[b].double().cpu().numpy()
    lp, lq = laws(zp, t, b), laws(zq, t, b)
    x = draft[b].cpu().numpy()
    want = np.minimum(1.0, lp[np.arange(G), x] / lq[np.arange(G), x])
    assert np.abs(got["alpha"].double().cpu().numpy().ravel() - want).max() <= ALPHA_TOL, (b, want)
    L = 0
    while L < G and uniform_bits(SEED, BASE + b, L, 1) * 2.0 ** -53 < want[L]:
        L += 1
    assert int(got["accept_len"]) == L
    assert lp[L, int(got["next_token"])] > 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_a_call_per_temperature(dtype):
    svd, p, q = problem(dtype)
    ask = dict(temperature=dev(TEMPS), top_k=dev(TOP_K), top_p=dev(TOP_P))
    fp, fq = svd.filter_logits(p, **ask), svd.filter_logits(q, **ask)
    draft = svd.sample(q, seed=77, **ask)["token"].view(B, G)
    for b in range(B):
        t = float(TEMPS[b])
        say("prefix", b, "at", t)
        # the largest logit alone is left at 0: any temperature has its law
        r = svd.verify(fp[b:b + 1], fq[b:b + 1], draft[b:b + 1], temp_p=t or 0.3, seed=SEED,
                       row_base=BASE + b, want_alpha=True)
        check(b, t, p, q, draft, r)


def test_divided_logits_in_one_call():
    svd, p, q = problem(torch.float32)
    t = dev(np.where(TEMPS == 0, np.float32(1), TEMPS)).view(B, 1, 1)
    p, q = p / t, q / t
    k = np.where(TEMPS == 0, np.int32(1), TOP_K)
    ask = dict(top_k=dev(k), top_p=dev(TOP_P))
    fp, fq = svd.filter_logits(p, **ask), svd.filter_logits(q, **ask)
    draft = svd.sample(q, seed=77, **ask)["token"].view(B, G)
    r = svd.verify(fp, fq, draft, seed=SEED, row_base=BASE, want_alpha=True)
    for b in range(B):
        say("prefix", b)
        one = {n: r[n][b:b + 1] for n in ("alpha", "accept_len", "next_token")}
        check(b, 0.0 if TEMPS[b] == 0 else 1.0, p, q, draft, one)
