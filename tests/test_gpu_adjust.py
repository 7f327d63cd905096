"""Penalties, biases and grammar masks against float64, token by token.
Tolerances: step_ref.adjust derives them (fp32 roundings, counted, and the output's own)."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def problem(B, T, V, H, seed, tree=True, bias=0, mask=True, pool=None):
    g = np.random.default_rng(seed)
    pool = min(V, 40) if pool is None else pool
    ids = g.permutation(V)[:pool]
    p = dict(history=ids[g.integers(0, pool, (B, H))].astype(np.int32),
             hist_len=g.integers(0, H + 1, B).astype(np.int32),
             tokens=ids[g.integers(0, pool, (B, T))].astype(np.int32),
             repetition=(0.7 + g.random(B)).astype(np.float32),
             frequency=(g.random(B) - 0.2).astype(np.float32),
             presence=(g.random(B) - 0.2).astype(np.float32))
    p["hist_len"][0] = H
    p["prompt_len"] = g.integers(0, H + 1, B).astype(np.int32)
    if H > 2:  # padding that no vocabulary has
        p["history"][:, 1] = -1
        p["history"][:, 2] = V
    on = np.zeros((B, T, T), bool)
    for b in range(B):
        for t in range(T):
            if t:
                on[b, t] = on[b, g.integers(max(0, t - 5), t)]
            on[b, t, t] = True
    p["anc"] = R.pack(on) if tree else None
    if bias:
        n = g.integers(0, bias + 1, B)
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        # some entries name the same token again, one no token at all
        tok = ids[g.integers(0, pool, off[-1])].astype(np.int32)
        if off[-1] > 3:
            tok[1] = -5
            tok[2] = V + 7
        p["bias"] = (off, tok, g.standard_normal(off[-1]).astype(np.float32))
    if mask:
        bits = g.random((5, V)) < np.array([[0.0], [0.02], [0.5], [0.98], [1.0]])
        p["allow"] = R.pack(bits)
        p["allow_index"] = g.integers(-1, 5, (B, T)).astype(np.int32)
    return p


def dev(x):
    if isinstance(x, tuple):
        return tuple(dev(y) for y in x)
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def check(svd, z, p, **kw):
    """Out of place, in place, and with the rows of n_rows only."""
    B, T, V = z.shape
    bf16 = z.dtype == torch.bfloat16
    want, tol = R.adjust(z.double().cpu().numpy(), bf16, **p)
    d = {n: dev(x) for n, x in p.items()}
    keep = z.clone()
    got = svd.adjust_logits(z, **d)
    assert torch.equal(z.view(torch.int16 if bf16 else torch.int32),
                       keep.view(torch.int16 if bf16 else torch.int32))
    R.close(got.double().cpu().numpy(), want, tol, "out of place")
    again = z.clone()
    assert svd.adjust_logits(again, out=again, **d) is again
    same = torch.int16 if bf16 else torch.int32
    assert torch.equal(again.view(same), got.view(same))
    n = torch.randint(0, T + 1, (B,), dtype=torch.int32, device="cuda")
    part = torch.full_like(z, 7.0)
    svd.adjust_logits(z, out=part, n_rows=n, **d)
    for b in range(B):
        k = int(n[b])
        assert (part[b, k:] == 7.0).all()
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [
    # B, T, V, H, bias, mask
    (1, 1, 1, 1, 0, False), (1, 1, 5, 3, 3, True), (2, 1, 1000, 50, 0, False),
    (3, 4, 1003, 200, 20, True), (2, 9, 8192, 64, 0, True), (2, 5, 8200, 64, 40, False),
    (1, 3, 20001, 300, 10, True), (1, 33, 4099, 100, 0, True), (2, 2, 152064, 40, 5, True),
    (1, 300, 515, 30, 8, True)],
    ids=lambda c: "B%d_T%d_V%d_H%d_b%d_%s" % (c[:5] + ("mask" if c[5] else "all",)))
def test_adjustments(dtype, case):
    svd = require_gpu()
    B, T, V, H, bias, mask = case
    say("adjust", dtype, case)
    p = problem(B, T, V, H, seed=sum(case[:5]), bias=bias, mask=mask, tree=T != 4)
    torch.manual_seed(V)
    z = (torch.randn(B, T, V, device="cuda") * 4).to(DT[dtype])
    check(svd, z, p)


@pytest.mark.parametrize("drop", ["repetition", "frequency", "presence", "prompt_len", "anc",
                                  "history", "tokens"])
def test_each_part_is_optional(drop):
    svd = require_gpu()
    p = problem(2, 6, 2050, 60, seed=3, bias=9)
    p.pop(drop)
    if drop == "history":
        p.pop("hist_len"), p.pop("prompt_len")
    if drop == "tokens":
        p.pop("anc")
    torch.manual_seed(1)
    check(svd, torch.randn(2, 6, 2050, device="cuda"), p)


def test_nothing_to_do_copies():
    svd = require_gpu()
    for dt, it in ((torch.bfloat16, torch.int16), (torch.float32, torch.int32)):
        raw = torch.randint(-2 ** 15, 2 ** 15, (2, 3, 1001 * (1 if it == torch.int16 else 2)),
                            device="cuda").to(torch.int16)
        z = raw.view(dt) if it == torch.int16 else raw.view(torch.int32).view(dt)
        got = svd.adjust_logits(z)
        assert torch.equal(got.view(it), z.view(it))  # NaN payloads too


def test_special_values():
    svd = require_gpu()
    V = 64
    z = torch.zeros(1, 1, V, device="cuda")
    z[0, 0, :6] = torch.tensor([float("inf"), -float("inf"), float("nan"), 0.0, -0.0, 5.0])
    p = dict(history=np.arange(6, dtype=np.int32).reshape(1, 6), hist_len=np.array([6], np.int32),
             repetition=np.array([2.0], np.float32), presence=np.array([0.5], np.float32),
             allow=R.pack(np.arange(V)[None] % 2 == 1), allow_index=np.array([[0]], np.int32))
    got = svd.adjust_logits(z, **{n: dev(x) for n, x in p.items()}).cpu().numpy()[0, 0]
    assert np.isneginf(got[0::2]).all()          # masked, whatever stood there
    assert np.isneginf(got[1]) and got[3] == -0.5 and got[5] == 2.0
    assert (got[7::2] == 0).all()


def test_counts_of_long_histories():
    svd = require_gpu()
    # one token thousands of times, so that counts and their sum are exact or nothing
    B, V, H = 2, 3000, 20000
    g = np.random.default_rng(5)
    h = g.integers(0, 4, (B, H)).astype(np.int32) * 700
    p = dict(history=h, hist_len=np.array([H, 12345], np.int32),
             prompt_len=np.array([0, 345], np.int32), frequency=np.array([1.0, 0.5], np.float32))
    z = torch.zeros(B, 1, V, device="cuda")
    got = svd.adjust_logits(z, **{n: dev(x) for n, x in p.items()}).cpu().numpy()
    for b in range(B):
        cnt = np.bincount(h[b, p["prompt_len"][b]:p["hist_len"][b]], minlength=V)
        assert np.array_equal(got[b, 0], -cnt * p["frequency"][b].astype(np.float64) + 0.0)


def test_repeated_bias_entries_add_in_order():
    svd = require_gpu()
    V = 9000
    tok = np.array([5, 8999, 5, 5, 17, 8999], np.int32)
    val = np.array([1e8, 1.0, 1.0, -1e8, 0.25, -3.0], np.float32)
    off = np.array([0, 6], np.int32)
    z = torch.zeros(1, 1, V, device="cuda")
    got = svd.adjust_logits(z, bias=(dev(off), dev(tok), dev(val))).cpu().numpy()[0, 0]
    s = np.float32(0)
    for x in (1e8, 1.0, -1e8):
        s = np.float32(s + np.float32(x))
    assert got[5] == s and got[8999] == -2.0 and got[17] == 0.25 and np.count_nonzero(got) <= 3


def test_offsets_of_the_bias_stay_in_its_list():
    svd = require_gpu()
    z = torch.zeros(3, 1, 100, device="cuda")
    off = torch.tensor([-4, 2, 50, 1], dtype=torch.int32, device="cuda")
    tok = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    val = torch.ones(3, device="cuda")
    got = svd.adjust_logits(z, bias=(off, tok, val)).cpu().numpy()[:, 0]
    assert np.flatnonzero(got[0]).tolist() == [1, 2]
    assert np.flatnonzero(got[1]).tolist() == [3] and not got[2].any()


def test_data_errors_give_nan_rows():
    svd = require_gpu()
    B, T, V = 5, 3, 777
    p = problem(B, T, V, 20, seed=8)
    p["allow_index"][:] = -1
    z = torch.randn(B, T, V, device="cuda").to(torch.bfloat16)
    base = svd.adjust_logits(z, **{n: dev(x) for n, x in p.items()})
    p["hist_len"][1] = -1
    p["hist_len"][2] = 21
    p["allow_index"][3, 1] = 5
    n = np.array([3, 3, 3, 3, 4], np.int32)
    got = svd.adjust_logits(z, n_rows=dev(n), **{n_: dev(x) for n_, x in p.items()})
    nan = torch.isnan(got)
    assert torch.equal(got[0], base[0]) and nan[1].all() and nan[2].all() and nan[4].all()
    assert nan[3, 1].all() and torch.equal(got[3, 0], base[3, 0]) and torch.equal(got[3, 2], base[3, 2])


def test_a_bad_history_leaves_the_rows_behind_n_rows():
    svd = require_gpu()
    z = torch.randn(2, 4, 100, device="cuda")
    h = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    n = torch.tensor([2, 3], dtype=torch.int32, device="cuda")
    out = torch.full_like(z, 7.0)
    svd.adjust_logits(z, history=h, hist_len=torch.tensor([6, 0], dtype=torch.int32, device="cuda"),
                      n_rows=n, out=out)
    assert torch.isnan(out[0, :2]).all() and (out[0, 2:] == 7.0).all()
    assert torch.equal(out[1, :3], z[1, :3]) and (out[1, 3:] == 7.0).all()


def test_rows_past_32_bits():
    svd = require_gpu()
    # 32768 rows of 152064: 5e9 elements; only the last rows change
    B, T, V = 8, 4096, 152064
    z = torch.zeros((B, T, V), dtype=torch.bfloat16, device="cuda")
    h = torch.full((B, 2), V - 1, dtype=torch.int32, device="cuda")
    n = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    f = torch.arange(1.0, B + 1, device="cuda")
    svd.adjust_logits(z, history=h, hist_len=n, frequency=f, out=z)
    assert torch.equal(z[:, :, V - 1].float(), (-2 * f).view(B, 1).expand(B, T))
    assert not z[:, :, 0].any() and not z[B - 1, T - 1, :V - 1].any()


def test_side_stream_and_repeatability():
    svd = require_gpu()
    p = problem(3, 9, 20001, 500, seed=21, bias=30)
    z = torch.randn(3, 9, 20001, device="cuda")
    d = {n: dev(x) for n, x in p.items()}
    a = svd.adjust_logits(z, **d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = svd.adjust_logits(z, **d)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
