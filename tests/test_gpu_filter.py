"""Filtered and sampled logits against 64-bit references: which tokens are kept, exactly,
and the draws among them."""
import math

import numpy as np
import pytest
import torch

import serve_ref as S
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DTYPES = pytest.mark.parametrize("dtype", sorted(TYPES))


def f32(x):
    return None if x is None else torch.tensor(np.asarray(x, np.float32), device="cuda")


def i32(x):
    return None if x is None else torch.tensor(np.asarray(x, np.int32), device="cuda")


def rows(g, B, T, V, dtype, spread=2.0):
    z = torch.from_numpy((g.standard_normal((B, T, V)) * spread).astype(np.float32)).cuda()
    return z.to(TYPES[dtype])


def ask(t, k, p, least):
    return dict(temperature=f32(t), top_k=i32(k), top_p=f32(p), min_p=f32(least))


def settings(t, k, p, least, b):
    """The settings of prefix b as the library has them, in fp32."""
    def one(x, off):
        return off if x is None else float(np.float32(x[b]))
    return one(t, 1.0), int(one(k, 0)), one(p, 1.0), one(least, 0.0)


def check(svd, z, t=None, k=None, p=None, least=None, n_rows=None, u=None):
    B, T, V = z.shape
    host = z.float().cpu().numpy()
    out = torch.full_like(z, 7.0)
    n = i32(n_rows)
    r = svd.filter_logits(z, n_rows=n, out=out, **ask(t, k, p, least))
    assert r is out
    K = 3 if u is None else u.shape[1]
    if u is None:
        u = np.random.default_rng(B + T + V).random((B, K, T))
    tok = torch.full((B, K, T), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((B, K, T), 7.0, device="cuda")
    svd.sample(z, torch.from_numpy(u).cuda(), n_rows=n, token=tok, logprob=lp,
               **ask(t, k, p, least))
    torch.cuda.synchronize()
    got, tok, lp = out.float().cpu().numpy(), tok.cpu().numpy(), lp.cpu().numpy()
    for b in range(B):
        mine = settings(t, k, p, least, b)
        m = T if n_rows is None else n_rows[b]
        for r in range(T):
            if 0 <= m <= T and r >= m:
                assert (got[b, r] == 7).all() and (tok[b, :, r] == -7).all()
                assert (lp[b, :, r] == 7).all()
                continue
            row = host[b, r].astype(np.float64)
            keep = S.kept(row, *mine) if 0 <= m <= T else None
            if keep is None:
                assert np.isnan(got[b, r]).all() and (tok[b, :, r] == -1).all(), (b, r)
                assert np.isnan(lp[b, :, r]).all()
                continue
            want = np.where(keep, host[b, r], -np.inf)
            assert np.array_equal(got[b, r], want), (b, r, int(keep.sum()),
                                                     int(np.isfinite(got[b, r]).sum()))
            for d in range(K):
                v, x = S.draw(row, keep, mine[0], u[b, d, r])
                assert tok[b, d, r] == v, (b, r, d)
                assert abs(lp[b, d, r] - x) <= S.logprob_tol(x, V), (b, r, d)
    return got, tok


@DTYPES
@pytest.mark.parametrize("V", [1, 2, 7, 63, 1000, 1003, 4097, 8192, 8200, 20011, 100003, 152064])
def test_all_settings_at_once(dtype, V):
    svd = require_gpu()
    say(dtype, V)
    g = np.random.default_rng(V)
    B = 9
    z = rows(g, B, 2, V, dtype)
    t = g.uniform(0.3, 1.5, B)
    k = g.integers(0, 200, B)
    p = g.uniform(0.3, 1.05, B)
    least = np.where(g.random(B) < 0.5, 0.0, g.uniform(0, 0.2, B))
    check(svd, z, t, k, p, least)


@DTYPES
@pytest.mark.parametrize("only", ["t", "k", "p", "least"])
def test_each_setting_alone(dtype, only):
    svd = require_gpu()
    g = np.random.default_rng(3)
    z = rows(g, 6, 3, 5003, dtype, 3.0)
    val = {"t": [0.1, 0.5, 1.0, 2.0, 30.0, 1e-3], "k": [1, 2, 50, 5002, 5003, 9999],
           "p": [0.01, 0.5, 0.9, 0.99, 0.9999, 0.999999], "least": [1.0, 0.5, 0.1, 0.01, 1e-6, 1e-30]}
    check(svd, z, **{only: val[only]})
    check(svd, z)  # nothing asked: all are kept


@DTYPES
def test_settings_out_of_the_ordinary(dtype):
    svd = require_gpu()
    g = np.random.default_rng(4)
    z = rows(g, 16, 1, 777, dtype)
    inf, nan = math.inf, math.nan
    t = [0.0, -0.0, -1.0, inf, nan, 1e-45, 1e-30, 3e38, 1, 1, 1, 1, 1, 1, 0.0, 1]
    k = [0, 5, 5, 5, 5, 5, 0, 0, -3, 1 << 31 - 1, 5, 5, 5, 0, 7, -(1 << 31)]
    p = [0.5, 1, 1, 1, 1, 1, 0.5, 0.5, 0.0, -1.0, nan, 2.0, inf, 1e-45, 0.1, -inf]
    least = [0, 0, 0, 0, 0, 0, 0, 0, 1.0, 2.0, 0, nan, inf, -1.0, 0.5, -inf]
    got, tok = check(svd, z, t, np.array(k, np.int64).clip(-(1 << 31), (1 << 31) - 1), p, least)
    assert (tok[[2, 3, 4, 10, 11]] == -1).all() and (np.isfinite(got[0]).sum() == 1)


@DTYPES
def test_rows_out_of_the_ordinary(dtype):
    svd = require_gpu()
    g = np.random.default_rng(5)
    V, inf, nan = 1009, math.inf, math.nan
    z = rows(g, 1, 14, V, dtype)[0]
    z[0] = -inf                       # nothing has a probability
    z[1, 500] = nan
    z[2, 1008] = inf
    z[3] = -inf
    z[3, 77] = -5.0                   # one token
    z[4, ::2] = -inf                  # a mask
    z[5] = 0.25                       # all equal
    z[6] = 0.0
    z[6, ::3] = -0.0                  # two zeros that are equal
    z[7] = torch.finfo(TYPES[dtype]).min   # masked with the lowest value, one token apart
    z[7, 3] = 1.0
    z[8] = torch.finfo(TYPES[dtype]).min   # nothing but that
    z[9, 9] = torch.finfo(TYPES[dtype]).max
    z[10] = z[10].abs() * -1000
    z[11] = -inf
    z[11, :20] = 1e-40                # below the least normal number
    z[12] = torch.arange(V, device="cuda").to(z.dtype) / 100
    z[13] = -torch.arange(V, device="cuda").to(z.dtype) / 100
    z = z.unsqueeze(0).contiguous()
    # 1.0 and 3.0 of the largest type are exact weights: sums of ties are decided exactly
    for one in (dict(), dict(k=[10]), dict(p=[0.5]), dict(p=[0.25], k=[100]), dict(t=[0.7], p=[0.9]),
                dict(least=[0.5]), dict(k=[1008], p=[0.999]), dict(t=[0.0])):
        check(svd, z, **one)


@DTYPES
def test_ties_go_to_the_lowest_index(dtype):
    svd = require_gpu()
    V = 30011
    z = torch.full((1, 4, V), -3.0, device="cuda", dtype=TYPES[dtype])
    z[0, 0, ::7] = 2.0     # 4288 equal ones
    z[0, 1] = 1.0
    z[0, 2, V // 2:] = 5.0
    z[0, 3, -1] = 9.0
    z[0, 3, 5:25] = 8.0
    for k in (1, 3, 100, 4287, 4288, 4289, 9000):
        got, _ = check(svd, z, k=[k])
        first = np.flatnonzero(np.isfinite(got[0, 0]))
        if k <= 4288:
            assert first.tolist() == list(range(0, 7 * k, 7))
    for p in (0.1, 0.5, 0.75, 0.999):
        check(svd, z, p=[p])
        check(svd, z, p=[p], k=[17])


@DTYPES
def test_some_rows_only(dtype):
    svd = require_gpu()
    g = np.random.default_rng(6)
    z = rows(g, 6, 5, 3001, dtype)
    check(svd, z, k=[9] * 6, p=[0.9] * 6, n_rows=[0, 1, 5, 6, -1, 3])


@DTYPES
def test_in_place_and_apart(dtype):
    svd = require_gpu()
    g = np.random.default_rng(7)
    for V in (2048, 2049):
        z = rows(g, 3, 4, V, dtype)
        kw = ask(None, [4, 0, 40], [0.9, 0.5, 1.0], None)
        want = svd.filter_logits(z, **kw)
        assert want.data_ptr() != z.data_ptr()
        same = z.clone()
        assert svd.filter_logits(same, out=same, **kw) is same
        assert torch.equal(same, want)
        # rows that do not begin at 16 bytes
        wide = torch.zeros(z.numel() + 1, dtype=z.dtype, device="cuda")
        off = wide[1:].view(z.shape)
        off.copy_(z)
        assert torch.equal(svd.filter_logits(off, **kw), want)
        with pytest.raises(svd.SvdError):
            svd.filter_logits(wide[:-1].view(z.shape), out=off, **kw)


def test_kept_bits_are_the_logits_own():
    # -0.0 stays -0.0, and what is filtered twice stays as it is
    svd = require_gpu()
    z = torch.tensor([[[-0.0, 0.0, -1.0, 3.0]]], device="cuda")
    out = svd.filter_logits(z, top_k=i32([3]))
    assert out.view(torch.int32).tolist() == [[[-(1 << 31), 0, -0x800000, 0x40400000]]]
    assert torch.equal(svd.filter_logits(out, top_k=i32([3])), out)


@DTYPES
def test_ends_of_the_unit_interval(dtype):
    svd = require_gpu()
    g = np.random.default_rng(8)
    z = rows(g, 2, 3, 9001, dtype)
    z[0, 0, :40] = -math.inf  # no weight at the ends
    z[0, 0, -40:] = -math.inf
    u = np.zeros((2, 6, 3))
    u[:, 1] = 1 - 2.0 ** -53
    u[:, 2] = 2.0 ** -53
    u[:, 3] = 0.5
    u[:, 4] = 2.0 ** -1074
    u[:, 5] = 1 - 2.0 ** -30
    _, tok = check(svd, z, u=u)
    assert tok[0, 0, 0] >= 40 and tok[0, 1, 0] < 9001 - 40
    check(svd, z, k=[5, 5], u=u)
    # a u outside [0, 1) has no token, and the others of its row have theirs
    bad = np.array([1.0, -1e-9, math.nan, math.inf, 0.25, 2.0]).reshape(1, 6, 1).repeat(3, 2)
    r = svd.sample(z[:1].contiguous(), torch.from_numpy(bad).cuda(), want_logprob=True)
    t, lp = r["token"].cpu().numpy(), r["logprob"].cpu().numpy()
    off = [0, 1, 2, 3, 5]
    assert (t[0, off] == -1).all() and np.isnan(lp[0, off]).all()
    assert (t[0, 4] >= 0).all() and (lp[0, 4] < 0).all()


@pytest.mark.parametrize("K", [1, 5, 64])
def test_draws_from_the_counter_hash(K):
    svd = require_gpu()
    g = np.random.default_rng(9)
    B, T, V, seed, base = 3, 2, 2003, 0x1234567890ABCDEF, (1 << 64) - 2
    z = rows(g, B, T, V, "bf16")
    u = np.array([[[S.hash_uniform(seed, base + b, k, t, T) for t in range(T)] for k in range(K)]
                  for b in range(B)])
    kw = ask([0.8] * B, [60] * B, None, None)
    want = svd.sample(z, torch.from_numpy(u).cuda(), want_logprob=True, **kw)
    got = svd.sample(z, K=K, seed=seed, row_base=base, want_logprob=True, **kw)
    assert torch.equal(got["token"], want["token"])
    assert torch.equal(got["logprob"], want["logprob"])
    assert svd.sample(z, K=K, seed=seed, row_base=base, **kw)["logprob"] is None


def test_draws_follow_the_law():
    # 64 equally spaced uniforms cut the law into 64 equal shares: a token of probability q is
    # drawn from 64 q - 1 to 64 q + 1 times, by the definition of the inverse
    svd = require_gpu()
    g = np.random.default_rng(10)
    T, V = 8, 40
    z = rows(g, 1, T, V, "f32", 1.0)
    u = ((np.arange(64) + 0.5) / 64).reshape(1, 64, 1).repeat(T, 2)
    tok = svd.sample(z, torch.from_numpy(u).cuda(), top_k=i32([12]))["token"].cpu().numpy()
    for t in range(T):
        row = z[0, t].double().cpu().numpy()
        q = np.where(S.kept(row, k=12), np.exp(row), 0)
        q /= q.sum()
        n = np.bincount(tok[0, :, t], minlength=V)
        assert (np.abs(n - 64 * q) <= 1 + 1e-9).all()


def test_a_vocabulary_of_many_parts():
    # more tokens than 1024 parts of 8192
    svd = require_gpu()
    V = 1024 * 8192 + 12345
    g = np.random.default_rng(11)
    z = rows(g, 1, 1, V, "bf16")
    u = np.array([0.0, 0.3, 0.77, 1 - 2.0 ** -53]).reshape(1, 4, 1)
    check(svd, z, p=[0.5], u=u)
    check(svd, z, k=[1 << 20], u=u)


def test_offsets_past_32_bits():
    # the last row begins behind 2^32 bytes and 2^31 elements
    svd = require_gpu()
    V = 152064
    T = (1 << 31) // V + 2
    if T > 4096:
        B, T = (T + 4095) // 4096, 4096
    else:
        B = 1
    z = torch.zeros((B, T, V), dtype=torch.bfloat16, device="cuda")
    g = np.random.default_rng(12)
    z[-1, -1] = rows(g, 1, 1, V, "bf16")[0, 0]
    z[0, 0] = rows(g, 1, 1, V, "bf16")[0, 0]
    say("rows", B * T)
    kw = ask(None, [50] * B, [0.9] * B, None)
    u = torch.full((B, 1, T), 0.4, dtype=torch.float64, device="cuda")
    tok = svd.sample(z, u, **kw)["token"]
    want = [svd.sample(z[i, j].view(1, 1, V), u[:1, :, :1].contiguous(), **ask(None, [50], [0.9], None))
            ["token"] for i, j in ((0, 0), (-1, -1))]
    assert int(tok[0, 0, 0]) == int(want[0]) and int(tok[-1, 0, -1]) == int(want[1])
    small = svd.filter_logits(z[-1, -1].view(1, 1, V), **ask(None, [50], [0.9], None))
    svd.filter_logits(z, out=z, **kw)
    assert torch.equal(z[-1, -1], small[0, 0])
    # equal logits: of the first 50 nine tenths, the first 45 (0.9 in fp32 is below nine tenths)
    assert int((z[0, 1] == 0).sum()) == 45 and (z[-1, 0, :45] == 0).all()
