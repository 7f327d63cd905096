"""Filtered and sampled logits of long rows against 64-bit references: every way in which a
row is held, and the values and ties that a held row can go wrong at."""
import math

import numpy as np
import pytest
import torch

import serve_ref as S
from gpu_util import require_gpu, say
from test_gpu_filter import DTYPES, TYPES, ask, check, rows

pytestmark = pytest.mark.gpu

# 16-byte pieces of 1024 threads end at 8192 bf16 (4096 fp32) tokens times 5, 10, 19 and 64;
# a row has one more where it begins between two
LONG = [8193, 8199, 40953, 40954, 40961, 81913, 81920, 81921, 155641, 155642, 155650, 262137,
        262138, 262144, 262145, 524281, 524282, 524289, 600001]


def lengths(*v):
    return pytest.mark.parametrize("V", v)


@DTYPES
@lengths(*LONG)
def test_lengths_at_which_the_way_changes(dtype, V):
    svd = require_gpu()
    say(dtype, V)
    g = np.random.default_rng(V)
    z = rows(g, 3, 1, V, dtype, 2.5)
    check(svd, z, [0.7, 1.0, 1.3], [0, 50, V - 1], [0.95, 1.0, 0.999], [0.0, 0.0, 1e-4])
    check(svd, z, p=[0.5, 0.9, 0.99])


def odd_rows(dtype, V):
    """Rows of values out of the ordinary, each with what it is."""
    g = np.random.default_rng(5)
    inf, t = math.inf, TYPES[dtype]
    low, top = torch.finfo(t).min, torch.finfo(t).max
    z = rows(g, 1, 24, V, dtype)[0]
    z[0] = -inf                       # nothing has a probability
    z[1, V // 2] = math.nan
    z[2, V - 1] = inf
    z[3] = -inf
    z[3, 7 * V // 8] = -5.0           # one token
    z[4, ::2] = -inf                  # a mask
    z[5] = 0.25                       # all equal
    z[6] = 0.0
    z[6, ::3] = -0.0                  # two zeros that are equal
    z[7] = low                        # masked with the lowest value, one token apart
    z[7, 3] = 1.0
    z[8] = low                        # nothing but that
    z[9, 9] = top
    z[10] = z[10].abs() * -1000       # all far below zero
    z[11] = -inf
    z[11, :20] = 1e-40                # below the least normal number
    z[12, V // 3:] = low              # a third is left
    z[13] *= 1e-9                     # smaller than the counters go
    z[14, 100:200] = 1e-12            # some of them
    z[15] = z[15] * 100 + 600         # past the counters
    z[16] -= 700                      # far down, with a maximum there too
    z[17] = 3.0
    z[17, 5] = 3.0 + 2.0 ** -6 * 4    # one above many equal ones
    z[18, :] = 511.0
    z[18, ::5] = 512.0                # across the counters' end
    z[19, 11] = -512.0
    z[20] = 2.0 ** -26
    z[20, ::2] = 2.0 ** -27
    z[21] = -(2.0 ** -26)
    z[21, 1] = 0.0
    z[22] = torch.arange(V, device="cuda").float().div(V).to(t)
    z[23] = -torch.arange(V, device="cuda").float().div(V / 16).to(t)
    return z.unsqueeze(0).contiguous()


ODD = [dict(), dict(k=[10]), dict(p=[0.5]), dict(p=[0.25], k=[100]), dict(t=[0.7], p=[0.9]),
       dict(least=[0.5]), dict(k=[-1], p=[0.999]), dict(t=[0.0]), dict(t=[200.0], p=[0.9])]


# the longest rows: four of the settings
@DTYPES
@pytest.mark.parametrize("V,one", [(V, one) for V in (8201, 20000, 50001, 100008, 200003)
                                   for one in range(len(ODD))
                                   if V <= 50001 or one in (1, 2, 4, 6)])
def test_rows_out_of_the_ordinary(dtype, V, one):
    svd = require_gpu()
    say(dtype, V, one)
    kw = {n: [V - 1 if n == "k" and x == -1 else x for x in v] for n, v in ODD[one].items()}
    # a bound on the mask's own tokens too: more are asked for than the mask leaves
    check(svd, odd_rows(dtype, V), u=np.random.default_rng(one).random((1, 1, 24)), **kw)


@DTYPES
@lengths(9000, 45001)
def test_more_tokens_asked_for_than_a_mask_leaves(dtype, V):
    svd = require_gpu()
    z = odd_rows(dtype, V)[:, [4, 7, 12, 3]].contiguous()
    for k in (V // 3 - 1, V // 3, V // 3 + 1, V // 2 + 1, V - 1, V):
        check(svd, z, k=[k])
        check(svd, z, k=[k], p=[0.9999999])


@DTYPES
@lengths(12001, 60000)
def test_ties_at_a_cut(dtype, V):
    """Equal tokens on both sides of a cut, spread over all waves' parts of the row."""
    svd = require_gpu()
    z = torch.full((1, 3, V), -3.0, device="cuda", dtype=TYPES[dtype])
    z[0, 0, 3::4] = 2.0
    z[0, 1, 1::1000] = 4.0
    z[0, 2, V // 2:] = 5.0
    m = z[0, 0].eq(2.0).sum().item()
    for k in (1, 2, m // 2, m - 1, m, m + 1, m + 1000):
        got, _ = check(svd, z, k=[k])
        if k <= m:
            assert np.flatnonzero(np.isfinite(got[0, 0])).tolist() == list(range(3, 3 + 4 * k, 4))
    for p in (1e-9, 0.1, 0.5, 0.9, 1 - 2.0 ** -20):
        check(svd, z, p=[p])


@lengths(30000, 270001)
def test_many_fp32_tokens_of_one_upper_half(V):
    """More tokens than can be listed around a cut, and a few, of different lower halves."""
    svd = require_gpu()
    g = np.random.default_rng(9)
    x = np.full((1, 3, V), -1.0, np.float32)
    low = g.permutation(1 << 15)
    x[0, 0] = 1.0 + np.resize(low, V) * 2.0 ** -23      # one upper half, every lower one
    x[0, 1, :3000] = 1.0 + low[:3000] * 2.0 ** -23
    x[0, 2] = -(1.0 + np.resize(low, V) * 2.0 ** -23)
    z = torch.from_numpy(x).cuda()
    for k in (1, 2, 1500, 2999, 3000, 3001, V // 2, V - 1):
        check(svd, z, k=[k])
    for p in (1e-6, 0.01, 0.3, 0.9):
        check(svd, z, p=[p])
        check(svd, z, p=[p], k=[2500])


@DTYPES
@lengths(8200, 8201, 33333, 90005, 160007)
def test_rows_begin_anywhere(dtype, V):
    """Rows that begin between two 16-byte pieces, in place and apart, and an output that
    begins elsewhere than its input."""
    svd = require_gpu()
    g = np.random.default_rng(V)
    z = rows(g, 1, 3, V, dtype)
    kw = ask([0.8], [77], [0.9], None)
    want = svd.filter_logits(z, **kw)
    check(svd, z, [0.8], [77], [0.9])
    for shift in (1, 3):
        wide = torch.full((z.numel() + 16,), 5.0, dtype=z.dtype, device="cuda")
        at = wide[shift:shift + z.numel()].view(z.shape)
        at.copy_(z)
        assert torch.equal(svd.filter_logits(at, **kw), want)      # apart, elsewhere
        assert svd.filter_logits(at, out=at, **kw) is at           # in place
        assert torch.equal(at, want)
        assert (wide[:shift] == 5).all() and (wide[shift + z.numel():] == 5).all()
        wide.fill_(5.0)
        svd.filter_logits(z, out=at, **kw)
        assert torch.equal(at, want)
        assert (wide[:shift] == 5).all() and (wide[shift + z.numel():] == 5).all()


@DTYPES
def test_many_rows_and_none(dtype):
    svd = require_gpu()
    g = np.random.default_rng(12)
    V = 8300
    z = rows(g, 70, 9, V, dtype)           # more rows than workgroups that fit at a time
    n = g.integers(0, 10, 70)
    n[:4] = [0, 9, -1, 10]
    check(svd, z, k=[20] * 70, p=[0.9] * 70, n_rows=n.tolist(), u=g.random((70, 1, 9)))


@DTYPES
def test_two_calls_at_once_and_replayed(dtype):
    """Calls on two streams at once, and a captured one replayed with other settings."""
    svd = require_gpu()
    g = np.random.default_rng(13)
    z = rows(g, 4, 3, 50021, dtype)
    y = rows(g, 4, 3, 50021, dtype)
    kw = ask([0.9] * 4, [300] * 4, [0.95] * 4, None)
    want_z, want_y = svd.filter_logits(z, **kw), svd.filter_logits(y, **kw)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, x in ((one, z), (two, y)):
            with torch.cuda.stream(s):
                got.append(svd.filter_logits(x, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want_y if i % 2 else want_z) for i, a in enumerate(got))
    out = torch.empty_like(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(one):
        svd.filter_logits(z, out=out, **kw)
        one.synchronize()
        with torch.cuda.graph(graph, stream=one):
            svd.filter_logits(z, out=out, **kw)
    for k in (5, 2000, 1):
        kw["top_k"].fill_(k)
        want = svd.filter_logits(z, **kw)
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@DTYPES
@lengths(1, 2, 7, 64, 511, 1000, 1003, 4097, 8191, 8192)
def test_many_rows_of_small_vocabularies(dtype, V):
    # more rows than are held at a time, with settings of their own
    svd = require_gpu()
    say(dtype, V)
    g = np.random.default_rng(V)
    B = 270
    z = rows(g, B, 1, V, dtype)
    t, k = g.uniform(0.3, 1.5, B), g.integers(0, 200, B)
    p, least = g.uniform(0.3, 1.05, B), np.where(g.random(B) < 0.5, 0.0, g.uniform(0, 0.2, B))
    check(svd, z, t, k, p, least, u=g.random((B, 2, 1)))


@DTYPES
@lengths(1009, 2048)
@pytest.mark.parametrize("one", range(len(ODD)))
def test_many_rows_out_of_the_ordinary(dtype, V, one):
    svd = require_gpu()
    say(dtype, V, one)
    z = odd_rows(dtype, V).repeat(11, 1, 1)
    kw = {n: [V - 1 if n == "k" and x == -1 else x for x in v] * 11 for n, v in ODD[one].items()}
    check(svd, z, u=np.random.default_rng(one).random((11, 1, 24)), **kw)
    # the same rows a few at a time are held: the same tokens
    few = svd.filter_logits(z[:1], **ask(*(None if kw.get(n) is None else kw[n][:1]
                                           for n in ("t", "k", "p", "least"))))
    many = svd.filter_logits(z, **ask(*(kw.get(n) for n in ("t", "k", "p", "least"))))
    same = (few[0] == many[5]) | (few[0].isnan() & many[5].isnan())
    assert same.all()


@DTYPES
@lengths(1009, 8201, 20000, 100008)
def test_rows_out_of_the_ordinary_in_place(dtype, V):
    svd = require_gpu()
    say(dtype, V)
    z = odd_rows(dtype, V)
    for one in (dict(), dict(top_k=[10]), dict(top_p=[0.5]), dict(temperature=[0.7], min_p=[0.3])):
        kw = {n: (torch.tensor(x, device="cuda") if n != "top_k" else
                  torch.tensor(x, dtype=torch.int32, device="cuda")) for n, x in one.items()}
        want = svd.filter_logits(z, **kw)
        same = z.clone()
        svd.filter_logits(same, out=same, **kw)
        assert ((same == want) | (same.isnan() & want.isnan())).all()
