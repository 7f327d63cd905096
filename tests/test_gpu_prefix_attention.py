"""Attention over shared prefixes and with shaped scores against float64, row by row.
Tolerances: serve_ref.attention derives them."""
import numpy as np
import pytest
import torch

import serve_ref as S
import step_ref as R
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
BOTH = pytest.mark.parametrize("kind", ["bf16", "e4m3"])


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def problem(groups, T, Hq, Hkv, D, page, kind, lo, hi, tree, seed, spread=1.0, alone=0):
    """groups: (sequences, shared tokens) of each; alone: sequences behind them without a
    group; lo..hi own tokens.  Places that nobody has hold NaN."""
    svd = require_gpu()
    g = np.random.default_rng(seed)
    ctx, first, off = [], [], [0]
    for n, shared in groups:
        first += [len(ctx)] * n
        ctx += (shared + g.integers(lo, hi + 1, n)).tolist()
        off.append(len(ctx))
    first += range(len(ctx), len(ctx) + alone)
    ctx += g.integers(lo, hi + 1, alone).tolist()
    B = len(ctx)
    ctx = np.array(ctx, np.int32)
    nodes = g.integers(max(1, T // 2), T + 1, B).astype(np.int32)
    nodes[0] = T
    mp = (int(ctx.max()) + T + page - 1) // page + 1
    tab = g.permutation(B * mp + 2)[:B * mp].reshape(B, mp).astype(np.int32)
    for i, (n, shared) in enumerate(groups):
        b = off[i]
        tab[b:b + n, :shared // page] = tab[b, :shared // page]
    n_pages = B * mp + 2
    c = svd.kv_cache(n_pages, Hkv, page, D, dtype=KINDS[kind])
    for n in ("k", "v"):
        x = torch.from_numpy(g.standard_normal((n_pages, Hkv, page, D)).astype(np.float32)).cuda()
        if kind == "bf16":
            c[n].copy_(x * spread)
        else:
            c[n].copy_((x * 100).clamp(-448, 448))
            c[n + "_scale"].copy_(torch.from_numpy(g.integers(119, 124, (n_pages, Hkv, page))))
    free = torch.ones((n_pages, page), dtype=torch.bool)
    for b in range(B):
        p = np.arange(int(ctx[b]) + int(nodes[b]))
        free[tab[b, p // page], p % page] = False
    idx = free.cuda().unsqueeze(1).unsqueeze(-1).expand(n_pages, Hkv, page, D)
    for n in ("k", "v"):
        if kind == "bf16":
            c[n].masked_fill_(idx, float("nan"))
        else:
            c[n].view(torch.uint8).masked_fill_(idx, 0x7F)
    anc = depth = None
    if tree:
        on = np.zeros((B, T, T), bool)
        for b in range(B):
            for t in range(T):
                if t:
                    on[b, t] = on[b, g.integers(max(0, t - 7), t)]
                on[b, t, t] = True
        anc, depth = R.pack(on), (on.sum(2) - 1).astype(np.int32)
    q = torch.from_numpy(g.standard_normal((B, T, Hq, D)).astype(np.float32) * spread).to(
        torch.bfloat16).cuda()
    return dict(c=c, tab=tab, ctx=ctx, nodes=nodes, anc=anc, depth=depth, q=q,
                off=np.array(off, np.int32) if groups else None)


def run(svd, p, **kw):
    B, T, Hq, D = p["q"].shape
    out = torch.full((B, T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, Hq), 7.0, device="cuda")
    kw.setdefault("share_off", dev(p["off"]))
    if kw.get("slopes") is not None:
        kw["slopes"] = dev(np.asarray(kw["slopes"], np.float32))
        kw.setdefault("depth", dev(p["depth"]))
    r = svd.prefix_attention(p["q"], p["c"], dev(p["tab"]), dev(p["ctx"]), anc=dev(p["anc"]),
                             n_nodes=dev(p["nodes"]), out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return r["out"].double().cpu().numpy(), r["lse"].double().cpu().numpy()


def check(svd, p, scale=None, cap=0.0, slopes=None, only=None, **kw):
    D = p["q"].shape[3]
    got, lse = run(svd, p, scale=scale, cap=cap, slopes=slopes, **kw)
    want, wl, tol, ltol = S.attention(
        p["q"].double().cpu().numpy(), R.cache_values(p["c"], "k"), R.cache_values(p["c"], "v"),
        p["tab"], p["ctx"], p["nodes"], p["anc"], p["depth"], D ** -0.5 if scale is None else scale,
        cap, None if slopes is None else np.asarray(slopes, np.float32))
    for b in range(len(p["ctx"])) if only is None else only:
        n = int(p["nodes"][b])
        R.close(got[b, :n], want[b, :n], tol[b, :n], ("out", b))
        R.close(lse[b, :n], wl[b, :n], ltol[b, :n], ("lse", b))
        assert (got[b, n:] == 7.0).all() and (lse[b, n:] == 7.0).all()
    return got, lse


def slopes_of(Hq):
    return [2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)]


@BOTH
@pytest.mark.parametrize("case", [
    # groups, T, Hq, Hkv, D, page, own tokens, tree, alone
    ([(2, 128)], 1, 1, 1, 64, 16, 0, 0, False, 0),
    ([(2, 128)], 1, 4, 1, 128, 16, 1, 5, False, 0),
    ([(4, 300)], 1, 8, 2, 128, 16, 1, 60, False, 0),
    ([(3, 256)], 9, 4, 2, 128, 64, 0, 70, False, 1),
    ([(3, 385)], 9, 4, 4, 64, 32, 0, 70, True, 2),
    ([(1, 200), (5, 130), (2, 700)], 5, 6, 2, 128, 16, 3, 40, True, 0),
    ([(7, 512)], 20, 8, 2, 128, 128, 1, 200, True, 1),
    ([(2, 1000), (3, 640)], 65, 4, 1, 64, 16, 0, 90, True, 0),
    ([(9, 1100)], 9, 8, 2, 128, 64, 0, 50, False, 0),
    ([(6, 100)], 3, 4, 2, 128, 16, 0, 200, True, 0)],      # too few to share
    ids=lambda c: "%s_T%d_H%d.%d_D%d_p%d_%s" % ("+".join("%dx%d" % x for x in c[0]), *c[1:6],
                                               "tree" if c[8] else "chain"))
def test_shared_prefixes(kind, case):
    svd = require_gpu()
    say("prefix", kind, case)
    p = problem(*case[:6], kind, *case[6:9], seed=sum(case[1:6]), alone=case[9])
    check(svd, p)


@BOTH
@pytest.mark.parametrize("tree", [False, True], ids=["chain", "tree"])
@pytest.mark.parametrize("cap,sloped", [(5.0, False), (30.0, True), (0.0, True), (0.5, True)])
@pytest.mark.parametrize("T,group,D", [(1, 1, 64), (3, 4, 128), (9, 4, 128), (17, 3, 64),
                                       (40, 2, 128), (70, 4, 64)])
def test_shaped_scores(kind, tree, cap, sloped, T, group, D):
    svd = require_gpu()
    say("shaped", kind, tree, cap, sloped, T, group, D)
    p = problem([(2, 256)], T, 2 * group, 2, D, 32, kind, 0, 90, tree, seed=T + D, spread=1.5,
                alone=1)
    sl = slopes_of(2 * group) if sloped else None
    check(svd, p, cap=cap, slopes=sl)
    check(svd, p, cap=cap, slopes=sl, share_off=None)


def test_nothing_asked_is_tree_attention():
    svd = require_gpu()
    p = problem([(2, 256)], 9, 8, 2, 128, 64, "e4m3", 0, 700, True, seed=4)
    got, lse = run(svd, p, share_off=None)
    r = svd.tree_attention(p["q"], p["c"], dev(p["tab"]), dev(p["ctx"]), anc=dev(p["anc"]),
                           n_nodes=dev(p["nodes"]), want_lse=True)
    for b in range(2):
        n = int(p["nodes"][b])
        assert np.array_equal(r["out"][b, :n].double().cpu().numpy(), got[b, :n])
        assert np.array_equal(r["lse"][b, :n].double().cpu().numpy(), lse[b, :n])


@BOTH
def test_wrong_groups_change_nothing(kind):
    # groups whose tables differ, from the first page on or later; offsets that are out of
    # order, out of range, or leave sequences out; every sequence a group of its own
    svd = require_gpu()
    p = problem([(3, 512), (3, 256)], 5, 4, 2, 128, 16, kind, 5, 60, True, seed=8)
    for off in ([0, 6], [0, 2, 5, 6], [1, 3, 4], [0, 0, 3, 3, 6], [0, 1, 2, 3, 4, 5, 6], [3, 0],
                [0, 7], [-1, 3], [0, 4, 3, 6], [2, 2]):
        say(off)
        check(svd, p, share_off=dev(np.array(off, np.int32)))
    p["tab"][1, 20] = p["tab"][0, 21]
    check(svd, p)


@BOTH
def test_sequences_without_rows_or_with_bad_lengths(kind):
    svd = require_gpu()
    p = problem([(6, 512)], 4, 4, 2, 128, 16, kind, 5, 60, False, seed=9)
    mp = p["tab"].shape[1]
    p["nodes"][2] = 0
    p["tab"][2] = 1 << 30        # no rows: whatever its table holds
    p["ctx"][3] = mp * 16 - 3    # past its pages with the nodes
    p["nodes"][3] = 4
    p["ctx"][4] = -1
    p["nodes"][5] = 5            # more than T
    q = p["nodes"].copy()
    got, lse = run(svd, p)
    assert (got[2] == 7).all()
    for b in (3, 4, 5):
        assert np.isnan(got[b]).all() and np.isnan(lse[b]).all()
    p["nodes"][[2, 3, 4, 5]] = 0
    p["ctx"][[2, 3, 4, 5]] = 0
    p["tab"][2] = 0
    want = S.attention(p["q"].double().cpu().numpy(), R.cache_values(p["c"], "k"),
                       R.cache_values(p["c"], "v"), p["tab"], p["ctx"], p["nodes"], None, None,
                       128 ** -0.5)
    for b in (0, 1):
        n = q[b]
        R.close(got[b, :n], want[0][b, :n], want[2][b, :n], b)
        R.close(lse[b, :n], want[1][b, :n], want[3][b, :n], b)


@BOTH
def test_a_bad_page_in_the_shared_tokens(kind):
    # the same index out of range in all tables: all rows attend to it
    svd = require_gpu()
    p = problem([(3, 512)], 4, 4, 2, 128, 16, kind, 5, 60, False, seed=10, alone=1)
    p["tab"][:3, 7] = 1 << 30
    got, lse = run(svd, p)
    for b in range(3):
        n = int(p["nodes"][b])
        assert np.isnan(got[b, :n]).all() and np.isnan(lse[b, :n]).all()
    n = int(p["nodes"][3])
    assert np.isfinite(got[3, :n]).all()


@BOTH
def test_values_that_are_not_finite_reach_their_rows(kind):
    # NaN in a node that only some rows attend to, with shaped scores and without
    svd = require_gpu()
    p = problem([(2, 256)], 6, 2, 1, 64, 16, kind, 3, 30, True, seed=11)
    on = R.bits(p["anc"], 6)
    b, node = 0, 2
    at = int(p["ctx"][b]) + node
    v = p["c"]["v"]
    if kind == "bf16":
        v[p["tab"][b, at // 16], :, at % 16] = float("nan")
    else:
        v.view(torch.uint8)[p["tab"][b, at // 16], :, at % 16] = 0x7F
    for kw in (dict(), dict(cap=10.0, slopes=slopes_of(2))):
        got, _ = run(svd, p, **kw)
        for t in range(int(p["nodes"][b])):
            assert np.isnan(got[b, t]).all() == on[b, t, node] == np.isnan(got[b, t]).any()
    clean = [x for x in range(int(p["nodes"][b])) if not on[b, x, node]]
    assert clean


@BOTH
def test_rows_that_attend_to_nothing(kind):
    svd = require_gpu()
    p = problem([(2, 0)], 4, 2, 1, 64, 16, kind, 0, 0, True, seed=12)
    on = R.bits(p["anc"], 4)
    on[0, 2] = False
    p["anc"] = R.pack(on)
    for kw in (dict(), dict(cap=10.0), dict(slopes=slopes_of(2))):
        got, lse = check(svd, p, **kw)
        assert (got[0, 2] == 0).all() and (lse[0, 2] == -np.inf).all()
    # next to rows that share a prefix
    p = problem([(3, 256)], 4, 2, 1, 64, 16, kind, 0, 9, False, seed=13)
    check(svd, p, cap=3.0)


def test_extreme_scores():
    svd = require_gpu()
    # far above the cap, and a cap far above the scores
    p = problem([(2, 256)], 3, 4, 2, 64, 16, "bf16", 5, 60, True, seed=14, spread=6.0)
    for cap in (0.01, 1.0, 50.0, 1e4):
        check(svd, p, scale=1.0, cap=cap)
    # a NaN key reaches every row through the cap as well
    k = p["c"]["k"]
    k[p["tab"][1, 2], :, 3] = float("nan")
    got, lse = run(svd, p, cap=5.0)
    for b in range(2):
        shared = p["tab"][0, 2] == p["tab"][1, 2]
        n = int(p["nodes"][b])
        assert shared and np.isnan(got[b, :n]).all()
    # slopes of zero, large, and negative (scores that grow with distance)
    p = problem([(2, 256)], 3, 4, 2, 64, 16, "bf16", 5, 60, True, seed=15)
    check(svd, p, slopes=[0.0, 30.0, -0.02, 1e-6])


def test_many_parts_and_wide_tables():
    # one kv head, few rows, a long prefix: the shared tokens are cut into many parts, and the
    # table has room for many more than there are
    svd = require_gpu()
    p = problem([(3, 4096)], 2, 2, 1, 128, 64, "e4m3", 5, 300, False, seed=16)
    wide = np.zeros((3, 400), np.int32)
    wide[:, :p["tab"].shape[1]] = p["tab"]
    p["tab"] = wide
    assert svd.svd_prefix_attention_workspace_bytes(3, 2, 2, 1, 128, 400 * 64, 1) > 10000
    check(svd, p)
    check(svd, p, cap=4.0, slopes=slopes_of(2))


def test_strided_queries_and_refusals():
    svd = require_gpu()
    p = problem([(3, 256)], 4, 4, 2, 64, 16, "bf16", 5, 60, True, seed=17)
    B, T, Hq, D = p["q"].shape
    fused = torch.randn(B, T, 3 * Hq * D, dtype=torch.bfloat16, device="cuda")
    fused[..., :Hq * D] = p["q"].flatten(2)
    p["q"] = fused[..., :Hq * D].unflatten(-1, (Hq, D))
    check(svd, p)
    t, c = dev(p["tab"]), dev(p["ctx"])
    with pytest.raises(ValueError):
        svd.prefix_attention(p["q"], p["c"], t, c, share_off=dev(np.zeros(1, np.int32)))
    with pytest.raises(ValueError):
        svd.prefix_attention(p["q"], p["c"], t, c, anc=dev(p["anc"]), slopes=dev(np.ones(4, np.float32)))
    with pytest.raises(ValueError):
        svd.prefix_attention(p["q"], p["c"], t, c, slopes=dev(np.ones(5, np.float32)))
    with pytest.raises(TypeError):
        svd.prefix_attention(p["q"], p["c"], t, c, share_off=dev(np.zeros(3, np.int64)))
    with pytest.raises(ValueError):
        svd.prefix_attention(p["q"], p["c"], t, c, share_off=dev(np.zeros(9, np.int32)))
    with pytest.raises(svd.SvdError):
        svd.prefix_attention(p["q"], p["c"], t, c, cap=-1.0)
    n = svd.prefix_attention_workspace(B, T, Hq, p["c"], t, 1).numel()
    with pytest.raises(svd.SvdError) as e:
        svd.prefix_attention(p["q"], p["c"], t, c, share_off=dev(p["off"]),
                             workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == svd.SVD_EWORKSPACE
    with pytest.raises(ValueError, match="workspace must be on"):
        svd.prefix_attention(p["q"], p["c"], t, c, workspace=torch.empty(n, dtype=torch.uint8))
