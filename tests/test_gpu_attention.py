"""Attention of a draft tree over the paged cache against float64, row by row.
Tolerances: step_ref.attention derives them (fp32 sums of the products, one
rounding of each probability to bf16, the output's rounding)."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def problem(B, T, Hq, Hkv, D, page, kind, lo, hi, tree, seed, spread=1.0, chain_nodes=True):
    """Random cache, table, lengths and tree; the pages no sequence owns and the places
    behind a sequence's end hold NaN."""
    g = np.random.default_rng(seed)
    ctx = g.integers(lo, hi + 1, B).astype(np.int32)
    nodes = g.integers(max(1, T // 2), T + 1, B).astype(np.int32)
    nodes[0] = T
    mp = (hi + T + page - 1) // page + 1
    n_pages = B * mp + 2
    svd = require_gpu()
    c = svd.kv_cache(n_pages, Hkv, page, D, dtype=KINDS[kind])
    for n in ("k", "v"):
        x = torch.from_numpy(g.standard_normal((n_pages, Hkv, page, D)).astype(np.float32)).cuda()
        if kind == "bf16":
            c[n].copy_(x * spread)
        else:
            c[n].copy_((x * 100).clamp(-448, 448))
            c[n + "_scale"].copy_(torch.from_numpy(g.integers(119, 124, (n_pages, Hkv, page))))
    tab = g.permutation(n_pages)[:B * mp].reshape(B, mp).astype(np.int32)
    nan = torch.ones((n_pages, page), dtype=torch.bool)
    for b in range(B):
        for p in range(int(ctx[b]) + int(nodes[b])):
            nan[tab[b, p // page], p % page] = False
    idx = nan.cuda().unsqueeze(1).unsqueeze(-1).expand(n_pages, Hkv, page, D)
    for n in ("k", "v"):
        if kind == "bf16":
            c[n].masked_fill_(idx, float("nan"))
        else:
            c[n].view(torch.uint8).masked_fill_(idx, 0x7F)
    anc = None
    if tree:
        on = np.zeros((B, T, T), bool)
        for b in range(B):
            for t in range(T):
                if t:
                    on[b, t] = on[b, g.integers(max(0, t - 7), t)]
                on[b, t, t] = True
        anc = R.pack(on)
    q = torch.from_numpy(g.standard_normal((B, T, Hq, D)).astype(np.float32) * spread).to(
        torch.bfloat16).cuda()
    return dict(c=c, tab=tab, ctx=ctx, nodes=nodes, anc=anc, q=q)


def dev(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def run(svd, p, scale=None, **kw):
    B, T, Hq, D = p["q"].shape
    out = torch.full((B, T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, Hq), 7.0, device="cuda")
    r = svd.tree_attention(p["q"], p["c"], dev(p["tab"]), dev(p["ctx"]), anc=dev(p["anc"]),
                           n_nodes=dev(p["nodes"]), scale=scale, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return r["out"].double().cpu().numpy(), r["lse"].double().cpu().numpy()


def check(svd, p, scale=None):
    D = p["q"].shape[3]
    got, lse = run(svd, p, scale)
    s = D ** -0.5 if scale is None else scale
    want, wl, tol, ltol = R.attention(
        p["q"].double().cpu().numpy(), R.cache_values(p["c"], "k"), R.cache_values(p["c"], "v"),
        p["tab"], p["ctx"], p["nodes"], p["anc"], s)
    for b in range(len(p["ctx"])):
        n = int(p["nodes"][b])
        R.close(got[b, :n], want[b, :n], tol[b, :n], ("out", b))
        R.close(lse[b, :n], wl[b, :n], ltol[b, :n], ("lse", b))
        assert (got[b, n:] == 7.0).all() and (lse[b, n:] == 7.0).all()
    return got, lse


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", [
    # B, T, Hq, Hkv, D, page, shortest, longest context, tree
    (1, 1, 1, 1, 64, 16, 0, 0, False), (1, 1, 8, 8, 128, 16, 1, 1, False),
    (2, 1, 8, 2, 128, 16, 31, 34, False), (3, 1, 16, 1, 64, 64, 200, 700, False),
    (3, 2, 7, 1, 128, 32, 15, 65, True), (2, 9, 8, 2, 128, 64, 0, 130, False),
    (4, 9, 4, 4, 64, 16, 0, 40, True), (2, 33, 4, 2, 128, 16, 3, 97, True),
    (2, 65, 6, 2, 64, 128, 0, 300, True), (1, 129, 8, 1, 128, 64, 100, 100, True),
    (1, 40, 5, 5, 128, 1024, 900, 900, True), (1, 17, 3, 1, 64, 32, 1500, 1500, False)],
    ids=lambda c: "B%d_T%d_H%d.%d_D%d_p%d_n%d-%d_%s" % (c[:8] + ("tree" if c[8] else "chain",)))
def test_attention(kind, case):
    svd = require_gpu()
    say("attention", kind, case)
    check(svd, problem(*case[:6], kind, *case[6:9], seed=sum(case[:8])))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_parts_of_a_long_context(kind):
    # one sequence with room for many more tokens than it has: the parts of its room
    # that hold nothing join as nothing
    svd = require_gpu()
    p = problem(2, 3, 4, 1, 128, 64, kind, 900, 1500, True, seed=5)
    wide = np.zeros((2, 400), np.int32)
    wide[:, :p["tab"].shape[1]] = p["tab"]
    p["tab"] = wide
    assert svd.svd_tree_attention_workspace_bytes(2, 3, 4, 1, 128, 400 * 64) > 4096
    check(svd, p)
    p["ctx"][:] = [0, 5]
    p["nodes"][:] = [1, 2]
    nan_tail = p  # the rest of its pages is unread
    check(svd, nan_tail)


def test_scales_and_large_scores():
    svd = require_gpu()
    for scale, spread in ((0.001, 1.0), (1.0, 4.0), (3.0, 6.0)):
        check(svd, problem(2, 5, 4, 2, 64, 16, "bf16", 50, 120, True, seed=9, spread=spread),
              scale=scale)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_rows_that_attend_to_nothing(kind):
    svd = require_gpu()
    p = problem(3, 6, 4, 2, 128, 16, kind, 0, 20, True, seed=12)
    p["ctx"][:] = [0, 0, 20]
    on = R.bits(p["anc"], 6)
    on[0, 2] = False
    on[1] = False
    on[2, 1] = False
    p["anc"] = R.pack(on)
    got, lse = check(svd, p)
    assert (got[0, 2] == 0).all() and np.isneginf(lse[0, 2]).all()
    # every row of a prefix without nodes stays
    p["nodes"][1] = 0
    got, lse = check(svd, p)
    assert (got[1] == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_masked_places_do_not_leak(kind, value):
    # a node with non-finite keys and values reaches the rows that attend to it only
    svd = require_gpu()
    T = 40
    p = problem(2, T, 4, 2, 128, 16, kind, 7, 50, True, seed=14)
    base, base_lse = check(svd, p)
    on = R.bits(p["anc"], T)
    for b in range(2):
        for node in (3, 11):
            pos = int(p["ctx"][b]) + node
            pg, pl = int(p["tab"][b, pos // 16]), pos % 16
            if kind == "bf16":
                p["c"]["v"][pg, :, pl, 5:9] = value
                if node == 11:
                    p["c"]["k"][pg, :, pl] = value
            else:  # the only code that is not finite
                p["c"]["v"].view(torch.uint8)[pg, :, pl, 5:9] = 0xFF
    got, lse = run(svd, p)
    for b in range(2):
        for t in range(int(p["nodes"][b])):
            hit = on[b, t, 3] or on[b, t, 11]
            if not hit:
                assert np.array_equal(got[b, t], base[b, t]), (b, t)
                assert np.array_equal(lse[b, t], base_lse[b, t])
            elif kind == "bf16" and on[b, t, 11]:
                # the reference's own arithmetic: exp(inf - inf), 0 * inf and NaN are NaN;
                # a score of -inf has no weight but a NaN product
                assert not np.isfinite(got[b, t, :, 5:9]).any()
            else:
                bad = ~np.isfinite(got[b, t])
                assert bad[:, 5:9].all() and not bad[:, :5].any() and not bad[:, 9:].any()
                if kind == "bf16" and not np.isnan(value):
                    assert (got[b, t, :, 5:9] == value).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("wide", [False, True])
def test_data_errors_give_nan(kind, wide):
    svd = require_gpu()
    p = problem(5, 4, 4, 2, 64, 16, kind, 40, 60, True, seed=15)
    if wide:  # room for parts
        t = np.zeros((5, 600), np.int32)
        t[:, :p["tab"].shape[1]] = p["tab"]
        p["tab"] = t
    base, base_lse = run(svd, p)
    p["ctx"][1] = -1
    p["nodes"][2] = 5
    p["ctx"][3] = p["tab"].shape[1] * 16 - 1
    p["nodes"][3] = 2
    p["tab"][4, 1] = 1 << 20
    got, lse = run(svd, p)
    assert np.array_equal(got[0], base[0]) and np.array_equal(lse[0], base_lse[0])
    for b in (1, 2, 3):
        assert np.isnan(got[b]).all() and np.isnan(lse[b]).all(), b
    n = int(p["nodes"][4])
    assert np.isnan(got[4, :n]).all() and np.isnan(lse[4, :n]).all() and (got[4, n:] == 7.0).all()
    p["tab"][4, 1] = -1
    got, _ = run(svd, p)
    assert np.isnan(got[4, :n]).all()


def test_strided_queries_and_streams():
    svd = require_gpu()
    p = problem(3, 9, 8, 2, 128, 16, "e4m3", 100, 200, False, seed=16)
    want, wl = run(svd, p)
    B, T, Hq, D = p["q"].shape
    fused = torch.zeros((B, T, Hq * D + 512), dtype=torch.bfloat16, device="cuda")
    fused[:, :, 256:256 + Hq * D] = p["q"].reshape(B, T, Hq * D)
    p["q"] = fused[:, :, 256:256 + Hq * D].view(B, T, Hq, D)
    assert not p["q"].is_contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, lse = run(svd, p)
    assert np.array_equal(got, want) and np.array_equal(lse, wl)
    got, lse = run(svd, p, stream=side.cuda_stream)
    assert np.array_equal(got, want)


def test_a_cache_past_32_bits():
    svd = require_gpu()
    n, H, page, D = 40000, 8, 64, 128   # 5.2 GB each of keys and values
    c = {x: torch.zeros((n, H, page, D), dtype=torch.bfloat16, device="cuda") for x in "kv"}
    c.update(k_scale=None, v_scale=None)
    small = svd.kv_cache(6, H, page, D)
    torch.manual_seed(2)
    for x in "kv":
        small[x].copy_(torch.randn(small[x].shape, device="cuda"))
    far = [n - 1, 33000, 0, n - 2, 20000, n - 3]
    for i, f in enumerate(far):
        for x in "kv":
            c[x][f] = small[x][i]
    q = torch.randn(1, 3, 16, D, device="cuda", dtype=torch.bfloat16)
    ctx = torch.tensor([370], dtype=torch.int32, device="cuda")
    a = svd.tree_attention(q, small, torch.arange(6, dtype=torch.int32, device="cuda").view(1, 6), ctx)
    b = svd.tree_attention(q, c, torch.tensor([far], dtype=torch.int32, device="cuda"), ctx)
    assert torch.equal(a["out"], b["out"])


def test_repeated_calls_are_bitwise_equal():
    svd = require_gpu()
    p = problem(2, 17, 8, 2, 128, 16, "bf16", 700, 1500, True, seed=17)
    a = run(svd, p)
    for _ in range(3):
        b = run(svd, p)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite_values_of_the_context_reach_every_row(kind, value):
    # in a whole tile of context, and in the tile that holds the context's end and the nodes
    svd = require_gpu()
    for rows in ((5, 4, 2), (40, 8, 2)):
        T, Hq, Hkv = rows
        for back in (1, 3, 150):
            p = problem(2, T, Hq, Hkv, 128, 16, kind, 200, 210, True, seed=18)
            for b in range(2):
                pos = int(p["ctx"][b]) - back
                pg, pl = int(p["tab"][b, pos // 16]), pos % 16
                if kind == "bf16":
                    p["c"]["v"][pg, :, pl, 5:9] = value
                else:
                    p["c"]["v"].view(torch.uint8)[pg, :, pl, 5:9] = 0x7F
            got, lse = run(svd, p)
            for b in range(2):
                n = int(p["nodes"][b])
                bad = ~np.isfinite(got[b, :n])
                assert bad[..., 5:9].all() and not bad[..., :5].any() and not bad[..., 9:].any()
                if kind == "bf16" and value == float("inf"):
                    assert (got[b, :n, :, 5:9] == value).all()
                assert np.isfinite(lse[b, :n]).all()


def test_sequences_that_share_pages():
    # a common prefix of two sequences is read from the same pages
    svd = require_gpu()
    p = problem(2, 6, 4, 2, 64, 16, "e4m3", 100, 100, True, seed=19)
    p["tab"][1, :4] = p["tab"][0, :4]
    check(svd, p)


@pytest.mark.parametrize("rows", [(1, 16, 1), (9, 8, 2), (33, 8, 2), (70, 8, 2), (129, 8, 1)])
def test_one_page_of_every_size(rows):
    svd = require_gpu()
    T, Hq, Hkv = rows
    for page in (16, 32, 64, 128, 256, 512, 1024):
        check(svd, problem(1, T, Hq, Hkv, 64, page, "bf16", page + 1, page + 9, True, seed=page))
