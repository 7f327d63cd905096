"""Attention over many shared prefixes at once, on two streams at once, and replayed with other
tables and lengths, against float64 and against the same call without groups."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu, say
from test_gpu_prefix_attention import BOTH, check, dev, problem, run, slopes_of

pytestmark = pytest.mark.gpu


@BOTH
@pytest.mark.parametrize("D,n", [(64, 70), (128, 70), (64, 1100)])
def test_many_groups(kind, D, n):
    # more than a ballot, and more than a workgroup, has lanes; some share nothing
    svd = require_gpu()
    say(kind, D, n)
    g = np.random.default_rng(n + D)
    groups = [(int(x), int(s)) for x, s in zip(g.integers(0, 4, n) if n < 100 else
                                               g.integers(0, 3, n), g.choice([0, 64, 128, 300], n))]
    p = problem(groups, 2 if n < 100 else 1, 2, 1, D, 16, kind, 0, 40, False, seed=n,
                alone=1 if n < 100 else 200)  # no more groups than sequences
    check(svd, p, only=range(0, len(p["ctx"]), 1 if n < 100 else 5))


@BOTH
def test_a_group_of_many_sequences(kind):
    # more sequences than a workgroup has threads, tables that part at different pages
    svd = require_gpu()
    say(kind)
    p = problem([(1100, 512)], 1, 2, 1, 64, 16, kind, 0, 40, False, seed=3)
    check(svd, p, only=range(0, 1100, 9))
    p["tab"][1090, 26] = p["tab"][0, 27]   # 26 pages of one in common: 384 tokens
    check(svd, p, only=[0, 511, 1089, 1090, 1091, 1099])
    p["tab"][7, 9] = p["tab"][0, 10]       # 9 pages: 128 tokens
    p["nodes"][5] = 0
    check(svd, p, only=[0, 5, 6, 7, 8, 700, 1090])
    p["tab"][1024, 0] = p["tab"][0, 1]     # nothing in common
    check(svd, p, only=[0, 1, 1023, 1024, 1025, 1099])


@BOTH
@pytest.mark.parametrize("T", [1, 9])
def test_two_streams_at_once(kind, T):
    svd = require_gpu()
    ps = [problem([(5, 700)], T, 8, 2, 128, 64, kind, 5, 300, False, seed=s) for s in (1, 2)]
    want = [run(svd, p, cap=20.0) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    args = [(p["q"], p["c"], dev(p["tab"]), dev(p["ctx"])) for p in ps]
    kws = [dict(n_nodes=dev(p["nodes"]), share_off=dev(p["off"]), cap=20.0) for p in ps]
    outs = [[torch.full(p["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
            for p in ps]
    torch.cuda.synchronize()
    for i in range(4):
        for s, a, kw, o in zip(streams, args, kws, outs):
            with torch.cuda.stream(s):
                svd.prefix_attention(*a, out=o[i], **kw)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for x in o:
            assert np.array_equal(x.double().cpu().numpy(), w[0])


@BOTH
def test_replays_follow_tables_lengths_and_groups(kind):
    svd = require_gpu()
    p = problem([(6, 512)], 5, 8, 2, 128, 32, kind, 5, 200, True, seed=5)
    tab, ctx, nodes, off = (dev(p[n]) for n in ("tab", "ctx", "nodes", "off"))
    anc, depth, slopes = dev(p["anc"]), dev(p["depth"]), dev(np.array(slopes_of(8), np.float32))
    out = torch.empty_like(p["q"])
    lse = torch.empty(p["q"].shape[:3], device="cuda")
    ws = svd.prefix_attention_workspace(6, 5, 8, p["c"], tab, 1)

    def call():
        svd.prefix_attention(p["q"], p["c"], tab, ctx, share_off=off, anc=anc, n_nodes=nodes,
                             depth=depth, cap=30.0, slopes=slopes, out=out, lse=lse, workspace=ws)

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        call()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            call()
    for step in range(6):
        if step == 1:
            p["nodes"] = np.minimum(p["nodes"], np.array([5, 4, 3, 2, 1, 0], np.int32))
        if step == 2:
            p["tab"][3, 9] = p["tab"][0, 10]     # fewer pages in common
        if step == 3:
            p["off"][:] = [2, 6]                 # two sequences leave the group
        if step == 4:
            p["ctx"][4] = 100                    # less than a tile of one is left to share
        if step == 5:
            p["off"][:] = [6, 0]                 # no group
        for t, n in ((tab, "tab"), (ctx, "ctx"), (nodes, "nodes"), (off, "off")):
            t.copy_(torch.from_numpy(p[n]))
        want, wl = check(svd, p, cap=30.0, slopes=slopes_of(8))
        out.fill_(7.0)
        lse.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want), step
        assert np.array_equal(lse.double().cpu().numpy(), wl), step
