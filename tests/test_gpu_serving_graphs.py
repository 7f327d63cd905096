"""Two captured graphs with one workspace between them, replayed in turn with eager work between:
every call fills what it reads."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu, say
from test_gpu_prefix_attention import BOTH, dev, problem, run

pytestmark = pytest.mark.gpu


def captured(call):
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        call()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            call()
    return graph


@BOTH
def test_two_attentions(kind):
    svd = require_gpu()
    # tiles of 64 rows in three groups, and of 256 in one
    ps = [problem([(2, 300), (3, 700), (1, 128)], 2, 8, 2, 64, 16, kind, 5, 90, False, seed=1),
          problem([(9, 900)], 9, 8, 2, 64, 16, kind, 5, 400, True, seed=2)]
    want = [run(svd, p) for p in ps]
    sizes = [svd.prefix_attention_workspace(len(p["ctx"]), p["q"].shape[1], 8, p["c"],
                                            dev(p["tab"]), len(p["off"]) - 1).numel() for p in ps]
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    outs, graphs, keep = [], [], []
    for p in ps:
        a = (p["q"], p["c"], dev(p["tab"]), dev(p["ctx"]))
        o = torch.empty_like(p["q"]), torch.empty(p["q"].shape[:3], device="cuda")
        kw = dict(n_nodes=dev(p["nodes"]), anc=dev(p["anc"]), share_off=dev(p["off"]), out=o[0],
                  lse=o[1], workspace=ws)
        keep.append((a, kw))
        outs.append(o)
        graphs.append(captured(lambda: svd.prefix_attention(*a, **kw)))
    for r in range(4):
        ws.fill_(0xFF if r % 2 else 0)
        for o in outs:
            o[0].fill_(7.0)
            o[1].fill_(7.0)
        for g in (graphs if r < 2 else graphs[::-1]):
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert np.array_equal(o[0].double().cpu().numpy(), w[0])
            assert np.array_equal(o[1].double().cpu().numpy(), w[1])
        say("replay", r, "matches")


def test_two_pools():
    svd = require_gpu()
    ws = torch.empty(svd.svd_cache_pages_workspace_bytes(1500), dtype=torch.uint8, device="cuda")
    g = np.random.default_rng(4)
    jobs = []
    for B in (1500, 7):
        pool = svd.page_pool(20 * B, B, 32)
        length = dev(g.integers(0, 500, B).astype(np.int32))
        to = {n: torch.empty_like(pool[n]) for n in ("table", "held", "state")}
        room = svd.cache_pages(pool, length, 16, out=to)  # apart from the pool: the same each time
        want = [room.clone()] + [to[n].clone() for n in to]
        assert (room >= length).all()
        jobs.append((pool, length, to, want))
    graphs = []
    for pool, length, to, _ in jobs:
        rooms = []
        graph = captured(lambda: rooms.append(svd.cache_pages(pool, length, 16, out=to,
                                                              workspace=ws)))
        graphs.append((graph, rooms[-1]))
    for r in range(4):
        ws.fill_(0xFF if r % 2 else 0)
        for _, _, to, _ in jobs:
            for x in to.values():
                x.fill_(-9)
        for graph, _ in (graphs if r < 2 else graphs[::-1]):
            graph.replay()
        torch.cuda.synchronize()
        for (graph, room), (_, _, to, want) in zip(graphs, jobs):
            for x, w in zip([room] + list(to.values()), want):
                assert torch.equal(x, w)
        say("replay", r, "matches")
