"""The operators of one speculative step together, as a serving loop runs them:
drafts -> tree -> the tree's keys and values into the cache -> attention -> a
vocabulary projection -> adjusted logits -> self-selection and verification over
the tree's rows -> the accepted nodes to their committed positions.  Eagerly, on a
side stream and as a captured graph; two streams at once with a workspace each."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

B, K, G, V, Hq, Hkv, D, PAGE = 6, 4, 5, 3001, 8, 2, 64, 16
T = 1 + K * G


def state(kind, seed):
    svd = require_gpu()
    g = np.random.default_rng(seed)
    t = {}
    cand = g.integers(0, V, (B, 1, G, 2))
    pick = g.integers(0, 2, (B, K, G, 1))
    t["drafts"] = np.take_along_axis(np.broadcast_to(cand, (B, K, G, 2)), pick, 3)[..., 0]
    t["root"] = g.integers(0, V, B)
    t["ctx"] = g.integers(0, 60, B)
    t["table"] = g.permutation(B * 8).reshape(B, 8)
    t["history"] = g.integers(0, V, (B, 64))
    s = {n: torch.from_numpy(np.ascontiguousarray(x.astype(np.int32))).cuda() for n, x in t.items()}
    torch.manual_seed(seed)
    s["cache"] = svd.kv_cache(B * 8, Hkv, PAGE, D, dtype=kind)
    old = torch.randn(2, B, 64, Hkv, D, device="cuda", dtype=torch.bfloat16)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    svd.cache_write(s["cache"], old[0], old[1], s["table"], zero)  # the contexts
    s["embed"] = torch.randn(V, (Hq + 2 * Hkv) * D, device="cuda", dtype=torch.bfloat16)
    s["head"] = torch.randn(Hq * D, V, device="cuda", dtype=torch.bfloat16) * 0.2
    s["q_rows"] = torch.randn(B, G, V, device="cuda", dtype=torch.bfloat16)
    s["q_index"] = (torch.arange(B * G, device="cuda", dtype=torch.int32).view(B, 1, G)
                    .expand(B, K, G).contiguous())
    s["repetition"] = torch.full((B,), 1.2, device="cuda")
    s["presence"] = torch.full((B,), 0.3, device="cuda")
    allow = g.random((3, V)) < 0.8
    s["allow"] = torch.from_numpy(R.pack(allow)).cuda()
    s["allow_index"] = torch.from_numpy(g.integers(-1, 3, (B, T)).astype(np.int32)).cuda()
    s["ws"] = svd.tree_attention_workspace(B, T, Hq, s["cache"], s["table"])
    s["vws"] = torch.empty(svd.svd_rows_workspace_bytes(B, K, G, V, B * T, B * G),
                           dtype=torch.uint8, device="cuda")
    return svd, s


def step(svd, s, seed=3):
    tree = svd.draft_tree(s["drafts"], root=s["root"])
    x = s["embed"][tree["tokens"].clamp(min=0).long()]  # [B, T, (Hq + 2 Hkv) D], fused q, k, v
    q = x[..., :Hq * D].unflatten(-1, (Hq, D))
    k = x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    v = x[..., (Hq + Hkv) * D:].unflatten(-1, (Hkv, D))
    svd.cache_write(s["cache"], k, v, s["table"], s["ctx"], n_new=tree["n_nodes"])
    out = torch.zeros(B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    svd.tree_attention(q, s["cache"], s["table"], s["ctx"], anc=tree["anc"],
                       n_nodes=tree["n_nodes"], out=out, workspace=s["ws"])
    logits = (out.view(B * T, Hq * D) @ s["head"]).view(B, T, V)
    svd.adjust_logits(logits, s["history"], s["ctx"], tokens=tree["tokens"], anc=tree["anc"],
                      n_rows=tree["n_nodes"], repetition=s["repetition"], presence=s["presence"],
                      allow=s["allow"], allow_index=s["allow_index"], out=logits)
    r = svd.select_and_verify_rows(logits.view(B * T, V), tree["p_index"], s["q_rows"].view(B * G, V),
                                   s["q_index"], s["drafts"], seed=seed, workspace=s["vws"])
    # the accepted nodes (root included) to the positions after the context
    path = tree["p_index"].gather(1, r["selected"].clamp(min=0).long().view(B, 1, 1).expand(
        B, 1, G + 1)).view(B, G + 1) - T * torch.arange(B, device="cuda", dtype=torch.int32).view(B, 1)
    depth = torch.arange(G + 1, device="cuda", dtype=torch.int32).expand(B, G + 1)
    dst = torch.full((B, T + 1), -1, dtype=torch.int32, device="cuda")
    dst.scatter_(1, torch.where(depth <= r["accept_len"].view(B, 1), path, T).long(), depth)
    dst = dst[:, :T].contiguous()
    svd.cache_write(s["cache"], k, v, s["table"], s["ctx"], dst=dst)
    kept = torch.zeros(2, B, 64, Hkv, D, device="cuda")
    svd.cache_read(s["cache"], s["table"], 64, count=(s["ctx"] + r["accept_len"] + 1).clamp(max=64),
                   out=(kept[0], kept[1]))
    return dict(tree, out=out, logits=logits, kept=kept, selected=r["selected"],
                accept_len=r["accept_len"], next_token=r["next_token"])


KINDS = pytest.mark.parametrize("kind", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "e4m3"])


@KINDS
def test_a_step_against_plain_steps(kind, orc):
    svd, s = state(kind, 4)
    before = {n: (None if x is None else x.clone()) for n, x in s["cache"].items()}
    got = step(svd, s)
    torch.cuda.synchronize()
    d = s["drafts"].cpu().numpy()
    tree = R.draft_tree(d, s["root"].cpu().numpy(), T)
    for n in tree:
        assert np.array_equal(got[n].cpu().numpy(), tree[n]), n
    n_nodes, ctx = tree["n_nodes"], s["ctx"].cpu().numpy()
    # attention over the cache as it was with the tree in it
    svd2, s2 = state(kind, 4)
    x = s["embed"][got["tokens"].clamp(min=0).long()]
    k = x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    v = x[..., (Hq + Hkv) * D:].unflatten(-1, (Hkv, D))
    for n, y in before.items():
        if y is not None:
            s2["cache"][n].copy_(y)
    svd.cache_write(s2["cache"], k, v, s["table"], s["ctx"], n_new=got["n_nodes"])
    q = x[..., :Hq * D].unflatten(-1, (Hq, D)).double().cpu().numpy()
    want, _, tol, _ = R.attention(q, R.cache_values(s2["cache"], "k"), R.cache_values(s2["cache"], "v"),
                                  s["table"].cpu().numpy(), ctx, n_nodes, tree["anc"], D ** -0.5)
    out = got["out"].double().cpu().numpy()
    for b in range(B):
        R.close(out[b, :n_nodes[b]], want[b, :n_nodes[b]], tol[b, :n_nodes[b]], b)
    # the adjusted rows, from the projection of the attention that was computed
    raw = (got["out"].view(B * T, Hq * D) @ s["head"]).view(B, T, V).double().cpu().numpy()
    adj, atol = R.adjust(raw, True, history=s["history"].cpu().numpy(), hist_len=ctx,
                         tokens=tree["tokens"], anc=tree["anc"],
                         repetition=s["repetition"].cpu().numpy(),
                         presence=s["presence"].cpu().numpy(), allow=s["allow"].cpu().numpy(),
                         allow_index=s["allow_index"].cpu().numpy())
    logits = got["logits"].double().cpu().numpy()
    for b in range(B):
        R.close(logits[b, :n_nodes[b]], adj[b, :n_nodes[b]], atol[b, :n_nodes[b]], b)
        assert np.array_equal(logits[b, n_nodes[b]:], raw[b, n_nodes[b]:])
    # verification of the same rows laid out densely, by the oracle's own library call
    px = got["p_index"].long().clamp(min=0)
    p = got["logits"].view(B * T, V)[px.view(-1)].view(B, K, G + 1, V).contiguous()
    qd = s["q_rows"].view(B, 1, G, V).expand(B, K, G, V).contiguous()
    dense = svd.select_and_verify(p, qd, s["drafts"], seed=3)
    for n in ("selected", "accept_len", "next_token"):
        assert torch.equal(dense[n], got[n]), n
    sel, L = got["selected"].cpu().numpy(), got["accept_len"].cpu().numpy()
    say("accepted", L.tolist(), "nodes", n_nodes.tolist())
    # the committed tokens' keys and values follow the context
    kept = got["kept"].cpu().numpy()
    for b in range(B):
        if L[b] < 0:
            continue
        for j in range(min(L[b] + 1, 64 - ctx[b])):
            node = tree["p_index"][b, sel[b], j] - b * T
            row = k[b, node].float().cpu().numpy()
            held = R.e4m3_values(row)[0] if kind == torch.float8_e4m3fn else row
            assert np.array_equal(kept[0, b, ctx[b] + j], held), (b, j)


@KINDS
def test_a_captured_step_replays(kind):
    svd, s = state(kind, 9)
    cache0 = {n: (None if x is None else x.clone()) for n, x in s["cache"].items()}

    def reset():
        for n, x in cache0.items():
            if x is not None:
                s["cache"][n].copy_(x)

    def same(a, b):
        # rows that are left as they were hold whatever a new tensor held, in `logits` too
        for n in a:
            if n != "logits":
                assert torch.equal(a[n], b[n]), n

    want = {n: x.clone() for n, x in step(svd, s).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        reset()
        same(step(svd, s), want)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    reset()
    with torch.cuda.graph(graph):
        got = step(svd, s)
    drafts = s["drafts"].clone()
    for r in range(4):
        # eager work of other drafts on the same cache and workspaces in between
        s["drafts"].copy_(drafts.roll(1 + r, 0))
        reset()
        other = {n: x.clone() for n, x in step(svd, s, seed=50 + r).items()}
        assert not torch.equal(other["tokens"], want["tokens"])
        s["drafts"].copy_(drafts)
        reset()
        graph.replay()
        torch.cuda.synchronize()
        same(got, want)
        say("replay", r, "matches")


@KINDS
def test_two_streams_with_a_workspace_each(kind):
    jobs = [state(kind, 20), state(kind, 21)]
    want = [{n: x.clone() for n, x in step(*j).items()} for j in jobs]
    jobs = [state(kind, 20), state(kind, 21)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for i, (svd, s) in enumerate(jobs):
        with torch.cuda.stream(streams[i]):
            for _ in range(3):
                got[i] = step(svd, s)
    torch.cuda.synchronize()
    for i in range(2):
        for n in ("tokens", "anc", "out", "selected", "accept_len", "next_token"):
            assert torch.equal(got[i][n], want[i][n]), (i, n)


def test_more_nodes_than_room_ends_as_a_data_error():
    # the tree's error reaches every later call: NaN rows, and -1 from the verification
    svd, s = state(torch.bfloat16, 5)
    full = svd.draft_tree(s["drafts"], root=s["root"])
    room = int(full["n_nodes"].max()) - 1
    tree = svd.draft_tree(s["drafts"], root=s["root"], n_max=room)
    bad = (tree["n_nodes"] < 0).cpu().numpy()
    assert bad.any()
    q = torch.randn(B, room, Hq, D, device="cuda", dtype=torch.bfloat16)
    out = svd.tree_attention(q, s["cache"], s["table"], s["ctx"], anc=tree["anc"],
                             n_nodes=tree["n_nodes"])["out"]
    z = svd.adjust_logits(torch.randn(B, room, V, device="cuda", dtype=torch.bfloat16),
                          s["history"], s["ctx"], tokens=tree["tokens"], anc=tree["anc"],
                          n_rows=tree["n_nodes"])
    r = svd.select_and_verify_rows(z.view(B * room, V), tree["p_index"], s["q_rows"].view(B * G, V),
                                   s["q_index"], s["drafts"])
    for b in range(B):
        assert torch.isnan(out[b]).all().item() == bad[b]
        assert torch.isnan(z[b]).all().item() == bad[b]
        assert (int(r["selected"][b]) == -1) == bad[b]
