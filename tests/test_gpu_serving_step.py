"""A serving loop's operators together, as it runs them: lengths -> block tables -> packed
prompts by slot -> drafts sampled from the drafter's marginals -> tree -> attention over
the shared prefix -> filtered logits -> verification -> the next lengths.  Eagerly against
the references, on a side stream, captured and replayed, and two at once."""
import numpy as np
import pytest
import torch

import serve_ref as S
import step_ref as R
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

B, K, G, V, Hq, Hkv, D, PAGE, MP = 5, 4, 4, 2003, 8, 2, 64, 16, 24
T = 1 + K * G
SHARED = 9 * PAGE
KINDS = pytest.mark.parametrize("kind", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "e4m3"])


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def state(kind, seed):
    svd = require_gpu()
    g = np.random.default_rng(seed)
    torch.manual_seed(seed)
    s = {"cache": svd.kv_cache(B * MP, Hkv, PAGE, D, dtype=kind),
         "pool": svd.page_pool(B * MP, B, MP)}
    # a common prefix in pages that the first nine of the ring name
    ids = s["pool"]["free"][:9].clone()
    s["pool"]["state"].copy_(i32([9, B * MP - 9]))
    s["pool"]["table"][:, :9] = ids
    s["pool"]["held"].fill_(9)
    s["shared"] = i32([9] * B)
    x = torch.randn(2, 1, SHARED, Hkv, D, device="cuda", dtype=torch.bfloat16)
    svd.cache_write(s["cache"], x[0], x[1], ids.view(1, 9), i32([0]))
    s["ctx"] = i32([SHARED] * B)
    s["prompt"] = i32(g.integers(0, 60, B))
    s["n"] = int(s["prompt"].sum())
    s["rows"] = torch.randn(2, s["n"], Hkv, D, device="cuda", dtype=torch.bfloat16)
    s["root"] = i32(g.integers(0, V, B))
    s["embed"] = torch.randn(V, (Hq + 2 * Hkv) * D, device="cuda", dtype=torch.bfloat16)
    s["head"] = torch.randn(Hq * D, V, device="cuda", dtype=torch.bfloat16) * 0.3
    s["marginals"] = torch.randn(B, G, V, device="cuda", dtype=torch.bfloat16) * 3
    s["q_index"] = i32(np.broadcast_to(np.arange(B * G).reshape(B, 1, G), (B, K, G)))
    s["off"] = i32([0, B])
    s["top_k"], s["temperature"] = i32([20, 0, 5, 40, 7]), torch.full((B,), 0.8, device="cuda")
    s["top_p"] = torch.tensor([1.0, 0.9, 0.8, 0.95, 0.5], device="cuda")
    s["slopes"] = torch.exp2(-torch.arange(1, Hq + 1, device="cuda").float())
    s["ws"] = svd.prefix_attention_workspace(B, T, Hq, s["cache"], s["pool"]["table"], 1)
    s["vws"] = torch.empty(svd.svd_rows_workspace_bytes(B, K, G, V, B * T, B * G),
                           dtype=torch.uint8, device="cuda")
    return svd, s


def copy_of(s):
    """Everything that a step changes."""
    return {"pool": {n: x.clone() for n, x in s["pool"].items()},
            "cache": {n: None if x is None else x.clone() for n, x in s["cache"].items()}}


def put_back(s, old):
    for what in old:
        for n, x in old[what].items():
            if x is not None:
                s[what][n].copy_(x)


def step(svd, s, seed=3):
    # room for the prompts and the tree behind them
    length = s["ctx"] + s["prompt"] + T
    room = svd.cache_pages(s["pool"], length, PAGE, shared=s["shared"])
    table = s["pool"]["table"]
    m = svd.cache_slots(s["cache"], table, s["ctx"], s["prompt"], s["n"])
    svd.cache_write_slots(s["cache"], s["rows"][0], s["rows"][1], m["slot"])
    ctx = s["ctx"] + s["prompt"]
    # the drafter's marginals, filtered: what the drafts are sampled from is what q is
    ask = dict(temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"])
    q_rows = svd.filter_logits(s["marginals"], **ask)
    drafts = svd.sample(s["marginals"], K=K, seed=seed, **ask)["token"]
    tree = svd.draft_tree(drafts, root=s["root"])
    x = s["embed"][tree["tokens"].clamp(min=0).long()]
    q = x[..., :Hq * D].unflatten(-1, (Hq, D))
    k = x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    v = x[..., (Hq + Hkv) * D:].unflatten(-1, (Hkv, D))
    svd.cache_write(s["cache"], k, v, table, ctx, n_new=tree["n_nodes"])
    out = torch.zeros(B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    svd.prefix_attention(q, s["cache"], table, ctx, share_off=s["off"], anc=tree["anc"],
                         n_nodes=tree["n_nodes"], depth=tree["depth"], cap=20.0,
                         slopes=s["slopes"], out=out, workspace=s["ws"])
    raw = (out.view(B * T, Hq * D) @ s["head"]).view(B, T, V)
    p_rows = svd.filter_logits(raw, n_rows=tree["n_nodes"], out=raw.clone(), **ask)
    r = svd.select_and_verify_rows(p_rows.view(B * T, V), tree["p_index"], q_rows.view(B * G, V),
                                   s["q_index"], drafts, temp_p=0.8, seed=seed,
                                   workspace=s["vws"])
    # what was not accepted gives its pages back
    kept = svd.cache_pages(s["pool"], ctx + r["accept_len"] + 1, PAGE, shared=s["shared"])
    return dict(tree, room=room, slot=m["slot"], q_rows=q_rows, drafts=drafts, q=q, k=k, v=v,
                out=out, raw=raw, p_rows=p_rows, selected=r["selected"], kept=kept,
                accept_len=r["accept_len"], next_token=r["next_token"])


@KINDS
def test_a_step_against_plain_steps(kind):
    svd, s = state(kind, 4)
    old = copy_of(s)
    got = step(svd, s)
    torch.cuda.synchronize()
    host = {n: x.float().cpu().numpy().astype(np.float64) if x.is_floating_point()
            else x.cpu().numpy() for n, x in got.items()}
    ctx0, prompt = s["ctx"].cpu().numpy(), s["prompt"].cpu().numpy()
    pool = {n: x.tolist() for n, x in old["pool"].items()}
    ring, st, held, table, room = S.pages(ctx0 + prompt + T, [9] * B, PAGE, pool["free"],
                                          pool["state"], pool["held"], pool["table"])
    assert host["room"].tolist() == room
    assert host["slot"].tolist() == S.slots(ctx0, prompt, table, PAGE, B * MP, s["n"])[3]
    top_k, top_p = s["top_k"].cpu().numpy(), s["top_p"].cpu().numpy()
    mine = [(float(np.float32(0.8)), int(top_k[b]), float(top_p[b]), 0.0) for b in range(B)]
    marg = s["marginals"].float().cpu().numpy().astype(np.float64)
    for b in range(B):
        for t in range(G):
            keep = S.kept(marg[b, t], *mine[b])
            assert np.array_equal(host["q_rows"][b, t], np.where(keep, marg[b, t], -np.inf))
            for d in range(K):
                assert host["drafts"][b, d, t] == S.draw(marg[b, t], keep, mine[b][0],
                                                        S.hash_uniform(3, b, d, t, G))[0]
    tree = R.draft_tree(host["drafts"], s["root"].cpu().numpy(), T)
    n, ctx = tree["n_nodes"], ctx0 + prompt
    assert np.array_equal(host["anc"], tree["anc"]) and np.array_equal(host["depth"], tree["depth"])
    want, _, tol, _ = S.attention(host["q"], R.cache_values(s["cache"], "k"),
                                  R.cache_values(s["cache"], "v"), np.array(table), ctx, n,
                                  tree["anc"], tree["depth"], D ** -0.5, 20.0,
                                  s["slopes"].cpu().numpy())
    for b in range(B):
        R.close(host["out"][b, :n[b]], want[b, :n[b]], tol[b, :n[b]], b)
        for t in range(T):
            row = host["raw"][b, t]
            if t < n[b]:
                row = np.where(S.kept(row, *mine[b]), row, -np.inf)
            assert np.array_equal(host["p_rows"][b, t], row)
    # verification of the same rows laid out densely
    px = got["p_index"].long()
    p = got["p_rows"].view(B * T, V)[px.view(-1)].view(B, K, G + 1, V).contiguous()
    qd = got["q_rows"].view(B, 1, G, V).expand(B, K, G, V).contiguous()
    dense = svd.select_and_verify(p, qd, got["drafts"], temp_p=0.8, seed=3)
    for name in ("selected", "accept_len", "next_token"):
        assert torch.equal(dense[name], got[name]), name
    L = host["accept_len"]
    say("accepted", L.tolist(), "nodes", n.tolist())
    assert (L >= 0).all()
    # every committed token is one that its filtered row keeps
    for b in range(B):
        row = px[b, host["selected"][b], L[b]] if L[b] < G else px[b, host["selected"][b], G]
        assert got["p_rows"].view(B * T, V)[row, int(host["next_token"][b])] > -float("inf")
    ring, st, held, table, kept = S.pages(ctx + L + 1, [9] * B, PAGE, ring, st, held, table)
    assert host["kept"].tolist() == kept
    for name, x in (("free", ring), ("state", st), ("held", held), ("table", table)):
        assert s["pool"][name].tolist() == list(x), name


def same(a, b):
    for n in a:
        if n not in ("k", "v", "q"):
            assert torch.equal(a[n], b[n]), n


@KINDS
def test_a_captured_step_replays(kind):
    svd, s = state(kind, 9)
    old = copy_of(s)
    want = {n: x.clone() for n, x in step(svd, s).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        put_back(s, old)
        same(step(svd, s), want)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    put_back(s, old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(svd, s)
    marginals = s["marginals"].clone()
    for r in range(4):
        # eager work of other drafts on the same cache, pool and workspaces in between
        s["marginals"].copy_(marginals.roll(1 + r, 0))
        put_back(s, old)
        other = {n: x.clone() for n, x in step(svd, s, seed=50 + r).items()}
        assert not torch.equal(other["drafts"], want["drafts"])
        s["marginals"].copy_(marginals)
        put_back(s, old)
        graph.replay()
        torch.cuda.synchronize()
        same(got, want)
        say("replay", r, "matches")


@KINDS
def test_two_streams_with_a_workspace_each(kind):
    jobs = [state(kind, 20), state(kind, 21)]
    want = [{n: x.clone() for n, x in step(*j).items()} for j in jobs]
    jobs = [state(kind, 20), state(kind, 21)]
    olds = [copy_of(s) for _, s in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for i, (svd, s) in enumerate(jobs):
        with torch.cuda.stream(streams[i]):
            for _ in range(3):
                put_back(s, olds[i])
                got[i] = step(svd, s)
    torch.cuda.synchronize()
    for i in range(2):
        same(got[i], want[i])


# -- the stream argument ----------------------------------------------------

SPIN = 20_000_000  # 8 ms, far more than the host takes for a call


def calls(svd):
    """(name, call(**kw) -> tuple of result tensors)."""
    torch.manual_seed(5)
    c = svd.kv_cache(300, Hkv, PAGE, D)
    for n in ("k", "v"):
        c[n].normal_()
    tab = torch.arange(300, dtype=torch.int32, device="cuda").view(5, 60)
    tab[:, :20] = tab[0, :20]
    ctx, new, off = i32([800, 400, 450, 320, 700]), i32([3, 0, 20, 7, 1]), i32([0, 5])
    q = torch.randn(5, 9, Hq, D, device="cuda", dtype=torch.bfloat16)
    z = torch.randn(5, 9, 5003, device="cuda")
    kw0 = dict(top_k=i32([5, 50, 0, 9, 7]), top_p=torch.full((5,), 0.9, device="cuda"))
    pool = svd.page_pool(300, 5, 60)
    to = {n: torch.zeros_like(pool[n]) for n in ("table", "held", "state")}

    def pages(**kw):
        return (svd.cache_pages(pool, ctx, PAGE, out=to, **kw),)

    def attention(**kw):
        r = svd.prefix_attention(q, c, tab, ctx, share_off=off, want_lse=True, **kw)
        return r["out"], r["lse"]

    return {"pages": pages, "attention": attention,
            "slots": lambda **kw: tuple(svd.cache_slots(c, tab, ctx, new, 40, **kw).values()),
            "filter": lambda **kw: (svd.filter_logits(z, **kw0, **kw),),
            "sample": lambda **kw: tuple(svd.sample(z, K=3, want_logprob=True, **kw0, **kw).values())}


@pytest.fixture(params=["pages", "attention", "slots", "filter", "sample"])
def job(request):
    svd = require_gpu()
    say(request.param)
    return calls(svd)[request.param]


def storages(r):
    return {x.untyped_storage().data_ptr(): x.untyped_storage().nbytes() for x in r}


def test_results_on_another_stream(job):
    want = [x.clone() for x in job()]
    side = torch.cuda.Stream()
    for stream in (side.cuda_stream, torch.cuda.current_stream().cuda_stream, 0):
        torch.cuda.synchronize()
        got = job(stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_dropped_results_go_back_after_the_call(job):
    sizes = storages(job())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    job(stream=side.cuda_stream)
    held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes.values()]
    torch.cuda.synchronize()
    for x in held:
        assert (x == 7).all()


def test_what_a_call_allocates_lasts_as_long_as_the_call(job, monkeypatch):
    want = [x.clone() for x in job()]
    made, empty = [], torch.empty

    def spy(*a, **kw):
        t = empty(*a, **kw)
        made.append((t.data_ptr(), max(t.numel() * t.element_size(), 1)))
        return t

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    monkeypatch.setattr(torch, "empty", spy)
    got = job(stream=side.cuda_stream)
    monkeypatch.undo()
    fill = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _, n in made for _ in range(4)]
    taken = {x.data_ptr() for x in fill}
    assert not any(at in taken for at, _ in made)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for x in fill:
        assert (x == 0xFF).all()
