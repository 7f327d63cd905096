"""The operators around a verification step, as they are measured: the prefix tree of
the K drafts, the paged cache that the tree's tokens are written to and read back from,
the attention of the tree over that cache, and the adjustments of the verifier's logits
(penalties, biases, grammar masks).

``run`` computes a case in elementary torch operations, or with ``own`` through this
repository's package.  Conventions of all cases: prefix b has ctx_len[b] cached tokens;
node 0 of its tree is the last committed token and the other nodes are drafted tokens,
every node after its parent; bit i of anc[b][t] says that node i is on node t's path
(t itself and the root are).
"""
import math

import torch

own = False

KINDS = ("bf16", "e4m3")


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one request drafting 8 candidates of 16 tokens: latency of the tree's bookkeeping
        dict(name="tree_one", op="tree", B=1, K=8, G=16, fan=2),
        # a batch of long windows with 16 drafts each
        dict(name="tree_batch", op="tree", B=64, K=16, G=32, fan=3),
        # one decode token of one request into the quantised cache and back: latency
        dict(name="cache_one_token", op="cache", B=1, T=1, Hkv=8, D=128, page=16, kind="e4m3",
             ctx_lo=37, ctx_hi=37, src="bf16"),
        # the tree tokens of a full serving batch, unaligned positions
        dict(name="cache_serving", op="cache", B=256, T=9, Hkv=8, D=128, page=64, kind="e4m3",
             ctx_lo=1, ctx_hi=4000, src="bf16"),
        # long prompts written in one go and read back for the next chunk
        dict(name="cache_prompt", op="cache", B=4, T=8192, Hkv=8, D=128, page=64, kind="e4m3",
             ctx_lo=0, ctx_hi=100, src="bf16"),
        # plain decoding of one request, a short context in small pages: latency
        dict(name="attn_one_token", op="attn", B=1, T=1, Hq=32, Hkv=8, D=128, page=16, kind="bf16",
             ctx_lo=777, ctx_hi=777, tree="chain", ragged=False),
        # batched serving: a window of 8 drafted tokens per request, quantised cache
        dict(name="attn_serving", op="attn", B=256, T=9, Hq=32, Hkv=8, D=128, page=64, kind="e4m3",
             ctx_lo=1, ctx_hi=4096, tree="chain", ragged=False),
        # trees of 8 drafts of 16 tokens over long contexts
        dict(name="attn_tree_long", op="attn", B=4, T=129, Hq=32, Hkv=8, D=128, page=128,
             kind="bf16", ctx_lo=30000, ctx_hi=32500, tree="tree", ragged=True),
        # one key head per query head, heads of 64, odd lengths
        dict(name="attn_heads64", op="attn", B=24, T=33, Hq=16, Hkv=16, D=64, page=32, kind="e4m3",
             ctx_lo=501, ctx_hi=5007, tree="tree", ragged=True),
        # one decode row of one request, penalties only: latency
        dict(name="adjust_one_row", op="adjust", B=1, T=1, V=152064, H=512, dtype="bf16", bias=0,
             mask="none"),
        # batched serving: every row of every window, a share of it under a grammar
        dict(name="adjust_serving", op="adjust", B=256, T=9, V=152064, H=1024, dtype="bf16",
             bias=0, mask="some"),
        # trees in fp32 with an odd vocabulary, long histories, biases and a grammar on every row
        dict(name="adjust_tree_odd", op="adjust", B=4, T=129, V=100003, H=32768, dtype="f32",
             bias=300, mask="all"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "cache", "attn", "attn", "adjust"])
    if op == "tree":
        K, G = _log_int(rng, 1, 16), _log_int(rng, 1, 32)
        return dict(op=op, B=_log_int(rng, 1, 64), K=K, G=G, fan=rng.randint(1, 4))
    if op == "cache":
        D, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 16])
        T = _log_int(rng, 1, 8192)
        room = 4 * 8192 * 8 * 128 // (T * Hkv * D)
        return dict(op=op, B=_log_int(rng, 1, max(1, min(256, room))), T=T, Hkv=Hkv, D=D,
                    page=rng.choice([16, 32, 64, 128]), kind=rng.choice(KINDS),
                    ctx_lo=0, ctx_hi=_log_int(rng, 1, 2000), src=rng.choice(["bf16", "f32"]))
    if op == "attn":
        D, Hkv, group = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 7, 8])
        T = _log_int(rng, 1, 129)
        hi = _log_int(rng, 1, 32500)
        # tokens and products bounded by the listed cases
        room = min(500_000 * 8 * 128 // (hi * Hkv * D),
                   4 * 32500 * 129 * 32 * 128 // (hi * T * Hkv * group * D))
        return dict(op=op, B=_log_int(rng, 1, max(1, min(256, room))), T=T, Hq=Hkv * group,
                    Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]), kind=rng.choice(KINDS),
                    ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                    tree=rng.choice(["chain", "tree"]), ragged=rng.random() < 0.5)
    V, T = _log_int(rng, 1000, 152064), _log_int(rng, 1, 129)
    room = 256 * 9 * 152064 // (V * T)
    return dict(op=op, B=_log_int(rng, 1, max(1, min(256, room))), T=T, V=V,
                H=_log_int(rng, 1, 32768), dtype=rng.choice(["bf16", "f32"]),
                bias=rng.choice([0, 0, 17, 300]), mask=rng.choice(["none", "some", "all"]))


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _ctx(case):
    return _spread(case["ctx_lo"], case["ctx_hi"], case["B"])


def _nodes(case):
    T = case["T"]
    return _spread((T + 1) // 2, T, case["B"]) if case["ragged"] else [T] * case["B"]


def _hist(case):
    return _spread((case["H"] + 1) // 2, case["H"], case["B"])


def work(case):
    op, B = case["op"], case["B"]
    if op == "tree":
        K, G = case["K"], case["G"]
        T = 1 + K * G
        return dict(bytes=4.0 * B * (K * G + 3 * T + T * ((T + 31) // 32) + 1 + K * (G + 1)),
                    flops=0.5 * B * K * K * G)
    if op == "cache":
        rows = 2.0 * B * case["T"] * case["Hkv"]
        D = case["D"]
        held = D + 1 if case["kind"] == "e4m3" else 2 * D
        src = D * (2 if case["src"] == "bf16" else 4)
        return dict(bytes=rows * (src + 2 * held + 2 * D), flops=rows * D * 4)
    if op == "attn":
        D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
        held = D + 1 if case["kind"] == "e4m3" else 2 * D
        nbytes = flops = 0.0
        for c, n in zip(_ctx(case), _nodes(case)):
            nbytes += 2.0 * (c + n) * Hkv * held + 2.0 * n * Hq * D * 2 + 4.0 * n * Hq
            path = n * (n + 1) / 2 if case["tree"] == "chain" else n * min(n, 9)
            flops += 4.0 * Hq * D * (n * c + path)
        return dict(bytes=nbytes, flops=flops)
    es = 2 if case["dtype"] == "bf16" else 4
    V, T = case["V"], case["T"]
    masked = {"none": 0.0, "some": 0.25, "all": 1.0}[case["mask"]]
    return dict(bytes=B * T * V * (2.0 * es + masked / 8) + 4.0 * sum(_hist(case)),
                flops=4.0 * B * T * V)


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _permuted(values, g):
    t = torch.tensor(values, dtype=torch.int32, device="cuda")
    return t[torch.randperm(len(values), generator=g, device="cuda")].contiguous()


def _pages(case, lens, g):
    """A block table whose sequences hold disjoint, shuffled pages."""
    B, page = case["B"], case["page"]
    need = [max(1, (n + page - 1) // page) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((B, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, n_pages


def _empty_cache(case, n_pages):
    shape = (n_pages, case["Hkv"], case["page"], case["D"])
    if case["kind"] == "bf16":
        return {"k": torch.zeros(shape, dtype=torch.bfloat16, device="cuda"),
                "v": torch.zeros(shape, dtype=torch.bfloat16, device="cuda"),
                "k_scale": None, "v_scale": None}
    return {"k": torch.zeros(shape, dtype=torch.float8_e4m3fn, device="cuda"),
            "v": torch.zeros(shape, dtype=torch.float8_e4m3fn, device="cuda"),
            "k_scale": torch.full(shape[:3], 127, dtype=torch.uint8, device="cuda"),
            "v_scale": torch.full(shape[:3], 127, dtype=torch.uint8, device="cuda")}


def _filled_cache(case, n_pages, g):
    c = _empty_cache(case, n_pages)
    for n in ("k", "v"):
        x = torch.randn(c[n].shape, generator=g, device="cuda", dtype=torch.bfloat16)
        if case["kind"] == "bf16":
            c[n].copy_(x)
        else:  # codes in the upper part of their range, as a scaled row has them
            c[n].copy_((x * 64).float().clamp(-448, 448))
            c[n + "_scale"].copy_(torch.randint(120, 123, c[n].shape[:3], generator=g,
                                                device="cuda", dtype=torch.uint8))
    return c


def _pack(bits):
    """bool [..., n] -> int32 words [..., ceil(n / 32)], bit i of word w = bits[32 w + i]."""
    n = bits.shape[-1]
    W = (n + 31) // 32
    b = torch.zeros(bits.shape[:-1] + (W * 32,), dtype=torch.int64, device=bits.device)
    b[..., :n] = bits
    b = (b.view(bits.shape[:-1] + (W, 32)) << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(b >= 1 << 31, b - (1 << 32), b).to(torch.int32)


def _random_tree(B, T, g):
    """anc of random trees in which a node's parent is one of the 16 before it, and
    branches are about as deep as a drafted window."""
    t = torch.arange(T, device="cuda")
    back = (torch.rand((B, T), generator=g, device="cuda") * 16).long() + 1
    parent = (t - back).clamp(min=0)
    reach = torch.zeros((B, T, T), device="cuda")
    reach.scatter_(2, parent.unsqueeze(-1), 1.0)
    reach[:, 0] = 0
    reach += torch.eye(T, device="cuda")
    for _ in range(max(1, math.ceil(math.log2(max(2, T))))):
        reach = (torch.bmm(reach, reach.contiguous()) > 0).float()
    return _pack(reach > 0)


def prepare(case, seed):
    g = _gen(seed)
    op, B = case["op"], case["B"]
    s = {"case": dict(case)}
    if op == "tree":
        K, G = case["K"], case["G"]
        # the drafts of one set of marginals: a few likely tokens a position, so prefixes are shared
        cand = torch.randint(0, 152064, (B, G, case["fan"]), generator=g, device="cuda")
        u = torch.rand((B, K, G), generator=g, device="cuda")
        pick = (u.square() * case["fan"]).long()
        s["drafts"] = cand.unsqueeze(1).expand(B, K, G, case["fan"]).gather(
            3, pick.unsqueeze(-1)).squeeze(-1).to(torch.int32).contiguous()
        s["root"] = torch.randint(0, 152064, (B,), generator=g, device="cuda", dtype=torch.int32)
        return s
    if op == "cache":
        T, Hkv, D = case["T"], case["Hkv"], case["D"]
        ctx = _ctx(case)
        s["table"], n_pages = _pages(case, [c + T for c in [max(ctx)] * B], g)
        s["ctx_len"] = _permuted(ctx, g)
        s["cache"] = _empty_cache(case, n_pages)
        dt = torch.bfloat16 if case["src"] == "bf16" else torch.float32
        for n in ("k", "v"):  # heads of different sizes, channels that stand out
            x = torch.randn((B, T, Hkv, D), generator=g, device="cuda", dtype=dt)
            x *= torch.rand((Hkv, D), generator=g, device="cuda").mul_(2).exp_().to(dt)
            s[n] = x
        return s
    if op == "attn":
        T, D = case["T"], case["D"]
        ctx, nodes = _ctx(case), _nodes(case)
        order = torch.randperm(B, generator=g, device="cuda").tolist()
        ctx, nodes = [ctx[i] for i in order], [nodes[i] for i in order]
        s["table"], n_pages = _pages(case, [c + n for c, n in zip(ctx, nodes)], g)
        s["cache"] = _filled_cache(case, n_pages, g)
        s["ctx_len"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["n_nodes"] = torch.tensor(nodes, dtype=torch.int32, device="cuda")
        s["q"] = torch.randn((B, T, case["Hq"], D), generator=g, device="cuda",
                             dtype=torch.bfloat16)
        s["anc"] = None if case["tree"] == "chain" else _random_tree(B, T, g)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((B, T, case["Hq"]), dtype=torch.float32, device="cuda")
        return s
    T, V, H = case["T"], case["V"], case["H"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    s["logits"] = torch.randn((B, T, V), generator=g, device="cuda", dtype=dt).mul_(3)
    s["out"] = torch.empty_like(s["logits"])
    # text repeats itself: token ranks with a heavy head, in an order of its own
    u = torch.rand((B, H), generator=g, device="cuda")
    rank = (V ** u - 1).long().clamp(0, V - 1)
    s["history"] = ((rank * 7919 + 13) % V).to(torch.int32).contiguous()
    s["hist_len"] = _permuted(_hist(case), g)
    s["prompt_len"] = (s["hist_len"].float() * torch.rand(B, generator=g, device="cuda")).to(
        torch.int32)
    u = torch.rand((B, T), generator=g, device="cuda")
    rank = (V ** u - 1).long().clamp(0, V - 1)
    s["tokens"] = ((rank * 7919 + 13) % V).to(torch.int32).contiguous()
    s["anc"] = _random_tree(B, T, g) if T > 16 else None
    s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device="cuda")
    s["frequency"] = 0.5 * torch.rand(B, generator=g, device="cuda")
    s["presence"] = 0.5 * torch.rand(B, generator=g, device="cuda")
    s["bias"] = None
    if case["bias"]:
        n = min(case["bias"], V)
        s["bias"] = (torch.arange(B + 1, device="cuda", dtype=torch.int32) * n,
                     torch.stack([torch.randperm(V, generator=g, device="cuda")[:n]
                                  for _ in range(B)]).to(torch.int32).reshape(-1).contiguous(),
                     torch.randn(B * n, generator=g, device="cuda"))
    s["allow"] = s["allow_index"] = None
    if case["mask"] != "none":
        W = (V + 31) // 32
        n = 16  # grammar states: some allow nearly everything, some nearly nothing
        share = torch.rand((n, 1), generator=g, device="cuda").mul_(8).sub_(4).sigmoid_()
        bits = torch.rand((n, W * 32), generator=g, device="cuda") < share
        s["allow"] = _pack(bits)
        idx = torch.randint(0, n, (B, T), generator=g, device="cuda", dtype=torch.int32)
        if case["mask"] == "some":
            idx[torch.rand((B, T), generator=g, device="cuda") < 0.75] = -1
        s["allow_index"] = idx
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        return _run_own(s)
    return {"tree": _plain_tree, "cache": _plain_cache, "attn": _plain_attn,
            "adjust": _plain_adjust}[s["case"]["op"]](s)


def _run_own(s):
    import lossless_draft_verification_verifier_amd as svd
    op = s["case"]["op"]
    if op == "tree":
        return svd.draft_tree(s["drafts"], root=s["root"])
    if op == "cache":
        svd.cache_write(s["cache"], s["k"], s["v"], s["table"], s["ctx_len"])
        k, v = svd.cache_read(s["cache"], s["table"], s["case"]["T"], start=s["ctx_len"])
        return {"k": k, "v": v}
    if op == "attn":
        return svd.tree_attention(s["q"], s["cache"], s["table"], s["ctx_len"], anc=s["anc"],
                                  n_nodes=s["n_nodes"], out=s["out"], lse=s["lse"])
    return svd.adjust_logits(s["logits"], s["history"], s["hist_len"],
                             prompt_len=s["prompt_len"], tokens=s["tokens"], anc=s["anc"],
                             repetition=s["repetition"], frequency=s["frequency"],
                             presence=s["presence"], bias=s["bias"], allow=s["allow"],
                             allow_index=s["allow_index"], out=s["out"])


# -- plain forms ------------------------------------------------------------

def _bits(words, n):
    """int32 words [..., W] -> bool [..., n]."""
    at = torch.arange(n, device=words.device)
    return (words[..., at // 32] >> (at % 32).to(torch.int32)) & 1 != 0


def _plain_tree(s):
    x = s["drafts"].long()
    B, K, G = x.shape
    T = 1 + K * G
    dev = x.device
    live = (x >= 0).long().cumprod(2).bool()
    same = (x.unsqueeze(2) == x.unsqueeze(1)) & live.unsqueeze(2) & live.unsqueeze(1)
    same = same.long().cumprod(3).bool()  # [B, k, k', j]: equal through position j
    k = torch.arange(K, device=dev)
    lead = torch.where(same, k.view(1, 1, K, 1), K).amin(2)  # smallest k' with this prefix
    mine = (lead == k.view(1, K, 1)) & live
    ids = mine.view(B, -1).long().cumsum(1)  # 1.., draft by draft
    node = ids.view(B, K, G).gather(1, lead.clamp(max=K - 1))
    node = torch.where(live, node, T)
    n = ids[:, -1] + 1
    to = torch.where(mine.view(B, -1), ids, T)  # T: a place that is cut off again
    j = torch.arange(G, device=dev)

    def put(values, fill):
        return torch.full((B, T + 1), fill, dtype=torch.int64, device=dev).scatter_(
            1, to, values.reshape(B, -1))[:, :T]

    tokens = put(x, -1)
    tokens[:, 0] = s["root"]
    owner = put(k.view(1, K, 1).expand(B, K, G), 0)
    depth = put((j + 1).expand(B, K, G), 0)
    above = torch.cat([torch.zeros((B, K, 1), dtype=torch.int64, device=dev), node[:, :, :-1]], 2)
    parent = put(above, -1)
    path = node.gather(1, owner.unsqueeze(-1).expand(B, T, G))
    path = torch.where(j < depth.unsqueeze(-1), path, T)
    bits = torch.zeros((B, T, T + 1), dtype=torch.bool, device=dev).scatter_(2, path, True)[..., :T]
    bits[:, :, 0] = torch.arange(T, device=dev) < n.view(B, 1)
    first = torch.zeros((B, K, 1), dtype=torch.int64, device=dev)
    p_index = torch.cat([first, node], 2)
    p_index = torch.where(p_index < T, p_index + T * torch.arange(B, device=dev).view(B, 1, 1), -1)
    return {"tokens": tokens.to(torch.int32), "parent": parent.to(torch.int32),
            "depth": depth.to(torch.int32), "anc": _pack(bits), "n_nodes": n.to(torch.int32),
            "p_index": p_index.to(torch.int32)}


def _where(s, start, n):
    """Page and place of the n positions from start[b] on."""
    page = s["case"]["page"]
    pos = start.long().view(-1, 1) + torch.arange(n, device=start.device)
    col = (pos // page).clamp(max=s["table"].shape[1] - 1)
    return pos, s["table"].long().gather(1, col), pos % page


def _e4m3(x):
    """Rows of x as codes and a power-of-two scale each: the smallest 2^e with
    amax <= 448 * 2^e; the scale is held as e + 127."""
    a = x.abs().amax(-1)
    m, e = torch.frexp(a)  # a = m * 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(a > 0, e, 0).clamp(-126, 127)
    return torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _value(c, name, at):
    """The fp32 values that the cache holds at `at` = (page, place): [B, n, Hkv, D]."""
    x = c[name][at[0], :, at[1]].float()
    if c[name + "_scale"] is None:
        return x
    e = c[name + "_scale"][at[0], :, at[1]].to(torch.int32) - 127
    return torch.ldexp(x, e.unsqueeze(-1))


def _plain_cache(s):
    c = s["cache"]
    _, pg, place = _where(s, s["ctx_len"], s["case"]["T"])
    got = {}
    for n in ("k", "v"):
        x = s[n].float()
        if c[n + "_scale"] is None:
            c[n][pg, :, place] = x.to(torch.bfloat16)
        else:
            code, e = _e4m3(x)
            c[n].view(torch.uint8)[pg, :, place] = code.view(torch.uint8)
            c[n + "_scale"][pg, :, place] = e
        got[n] = _value(c, n, (pg, place)).to(torch.bfloat16)
    return got


def _plain_attn(s):
    case = s["case"]
    B, T, Hq, D = s["q"].shape
    Hkv = case["Hkv"]
    group = Hq // Hkv
    N = s["table"].shape[1] * case["page"]
    pos, pg, place = _where(s, torch.zeros_like(s["ctx_len"]), N)
    ctx, nodes = s["ctx_len"].long().view(B, 1), s["n_nodes"].long().view(B, 1)
    there = pos < ctx + nodes
    q = s["q"].float().view(B, T, Hkv, group, D).permute(0, 2, 1, 3, 4).reshape(
        B * Hkv, T * group, D)
    k = _value(s["cache"], "k", (pg, place)).permute(0, 2, 3, 1).reshape(B * Hkv, D, N)
    z = torch.bmm(q, k).view(B, Hkv, T, group, N) * (1.0 / math.sqrt(D))
    del k
    t = torch.arange(T, device=q.device)
    node = (pos - ctx).clamp(0, T - 1)  # the node that a position past the context holds
    if s["anc"] is None:
        sees = node.unsqueeze(1) <= t.view(1, T, 1)
    else:
        sees = _bits(s["anc"], T).gather(2, node.unsqueeze(1).expand(B, T, N))
    sees = (pos < ctx).unsqueeze(1) | (sees & there.unsqueeze(1))  # [B, T, N]
    z = z.masked_fill(~sees.view(B, 1, T, 1, N), -math.inf)
    m = z.amax(-1, keepdim=True)
    safe = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(z - safe)
    del z
    total = p.sum(-1, keepdim=True)
    v = torch.where(there.view(B, N, 1, 1), _value(s["cache"], "v", (pg, place)), 0.0)
    v = v.permute(0, 2, 1, 3).reshape(B * Hkv, N, D)
    o = torch.bmm(p.view(B * Hkv, T * group, N), v).view(B, Hkv, T, group, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (safe + torch.log(total)).squeeze(-1)
    valid = (t < nodes).view(B, T, 1)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(torch.bfloat16)
    lse = lse.permute(0, 2, 1, 3).reshape(B, T, Hq)
    s["out"].copy_(torch.where(valid.unsqueeze(-1), o, s["out"]))
    s["lse"].copy_(torch.where(valid, lse, s["lse"]))
    return {"out": s["out"], "lse": s["lse"]}


def _counts(s):
    """Occurrences: in the whole history [B, V], in its generated part [B, V] and on
    each row's path [B, T, V]."""
    B, T, V = s["logits"].shape
    dev = s["logits"].device
    at = torch.arange(s["history"].shape[1], device=dev)
    inside = at < s["hist_len"].view(B, 1)
    made = inside & (at >= s["prompt_len"].view(B, 1))
    h = s["history"].long()
    seen = torch.zeros((B, V), dtype=torch.int32, device=dev).scatter_add_(1, h, inside.int())
    count = torch.zeros((B, V), dtype=torch.int32, device=dev).scatter_add_(1, h, made.int())
    if s["anc"] is None:
        t = torch.arange(T, device=dev)
        on = (t.view(1, T, 1) >= t.view(1, 1, T)).expand(B, T, T)
    else:
        on = _bits(s["anc"], T)
    path = torch.zeros((B, T, V), dtype=torch.int32, device=dev).scatter_add_(
        2, s["tokens"].long().unsqueeze(1).expand(B, T, T), on.int())
    return seen, count, path


def _plain_adjust(s):
    B, T, V = s["logits"].shape
    z = s["logits"].float()
    seen, count, path = _counts(s)
    r = s["repetition"].view(B, 1, 1)
    z = torch.where(seen.unsqueeze(1) + path > 0, torch.where(z > 0, z / r, z * r), z)
    c = count.unsqueeze(1) + path
    z = z - s["frequency"].view(B, 1, 1) * c
    z = torch.where(c > 0, z - s["presence"].view(B, 1, 1), z)
    if s["bias"] is not None:
        off, tok, val = s["bias"]
        n = tok.numel() // B
        z = z + torch.zeros((B, V), device=z.device).scatter_add_(
            1, tok.view(B, n).long(), val.view(B, n)).unsqueeze(1)
    if s["allow"] is not None:
        idx = s["allow_index"].long()
        ok = _bits(s["allow"], V)[idx.clamp(min=0)] | (idx < 0).unsqueeze(-1)
        z = z.masked_fill(~ok, -math.inf)
    s["out"].copy_(z)
    return s["out"]


# ---------------------------------------------------------------------------
# the definitions in 64 bits, a prefix at a time

def _exact_e4m3(x):
    """What the quantised cache gives back for the rows of x (float64)."""
    a = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(a > 0, a, 448.0) / 448.0))
    e = torch.where(a <= 448.0 * torch.exp2(e - 1), e - 1, e)  # log2 next to a whole number
    e = torch.where(a > 448.0 * torch.exp2(e), e + 1, e)
    y = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(e)


def exact(case, seed):
    if case["op"] == "tree":
        return None  # whole numbers
    s = prepare(case, seed)
    B = case["B"]
    if case["op"] == "cache":
        if case["kind"] == "e4m3":
            return {n: _exact_e4m3(s[n].double()) for n in ("k", "v")}
        return {n: s[n].double() for n in ("k", "v")}
    if case["op"] == "attn":
        T, Hq, D = s["q"].shape[1:]
        Hkv, page = case["Hkv"], case["page"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros((B, T, Hq), dtype=torch.float64, device="cuda")
        c = s["cache"]
        for b in range(B):
            n0, n1 = int(s["ctx_len"][b]), int(s["n_nodes"][b])
            pages = s["table"][b, :(n0 + n1 + page - 1) // page].long()
            kv = []
            for name in ("k", "v"):
                x = c[name][pages].double()
                if case["kind"] == "e4m3":
                    x = x * torch.exp2(c[name + "_scale"][pages].double() - 127).unsqueeze(-1)
                kv.append(x.transpose(0, 1).reshape(Hkv, -1, D)[:, :n0 + n1])
            k, v = (x.repeat_interleave(Hq // Hkv, 0).contiguous() for x in kv)
            q = s["q"][b, :n1].double().transpose(0, 1).contiguous()
            z = torch.bmm(q, k.transpose(1, 2).contiguous()) / math.sqrt(D)
            if s["anc"] is None:
                ok = torch.ones((n1, n1), device="cuda").tril() > 0
            else:
                w = s["anc"][b, :n1].long()
                i = torch.arange(n1, device="cuda")
                ok = torch.bitwise_and(torch.bitwise_right_shift(w[:, i // 32], i % 32), 1) > 0
            z[:, :, n0:] = torch.where(ok, z[:, :, n0:], -math.inf)
            lse[b, :n1] = torch.logsumexp(z, -1).transpose(0, 1)
            out[b, :n1] = torch.bmm(torch.softmax(z, -1), v).transpose(0, 1)
        return {"out": out, "lse": lse}
    T, V = case["T"], case["V"]
    out = torch.empty((B, T, V), dtype=torch.float64, device="cuda")
    for b in range(B):
        n, p = int(s["hist_len"][b]), int(s["prompt_len"][b])
        h = s["history"][b, :n].long()
        every = torch.bincount(h, minlength=V)
        made = torch.bincount(h[p:], minlength=V)
        if s["anc"] is None:
            on = torch.ones((T, T), device="cuda").tril()
        else:
            w = s["anc"][b].long()
            i = torch.arange(T, device="cuda")
            on = torch.bitwise_and(torch.bitwise_right_shift(w[:, i // 32], i % 32), 1).float()
        z = s["logits"][b].double()
        extra = torch.zeros((T, V), device="cuda", dtype=torch.float64)
        extra.index_add_(1, s["tokens"][b].long(), on.double())
        total = made + extra
        r = s["repetition"][b].double()
        z = torch.where((every + extra) > 0, torch.where(z > 0, z / r, z * r), z)
        z = z - s["frequency"][b].double() * total - s["presence"][b].double() * (total > 0)
        if s["bias"] is not None:
            off, tok, val = s["bias"]
            i, j = int(off[b]), int(off[b + 1])
            z[:, tok[i:j].long()] += val[i:j].double()
        if s["allow"] is not None:
            for t, a in enumerate(s["allow_index"][b].tolist()):
                if a >= 0:
                    w = s["allow"][a].long().unsqueeze(1)
                    bit = torch.bitwise_right_shift(w, torch.arange(32, device="cuda")) & 1
                    z[t][bit.reshape(-1)[:V] == 0] = -math.inf
        out[b] = z
    return out
