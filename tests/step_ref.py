"""Plain references of the operators around a verification step, in numpy and
64 bits: the draft tree as a dictionary of prefixes, the quantised cache by its
definition, attention and logit adjustments row by row."""
from __future__ import annotations

import math

import numpy as np
import torch

BF16 = 2.0 ** -8   # half a step of each type, relative to the value
F32 = 2.0 ** -24


# -- draft tree -------------------------------------------------------------

def draft_tree(drafts, root, T):
    """The arrays of svd_draft_tree for drafts [B,K,G]."""
    B, K, G = drafts.shape
    W = (T + 31) // 32
    out = {"tokens": np.full((B, T), -1, np.int32), "parent": np.full((B, T), -1, np.int32),
           "depth": np.zeros((B, T), np.int32), "anc": np.zeros((B, T, W), np.uint32),
           "n_nodes": np.zeros(B, np.int32), "p_index": np.full((B, K, G + 1), -1, np.int32)}
    for b in range(B):
        node = {(): 0}
        where = {}
        for k in range(K):
            path = ()
            where[k, 0] = 0
            for j in range(G):
                x = int(drafts[b, k, j])
                if x < 0:
                    break
                path = path + (x,)
                node.setdefault(path, len(node))
                where[k, j + 1] = node[path]
        n = len(node)
        if n > T:
            out["n_nodes"][b] = -1
            continue
        out["n_nodes"][b] = n
        for (k, j), i in where.items():
            out["p_index"][b, k, j] = b * T + i
        for path, i in node.items():
            out["tokens"][b, i] = path[-1] if path else (-1 if root is None else root[b])
            out["parent"][b, i] = node[path[:-1]] if path else -1
            out["depth"][b, i] = len(path)
            for d in range(len(path) + 1):
                a = node[path[:d]]
                out["anc"][b, i, a // 32] |= np.uint32(1 << (a % 32))
    out["anc"] = out["anc"].view(np.int32)
    return out


def bits(words, n):
    """[..., W] words -> bool [..., n]."""
    w = np.asarray(words).astype(np.int64) & 0xFFFFFFFF
    i = np.arange(n)
    return ((w[..., i // 32] >> (i % 32)) & 1) != 0


def pack(b):
    """bool [..., n] -> int32 words."""
    b = np.asarray(b)
    n = b.shape[-1]
    W = (n + 31) // 32
    full = np.zeros(b.shape[:-1] + (W * 32,), np.uint64)
    full[..., :n] = b
    full = full.reshape(b.shape[:-1] + (W, 32)) << np.arange(32, dtype=np.uint64)
    return full.sum(-1).astype(np.uint32).view(np.int32)


# -- quantised cache --------------------------------------------------------

def e4m3_values(x):
    """What the E4M3 cache holds for the rows (last axis) of x: (values, scale bytes)."""
    x = np.asarray(x, np.float64)
    finite = np.isfinite(x)
    a = np.where(finite, np.abs(x), 0.0).max(-1)
    e = np.zeros(a.shape, np.int64)
    for i in np.ndindex(a.shape):
        if a[i] > 0:
            k = math.frexp(a[i] / 448.0)  # a / 448 = m * 2^k, m in [0.5, 1)
            e[i] = k[1] if k[0] > 0.5 else k[1] - 1
    e = np.maximum(e, -126)
    y = np.where(finite, x, 0.0) / np.exp2(e)[..., None]
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    y = np.round(y / step) * step  # np.round: ties to even
    # 256 * 2^120 would be past the largest number: 240 is the code below
    y = np.where((e == 120)[..., None], np.clip(y, -240.0, 240.0), y)
    v = y * np.exp2(e)[..., None]
    return np.where(finite, v, np.nan), (e + 127).astype(np.uint8)


def cache_values(cache, name):
    """float64 values of a whole cache on the host."""
    x = cache[name].detach().cpu().float().double()
    s = cache.get(name + "_scale")
    if s is None:
        return x.numpy()
    return (x * torch.exp2(s.cpu().double() - 127).unsqueeze(-1)).numpy()


# -- attention --------------------------------------------------------------

def attention(q, k_pages, v_pages, table, ctx, n_nodes, anc, scale):
    """q [B,T,Hq,D] float64, pages [n,Hkv,page,D].  Returns out, lse and the bounds of
    their errors: the products' fp32 sums, p rounded to bf16, the output's rounding."""
    B, T, Hq, D = q.shape
    Hkv, page = k_pages.shape[1:3]
    out, lse = np.zeros((B, T, Hq, D)), np.full((B, T, Hq), -np.inf)
    tol, ltol = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq))
    for b in range(B):
        n = int(n_nodes[b])
        total = int(ctx[b]) + n
        pg = table[b, np.arange(total) // page]
        place = np.arange(total) % page
        for t in range(n):
            see = np.ones(total, bool)
            see[ctx[b]:] = bits(anc[b, t], n) if anc is not None else np.arange(n) <= t
            if not see.any():
                continue
            for h in range(Hq):
                kh = h // (Hq // Hkv)
                k = k_pages[pg[see], kh, place[see]]
                v = v_pages[pg[see], kh, place[see]]
                z = scale * (k @ q[b, t, h])
                size = scale * (np.abs(k) @ np.abs(q[b, t, h])).max()
                m = z.max()
                p = np.exp(z - m)
                s = p.sum()
                w = p / s
                o = w @ v
                A = w @ np.abs(v)
                out[b, t, h], lse[b, t, h] = o, m + math.log(s)
                # exponent: D products and sums, the scaling, its rounding; then exp2 and the sums
                dz = F32 * ((D + 4) * size + 4 * abs(m))
                rel = 2 * dz + F32 * (see.sum() + 16)
                tol[b, t, h] = BF16 * A + BF16 * (np.abs(o) + BF16 * A) + rel * A
                ltol[b, t, h] = rel + 4 * F32 * abs(lse[b, t, h])
    return out, lse, tol, ltol


# -- logit adjustments ------------------------------------------------------

def adjust(z, bf16, history=None, hist_len=None, prompt_len=None, tokens=None, anc=None,
           repetition=None, frequency=None, presence=None, bias=None, allow=None,
           allow_index=None):
    """z [B,T,V] float64: the adjusted rows and the bound of their errors."""
    B, T, V = z.shape
    out, size = z.copy(), np.abs(z)
    # 1 / r, f * count, the two sums, then the factor and the summand at once: five
    # roundings of values no larger than `size`, and one for each bias entry of a token
    roundings = np.full(z.shape, 5.0)
    for b in range(B):
        for t in range(T):
            toks, made = [], []
            if history is not None:
                h = history[b, :hist_len[b]].tolist()
                p = 0 if prompt_len is None else int(prompt_len[b])
                toks += h
                made += h[max(p, 0):]
            if tokens is not None:
                on = bits(anc[b, t], T) if anc is not None else np.arange(T) <= t
                way = tokens[b, on].tolist()
                toks += way
                made += way
            row, mag = out[b, t], size[b, t]
            for v in {x for x in toks if 0 <= x < V}:
                c = made.count(v)
                if repetition is not None:
                    r = float(repetition[b])
                    row[v] = row[v] / r if row[v] > 0 else row[v] * r
                f = 0.0 if frequency is None else float(frequency[b])
                pr = 0.0 if presence is None else float(presence[b])
                mag[v] = abs(row[v]) + abs(f * c) + abs(pr)
                if c > 0:
                    row[v] = row[v] - f * c - pr
            if bias is not None:
                for i in range(int(bias[0][b]), int(bias[0][b + 1])):
                    v = int(bias[1][i])
                    if 0 <= v < V:
                        row[v] += float(bias[2][i])
                        mag[v] += abs(float(bias[2][i]))
                        roundings[b, t, v] += 1
            if allow is not None and allow_index[b, t] >= 0:
                row[~bits(allow[allow_index[b, t]], V)] = -np.inf
    tol = roundings * F32 * size
    if bf16:
        tol = tol + BF16 * (np.where(np.isfinite(out), np.abs(out), 0.0) + tol)
    return out, tol


def close(got, want, tol, what=""):
    """got and want agree: infinities and NaN in place, the rest within tol."""
    got = np.asarray(got, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    ok = np.isfinite(want)
    over = np.abs(got[ok] - want[ok]) - tol[ok]
    assert over.size == 0 or over.max() <= 0, (what, float(over.max()), int((over > 0).sum()))
