"""Plain references of a serving loop's other operators, in numpy and 64 bits: filtered
and sampled logits, block tables and slot maps, attention with shaped scores."""
from __future__ import annotations

import math

import numpy as np

import step_ref as R
from hash_ref import uniform_bits

BF16, F32 = R.BF16, R.F32
SAMPLE = 4  # the purpose of a draw's uniforms


# -- filtered and sampled logits --------------------------------------------

def scale_bits(V):
    """s: weights are whole multiples of 2^-s of the largest."""
    return min(62 - (V - 1).bit_length(), 50)


def weights(z, t):
    """The weights of a row as whole numbers (int64)."""
    with np.errstate(invalid="ignore"):
        x = (z - z.max()) / t
    return np.rint(np.exp(x) * 2.0 ** scale_bits(z.size)).astype(np.int64)


def answers(z, t, p, least):
    return (t >= 0 and t < math.inf and p == p and least == least and
            not np.isnan(z).any() and z.max() < math.inf and z.max() > -math.inf)


def kept(z, t=1.0, k=0, p=1.0, least=0.0):
    """Which tokens of a row (float64) are kept, or None for a row without an answer."""
    V = z.size
    if not answers(z, t, p, least):
        return None
    if t == 0:
        t, k = 1.0, 1
    order = np.lexsort((np.arange(V), -z))
    zs = z[order]
    n = V
    if least > 0:
        n = max(int((zs >= z.max() + t * math.log(least)).sum()), int((zs == zs[0]).sum()))
    if k > 0:
        n = min(n, k)
    if p < 1:
        w = weights(z, t)[order[:n]]
        total = int(w.sum())
        target = min(max(math.ceil(max(p, 0.0) * float(total)), 1), total)
        n = int((np.cumsum(w) < target).sum()) + 1
    keep = np.zeros(V, bool)
    keep[order[:n]] = True
    return keep


def draw(z, keep, t, u):
    """(token, log-probability) of a row's draw."""
    t = 1.0 if t == 0 else t
    w = np.where(keep, weights(z, t), 0)
    upto = np.cumsum(w)
    total = int(upto[-1])
    x = min(int(u * float(total)), total - 1)
    v = int((upto <= x).sum())
    exact = np.where(keep, np.exp((z - z.max()) / t), 0.0).sum()
    return v, (z[v] - z.max()) / t - math.log(exact)


def logprob_tol(lp, V):
    # one rounding to fp32; weights are off by half a unit each, of which the largest has 2^s
    return F32 * abs(lp) + V * 2.0 ** -(scale_bits(V) + 1) + 1e-13


def hash_uniform(seed, row, k, t, T):
    return uniform_bits(seed, row, k * T + t, SAMPLE) * 2.0 ** -53


# -- block tables and slots -------------------------------------------------

def pages(length, shared, page, ring, state, held, table):
    """(ring, state, held, table, room) after a call, as lists of ints."""
    n, B, mp = len(ring), len(length), len(table[0])
    ring, held, table = list(ring), list(held), [list(r) for r in table]
    head, count = int(state[0]), int(state[1])
    need, room = [None] * B, [-1] * B
    for b in range(B):
        sh = 0 if shared is None else int(shared[b])
        x = max(sh, -(-int(length[b]) // page))
        if length[b] >= 0 and x <= mp and 0 <= held[b] <= mp and 0 <= sh <= held[b]:
            need[b] = x
    back = sum(max(held[b] - need[b], 0) for b in range(B) if need[b] is not None)
    if not (0 <= head < n and 0 <= count <= n and count + back <= n):
        return ring, [head, count], held, table, room
    end, asked, taken, given = head + count, 0, 0, 0
    new_ring = list(ring)
    for b in range(B):
        if need[b] is None:
            continue
        grow = need[b] - held[b]
        if grow > 0:
            asked += grow
            if asked <= count:
                for j in range(held[b], need[b]):
                    table[b][j] = ring[(head + taken) % n]
                    taken += 1
                held[b] = need[b]
        else:
            for j in range(need[b], held[b]):
                new_ring[(end + given) % n] = table[b][j]
                table[b][j] = -1
                given += 1
            held[b] = need[b]
        room[b] = held[b] * page
    return new_ring, [(head + taken) % n, count - taken + given], held, table, room


def slots(ctx, new, table, page, n_pages, N):
    off, seq, pos, slot = [], [], [], []
    for b in range(len(ctx)):
        off.append(len(seq))
        n, c = int(new[b]), int(ctx[b])
        if n < 0 or c < 0 or n + c > 2 ** 31 - 1:
            continue
        for p in range(c, c + n):
            seq.append(b)
            pos.append(p)
            pg = int(table[b][p // page]) if p // page < len(table[b]) else -1
            slot.append(pg * page + p % page if 0 <= pg < n_pages else -1)
    off.append(len(seq))
    fill = [-1] * max(0, N - len(seq))
    return off, (seq + fill)[:N], (pos + fill)[:N], (slot + fill)[:N]


# -- attention --------------------------------------------------------------

def attention(q, k_pages, v_pages, table, ctx, n_nodes, anc, depth, scale, cap=0.0, slopes=None,
              parts=64):
    """As step_ref.attention, with capped scores and slopes.  parts: how many partial sums a
    row may be joined from."""
    B, T, Hq, D = q.shape
    Hkv, page = k_pages.shape[1:3]
    out, lse = np.zeros((B, T, Hq, D)), np.full((B, T, Hq), -np.inf)
    tol, ltol = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq))
    for b in range(B):
        n, c = int(n_nodes[b]), int(ctx[b])
        total = c + n
        pg, place = table[b, np.arange(total) // page], np.arange(total) % page
        d = np.arange(n) if anc is None or depth is None else depth[b, :n]
        at = np.concatenate([np.arange(c), c + d])
        for t in range(n):
            see = np.ones(total, bool)
            see[c:] = R.bits(anc[b, t], n) if anc is not None else np.arange(n) <= t
            if not see.any():
                continue
            for kh in range(Hkv):
                k, v = k_pages[pg[see], kh, place[see]], v_pages[pg[see], kh, place[see]]
                for h in range(kh * (Hq // Hkv), (kh + 1) * (Hq // Hkv)):
                    z = scale * (k @ q[b, t, h])
                    # products, sums, scaling; then the roundings of the steps after them
                    dz = F32 * (D + 4) * scale * (np.abs(k) @ np.abs(q[b, t, h])).max()
                    if cap:
                        z = cap * np.tanh(z / cap)
                        # exp2 and its argument, 1 + e, the reciprocal, the last sum
                        dz += 8 * F32 * cap
                    if slopes is not None:
                        far = float(slopes[h]) * (c + d[t] - at[see])
                        z = z - far
                    m = z.max()
                    if slopes is not None:  # of the tokens that weigh anything
                        dz += 4 * F32 * np.abs(far[z > m - 40]).max()
                    dz += 4 * F32 * abs(m)
                    p = np.exp(z - m)
                    s = p.sum()
                    w = p / s
                    o, A = w @ v, w @ np.abs(v)
                    out[b, t, h], lse[b, t, h] = o, m + math.log(s)
                    rel = 2 * dz + F32 * (see.sum() + 16 + 2 * parts)
                    tol[b, t, h] = BF16 * A + BF16 * (np.abs(o) + BF16 * A) + rel * A
                    ltol[b, t, h] = rel + 4 * F32 * abs(lse[b, t, h])
    return out, lse, tol, ltol
