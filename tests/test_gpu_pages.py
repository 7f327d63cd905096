"""Block tables and slot maps of the paged cache against plain references."""
import numpy as np
import pytest
import torch

import serve_ref as S
import step_ref as R
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x, np.int64).clip(-(1 << 31), (1 << 31) - 1).astype(np.int32),
                        device="cuda")


def pool_of(ring, state, held, table):
    return {"free": i32(ring), "state": i32(state), "held": i32(held), "table": i32(table)}


def check(svd, length, shared, page, ring, state, held, table, apart=False):
    pool = pool_of(ring, state, held, table)
    want = S.pages(length, shared, page, ring, state, held, table)
    to = None
    if apart:
        to = {n: torch.full_like(pool[n], 99) for n in ("table", "held", "state")}
        before = {n: pool[n].clone() for n in to}
    room = svd.cache_pages(pool, i32(length), page, shared=None if shared is None else i32(shared),
                           out=to)
    if apart:
        for n in to:
            assert torch.equal(pool[n], before[n]), n
    got = dict(pool, **(to or {}))
    for n, w in zip(("free", "state", "held", "table"), want):
        assert got[n].tolist() == list(w), n
    assert room.tolist() == want[4]
    return want


def state_of(g, B, mp, spare):
    """A pool in the middle of its life: B sequences, a ring that begins anywhere."""
    held = g.integers(0, mp + 1, B)
    n = int(held.sum()) + spare
    ids = g.permutation(n)
    table, at = np.full((B, mp), -1), 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    head = int(g.integers(0, n))
    ring = np.full(n, -5)
    ring[(head + np.arange(spare)) % n] = ids[at:]
    return ring.tolist(), [head, spare], held.tolist(), table.tolist()


@pytest.mark.parametrize("apart", [False, True], ids=["in_place", "apart"])
@pytest.mark.parametrize("B,mp,spare,page", [(1, 1, 1, 16), (1, 5, 3, 32), (7, 9, 20, 16),
                                             (64, 40, 700, 64), (1024, 11, 3000, 16),
                                             (1025, 3, 100, 1024), (3000, 17, 9000, 128)])
def test_pages(B, mp, spare, page, apart):
    svd = require_gpu()
    say(B, mp, spare, page)
    for seed in range(3):
        g = np.random.default_rng([B, mp, seed])
        ring, state, held, table = state_of(g, B, mp, spare)
        length = g.integers(0, mp * page + 1, B)
        if seed == 2:  # some settings that no sequence has
            length[g.random(B) < 0.2] = -1
            length[g.random(B) < 0.2] = mp * page + 1
        shared = None if seed == 0 else (np.array(held) * g.random(B)).astype(int)
        check(svd, length, shared, page, ring, state, held, table, apart)


def test_a_ring_that_runs_out():
    svd = require_gpu()
    # three pages free: the first sequence takes two, the second would need two more and gets
    # none, and so does the third, which would need one
    r = check(svd, [32, 32, 16, 0], None, 16, [9, 8, 7, 6, 5, 4], [5, 3], [0, 0, 0, 1],
              [[-1] * 4, [-1] * 4, [-1] * 4, [1, -1, -1, -1]])
    assert r[2] == [2, 0, 0, 0] and r[4] == [32, 0, 0, 0]
    # what one gives back is for the next call
    check(svd, [16, 0], None, 16, [1], [0, 0], [0, 1], [[-1], [0]])


def test_states_out_of_range_change_nothing():
    svd = require_gpu()
    table, held = [[0, 1], [2, -1]], [2, 1]
    for state in ([-1, 2], [5, 2], [0, -1], [0, 6], [(1 << 31) - 1, 0], [4, 4]):
        r = check(svd, [0, 32], None, 16, [4, 3, 2, 1, 0], state, held, table)
        assert r[4] == [-1, -1]
    for held in ([-1, 1], [3, 1]):  # of one sequence: that one alone
        r = check(svd, [32, 32], None, 16, [4, 3, 2, 1, 0], [1, 2], held, table)
        assert r[4] == [-1, 32]
    r = check(svd, [32, 32], [0, 2], 16, [4, 3, 2, 1, 0], [1, 2], [2, 1], table)
    assert r[4] == [32, -1]
    r = check(svd, [32, 32], [-1, 1], 16, [4, 3, 2, 1, 0], [1, 2], [2, 1], table)
    assert r[4] == [-1, 32]
    check(svd, [(1 << 31) - 1, 0], None, 16, [4, 3, 2, 1, 0], [1, 2], [2, 1], table)


def test_a_pool_through_many_calls():
    # no page is ever in two places, and none is lost
    svd = require_gpu()
    g = np.random.default_rng(2)
    B, mp, page, n = 40, 30, 16, 500
    pool = svd.page_pool(n, B, mp)
    ws = torch.empty(svd.svd_cache_pages_workspace_bytes(B), dtype=torch.uint8, device="cuda")
    for step in range(30):
        length = g.integers(0, mp * page + 1, B) * (g.random(B) < 0.7)
        before = pool["held"].tolist()
        room = svd.cache_pages(pool, i32(length), page, workspace=ws).tolist()
        head, count = pool["state"].tolist()
        held, ring, table = pool["held"].tolist(), pool["free"].tolist(), pool["table"].tolist()
        ids = [ring[(head + i) % n] for i in range(count)]
        for b in range(B):
            ids += table[b][:held[b]]
            assert all(x == -1 for x in table[b][held[b]:])
            need = -(-int(length[b]) // page)
            assert held[b] == need or (held[b] == before[b] and need > held[b])
            assert room[b] == held[b] * page
        assert sorted(ids) == list(range(n)), step


def test_pages_of_many_sequences_captured():
    svd = require_gpu()
    g = np.random.default_rng(3)
    B, mp, page = 300, 50, 16
    ring, state, held, table = state_of(g, B, mp, 4000)
    pool = pool_of(ring, state, held, table)
    to = {n: torch.zeros_like(pool[n]) for n in ("table", "held", "state")}
    length = i32(g.integers(0, mp * page, B))
    svd.cache_pages(pool, length, page, out=to)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        room = svd.cache_pages(pool, length, page, out=to)
    for r in range(4):
        length.copy_(i32(g.integers(0, mp * page, B)))
        svd.cache_pages(pool_of(ring, state, held, table), length, page)  # eager work between
        pool["free"].copy_(i32(ring))
        graph.replay()
        torch.cuda.synchronize()
        want = S.pages(length.tolist(), None, page, ring, state, held, table)
        for n, w in zip(("free", "state", "held", "table"), want):
            assert dict(pool, **to)[n].tolist() == list(w), (r, n)
        assert room.tolist() == want[4]


# -- packed tokens ----------------------------------------------------------

@pytest.mark.parametrize("B,most,page", [(1, 1, 16), (1, 5000, 64), (5, 40, 16), (300, 30, 32),
                                         (1024, 3, 16), (1025, 2, 128), (4000, 5, 16)])
def test_slots(B, most, page):
    svd = require_gpu()
    say(B, most, page)
    g = np.random.default_rng([B, most])
    mp, n_pages = (most + 200) // page + 2, 1000
    c = svd.kv_cache(n_pages, 1, page, 64)
    for seed in range(3):
        new = g.integers(0, most + 1, B)
        ctx = g.integers(0, 200, B)
        table = g.integers(0, n_pages, (B, mp))
        if seed == 1:  # pages and lengths that are none
            table[g.random((B, mp)) < 0.3] = -1
            table[g.random((B, mp)) < 0.1] = n_pages
            new[g.random(B) < 0.1] = -4
            ctx[g.random(B) < 0.1] = -1
            ctx[g.random(B) < 0.1] = (1 << 31) - 1
        if seed == 2:
            new[:] = 0
            new[B // 2] = most
        total = int(np.where((new > 0) & (ctx >= 0) & (ctx + new < 1 << 31), new, 0).sum())
        for N in {max(1, total), total + 1500, max(1, total // 2), 1}:
            m = svd.cache_slots(c, i32(table), i32(ctx), i32(new), N)
            off, seq, pos, slot = S.slots(ctx, new, table, page, n_pages, N)
            assert m["row_off"].tolist() == off
            assert m["seq"].tolist() == seq and m["pos"].tolist() == pos
            assert m["slot"].tolist() == slot and m["slot"].dtype == torch.int64


def test_slots_past_32_bits():
    # a page index whose slots need more than 32 bits, a number of tokens that does, too
    svd = require_gpu()
    n_pages, page = (1 << 31) - 1, 1024
    table, ctx, new = i32([[n_pages - 1, 3]]), i32([1022]), i32([4])
    o = torch.zeros(8, dtype=torch.int64, device="cuda")
    i = torch.zeros(32, dtype=torch.int32, device="cuda")
    svd._torch()
    svd._call(svd._c.svd_cache_slots, "svd_cache_slots", 0, ctx.data_ptr(),
              new.data_ptr(), table.data_ptr(), 1, 2, page, n_pages, 5, i.data_ptr(),
              i[8:].data_ptr(), i[16:].data_ptr(), o.data_ptr())
    torch.cuda.synchronize()
    base = (n_pages - 1) * page
    assert o.tolist()[:5] == [base + 1022, base + 1023, 3 * page, 3 * page + 1, -1]
    c = svd.kv_cache(4, 1, 16, 64)
    big = (1 << 31) - 1
    m = svd.cache_slots(c, i32([[0], [1], [2]]), i32([0, 0, 5]), i32([big, big, 2]), 3)
    assert m["row_off"].tolist() == [0, big, big, big] and m["seq"].tolist() == [0, 0, 0]
    assert m["pos"].tolist() == [0, 1, 2] and m["slot"].tolist() == [0, 1, 2]


KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32], ids=["from_bf16", "from_f32"])
@pytest.mark.parametrize("Hkv,D,page", [(1, 64, 16), (3, 128, 32), (8, 64, 128)])
def test_write_by_slot(kind, src, Hkv, D, page):
    # the same bits as a write by position, and nothing else touched
    svd = require_gpu()
    g = np.random.default_rng(5)
    B, T = 5, 40
    new, ctx = g.integers(0, T + 1, B), g.integers(0, 50, B)
    mp = (50 + T) // page + 1
    table = g.permutation(B * mp + 3)[:B * mp].reshape(B, mp)
    x = torch.randn(2, B, T, Hkv, D, device="cuda").to(src) * 5
    x[0, 0, :3, 0, 7] = float("inf")
    both = []
    for packed in (False, True):
        c = svd.kv_cache(B * mp + 3, Hkv, page, D, dtype=KINDS[kind])
        for n in ("k", "v"):
            c[n].view(torch.uint8).fill_(0x11)
        if packed:
            m = svd.cache_slots(c, i32(table), i32(ctx), i32(new), int(new.sum()) + 7)
            rows = [torch.cat([x[i, b, :new[b]] for b in range(B)] + [x[i, 0, :7]]) for i in (0, 1)]
            fused = torch.cat([rows[0].flatten(1), rows[1].flatten(1)], 1)  # strided tokens
            k = fused[:, :Hkv * D].unflatten(1, (Hkv, D))
            v = fused[:, Hkv * D:].unflatten(1, (Hkv, D))
            svd.cache_write_slots(c, k, v, m["slot"])
        else:
            svd.cache_write(c, x[0], x[1], i32(table), i32(ctx), n_new=i32(new))
        both.append(c)
    for n in ("k", "v", "k_scale", "v_scale"):
        if both[0][n] is not None:
            assert torch.equal(both[0][n].view(torch.uint8), both[1][n].view(torch.uint8)), n


def test_slots_that_are_none_are_skipped():
    svd = require_gpu()
    c = svd.kv_cache(3, 1, 16, 64)
    x = torch.ones(6, 1, 64, dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([-1, 48, 1 << 40, -(1 << 40), 47, 0], device="cuda")
    svd.cache_write_slots(c, x, x, slot)
    assert int((c["k"] == 1).sum()) == 128 and int((c["v"] == 1).sum()) == 128
    assert (c["k"][2, 0, 15] == 1).all() and (c["k"][0, 0, 0] == 1).all()
    with pytest.raises(ValueError):
        svd.cache_write_slots(c, x, x[:5], slot)
    with pytest.raises(ValueError):
        svd.cache_write_slots(c, x, x, slot[:5])
    with pytest.raises(TypeError):
        svd.cache_write_slots(c, x, x, slot.int())
