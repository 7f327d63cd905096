"""Refusals and references of a serving loop's other operators, without a GPU: every
rejection happens on the host before any HIP call (the addresses are fake)."""
import math

import numpy as np
import pytest
import torch

import serve_ref as S


@pytest.fixture(scope="module")
def svd():
    import lossless_draft_verification_verifier_amd as m
    return m


def cache(svd, **kw):
    a = dict(k=4096, v=8192, k_scale=None, v_scale=None, block_table=12288, n_pages=10,
             max_pages=4, page=16, kv_heads=2, head_dim=64, dtype=svd.SVD_CACHE_BF16)
    a.update(kw)
    return svd.CacheStruct(*[a[n] for n, _ in svd.CacheStruct._fields_])


def pages(svd, **kw):
    a = dict(length=64, shared=None, B=4, mp=8, page=16, n=10, ring=1 << 12, state=1 << 13,
             held=1 << 14, table=1 << 15, so=1 << 16, ho=1 << 17, to=1 << 18, room=1 << 19,
             ws=1 << 20, wb=1 << 12)
    a.update(kw)
    return svd.svd_cache_pages(a["length"], a["shared"], a["B"], a["mp"], a["page"], a["n"],
                               a["ring"], a["state"], a["held"], a["table"], a["so"], a["ho"],
                               a["to"], a["room"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(length=None), -1), (dict(ring=None), -1), (dict(state=None), -1), (dict(held=None), -1),
    (dict(table=None), -1), (dict(so=None), -1), (dict(ho=None), -1), (dict(to=None), -1),
    (dict(room=None), -1), (dict(ws=None), -1), (dict(ws=(1 << 20) + 128), -1), (dict(B=0), -1),
    (dict(B=1 << 31), -1), (dict(B=1 << 29), -1), (dict(mp=0), -1), (dict(mp=1 << 27), -1),
    (dict(page=8), -1), (dict(page=48), -1), (dict(page=2048), -1), (dict(page=-16), -1),
    (dict(n=0), -1), (dict(n=1 << 31), -1), (dict(wb=0), -3), (dict(wb=511), -3),
    # an output that meets its input without being it
    (dict(so=(1 << 13) + 4), -1), (dict(ho=(1 << 14) - 12), -1), (dict(to=(1 << 15) + 124), -1)])
def test_pages_refusals(svd, kw, want):
    assert pages(svd, **kw) == want


def test_pages_workspace(svd):
    f = svd.svd_cache_pages_workspace_bytes
    assert f(1) == 512 and f(16) == 512 and f(17) == 768
    assert f(0) == f(-1) == f(1 << 31) == f(-(1 << 63)) == 0


@pytest.mark.parametrize("kw", [
    dict(c=None), dict(new=None), dict(table=None), dict(off=None), dict(seq=None), dict(pos=None),
    dict(slot=None), dict(B=0), dict(B=1 << 30), dict(mp=0), dict(mp=1 << 28), dict(page=17),
    dict(n=0), dict(n=1 << 31), dict(N=0), dict(N=-1), dict(N=1 << 31)])
def test_slots_refusals(svd, kw):
    a = dict(c=64, new=128, table=256, B=4, mp=8, page=16, n=10, N=30, off=512, seq=1024, pos=2048,
             slot=4096)
    a.update(kw)
    assert svd.svd_cache_slots(a["c"], a["new"], a["table"], a["B"], a["mp"], a["page"], a["n"],
                               a["N"], a["off"], a["seq"], a["pos"], a["slot"],
                               None) == svd.SVD_EINVAL


def write_slots(svd, c, **kw):
    a = dict(k=4096, v=8192, dtype=svd.SVD_BF16, ks=128, vs=128, slot=64, N=3)
    a.update(kw)
    return svd.svd_cache_write_slots(c, a["k"], a["v"], a["dtype"], a["ks"], a["vs"], a["slot"],
                                     a["N"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(slot=None), -1), (dict(dtype=2), -2),
    (dict(ks=127), -1), (dict(vs=-1), -1), (dict(k=4097), -1), (dict(dtype=0, v=8194), -1),
    (dict(N=0), -1), (dict(N=1 << 31), -1)])
def test_write_slots_refusals(svd, kw, want):
    assert write_slots(svd, cache(svd, block_table=None, max_pages=0), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(dtype=2), -2), (dict(dtype=1), -1),
    (dict(head_dim=96), -1), (dict(page=48), -1), (dict(n_pages=0), -1), (dict(n_pages=1 << 31), -1),
    (dict(kv_heads=0), -1), (dict(kv_heads=4097), -1), (dict(k=4100), -1)])
def test_write_slots_refuses_bad_caches(svd, kw, want):
    assert write_slots(svd, cache(svd, **kw)) == want
    assert write_slots(svd, None) == svd.SVD_EINVAL


def filt(svd, **kw):
    a = dict(z=4096, out=1 << 20, dtype=svd.SVD_BF16, B=2, T=3, V=100)
    a.update(kw)
    return svd.svd_filter_logits(a["z"], a["out"], a["dtype"], a["B"], a["T"], a["V"], None, None,
                                 None, None, None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(z=None), -1), (dict(out=None), -1), (dict(dtype=2), -2), (dict(dtype=-9), -2),
    (dict(B=0), -1), (dict(B=1 << 30, T=1), -1), (dict(B=1 << 22, T=1), -1), (dict(T=0), -1),
    (dict(T=4097), -1), (dict(V=0), -1), (dict(V=-5), -1), (dict(z=4097), -1),
    (dict(out=(1 << 20) + 1), -1), (dict(dtype=0, z=4098), -1),
    # an out that meets the logits without being them
    (dict(out=4096 + 2), -1), (dict(out=4096 + 1198), -1), (dict(z=8192, out=8192 - 1198), -1)])
def test_filter_refusals(svd, kw, want):
    assert filt(svd, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(z=None), -1), (dict(token=None), -1), (dict(dtype=3), -2), (dict(B=0), -1),
    (dict(T=4097), -1), (dict(V=0), -1), (dict(z=4097), -1), (dict(K=0), -1), (dict(K=65), -1),
    (dict(B=1 << 21, T=2), -1), (dict(B=1 << 22, T=1), -1)])
def test_sample_refusals(svd, kw, want):
    a = dict(z=4096, dtype=svd.SVD_BF16, B=2, T=3, V=100, K=2, token=1 << 20)
    a.update(kw)
    assert svd.svd_sample(a["z"], a["dtype"], a["B"], a["T"], a["V"], a["K"], None, None, None,
                          None, None, None, 0, 0, a["token"], None, None) == want


def attend(svd, c, **kw):
    a = dict(q=4096, qs=256, ctx=64, anc=None, depth=None, off=None, G=0, scale=0.125, cap=0.0,
             slopes=None, B=2, T=3, Hq=4, out=1 << 16, ws=1 << 20, n=0)
    a.update(kw)
    return svd.svd_prefix_attention(c, a["q"], a["qs"], a["ctx"], None, a["anc"], a["depth"],
                                    a["off"], a["G"], a["scale"], a["cap"], a["slopes"], a["B"],
                                    a["T"], a["Hq"], a["out"], None, a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), -1), (dict(ctx=None), -1), (dict(out=None), -1), (dict(ws=None), -1),
    (dict(q=4104), -1), (dict(out=(1 << 16) + 8), -1), (dict(ws=(1 << 20) + 64), -1),
    (dict(qs=255), -1), (dict(qs=260), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1),
    (dict(B=0), -1), (dict(T=0), -1), (dict(T=4097), -1), (dict(Hq=3), -1), (dict(B=1 << 30), -1),
    (dict(cap=-1.0), -1), (dict(cap=float("nan")), -1), (dict(cap=float("inf")), -1),
    (dict(cap=1e-39), -1), (dict(cap=3e38), -1), (dict(off=64), -1), (dict(G=1), -1),
    (dict(off=64, G=-1), -1), (dict(off=64, G=3), -1), (dict(slopes=64, anc=64), -1),
    (dict(out=4096 + 512, n=1 << 40), -1),
    (dict(), -3), (dict(off=64, G=2), -3), (dict(slopes=64), -3), (dict(cap=30.0), -3),
    (dict(slopes=64, anc=64, depth=64), -3)])
def test_prefix_attention_refusals(svd, kw, want):
    assert attend(svd, cache(svd), **kw) == want


@pytest.mark.parametrize("cap,scale,want", [
    (16384.0, 0.125, -3), (16385.0, 0.125, -1), (1e6, 0.125, -1), (1e30, 0.125, -1),
    (2.0 ** -10, 0.125, -3), (16384.0, 1e-35, -1), (1e-30, 1e30, -1)])
def test_prefix_attention_refuses_caps_it_cannot_keep(svd, cap, scale, want):
    # scores would be off by a few 2^-24 of the cap; or scale / cap is no normal number
    assert attend(svd, cache(svd), cap=cap, scale=scale) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), -1), (dict(block_table=None), -1), (dict(dtype=2), -2), (dict(dtype=1), -1),
    (dict(head_dim=96), -1), (dict(page=8), -1), (dict(max_pages=0), -1), (dict(kv_heads=0), -1)])
def test_prefix_attention_refuses_bad_caches(svd, kw, want):
    assert attend(svd, cache(svd, **kw)) == want
    assert attend(svd, None) == svd.SVD_EINVAL


def test_prefix_attention_workspace(svd):
    f, tree = svd.svd_prefix_attention_workspace_bytes, svd.svd_tree_attention_workspace_bytes
    for a in ((1, 1, 32, 8, 128, 4096), (256, 9, 32, 8, 128, 4096), (3, 5, 4, 4, 64, 100)):
        assert f(*a, 0) == tree(*a)
        assert f(*a, 1) > tree(*a) and f(*a, 1) % 256 == 0
    for bad in [(0, 1, 8, 8, 64, 64, 0), (1, 1, 8, 3, 64, 64, 0), (2, 1, 8, 8, 64, 64, 3),
                (2, 1, 8, 8, 64, 64, -1), (1, 1, 8, 8, 80, 64, 1), (1, 1, 8, 8, 64, 1 << 31, 1),
                (1 << 17, 4096, 8, 1, 64, 64, 1), (1 << 20, 512, 65536, 1, 64, 64, 1),
                ((1 << 63) - 1, 1, 8, 8, 64, 64, 1)]:
        assert f(*bad) == 0, bad


def test_conveniences_refuse_host_tensors(svd):
    c = {"k": torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16),
         "v": torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)}
    i = torch.zeros(1, 1, dtype=torch.int32)
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    pool = svd.page_pool(5, 2, 3, device="cpu")
    assert pool["table"].shape == (2, 3) and pool["state"].tolist() == [0, 5]
    assert pool["free"].tolist() == [0, 1, 2, 3, 4] and not pool["held"].any()
    with pytest.raises(ValueError):
        svd.cache_pages(pool, i[0], 16)
    with pytest.raises(ValueError):
        svd.cache_slots(c, i, i[0], i[0], 4)
    with pytest.raises(ValueError):
        svd.cache_write_slots(c, x[0], x[0], torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        svd.filter_logits(torch.zeros(1, 1, 4))
    with pytest.raises(ValueError):
        svd.sample(torch.zeros(1, 1, 4))
    with pytest.raises(ValueError):
        svd.filter_logits(torch.zeros(1, 4))
    with pytest.raises(ValueError):
        svd.prefix_attention(x, c, i, i[0])


# -- the references themselves ----------------------------------------------

def test_reference_filter_by_hand():
    z = np.array([1.0, 3.0, 3.0, -np.inf, 2.0])
    assert S.kept(z).all()
    assert S.kept(z, k=1).tolist() == [False, True, False, False, False]
    assert S.kept(z, k=2).tolist() == [False, True, True, False, False]
    assert S.kept(z, t=0.0).tolist() == [False, True, False, False, False]
    assert S.kept(z, k=3).tolist() == [False, True, True, False, True]
    # weights 1, 1, e^-1, e^-2: half of the mass is one token and a quarter of the next
    assert S.kept(z, p=0.3).tolist() == [False, True, False, False, False]
    assert S.kept(z, p=0.5).tolist() == [False, True, True, False, False]
    assert S.kept(z, p=0.0).tolist() == [False, True, False, False, False]
    assert S.kept(z, least=math.exp(-1.5)).tolist() == [False, True, True, False, True]
    assert S.kept(z, least=7.0).tolist() == [False, True, True, False, False]
    assert S.kept(z, t=-1.0) is None and S.kept(z, p=math.nan) is None
    assert S.kept(np.array([0.0, np.nan])) is None and S.kept(np.full(3, -np.inf)) is None
    keep = S.kept(z, k=3)
    assert [S.draw(z, keep, 1.0, u)[0] for u in (0.0, 0.4, 0.45, 0.8, 0.9, 1 - 2.0 ** -53)] == [
        1, 1, 2, 2, 4, 4]
    assert abs(S.draw(z, keep, 1.0, 0.0)[1] + math.log(2 + math.exp(-1))) < 1e-15


def test_reference_pages_by_hand():
    table = [[0, -1, -1], [1, 2, -1], [3, -1, -1], [-1, -1, -1], [-1, -1, -1]]
    args = [33, 0, 10, 200, -1], [0, 0, 1, 0, 0], 16
    held = [1, 2, 1, 0, 0]
    ring, state, now, tab, room = S.pages(*args, [7, 8, 9, 4, 5, 6, 10, 11], [4, 4], held, table)
    # two pages from places 4 and 5; the second sequence's two behind the ring's end, places
    # 0 and 1; 200 tokens have no room in three entries, and a length below zero is none
    assert tab == [[0, 5, 6], [-1, -1, -1], [3, -1, -1], [-1] * 3, [-1] * 3]
    assert ring == [1, 2, 9, 4, 5, 6, 10, 11] and state == [6, 4]
    assert room == [48, 0, 16, -1, -1] and now == [3, 0, 1, 0, 0]
    # one page for a sequence that needs two: it gets none, and so does a later one
    _, state, now, tab, room = S.pages([33, 5], None, 16, [4, 5, 6, 7], [3, 1], [1, 0],
                                       [[0, -1, -1], [-1, -1, -1]])
    assert now == [1, 0] and room == [16, 0] and state == [3, 1]
    # four free pages and two given back in a ring of five: nothing moves
    _, state, now, tab2, room = S.pages(*args, [7, 8, 9, 4, 5], [4, 4], held, table)
    assert state == [4, 4] and now == held and tab2 == table and room == [-1] * 5


def test_reference_slots_by_hand():
    off, seq, pos, slot = S.slots([15, 0, 3], [2, 0, 3], [[4, 9], [1, 1], [2, 0]], 16, 5, 7)
    assert off == [0, 2, 2, 5] and seq == [0, 0, 2, 2, 2, -1, -1]
    assert pos == [15, 16, 3, 4, 5, -1, -1] and slot == [79, -1, 35, 36, 37, -1, -1]
