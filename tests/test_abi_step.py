"""Refusals of the operators around a verification step, without a GPU: every
rejection happens on the host before any HIP call (the addresses are fake)."""
import ctypes

import numpy as np
import pytest
import torch

import step_ref as R


@pytest.fixture(scope="module")
def svd():
    import lossless_draft_verification_verifier_amd as m
    return m


def cache(svd, **kw):
    a = dict(k=4096, v=8192, k_scale=None, v_scale=None, block_table=12288, n_pages=10,
             max_pages=4, page=16, kv_heads=2, head_dim=64, dtype=svd.SVD_CACHE_BF16)
    a.update(kw)
    return svd.CacheStruct(*[a[n] for n, _ in svd.CacheStruct._fields_])


BAD_CACHE = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(block_table=None), -1), (dict(dtype=2), -2),
    (dict(dtype=-7), -2), (dict(dtype=1), -1), (dict(dtype=1, k_scale=64), -1),
    (dict(head_dim=96), -1), (dict(head_dim=0), -1), (dict(page=8), -1), (dict(page=48), -1),
    (dict(page=2048), -1), (dict(page=0), -1), (dict(page=-16), -1), (dict(n_pages=0), -1),
    (dict(n_pages=1 << 31), -1), (dict(max_pages=0), -1), (dict(max_pages=1 << 27), -1),
    (dict(kv_heads=0), -1), (dict(kv_heads=4097), -1), (dict(k=4100), -1), (dict(v=8200), -1),
]


def write(svd, c, **kw):
    a = dict(k=4096, v=8192, dtype=svd.SVD_BF16, ks=128, vs=128, ctx=64, B=2, T=3)
    a.update(kw)
    return svd.svd_cache_write(c, a["k"], a["v"], a["dtype"], a["ks"], a["vs"], a["ctx"], None,
                               None, a["B"], a["T"], None)


def read(svd, c, **kw):
    a = dict(B=2, N=3, dtype=svd.SVD_BF16, k=4096, v=8192)
    a.update(kw)
    return svd.svd_cache_read(c, None, None, a["B"], a["N"], a["dtype"], a["k"], a["v"], None)


def attend(svd, c, **kw):
    a = dict(q=4096, qs=256, ctx=64, scale=0.125, B=2, T=3, Hq=4, out=8192, ws=1 << 20, n=0)
    a.update(kw)
    return svd.svd_tree_attention(c, a["q"], a["qs"], a["ctx"], None, None, a["scale"], a["B"],
                                  a["T"], a["Hq"], a["out"], None, a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_bad_caches_are_refused_everywhere(svd, kw, want):
    c = cache(svd, **kw)
    assert write(svd, c) == want
    assert read(svd, c) == want
    assert attend(svd, c) == want


def test_no_cache(svd):
    assert write(svd, None) == read(svd, None) == attend(svd, None) == svd.SVD_EINVAL


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(ctx=None), -1), (dict(dtype=2), -2),
    (dict(ks=127), -1), (dict(vs=0), -1), (dict(k=4097), -1), (dict(v=8193), -1),
    (dict(dtype=0, k=4098), -1), (dict(B=0), -1), (dict(T=0), -1), (dict(T=1 << 31), -1),
    (dict(B=1 << 30, T=4), -1)])
def test_write_refusals(svd, kw, want):
    assert write(svd, cache(svd), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(dtype=2), -2), (dict(k=4104), -1),
    (dict(v=8200), -1), (dict(B=0), -1), (dict(N=0), -1), (dict(B=1 << 30, N=4), -1)])
def test_read_refusals(svd, kw, want):
    assert read(svd, cache(svd), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), -1), (dict(ctx=None), -1), (dict(out=None), -1), (dict(ws=None), -1),
    (dict(q=4104), -1), (dict(out=8200), -1), (dict(ws=(1 << 20) + 64), -1), (dict(qs=255), -1),
    (dict(qs=260), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(scale=3e38), -1),
    (dict(B=0), -1), (dict(T=0), -1), (dict(T=4097), -1), (dict(Hq=3), -1), (dict(Hq=0), -1),
    (dict(B=1 << 30), -1), (dict(), -3)])
def test_attention_refusals(svd, kw, want):
    assert attend(svd, cache(svd), **kw) == want


def test_attention_workspace(svd):
    f = svd.svd_tree_attention_workspace_bytes
    assert f(1, 1, 32, 8, 128, 4096) > 0 and f(1, 1, 32, 8, 128, 4096) % 256 == 0
    # a full batch needs no parts; one long sequence does
    assert f(256, 9, 32, 8, 128, 4096) == 256
    assert f(1, 1, 32, 8, 128, 1 << 17) > f(1, 1, 32, 8, 128, 512)
    for bad in [(0, 1, 8, 8, 64, 64), (1, 0, 8, 8, 64, 64), (1, 4097, 8, 8, 64, 64),
                (1, 1, 8, 3, 64, 64), (1, 1, 8, 0, 64, 64), (1, 1, 8, 8, 80, 64),
                (1, 1, 8, 8, 64, 0), (1, 1, 8, 8, 64, 1 << 31), (1, 1, 4, 8, 64, 64)]:
        assert f(*bad) == 0, bad


@pytest.mark.parametrize("kw", [
    dict(d=None), dict(tok=None), dict(par=None), dict(dep=None), dict(anc=None), dict(nn=None),
    dict(px=None), dict(B=0), dict(B=1 << 30), dict(K=0), dict(K=65), dict(G=0), dict(G=4097),
    dict(T=0), dict(T=4097)])
def test_draft_tree_refusals(svd, kw):
    a = dict(d=64, tok=128, par=192, dep=256, anc=320, nn=384, px=448, B=2, K=2, G=3, T=7)
    a.update(kw)
    assert svd.svd_draft_tree(a["d"], None, a["B"], a["K"], a["G"], a["T"], a["tok"], a["par"],
                              a["dep"], a["anc"], a["nn"], a["px"], None) == svd.SVD_EINVAL


@pytest.mark.parametrize("kw,want", [
    (dict(z=None), -1), (dict(out=None), -1), (dict(dtype=2), -2), (dict(B=0), -1),
    (dict(T=0), -1), (dict(T=4097), -1), (dict(V=0), -1), (dict(hist=64), -1),
    (dict(hist=64, hlen=64, hs=0), -1), (dict(hist=64, hlen=64, hs=1 << 30), -1),
    (dict(anc=64), -1), (dict(boff=64, nb=-1), -1), (dict(boff=64, nb=2), -1),
    (dict(boff=64, nb=2, btok=64), -1), (dict(allow=64), -1), (dict(allow=64, nm=1), -1),
    (dict(allow=64, ai=64, nm=0), -1), (dict(z=4097), -1), (dict(out=8193), -1),
    (dict(dtype=0, z=4098), -1), (dict(B=1 << 29, V=1 << 20), -1)])
def test_adjust_refusals(svd, kw, want):
    a = dict(z=4096, out=8192, dtype=svd.SVD_BF16, B=2, T=3, V=100, hist=None, hs=0, hlen=None,
             tok=None, anc=None, boff=None, btok=None, bval=None, nb=0, allow=None, ai=None, nm=0)
    a.update(kw)
    assert svd.svd_adjust_logits(a["z"], a["out"], a["dtype"], a["B"], a["T"], a["V"], None,
                                 a["hist"], a["hs"], a["hlen"], None, a["tok"], a["anc"], None,
                                 None, None, a["boff"], a["btok"], a["bval"], a["nb"],
                                 a["allow"], a["ai"], a["nm"], None) == want


def test_conveniences_refuse_host_tensors(svd):
    c = {"k": torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16),
         "v": torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)}
    i = torch.zeros(1, 1, dtype=torch.int32)
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        svd.draft_tree(torch.zeros(1, 1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        svd.cache_write(c, x, x, i, i[0])
    with pytest.raises(ValueError):
        svd.cache_read(c, i, 1)
    with pytest.raises(ValueError):
        svd.tree_attention(x, c, i, i[0])
    with pytest.raises(ValueError):
        svd.adjust_logits(torch.zeros(1, 1, 4))
    with pytest.raises(TypeError):
        svd.kv_cache(1, 1, 16, 64, dtype=torch.float16, device="cpu")
    e = svd.kv_cache(3, 2, 16, 64, dtype=torch.float8_e4m3fn, device="cpu")
    assert e["k"].shape == (3, 2, 16, 64) and e["v_scale"].shape == (3, 2, 16)
    assert int(e["k_scale"].min()) == 127


def test_cache_struct_is_the_headers(svd):
    # five pointers, an int64, four int32 and the enum: no padding but the tail's
    assert ctypes.sizeof(svd.CacheStruct) == 5 * 8 + 8 + 5 * 4 + 4
    assert svd.CacheStruct.n_pages.offset == 40 and svd.CacheStruct.dtype.offset == 64


def test_reference_quantiser_agrees_with_torch():
    # the reference of the GPU tests, against torch's own conversion on scaled rows
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((50, 64)) * np.exp2(rng.integers(-30, 30, (50, 1)))).astype(np.float32)
    x[0] = 0
    x[1, 0] = 448.0
    x[1, 1:] = 1.0
    v, s = R.e4m3_values(x)
    e = s.astype(np.int64) - 127
    y = np.ldexp(x, -e[:, None]).astype(np.float32)
    assert np.abs(y).max() <= 448 and s[0] == 127 and s[1] == 127
    assert np.all(np.abs(y).max(1)[2:] > 224 - 1)
    t = torch.from_numpy(y).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.ldexp(t.astype(np.float64), e[:, None]), v)


def test_reference_tree_by_hand():
    d = np.array([[[5, 6, 7], [5, 6, 8], [5, 9, 7], [4, 6, 7]]], np.int32)
    r = R.draft_tree(d, [2], 13)
    assert r["n_nodes"][0] == 10
    assert r["tokens"][0, :10].tolist() == [2, 5, 6, 7, 8, 9, 7, 4, 6, 7]
    assert r["parent"][0, :10].tolist() == [-1, 0, 1, 2, 2, 1, 5, 0, 7, 8]
    assert r["p_index"][0].tolist() == [[0, 1, 2, 3], [0, 1, 2, 4], [0, 1, 5, 6], [0, 7, 8, 9]]
    assert np.flatnonzero(R.bits(r["anc"][0, 6], 13)).tolist() == [0, 1, 5, 6]
