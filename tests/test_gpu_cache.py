"""The paged cache on the GPU: what is written is read back as the values that the
codes stand for, bit for bit (the scale is a power of two, so x * 2^-e, the code
and code * 2^e are each exact or rounded once, to nearest even)."""
import numpy as np
import pytest
import torch

import step_ref as R
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def table(B, max_pages, n_pages, seed):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.permutation(n_pages)[:B * max_pages].reshape(B, max_pages)
                            .astype(np.int32)).cuda()


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def held(x, kind):
    """float64 values that a cache of this kind holds for the rows of x."""
    if kind == "e4m3":
        return R.e4m3_values(x.float().cpu().numpy())[0]
    return x.float().to(torch.bfloat16).double().cpu().numpy()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,D,page", [(1, 1, 1, 64, 16), (3, 37, 2, 128, 16), (2, 5, 8, 128, 64),
                                          (4, 100, 3, 64, 32), (1, 300, 5, 128, 1024)],
                         ids=lambda v: str(v))
def test_written_tokens_read_back(kind, src, B, T, H, D, page):
    svd = require_gpu()
    torch.manual_seed(B + T)
    say("cache", kind, src, B, T, H, D, page)
    ctx = torch.randint(0, 50, (B,), dtype=torch.int32, device="cuda")
    mp = (50 + T + page - 1) // page
    tab = table(B, mp, B * mp + 5, T)
    c = svd.kv_cache(B * mp + 5, H, page, D, dtype=KINDS[kind])
    # rows of very different sizes, a zero row, a row of one value
    k = torch.randn(B, T, H, D, device="cuda") * torch.exp2(
        torch.randint(-40, 40, (B, T, H, 1), device="cuda").float())
    v = torch.randn(B, T, H, D, device="cuda")
    k[0, 0, 0] = 0
    v[0, 0, 0] = 1.75
    k, v = k.to(src), v.to(src)
    svd.cache_write(c, k, v, tab, ctx)
    for dt in (torch.float32, torch.bfloat16):
        gk, gv = svd.cache_read(c, tab, T, start=ctx, dtype=dt)
        for got, x in ((gk, k), (gv, v)):
            assert np.array_equal(got.double().cpu().numpy(), held(x, kind))
    # the pages that no sequence has, and the positions around the written ones, stay
    used = set(tab.flatten().tolist())
    for p in range(c["k"].shape[0]):
        if p not in used:
            assert not c["k"][p].view(torch.uint8).any() and not c["v"][p].view(torch.uint8).any()
    before, _ = svd.cache_read(c, tab, 50, count=ctx, out=(
        torch.full((B, 50, H, D), 7.0, device="cuda"),
        torch.full((B, 50, H, D), 7.0, device="cuda")))
    for b in range(B):
        n = int(ctx[b])
        assert not before[b, :n].any() and (before[b, n:] == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_destinations_counts_and_strides(kind):
    svd = require_gpu()
    torch.manual_seed(4)
    B, T, H, D, page = 3, 9, 2, 128, 16
    tab = table(B, 4, 20, 1)
    ctx = i32(0, 13, 31)
    n_new = i32(9, 0, 4)
    dst = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    dst[0, 0], dst[0, 3], dst[0, 8], dst[2, 1], dst[2, 5] = 0, 1, 2, 0, 1
    # keys and values as parts of one fused projection; 3 elements off alignment too
    for off in (0, 3):
        c = svd.kv_cache(20, H, page, D, dtype=KINDS[kind])
        width = 5 * H * D + 8
        qkv = torch.randn(B * T * width + 8, device="cuda", dtype=torch.bfloat16)[off:]
        k = qkv.as_strided((B, T, H, D), (T * width, width, D, 1), qkv.storage_offset())
        v = qkv.as_strided((B, T, H, D), (T * width, width, D, 1), qkv.storage_offset() + 3 * H * D)
        svd.cache_write(c, k, v, tab, ctx, n_new=n_new, dst=dst)
        gk, gv = svd.cache_read(c, tab, 64, dtype=torch.float32)
        want = np.zeros((B, 64, H, D))
        for b, t, p in ((0, 0, 0), (0, 3, 1), (0, 8, 2), (2, 1, 31)):
            want[b, p] = held(k[b, t], kind)
        assert np.array_equal(gk.double().cpu().numpy(), want)
        for b, t, p in ((0, 0, 0), (0, 3, 1), (0, 8, 2), (2, 1, 31)):
            want[b, p] = held(v[b, t], kind)
        assert np.array_equal(gv.double().cpu().numpy(), want)


def test_rounding_of_every_code_and_tie():
    # all e4m3 values and the midpoints between them, under a scale of one
    svd = require_gpu()
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (codes[1:] + codes[:-1]) / 2
    x = torch.cat([codes, mid, -codes, -mid, torch.nextafter(mid, mid * 2),
                   torch.nextafter(mid, mid * 0)])
    x = x[:x.numel() // 63 * 63].view(-1, 63)
    x = torch.cat([torch.full((x.shape[0], 1), 448.0), x], 1)
    n = x.shape[0]
    c = svd.kv_cache(1 + n // 16, 1, 16, 64, dtype=torch.float8_e4m3fn)
    tab = torch.arange(1 + n // 16, dtype=torch.int32, device="cuda").view(1, -1)
    k = x.view(1, n, 1, 64).cuda()
    svd.cache_write(c, k, -k, tab, i32(0))
    gk, gv = svd.cache_read(c, tab, n, dtype=torch.float32)
    want = R.e4m3_values(x.numpy())[0]
    assert np.array_equal(gk.view(n, 64).double().cpu().numpy(), want)
    assert np.array_equal(gv.view(n, 64).double().cpu().numpy(), -want)


def test_extreme_and_non_finite_rows():
    svd = require_gpu()
    D = 64
    x = torch.zeros(8, D)
    x[0, :3] = torch.tensor([3.4028235e38, -1e30, 1.0])
    x[1, :3] = torch.tensor([1e-45, 2e-45, -3e-45])   # subnormal inputs: 2^-126 is the least scale
    x[2, :3] = torch.tensor([2.0 ** -126, -2.0 ** -130, 0.0])
    x[3, :4] = torch.tensor([float("inf"), 3.0, -1.0, 0.5])
    x[4, :4] = torch.tensor([float("nan"), 3.0, -1.0, 0.5])
    x[5] = float("-inf")
    x[6, :2] = torch.tensor([448.0, 1.0])
    x[7, :2] = torch.tensor([448.00003, 1.0])
    c = svd.kv_cache(1, 1, 16, D, dtype=torch.float8_e4m3fn)
    tab = i32(0).view(1, 1)
    k = x.view(1, 8, 1, D).cuda()
    svd.cache_write(c, k, k, tab, i32(0))
    gk, _ = svd.cache_read(c, tab, 8, dtype=torch.float32)
    want, scale = R.e4m3_values(x.numpy())
    got = gk.view(8, D).double().cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(c["k_scale"].cpu().numpy()[0, 0, :8], scale)
    assert scale[6] == 127 and scale[7] == 128 and scale[1] == 1


def test_positions_without_a_page():
    svd = require_gpu()
    torch.manual_seed(6)
    B, T, H, D, page = 5, 20, 2, 64, 16
    for kind in KINDS.values():
        c = svd.kv_cache(8, H, page, D, dtype=kind)
        # a bad page index on either side, a negative length, a length past the table
        tab = i32(0, 1, -1, 2, 8, 3, 4, 5, 6, 7).view(B, 2)
        ctx = i32(5, 0, 0, -3, 25)
        k = torch.randn(B, T, H, D, device="cuda")
        svd.cache_write(c, k, k, tab, ctx)
        got, _ = svd.cache_read(c, tab, T, start=ctx, dtype=torch.float32)
        got = got.cpu().numpy()
        want = held(k, "bf16" if kind == torch.bfloat16 else "e4m3")
        nan = np.zeros((B, T), bool)
        nan[1, :16] = nan[2, :16] = True   # their first page is out of range
        nan[3] = True
        nan[4, 7:] = True                  # positions 32.. have no page
        assert np.isnan(got[nan]).all()
        assert np.array_equal(got[~nan], want[~nan])


def test_a_cache_past_32_bits():
    svd = require_gpu()
    # 40000 pages of 128 KiB: the last pages start beyond 2^32 bytes and 2^31 elements
    n, H, page, D = 40000, 8, 64, 128
    c = {x: torch.empty((n, H, page, D), dtype=torch.bfloat16, device="cuda") for x in "kv"}
    c.update(k_scale=None, v_scale=None)
    tab = i32(n - 1, 17, n - 2, 33000).view(1, 4)
    k = torch.randn(1, 256, H, D, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(1, 256, H, D, device="cuda", dtype=torch.bfloat16)
    svd.cache_write(c, k, v, tab, i32(0))
    gk, gv = svd.cache_read(c, tab, 256)
    assert torch.equal(gk, k) and torch.equal(gv, v)
    assert torch.equal(c["k"][n - 2].transpose(0, 1), k[0, 128:192])
    assert torch.equal(c["v"][33000].transpose(0, 1), v[0, 192:])
