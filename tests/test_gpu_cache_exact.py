"""What bf16 makes of the cache's values at the ends of its range: exact for scales of 2^-124
and more, rounded to the nearest multiple of 2^-133 (ties to even) below, in a read as in the
attention."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("byte", [1, 2, 3, 4, 127, 247])
def test_every_code_in_bf16(byte):
    svd = require_gpu()
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    codes[0x7F] = codes[0xFF] = 0           # NaN
    if byte == 247:                         # 256 * 2^120 and more are no numbers
        codes[(codes & 0x7F) > 0x77] = 0
    exact = codes.view(torch.float8_e4m3fn).double().cpu().numpy() * 2.0 ** (byte - 127)
    step = 2.0 ** -133
    bf16 = exact if byte >= 3 else np.round(exact / step) * step
    assert (bf16 != exact).any() == (byte < 3)
    tab = i32(0).view(1, 1)
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    for part in range(4):
        c = svd.kv_cache(1, 1, 16, 64, dtype=torch.float8_e4m3fn)
        for n in "kv":
            c[n].view(torch.uint8)[0, 0, 0] = codes[64 * part:64 * part + 64]
            c[n + "_scale"][0, 0, 0] = byte
        want = bf16[64 * part:64 * part + 64]
        for got in svd.cache_read(c, tab, 1, dtype=torch.float32):
            assert np.array_equal(got.double().cpu().numpy().ravel(), exact[64 * part:64 * part + 64])
        for got in svd.cache_read(c, tab, 1):
            assert np.array_equal(got.double().cpu().numpy().ravel(), want)
        # one token: its weight is 1
        got = svd.tree_attention(q, c, tab, i32(0))["out"]
        assert np.array_equal(got.double().cpu().numpy().ravel(), want)


def test_the_least_rows_as_they_are_written():
    svd = require_gpu()
    x = torch.zeros(1, 3, 1, 64, device="cuda")
    x[0, 0, 0, :3] = torch.tensor([1e-45, 2e-45, -3e-45])
    x[0, 1, 0, :4] = torch.tensor([2.0 ** -126, -(2.0 ** -130), 2.0 ** -134, 2.0 ** -133])
    x[0, 2, 0, :3] = torch.tensor([448 * 2.0 ** -125, 2.0 ** -134, 3 * 2.0 ** -134])
    c = svd.kv_cache(1, 1, 16, 64, dtype=torch.float8_e4m3fn)
    svd.cache_write(c, x, x, i32(0).view(1, 1), i32(0))
    assert c["k_scale"][0, 0, :3].tolist() == [1, 1, 2]
    wide, _ = svd.cache_read(c, i32(0).view(1, 1), 3, dtype=torch.float32)
    got, _ = svd.cache_read(c, i32(0).view(1, 1), 3)
    step = 2.0 ** -133
    want = np.round(wide.double().cpu().numpy() / step) * step
    assert np.array_equal(got.double().cpu().numpy(), want)
    assert float(wide[0, 1, 0, 2]) == 2.0 ** -134 and float(got[0, 1, 0, 2]) == 0


def test_bf16_rows_are_held_bit_for_bit():
    # every bf16 number, subnormal ones too; a NaN stays a NaN of its sign
    svd = require_gpu()
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
    x = bits.view(torch.bfloat16).view(1, 1024, 1, 64)
    c = svd.kv_cache(64, 1, 16, 64)
    tab = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64)
    for src in (x, x.float()):
        svd.cache_write(c, src, src, tab, i32(0))
        for got in svd.cache_read(c, tab, 1024):
            nan = torch.isnan(x)
            assert torch.equal(torch.isnan(got), nan)
            assert torch.equal(got.view(torch.int16)[~nan], x.view(torch.int16)[~nan])
