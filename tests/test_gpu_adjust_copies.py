"""Logits that no adjustment applies to keep their bits: payloads of NaN and signs of zero,
also where the token occurs in the history or on the path without any effect."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

KINDS = pytest.mark.parametrize("dt,it", [(torch.bfloat16, torch.int16), (torch.float32, torch.int32)],
                                ids=["bf16", "f32"])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def raw(B, T, V, dt, it):
    """Rows of -0, with NaN payloads of both signs and infinities."""
    bits = torch.iinfo(it).bits
    z = torch.full((B, T, V), -(1 << (bits - 1)), dtype=it, device="cuda")  # -0
    nan = 0x7F81 if it == torch.int16 else 0x7F800123
    z[..., 1::5] = nan
    z[..., 2::5] = nan - (1 << (bits - 1))
    z[..., 3::5] = 0x7F80 if it == torch.int16 else 0x7F800000
    return z


@KINDS
@pytest.mark.parametrize("V", [64, 61, 4103])
@pytest.mark.parametrize("args", [
    {},                                             # occurs, and nothing is asked for
    dict(repetition=1.0),                           # a factor of one
    dict(frequency=0.0, presence=0.0),              # counts without a price
    dict(repetition=1.0, frequency=0.0, presence=0.0, bias=True),  # biases of zero
], ids=["plain", "factor", "prices", "biases"])
@pytest.mark.parametrize("path", [False, True])
def test_tokens_without_an_effect(dt, it, V, args, path):
    svd = require_gpu()
    B, T = 2, 3
    z = raw(B, T, V, dt, it)
    h = torch.arange(40, dtype=torch.int32, device="cuda").expand(B, 40).contiguous() + V - 45
    kw = dict(history=h, hist_len=i32([40, 25]))
    if path:
        kw["tokens"] = i32([[0, V - 1, 7], [5, 5, 6]])
    for n, x in args.items():
        kw[n] = torch.full((B,), x, device="cuda") if n != "bias" else (
            i32([0, 4, 8]), i32([0, 1, V - 1, 30] * 2), torch.zeros(8, device="cuda"))
    got = svd.adjust_logits(z.view(dt), **kw)
    assert torch.equal(got.view(it), z)
    same = z.clone()
    svd.adjust_logits(same.view(dt), out=same.view(dt), **kw)
    assert torch.equal(same, z)


@KINDS
def test_a_prompt_has_no_count(dt, it):
    # frequency and presence price the tokens behind the prompt only
    svd = require_gpu()
    V = 64
    z = raw(1, 1, V, dt, it)
    kw = dict(history=i32([list(range(10))]), hist_len=i32([10]), prompt_len=i32([8]),
              frequency=torch.ones(1, device="cuda"), presence=torch.ones(1, device="cuda"))
    got = svd.adjust_logits(z.view(dt), **kw).view(it)
    keep = np.ones(V, bool)
    keep[[8, 9]] = False
    assert np.array_equal(got.cpu().numpy()[0, 0, keep], z.cpu().numpy()[0, 0, keep])
    assert float(got.view(dt)[0, 0, 9]) == -2.0 and float(got.view(dt)[0, 0, 8]) == np.inf


@KINDS
def test_a_factor_keeps_the_sign_of_zero(dt, it):
    svd = require_gpu()
    z = torch.zeros(1, 1, 16, dtype=dt, device="cuda")
    z[..., ::2] = -0.0
    got = svd.adjust_logits(z, i32([list(range(16))]), i32([16]), prompt_len=i32([16]),
                            repetition=torch.full((1,), 1.5, device="cuda"))
    assert torch.equal(got.view(it), z.view(it))
