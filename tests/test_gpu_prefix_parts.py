"""Attention over shared prefixes at its longest: a row joined from a part of every workgroup that
the shared tokens are cut over, and prompts of hundreds of new tokens behind a prefix, against
float64.  serve_ref.attention derives the tolerances, with the number of parts that these
lengths make."""
import pytest

import serve_ref as S
import step_ref as R
from gpu_util import require_gpu, say
from test_gpu_prefix_attention import BOTH, check, problem, run, slopes_of

pytestmark = pytest.mark.gpu


@BOTH
@pytest.mark.parametrize("D,shared,want", [(64, 32768, 256), (128, 33024, 172), (128, 16000, 125)])
@pytest.mark.parametrize("cap,sloped", [(0.0, False), (20.0, True)])
def test_a_row_of_many_parts(kind, D, shared, want, cap, sloped):
    # one kv head and one row tile: the line is one unit of shared / 64 steps, at least two of
    # them, and a 256th of them, in a piece
    steps = shared // 64
    per = max(2, -(-steps // 256))
    assert -(-steps // per) == want
    svd = require_gpu()
    say("parts", kind, D, shared, cap)
    p = problem([(3, shared)], 2, 2, 1, D, 128, kind, 0, 300, False, seed=D + want)
    sl = slopes_of(2) if sloped else None
    got, lse = run(svd, p, cap=cap, slopes=sl)
    # up to 64 parts of the rest besides
    ref, wl, tol, ltol = S.attention(
        p["q"].double().cpu().numpy(), R.cache_values(p["c"], "k"), R.cache_values(p["c"], "v"),
        p["tab"], p["ctx"], p["nodes"], None, None, D ** -0.5, cap, sl, parts=want + 64)
    for b in range(3):
        n = int(p["nodes"][b])
        R.close(got[b, :n], ref[b, :n], tol[b, :n], ("out", b))
        R.close(lse[b, :n], wl[b, :n], ltol[b, :n], ("lse", b))


@BOTH
@pytest.mark.parametrize("T,tree", [(130, False), (300, True), (513, False)])
def test_prompts_behind_a_prefix(kind, T, tree):
    svd = require_gpu()
    say("prompts", kind, T, tree)
    p = problem([(2, 390), (3, 128)], T, 4, 2, 128 if tree else 64, 16, kind, 0, 40, tree, seed=T)
    check(svd, p)
    check(svd, p, cap=15.0, slopes=slopes_of(4), only=[1, 4])
