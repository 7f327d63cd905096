"""Attention over shared prefixes where groups have few rows on average and many in one, and the
other way round: row tiles of 64 and of 256 against float64."""
import pytest

from gpu_util import require_gpu, say
from test_gpu_prefix_attention import BOTH, check, problem, slopes_of

pytestmark = pytest.mark.gpu


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,groups,alone", [
    # 4 query heads per kv head.  15 groups, 26 sequences of 36 rows: 62 on average, 432 in one
    (9, [(12, 400)] + [(1, 0)] * 11 + [(2, 256), (0, 0), (1, 130)], 0),
    # the same with two sequences more: 67 on average
    (9, [(12, 400)] + [(1, 0)] * 11 + [(2, 256), (0, 0), (1, 130)], 2),
    # pairs and fours of a token each
    (1, [(2, 300)] * 20 + [(4, 700)] * 9 + [(17, 128), (33, 1100)], 3)])
def test_uneven_groups(kind, D, T, groups, alone):
    svd = require_gpu()
    say("uneven", kind, D, T, len(groups), alone)
    p = problem(groups, T, 8, 2, D, 16, kind, 0, 50, T > 1, seed=D + T, alone=alone)
    check(svd, p)
    check(svd, p, cap=20.0)
    check(svd, p, cap=20.0, slopes=slopes_of(8))
