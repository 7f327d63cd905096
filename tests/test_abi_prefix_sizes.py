"""Workspaces of the attention over shared prefixes, without a GPU."""
import pytest


@pytest.fixture(scope="module")
def svd():
    import lossless_draft_verification_verifier_amd as m
    return m


@pytest.mark.parametrize("B,T,Hq,Hkv,D,G", [
    (1024, 1, 32, 8, 128, 512), (256, 1, 32, 8, 128, 64), (512, 1, 8, 1, 64, 512),
    (64, 3, 16, 4, 128, 16), (1024, 1, 32, 32, 128, 512), (16, 1, 32, 8, 128, 1)])
def test_groups_of_few_rows_take_parts_of_64_rows(svd, B, T, Hq, Hkv, D, G):
    # no group has more than 64 rows on average: a part per kv head and tile of a group, and
    # one per piece of the line of 256, each of 64 rows with D elements, an exponent and a sum
    group = Hq // Hkv
    assert B * T * group <= 64 * G
    parts = (B * T * group // 64 + G) * Hkv + 256
    plans = 64 * (B + G) + 4 * B * T + 256 * 8
    own = svd.svd_tree_attention_workspace_bytes(B, T, Hq, Hkv, D, 4096)
    got = svd.svd_prefix_attention_workspace_bytes(B, T, Hq, Hkv, D, 4096, G)
    assert got <= parts * 64 * (D + 2) * 4 + plans + own


def test_groups_of_many_rows_take_parts_of_256(svd):
    # just past 64 rows on average: no less than a whole part of 256 rows per kv head
    f = svd.svd_prefix_attention_workspace_bytes
    few, many = f(32, 1, 64, 4, 128, 4096, 8), f(33, 1, 64, 4, 128, 4096, 8)
    assert many >= (8 * 4 + 256) * 256 * (128 + 2) * 4 > few
