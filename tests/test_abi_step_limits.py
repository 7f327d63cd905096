"""More refusals of the operators around a verification step, without a GPU: the
addresses are fake, and every rejection happens before any HIP call."""
import pytest

from test_abi_step import attend, cache, read, svd, write  # noqa: F401  (svd: the fixture)


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("name", ["k_scale", "v_scale"])
def test_scales_are_words(svd, name, off):  # noqa: F811
    good = dict(dtype=svd.SVD_CACHE_E4M3, k_scale=4096, v_scale=8192)
    c = cache(svd, **{**good, name: good[name] + off})
    assert write(svd, c) == read(svd, c) == attend(svd, c) == svd.SVD_EINVAL
    # the next check of an attention call is its workspace
    assert attend(svd, cache(svd, **good)) == svd.SVD_EWORKSPACE
    # a bf16 cache has no scales to check
    c = cache(svd, **{name: 4096 + off})
    assert attend(svd, c) == svd.SVD_EWORKSPACE


# a launch holds fewer than 2^32 threads: the least batch that is too large

def tree(svd, B):  # noqa: F811
    return svd.svd_draft_tree(64, None, B, 1, 1, 2, 128, 192, 256, 320, 384, 448, None)


def adjust(svd, B, V):  # noqa: F811
    return svd.svd_adjust_logits(4096, 8192, svd.SVD_BF16, B, 1, V, None, None, 0, None, None,
                                 None, None, None, None, None, None, None, None, 0, None, None, 0,
                                 None)


def test_more_threads_than_a_launch_holds(svd):  # noqa: F811
    assert tree(svd, 1 << 22) == svd.SVD_EINVAL                   # 1024 threads a prefix
    # 2 heads of 64, k and v: 32 threads a token
    assert write(svd, cache(svd), B=1, T=1 << 27) == svd.SVD_EINVAL
    assert read(svd, cache(svd), B=1, N=1 << 27) == svd.SVD_EINVAL
    assert write(svd, cache(svd), B=1 << 26, T=2) == svd.SVD_EINVAL
    # one row a head: waves for 16 rows in two halves and 256 threads, 384 a head
    f = svd.svd_tree_attention_workspace_bytes
    most = ((1 << 32) - 1) // 384 // 8 * 8
    assert f(most // 2, 1, 2, 2, 64, 64) > 0 and f(most // 2 + 1, 1, 2, 2, 64, 64) == 0
    assert attend(svd, cache(svd), B=most // 2 + 1, T=1, Hq=2) == svd.SVD_EINVAL
    assert attend(svd, cache(svd), B=most // 2, T=1, Hq=2) == svd.SVD_EWORKSPACE
    assert adjust(svd, 1 << 24, 100) == svd.SVD_EINVAL            # 256 a prefix and range


@pytest.mark.parametrize("out", [1 << 16, (1 << 16) + 512, (1 << 16) - 2560, (1 << 16) + 5 * 768 + 256])
def test_attention_does_not_write_over_its_queries(svd, out):  # noqa: F811
    # 6 tokens of 4 heads of 64, 384 elements apart: q from 65536 to 65536 + 5 * 768 + 512
    kw = dict(q=1 << 16, qs=384, ws=1 << 20, n=1 << 20)
    assert attend(svd, cache(svd), out=out, **kw) == svd.SVD_EINVAL
