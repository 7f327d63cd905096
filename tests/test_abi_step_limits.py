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
