"""A caller's workspace is checked like every other tensor: its device and that it is
contiguous.  On the host, where no call can reach a kernel."""
import pytest
import torch


@pytest.fixture(scope="module")
def svd():
    import lossless_draft_verification_verifier_amd as m
    return m


def test_a_workspace_elsewhere_is_refused(svd):
    with pytest.raises(ValueError, match="workspace must be on cuda:0"):
        svd._workspace(torch.empty(256, dtype=torch.uint8), 0)


def test_a_workspace_with_gaps_is_refused(svd):
    # (-1 is what a host tensor's get_device gives)
    with pytest.raises(ValueError, match="contiguous"):
        svd._workspace(torch.empty(512, dtype=torch.uint8)[::2], -1)
    whole = torch.empty(64, dtype=torch.float32)
    assert svd._workspace(whole, -1) == (whole.data_ptr(), 256)


@pytest.mark.gpu
def test_tree_attention_refuses_a_bad_workspace(svd):
    c = svd.kv_cache(4, 2, 16, 64)
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    tab = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    ctx = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = svd.tree_attention_workspace(1, 2, 4, c, tab).numel()
    with pytest.raises(ValueError, match="workspace must be on"):
        svd.tree_attention(q, c, tab, ctx, workspace=torch.empty(n, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        svd.tree_attention(q, c, tab, ctx,
                           workspace=torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(svd.SvdError) as e:
        svd.tree_attention(q, c, tab, ctx,
                           workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == svd.SVD_EWORKSPACE
