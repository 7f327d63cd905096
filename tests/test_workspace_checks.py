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


def verifications(svd, dev):
    """(call, bytes it needs) for each verification with a workspace, one prefix of 2 drafts."""
    i32 = dict(dtype=torch.int32, device=dev)
    p, q = torch.zeros(1, 2, 4, 32, device=dev), torch.zeros(1, 2, 3, 32, device=dev)
    d = torch.zeros(1, 2, 3, **i32)
    one, two = svd.workspace_bytes(1, 1, 3, 32), svd.workspace_bytes(1, 2, 3, 32)
    px = torch.arange(8, **i32).view(1, 2, 4)
    qx = torch.arange(6, **i32).view(1, 2, 3)
    rows = svd.svd_rows_workspace_bytes(1, 2, 3, 32, 8, 6)
    return [
        (lambda w: svd.select_and_verify(p, q, d, workspace=w), two),
        (lambda w: svd.verify(p[:, 0], q[:, 0], d[:, 0], workspace=w), one),
        (lambda w: svd.greedy_select_and_verify(p, d, workspace=w), two),
        (lambda w: svd.greedy_verify(p[:, 0], d[:, 0], workspace=w), one),
        (lambda w: svd.verify_window(p, q, d, workspace=w), two),
        (lambda w: svd.select_and_verify_rows(p.view(8, 32), px, q.view(6, 32), qx, d,
                                              workspace=w), rows),
    ]


def test_verifications_check_their_workspace(svd, monkeypatch):
    # the checks see the workspace before the library's call, which is kept out here
    seen = []
    monkeypatch.setattr(svd, "_check", lambda t, name, dev: seen.append((t, name)))
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda dev=None: type("S", (), {"cuda_stream": 0}))
    for name in svd.C_EXPORTS:
        if "verify" in name:
            monkeypatch.setattr(svd, name, lambda *a: svd.SVD_OK)
    for call, n in verifications(svd, "cpu"):
        w = torch.empty(n, dtype=torch.uint8)
        seen.clear()
        call(w)
        assert any(t is w and name == "workspace" for t, name in seen)


@pytest.mark.gpu
def test_verifications_refuse_a_bad_workspace(svd):
    for call, n in verifications(svd, "cuda:0"):
        with pytest.raises(ValueError, match="workspace must be on"):
            call(torch.empty(n, dtype=torch.uint8))
        with pytest.raises(ValueError, match="contiguous"):
            call(torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2])
        assert int(call(torch.empty(n, dtype=torch.uint8, device="cuda"))["accept_len"][0]) >= 0


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
