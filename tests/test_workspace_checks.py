"""A workspace that the caller passes is as many bytes as the call may write, on the call's device."""
import pytest
import torch


def test_workspace():
    import ssm_sequence_models_amd as ssm
    cpu = torch.device("cpu")
    assert ssm._workspace(None, 0, cpu) == (None, 0)
    ws = torch.empty(1024, dtype=torch.float32)
    assert ssm._workspace(ws, 4096, cpu) == (ws, 4096)
    for bad in (ws[1:], torch.empty(1, dtype=torch.uint8).expand(4096), torch.empty(8192, dtype=torch.uint8)[::2],
                torch.empty(4096, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            ssm._workspace(bad, 4096, cpu)


def test_sizes_that_the_calls_refuse_need_nothing():
    """Sizes whose products leave 64 bits (a batch expanded to 2^62, say) are refused by the calls; the
    size queries that come first answer 0 for them."""
    import ssm_sequence_models_amd as ssm
    big = 1 << 62
    for B, L, C in ((big, 1, 256), (1 << 32, 1, 1 << 38), (1, big, 1), (1, 1, big), (1 << 31, 1, 1)):
        assert ssm.gated_scan_fwd_workspace_size(B, L, C) == 0
        assert ssm.gated_scan_bwd_workspace_size(B, L, C) == 0
    for B, L, H in ((big, 1, 4), (1 << 40, 1 << 40, 4), (1, 1, 1 << 60), (1, big, 1), (1 << 30, 1 << 30, 64)):
        for dtype in (torch.bfloat16, torch.float32):
            assert ssm.scan_bwd_workspace_size(B, L, H, 64, 1, 128, dtype) == 0
    assert ssm.norm_bwd_workspace_size(4, 1 << 60) == 0
    # the largest that the calls take
    assert ssm.gated_scan_bwd_workspace_size(1 << 20, 1 << 10, 1 << 10) > 1 << 33
    assert ssm.scan_bwd_workspace_size(1 << 10, 1 << 20, 64, 64, 1, 128) > 1 << 40
