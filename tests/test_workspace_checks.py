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
