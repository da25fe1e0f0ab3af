"""decode_step and conv_scan_fwd with a norm, on tensors of a device that is not the current one: the
step and the norm that reads its output are launched on one stream, that device's.  On the CPU, with
the library and the device switch replaced by recorders."""
import contextlib

import pytest
import torch


class _Library:
    def __init__(self, calls, where):
        self.calls, self.where = calls, where

    def __getattr__(self, name):
        def call(*args):
            if not name.endswith("workspace_size"):
                self.calls.append((name, self.where[-1], args[-1]))
            return 0
        return call


@pytest.fixture
def recorded(monkeypatch):
    import ssm_sequence_models_amd as ssm
    calls, where = [], ["current"]

    @contextlib.contextmanager
    def on(device):
        where.append(device)
        yield
        where.pop()
    monkeypatch.setattr(ssm, "_need", lambda *a, **k: None)
    monkeypatch.setattr(ssm, "_on", on)
    monkeypatch.setattr(ssm, "_stream", lambda: ("stream of", where[-1]))
    monkeypatch.setattr(ssm, "_lib", _Library(calls, where))
    return ssm, calls


def test_step_and_norm_on_one_stream(recorded):
    ssm, calls = recorded
    H, P, N, G, K = 2, 4, 4, 1, 4
    C, dev = H * P + 2 * G * N, torch.device("cpu")
    z = torch.zeros
    ssm.decode_step(z(3, C, 1), z(5, C, K), z(C, K), z(C), z(3, 1, H), z(H), z(5, H, P, N), H, P, G, N,
                    norm=dict(z=z(3, 1, H * P)))
    ssm.conv_scan_fwd(z(3, 2, C), z(C, K), z(C), z(3, 2, H), z(H), H, P, G, N, norm=dict(z=z(3, 2, H * P)))
    assert [c[0] for c in calls] == ["ssm_decode_step", "ssm_norm_fwd", "ssm_conv_scan_fwd", "ssm_norm_fwd"]
    assert all(c[1] == dev and c[2] == ("stream of", dev) for c in calls), calls
