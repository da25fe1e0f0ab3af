"""The gated delta rule and the queries' and keys' norm on tensors of a device that is not the current one:
each is launched on that device's stream, with a workspace there.  On the CPU, with the library and
the device switch replaced by recorders."""
import contextlib

import pytest
import torch


class _Library:
    def __init__(self, calls, where):
        self.calls, self.where = calls, where

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_size"):
                return 64
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


def test_calls_on_the_tensors_stream(recorded):
    ssm, calls = recorded
    B, L, H, G, P, N, dev = 2, 3, 4, 2, 8, 16, torch.device("cpu")
    z = torch.zeros
    q, k, v, beta = z(B, L, G, N), z(B, L, G, N), z(B, L, H, P), z(B, L, H)
    ssm.delta_scan_fwd(q, k, v, beta)
    ssm.delta_scan_bwd(q, k, v, beta, z(B, L, H, P))
    ssm.delta_scan_step(q, k, v, beta, z(5, H, P, N))
    ssm.qk_norm_fwd(q, k)
    ssm.qk_norm_bwd(q, k, q, k, q_weight=z(N))
    assert [c[0] for c in calls] == ["ssm_delta_scan_fwd", "ssm_delta_scan_bwd", "ssm_delta_scan_step",
                                     "ssm_qk_norm_fwd", "ssm_qk_norm_bwd"]
    assert all(c[1] == dev and c[2] == ("stream of", dev) for c in calls), calls
