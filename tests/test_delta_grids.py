"""Sizes whose launches would have 2^32 threads or more are refused by the delta rule's calls over rows, and
have no workspace size; on the CPU."""
import pytest
import torch

from test_delta_refusals import _bwd, _fwd, lib  # noqa: F401

F32, BF16 = 0, 1


@pytest.mark.parametrize("what,dtype,most,call", [
    ("a block a chunk and head", F32, dict(b=1 << 16, L=97, H=128, P=16, G=128, N=16), _fwd),
    ("a block a chunk and two heads", F32, dict(b=1 << 16, L=225, H=128, P=4, G=64, N=4), _fwd),
    ("a block a head", F32, dict(b=1 << 18, L=32, H=52, P=16, G=52, N=16), _fwd),
    ("a block a head and 64 channels", BF16, dict(b=1 << 12, L=1, H=32, P=103 * 64, G=1, N=16), _fwd),
    ("a block a chunk and key head", F32, dict(b=1 << 18, L=32, H=32, P=16, G=32, N=16), _bwd)])
def test_more_threads_than_a_launch_has(lib, what, dtype, most, call):  # noqa: F811
    import ssm_sequence_models_amd as s
    size = s.delta_scan_fwd_workspace_size if call is _fwd else s.delta_scan_bwd_workspace_size
    args = lambda d: (d["b"], d["L"], d["H"], d["P"], d["G"], d["N"], torch.float32 if dtype == F32 else torch.bfloat16)  # noqa: E731
    rows = {f"{n}_row": 1 << 24 for n in ("q", "k", "v", "y", "dy", "dq", "dk", "dv")}
    assert size(*args(most)) == 0
    assert call(lib, **most, **rows, dtype=dtype, wsb=1 << 62) == 2 and lib.ssm_last_error()
    less = dict(most, b=most["b"] - (most["b"] >> 5))  # just below, there is a size, and too small a workspace is seen
    assert size(*args(less)) > 0
    assert call(lib, **less, **rows, dtype=dtype, wsb=1) == 4


def test_states_without_tokens(lib):  # noqa: F811
    """Nothing to do but the states' copy, whose number of values must be one."""
    from test_delta_refusals import P as p
    assert _fwd(lib, b=1 << 30, L=0, H=1 << 30, P=65536, G=1, N=256, hT=p, h0=p) == 2
