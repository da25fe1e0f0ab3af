"""GPU tests of the gated recurrence with its final state in place of the initial one, where a
group of channels ends on an odd channel of its own, and of those widths in general."""
import pytest
import torch

from test_gpu_b_gated_scan import BF16, F32, _compare, _inputs, _seq
from train_ref import check_err, gated64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("C", [65, 129, 127, 1025])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_final_state_over_initial(C, dtype):
    """More rows of a few tokens than the GPU runs blocks at a time: the rows' blocks end at
    different times."""
    import ssm_sequence_models_amd as ssm
    for B, L in ((900, 3), (700, 9)) if C < 1000 else ((100, 3),):
        x, gate, dy, h0, dhT = _inputs(B, L, C, "sigmoid", dtype, True, seed=C + L)
        xg, gg = x.cuda(), gate.cuda()
        want, want_state = ssm.gated_scan_fwd(xg, gg, initial_state=h0.cuda())
        ref = gated64(x, gate, "sigmoid", h0)
        for _ in range(4):
            state = h0.cuda()
            y, final = ssm.gated_scan_fwd(xg, gg, initial_state=state, final_state=state)
            torch.cuda.synchronize()
            assert final is state and torch.equal(y, want) and torch.equal(state, want_state)
        check_err(y, ref, "y", dtype)
        check_err(state, ref, "final", F32)


@pytest.mark.parametrize("C", [65, 129, 193])
@pytest.mark.parametrize("form", ["log", "sigmoid"])
def test_odd_last_channel(C, form):
    """Whole and ragged tiles, cut and uncut rows, packed or not, where 64 divides C - 1."""
    for L, dtype, kind in ((300, BF16, "random"), (256, F32, None), (2600, F32, "tiles"), (3000, BF16, None)):
        x, gate, dy, h0, dhT = _inputs(2, L, C, form, dtype, True, seed=C + L)
        _compare(x, gate, dy, h0, dhT, form, _seq(2, L, kind, seed=L))
