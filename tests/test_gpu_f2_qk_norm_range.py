"""GPU parity of ssm_qk_norm_fwd / _bwd for heads whose squares leave fp32's range, beside ordinary ones."""
import pytest
import torch

from delta_ref import check_qk, qk_norm64
from test_gpu_f_qk_norm import BF16, F32, _inputs, _run

pytestmark = pytest.mark.gpu
SIZES = [1.0, 1e15, 1e19, 1e25, 3e37, 1e-15, 1e-19, 1e-25, 1e-36, 1e-39]  # the last one is subnormal
SMALL = 1e-8  # of the gradients: those of the smallest heads stay finite


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["l2", "rms"])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30, 1e30])
@pytest.mark.parametrize("D,R,interleaved", [(64, 32, False), (128, 128, True), (80, 18, False), (7, 4, True), (256, 0, False)])
def test_any_finite_values(D, R, interleaved, eps, kind, dtype):
    s = _inputs(2, len(SIZES) + 1, 3, 2, D, R, dtype, seed=D)
    for t, f in enumerate(SIZES):
        # around their middle, so that none is past the type's range
        for n in ("q", "k"):
            s[n][:, t] = (s[n][:, t].double().clamp(-4, 4) * f).to(dtype)
    s["q"][0, 3, 1, D // 2:] = (torch.linspace(-1, 1, D - D // 2) * 1e-5).to(dtype)  # large and small in a head
    s["q"][:, -1], s["k"][:, -1] = 0.0, 0.0
    for n in ("dq", "dk"):
        s[n] = (s[n].double() * SMALL).to(dtype)
    q, k, dq, dk, dwq, dwk = _run(s, dict(kind=kind, eps=eps, interleaved=interleaved))
    for x, w, dy, out, dx, dw in ((s["q"], s["wq"], s["dq"], q, dq, dwq), (s["k"], s["wk"], s["dk"], k, dk, dwk)):
        ref = qk_norm64(x, w, eps, kind, s["freq"], s["pos"], interleaved, dy)
        check_qk(out, ref, "out", dtype, D)
        check_qk(dx, ref, "dx", dtype, D)
        check_qk(dw, ref, "dw", F32, D, x[..., 0].numel())
    assert not q[:, -1].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_unit_length(dtype):
    """A head times a power of 2 has the same bits."""
    s = _inputs(1, 8, 2, 2, 128, 64, dtype, seed=1)
    one = _run(s, dict(eps=0.0))
    for e in (100, -110):
        got = _run(dict(s, **{n: torch.ldexp(s[n].float(), torch.tensor(e)).to(dtype) for n in ("q", "k")}), dict(eps=0.0))
        assert torch.equal(got[0], one[0]) and torch.equal(got[1], one[1])


def test_not_finite_values_reach_their_head_only():
    s = _inputs(1, 4, 2, 2, 64, 32, F32, seed=2)
    one = _run(s, {})
    for bad in (float("inf"), float("nan")):
        t = dict(s, q=s["q"].clone())
        t["q"][0, 1, 1, 5] = bad
        got = _run(t, {})
        other = torch.ones(1, 4, 2, dtype=torch.bool)
        other[0, 1, 1] = False
        for a, b in ((got[0], one[0]), (got[2], one[2])):
            assert torch.equal(a[other], b[other])
        assert torch.isnan(got[0][0, 1, 1, 5]) and torch.equal(got[1], one[1])
