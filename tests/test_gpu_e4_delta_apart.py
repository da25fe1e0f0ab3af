"""GPU test that forward a value that is not finite reaches its own sequence only, in the chunks that
other sequences share with it too."""
import pytest
import torch

from test_gpu_e_delta import BF16, F32, _cuda, _inputs

pytestmark = pytest.mark.gpu
ENDS = (70, 76, 90, 150, 190)  # sequences 0 .. 5; the second and third lie within chunks


def _forward(s, seq):
    import ssm_sequence_models_amd as ssm
    c = {n: _cuda(t) for n, t in s.items()}
    y, final = ssm.delta_scan_fwd(c["q"], c["k"], c["v"], c["beta"], gate=c["gate"], scale=1.0,
                                  initial_state=c["h0"], seq_idx=_cuda(seq))
    torch.cuda.synchronize()
    return y, final


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("P,N", [(32, 64), (80, 128), (20, 132), (36, 44)])
def test_other_sequences_do_not_see_it(P, N, bad, dtype):
    B, L, H = 2, 260, 2
    s = _inputs(B, L, H, 1, P, N, dtype, seed=33)
    seq = torch.zeros(B, L, dtype=torch.int32)
    for e in ENDS:
        seq[:, e:] += 1
    clean = _forward(s, seq)
    for name in ("q", "k", "v", "beta", "gate", "h0"):
        for at in ((10, 69, 72, 80, 149, 151, 230) if name != "h0" else (0,)):
            t = dict(s, **{name: s[name].clone()})
            if name == "h0":
                t["h0"][0, :, 3, 5] = bad
            else:
                t[name].view(B, L, -1)[0, at, :] = bad
            y, final = _forward(t, seq)
            other = seq != seq[0, at]
            other[1] = True
            assert torch.equal(y[other], clean[0][other]), (name, at)
            assert torch.equal(final[1], clean[1][1]), (name, at)
            assert at >= ENDS[-1] or torch.equal(final[0], clean[1][0]), (name, at)
            if name != "q" and not (name == "gate" and bad < 0):  # and its own tokens from there on do
                assert torch.isnan(y[0, at:][~other[0, at:]]).any(), (name, at)
