"""GPU test of the gated delta rule with gates above 0, in rows uncut and cut into segments: what a
segment makes of the state before it may pass fp32's range where the states themselves do not."""
import math

import pytest
import torch

from delta_ref import check_delta, delta64
from test_gpu_e_delta import BF16, F32, STATE, _inputs, _run

pytestmark = pytest.mark.gpu
SHAPES = [(BF16, 1, 2100, 1, 64, 128), (BF16, 9, 2100, 30, 16, 16), (BF16, 1, 1100, 2, 24, 64), (F32, 1, 1100, 2, 40, 48),
          (BF16, 2, 1100, 1, 16, 200), (F32, 1, 900, 1, 32, 256)]


@pytest.mark.parametrize("dtype,B,L,H,P,N", SHAPES)
def test_growth_of_nothing(dtype, B, L, H, P, N):
    """A sequence of gates above 0 that writes nothing, and whose state is 0, between two others."""
    s = _inputs(B, L, H, 1, P, N, dtype, seed=L + P)
    seq = torch.zeros(B, L, dtype=torch.int32)
    seq[:, L // 5:] = 1
    seq[:, L - 150:] = 2
    zone = slice(L // 5, L - 150)
    s["gate"][:, zone] = 0.5
    s["beta"][:, zone] = 0.0
    s["dy"][:, zone] = 0.0
    got = _run(s, 1.0, seq)
    assert not got["y"][:, zone].any() and not got["dgate"][:, zone].any()
    few = {n: t[:1].contiguous() for n, t in s.items()}
    ref = delta64(few["q"], few["k"], few["v"], few["beta"], few["gate"], 1.0, few["h0"], seq[:1], few["dy"], few["dhT"])
    for n, t in got.items():
        check_delta(t[:1], ref, n, F32 if n in STATE else dtype, N + P + 256, -(-L // 32))


@pytest.mark.parametrize("dtype,B,L,H,P,N", SHAPES)
def test_growth_and_decay_of_a_state(dtype, B, L, H, P, N):
    """Columns that no key touches, up by 2^216 and down again, or the other way in the gradient: relative to
    the result an exponential (two roundings) and its product a chunk, and as many a segment."""
    s = _inputs(B, L, H, 1, P, N, dtype, seed=L + N)
    s["k"][..., 9:11], s["q"][..., 9:11] = 0.0, 0.0
    s["beta"][:, :500] = 0.0  # what tokens write would grow too
    s["dy"], s["h0"], s["dhT"] = torch.zeros_like(s["dy"]), torch.zeros(B, H, P, N), torch.zeros(B, H, P, N)
    s["gate"][:, :500] = 0.3
    s["gate"][:, 500:] = -120 * math.log(2) / (L - 500)
    s["h0"][..., 9], s["dhT"][..., 10] = 2.0 ** -120, 2.0 ** 10
    got = _run(s, 1.0, None)
    through = math.exp(float(s["gate"][0, :, 0].double().sum()))
    for n, at, start in (("final", 9, 2.0 ** -120), ("dh0", 10, 2.0 ** 10)):
        rel = float((got[n][..., at].double().cpu() / (start * through) - 1).abs().max())
        assert rel <= 4 * (L // 32 + 65) * 2.0 ** -24, (n, rel)
