"""GPU test that the scan's backward is linear in the gradients that it is given, whatever their
size: dy and dfinal_state times 2^-80 give every fp32 gradient times 2^-80.

A power of two changes no rounding, so what differs is only what falls below fp32's smallest normal
number: terms 2^-46 of the inputs' size and less, over at most 2^13 of them, and the bound that a
carried product is held to, whose rest is 2^-29 of it.  2^-20 of the output's norm is far above both
and far below what a lost product changes."""
import pytest
import torch

from test_gpu_c_scan_bwd import BF16, F32, _inputs, _run, _seq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,N,dtype,kind", [(64, 128, BF16, None), (64, 64, BF16, "random"), (16, 16, F32, None)])
def test_small_gradients(P, N, dtype, kind):
    L = 1300  # more than one range of chunks that share a carried product
    i = _inputs(1, L, 4, 2, P, N, dtype, True, seed=37, A=torch.tensor([-0.02, -0.1, -0.5, -2.0]))
    i["seq"] = _seq(1, L, kind, 5)
    want = _run(i)
    small = dict(i, dy=i["dy"] * 2.0 ** -80, dhT=i["dhT"] * 2.0 ** -80)
    got = _run(small)
    torch.cuda.synchronize()
    for k, name in ((1, "ddt"), (2, "dA"), (5, "dh0")):
        a, b = got[k].cpu().double() * 2.0 ** 80, want[k].cpu().double()
        if name == "ddt":  # head by head, each with its own decay
            a, b = a[0].t(), b[0].t()
        elif name == "dh0":
            a, b = a.reshape(4, -1), b.reshape(4, -1)
        else:
            a, b = a[:, None], b[:, None]
        off = (a - b).norm(dim=1) / b.norm(dim=1)
        assert float(off.max()) <= 2.0 ** -20, (name, off.tolist())
