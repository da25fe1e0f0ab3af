"""GPU test that no fp32 operand of the scan backward's products loses bits: sums that cancel down to
the last bit of a 21-bit number.  A = 0 and dt = 1, so every decay is 1, and all products are whole
numbers below 2^24: the outputs are exact."""
import pytest
import torch

from test_gpu_c_scan_bwd import BF16, F32, _run

pytestmark = pytest.mark.gpu
PARTS = (1024.0, 32.0, 1.0)  # the squares' sum, 2^20 + 2^10 + 1, needs three bf16 numbers
LESS = (1024.0, 32.0, 0.0)
WHERE = [(0, 1, 2), (5, 6, 9), (5, 20, 70), (100, 126, 127), (15, 16, 112), (33, 64, 65)]


def _zeros(L, P, N, dtype):
    z = lambda *s: torch.zeros(*s, dtype=dtype)  # noqa: E731
    return dict(x=z(1, L, 1, P), dt=torch.ones(1, L, 1), A=torch.zeros(1), Bm=z(1, L, 1, N), Cm=z(1, L, 1, N),
                dy=z(1, L, 1, P), h0=None, dhT=None, seq=None)


def _set(t, token, values, last):
    t[0, token, 0, :2] = torch.tensor(values[:2], dtype=t.dtype)
    t[0, token, 0, last] = values[2]


@pytest.mark.parametrize("P,N,dtype", [(64, 128, BF16), (64, 64, BF16), (32, 64, BF16), (16, 16, F32)])
def test_last_bit(P, N, dtype):
    L = 128
    for a, b, c in WHERE:
        # dx of a: (C_b.B_a) dy_b + (C_c.B_a) dy_c
        i = _zeros(L, P, N, dtype)
        _set(i["Bm"], a, PARTS, N - 1)
        _set(i["Cm"], b, PARTS, N - 1)
        _set(i["Cm"], c, LESS, N - 1)
        i["dy"][0, b], i["dy"][0, c] = 1.0, -1.0
        dx = _run(i)[0].float().cpu()
        assert (dx[0, a] == 1.0).all(), ("dx", a, b, c)
        # dB of a: (dy_b.x_a) C_b + (dy_c.x_a) C_c
        i = _zeros(L, P, N, dtype)
        _set(i["x"], a, PARTS, P - 1)
        _set(i["dy"], b, PARTS, P - 1)
        _set(i["dy"], c, LESS, P - 1)
        i["Cm"][0, b], i["Cm"][0, c] = 1.0, -1.0
        dB = _run(i)[3].float().cpu()
        assert (dB[0, a] == 1.0).all(), ("dB", a, b, c)
        # dC of c: (dy_c.x_a) B_a + (dy_c.x_b) B_b
        i = _zeros(L, P, N, dtype)
        _set(i["dy"], c, PARTS, P - 1)
        _set(i["x"], a, PARTS, P - 1)
        _set(i["x"], b, LESS, P - 1)
        i["Bm"][0, a], i["Bm"][0, b] = 1.0, -1.0
        dC = _run(i)[4].float().cpu()
        assert (dC[0, c] == 1.0).all(), ("dC", a, b, c)


@pytest.mark.parametrize("P,N,dtype", [(64, 128, BF16), (64, 64, BF16), (32, 64, BF16), (16, 16, F32)])
def test_last_bit_of_states(P, N, dtype):
    """The final state's gradient into dx and dB, the initial state into dC."""
    L, whole = 200, sum(v * v for v in PARTS)
    for t in (0, 17, 127, 128, 199):
        i = _zeros(L, P, N, dtype)
        i["dhT"] = torch.zeros(1, 1, P, N)
        i["dhT"][..., 0], i["dhT"][..., N - 1] = whole, whole - 1.0
        i["Bm"][0, t, 0, 0], i["Bm"][0, t, 0, N - 1] = 1.0, -1.0
        assert (_run(i)[0][0, t].float() == 1.0).all(), ("dx", t)
        i = _zeros(L, P, N, dtype)
        i["dhT"], i["h0"] = torch.zeros(1, 1, P, N), torch.zeros(1, 1, P, N)
        for k in ("dhT", "h0"):
            i[k][:, :, 0], i[k][:, :, P - 1] = whole, whole - 1.0
        for k in ("x", "dy"):
            i[k][0, t, 0, 0], i[k][0, t, 0, P - 1] = 1.0, -1.0
        got = _run(i)
        assert (got[3][0, t].float() == 1.0).all() and (got[4][0, t].float() == 1.0).all(), ("dB, dC", t)
