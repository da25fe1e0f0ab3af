"""GPU accuracy of the scan backward's fp32 outputs: ddt and dA by norms (scan_bwd_sharp.py), over
several ranges of chunks that share a carried product, packed and not, decays from slow to fast; and
on the CPU that the bounds see what is wrong."""
import pytest
import torch

from scan_bwd_sharp import carried, ddt_dA64, errors, tol, tol_dA
from test_gpu_c_scan_bwd import BF16, F32, _inputs, _run, _seq

A4 = torch.tensor([-0.03, -0.4, -3.0, -16.0])
CASES = [  # B, L, H, G, P, N, dtype, packed
    (1, 1300, 4, 2, 64, 128, BF16, None), (1, 1300, 4, 1, 64, 128, BF16, "random"),
    (1, 2500, 4, 2, 64, 64, BF16, None), (1, 1300, 4, 4, 64, 64, BF16, "edges"),
    (2, 1100, 48, 1, 64, 64, BF16, None), (1, 1300, 96, 2, 64, 128, BF16, "random"),
    (1, 129, 4, 1, 64, 128, BF16, None), (1, 64, 4, 1, 64, 64, BF16, None),
    (1, 700, 4, 2, 32, 64, BF16, "random"), (1, 700, 4, 1, 16, 16, F32, None), (1, 300, 4, 1, 64, 128, F32, None),
]


def _case(B, L, H, G, P, N, dtype, kind):
    i = _inputs(B, L, H, G, P, N, dtype, True, seed=L + H + N, A=A4.repeat(H // 4))
    i["seq"] = _seq(B, L, kind, 7)
    heads = range(4) if H == 4 else (0, 1, H // 2 + 2, H - 1)
    return i, heads


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_ddt_and_dA(case):
    i, heads = _case(*case)
    got = _run(i)
    torch.cuda.synchronize()
    e = errors(got[1], got[2], ddt_dA64(i, heads), heads)
    assert e[0] <= tol(case[4], case[5]) and e[1] <= tol_dA(case[4], case[5], carried(i)), e


@pytest.mark.parametrize("case", [CASES[1], CASES[3], CASES[6], CASES[7], CASES[9]], ids=str)
def test_bounds_reject(case):
    """What is 0 or one percent off is far over the bound, for every head; what is formed from initial
    states rounded to bf16 (which only the row's ends see) over it."""
    i, heads = _case(*case)
    ref = ddt_dA64(i, heads)
    B, L, H = i["dt"].shape
    ddt, dA = torch.zeros(B, L, H, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
    for h, (d, s, _) in zip(heads, ref):
        ddt[:, :, h], dA[h] = d, s
    bound = tol_dA(case[4], case[5], carried(i))
    for h, r in zip(heads, ref):
        assert max(errors(ddt, dA, [r], [h])) == 0.0
        for k in (0.0, 0.99):
            assert min(errors(k * ddt, k * dA, [r], [h])) > 10 * bound, (h, k)
    rough = dict(i, dhT=i["dhT"].to(BF16).float(), h0=i["h0"].to(BF16).float())
    off = errors(ddt, dA, ddt_dA64(rough, heads), heads)
    assert off[0] > 10 * tol(case[4], case[5]) and off[1] > bound, off
