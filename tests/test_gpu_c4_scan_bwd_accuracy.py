"""GPU accuracy of the scan backward's fp32 outputs: ddt and dA by norms (scan_bwd_sharp.py), over
several ranges of chunks that share a carried product, packed and not, decays from slow to fast; and
on the CPU that the bounds see what is wrong."""
import math

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
    """What is 0, one percent off, or formed from operands rounded to 8 bits (as if fp32 states had gone
    through bf16: here dy and x, each element up to 2^-9 off) is over the bound."""
    i, heads = _case(*case)
    ref = ddt_dA64(i, heads)
    r = torch.Generator().manual_seed(1)
    off = {k: i[k].double() * (1 + 2.0 ** -9 * (2 * torch.rand(i[k].shape, generator=r) - 1)) for k in ("x", "dy")}
    rough = ddt_dA64(dict(i, **off), heads)
    B, L, H = i["dt"].shape

    def whole(values):
        ddt, dA = torch.zeros(B, L, H, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
        for h, (d, s, _) in zip(heads, values):
            ddt[:, :, h], dA[h] = d, s
        return ddt, dA
    ddt, dA = whole(ref)
    bound, bound_dA = tol(case[4], case[5]), tol_dA(case[4], case[5], carried(i))
    for h, one in zip(heads, ref):
        assert max(errors(ddt, dA, [one], [h])) == 0.0
        for k in (0.0, 0.99):
            e = errors(k * ddt, k * dA, [one], [h])
            assert e[0] > 10 * bound and e[1] > 2 * bound_dA, (h, k, e)
    e = [errors(*whole(rough), [one], [h]) for h, one in zip(heads, ref)]
    assert min(x[0] for x in e) > 10 * bound, e
    # one random error may cancel in one head's sum: the heads together
    assert math.sqrt(sum(x[1] ** 2 for x in e) / len(e)) > bound_dA, e
