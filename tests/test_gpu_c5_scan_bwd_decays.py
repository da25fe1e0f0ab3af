"""GPU test of the decay factors of the scan's backward: what a whole row's decays leave of the final
state's gradient."""
import pytest
import torch

from test_gpu_c_scan_bwd import BF16, F32, _inputs, _run


@pytest.mark.gpu
@pytest.mark.parametrize("P,N,dtype,L", [(64, 128, BF16, 128), (64, 64, BF16, 384), (16, 16, F32, 64), (16, 16, BF16, 192)])
def test_decay_through_chunks(P, N, dtype, L):
    """dy = 0: dinitial_state is dfinal_state times the decay of the whole row, e^-0.1 to e^-40.  A
    chunk's factor is off by the instruction's step (two half-steps), its rest (one) and their product
    (one), and by the product with the gradient (one)."""
    H = 16
    i = _inputs(1, L, H, 1, P, N, dtype, True, seed=1, A=-torch.logspace(-1, 1.6, H))
    i["dt"][:] = torch.rand(1, L, H, generator=torch.Generator().manual_seed(2)) * 2 / L
    i["dy"] = torch.zeros_like(i["dy"])
    got = _run(i)[5].cpu().double()
    want = i["dhT"].double() * torch.exp((i["dt"].double() * i["A"].double()).sum(1))[..., None, None]
    chunks = -(-L // (128 if P == 64 else 64))
    off = ((got - want).abs() / want.abs()).amax((0, 2, 3))
    assert float(off.max()) <= (5 * chunks + 1) * 2.0 ** -24, off.tolist()
