"""A norm that is the last step of a call on state pools is refused before the call moves them: the
binding's checks against the C entry point's own, on the CPU, and the pools after a refused
decode_step and conv_scan_fwd on the GPU."""
import ctypes
import itertools

import pytest
import torch

BF16 = torch.bfloat16
P = ctypes.c_void_p(256)


def test_limits_are_the_entry_points():
    import ssm_sequence_models_amd as ssm
    widths = ((64, 1), (16384, 1), (16385, 1), (16392, 1), (32768, 2), (32768, 1), (1 << 32, 1 << 32), (1 << 37, 1 << 30))
    for (C, g), eps, rows, row in itertools.product(
            widths, (1e-5, 0.0, -0.0, -1.0, float("nan"), float("inf"), -1e-60, 1e60), (1, 2), (-1, 0, 1)):
        out_row = C + row
        # an x that is not there is refused last: no call reaches a launch
        status = ssm._lib.ssm_norm_fwd(P, C, None, 0, None, None, P, out_row, 0 if row >= 0 or rows < 2 else rows, C, g,
                                       eps, 0, 0, 1, None)
        try:
            ssm._norm_limits(C, g, eps, rows, out_row)
            assert status == 0, (C, g, eps, rows, out_row)
        except ssm.SSMError as e:
            assert e.status == status, (C, g, eps, rows, out_row, e)
    with pytest.raises(TypeError):
        ssm._norm_limits(64, 2.0, 1e-5, 1, 64)


def _bits(t):
    return t.view(torch.int16 if t.dtype == BF16 else torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("H,how", [(4, dict(eps=-1.0)), (4, dict(eps=float("nan"))), (264, dict()),
                                   (4, dict(ngroups=2.0)), (4, dict(out="rows"))], ids=str)
def test_refused_norm_leaves_the_pools(H, how):
    import ssm_sequence_models_amd as ssm
    P_, N, G, K, n = 64, 16, 1, 4, 5
    C = H * P_ + 2 * G * N
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    pool, spool = r(n, C, K).to(BF16), r(n, H, P_, N)
    keep, skeep = pool.clone(), spool.clone()
    w, b, dt, A = r(C, K), r(C), r(3, 1, H).abs(), -r(H).abs()
    norm = dict(how)
    if "out" in how:  # rows that overlap
        norm["out"] = torch.empty(3 * H * P_, dtype=BF16, device="cuda").as_strided((3, 1, H * P_), (8, 8, 1))
    with pytest.raises((ssm.SSMError, TypeError)):
        ssm.decode_step(r(3, C, 1).to(BF16), pool, w, b, dt, A, spool, H, P_, G, N, norm=norm)
    torch.cuda.synchronize()
    assert torch.equal(_bits(pool), _bits(keep)) and torch.equal(_bits(spool), _bits(skeep))
    conv, state = torch.full((3, C, K - 1), 7.0, dtype=BF16, device="cuda"), torch.full((3, H, P_, N), 7.0, device="cuda")
    with pytest.raises((ssm.SSMError, TypeError)):
        ssm.conv_scan_fwd(r(3, 1, C).to(BF16), w, b, dt, A, H, P_, G, N, conv_final_state=conv, final_state=state,
                          norm=norm)
    torch.cuda.synchronize()
    assert (conv == 7.0).all() and (state == 7.0).all()
