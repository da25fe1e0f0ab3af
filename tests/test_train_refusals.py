"""Refusals of the training operators, on the CPU: status codes of the C entry points for
arguments that fail their host-side checks (no call reaches a launch), and the 64-bit plain
forms against differences."""
import ctypes

import pytest
import torch

from train_ref import norm64


@pytest.fixture(scope="module")
def lib():
    import ssm_sequence_models_amd as s
    return s._lib


P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(257)
F = ctypes.c_float


def _norm_fwd(lib, x=P, x_row=64, z=None, z_row=64, w=P, b=None, out=P, out_row=64, rows=2, C=64,
              g=1, eps=1e-5, kind=0, after=0, dtype=1):
    return lib.ssm_norm_fwd(x, x_row, z, z_row, w, b, out, out_row, rows, C, g, F(eps), kind, after,
                            dtype, None)


def _norm_bwd(lib, x=P, x_row=64, z=None, z_row=64, d=P, d_row=64, w=P, b=None, dx=P, dx_row=64,
              dz=None, dz_row=64, dw=P, db=None, ws=P, wsb=1 << 30, rows=2, C=64, g=1, eps=1e-5,
              kind=0, after=0, dtype=1):
    return lib.ssm_norm_bwd(x, x_row, z, z_row, d, d_row, w, b, dx, dx_row, dz, dz_row, dw, db, ws,
                            wsb, rows, C, g, F(eps), kind, after, dtype, None)


@pytest.mark.parametrize("call", [_norm_fwd, _norm_bwd])
def test_norm_refusals(lib, call):
    for status, how in ((1, dict(dtype=7)), (1, dict(kind=2)), (1, dict(kind=-1)), (1, dict(rows=-1)),
                        (1, dict(C=0)), (1, dict(g=0)), (1, dict(g=3)), (1, dict(eps=-1.0)),
                        (1, dict(eps=float("nan"))), (2, dict(C=16392)), (1, dict(x=None)),
                        (3, dict(x=ODD)), (3, dict(w=ODD)), (3, dict(z=ODD)), (1, dict(x_row=-64)),
                        (1, dict(z=P, z_row=-1))):
        assert call(lib, **how) == status, how
        assert lib.ssm_last_error()
    # a group of 16384 is the largest; rows = 0 is a no-op that needs no pointers
    if call is _norm_fwd:
        assert call(lib, out=None) == 1
        assert call(lib, out_row=63) == 1
        assert call(lib, x=None, out=None, rows=0) == 0
    else:
        assert call(lib, dx=None) == 1
        assert call(lib, d=None) == 1
        assert call(lib, dx_row=63) == 1
        assert call(lib, z=P, dz=P, dz_row=63) == 1
        assert call(lib, ws=None) == 4
        assert call(lib, wsb=16) == 4
        assert call(lib, x=None, d=None, dx=None, dw=None, rows=0) == 0


def test_norm_workspace_size(lib):
    import ssm_sequence_models_amd as s
    # 1024 blocks over the groups, of at least four rows a team; four teams a block up to 1024
    # channels a group, one above
    assert s.norm_bwd_workspace_size(32768, 4096, 1) == 2 * 1024 * 4096 * 4
    assert s.norm_bwd_workspace_size(32768, 4096, 8) == 2 * 128 * 4096 * 4
    assert s.norm_bwd_workspace_size(10, 4096, 1) == 2 * 3 * 4096 * 4
    assert s.norm_bwd_workspace_size(10, 64, 1) == 2 * 1 * 64 * 4
    assert s.norm_bwd_workspace_size(33, 1024, 1) == 2 * 3 * 1024 * 4
    assert s.norm_bwd_workspace_size(0, 64, 1) == 0


def test_norm_binding_refusals():
    import ssm_sequence_models_amd as ssm
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        ssm.norm_fwd(x)
    with pytest.raises(ValueError, match="kind"):
        ssm.norm_fwd(x, kind="batch")
    with pytest.raises(ValueError, match="ngroups"):
        ssm.norm_fwd(x, ngroups=3)
    # the row view: one stride for all leading dimensions, consecutive channels
    assert ssm._rows(torch.zeros(3, 4, 8), "x", 8) == (12, 8)
    assert ssm._rows(torch.zeros(3, 4, 20)[:, :, 2:10], "x", 8) == (12, 20)
    assert ssm._rows(torch.zeros(6, 4, 8)[::2, :1], "x", 8) == (3, 64)
    assert ssm._rows(torch.zeros(1, 8).expand(5, 8), "x", 8) == (5, 0)
    assert ssm._rows(torch.zeros(0, 8), "x", 8)[0] == 0
    assert ssm._rows(torch.zeros(8), "x", 8) == (1, 8)
    with pytest.raises(ValueError, match="one stride"):
        ssm._rows(torch.zeros(3, 5, 8)[:, :4], "x", 8)
    with pytest.raises(ValueError, match="consecutive"):
        ssm._rows(torch.zeros(8, 4).t(), "x", 8)
    with pytest.raises(ValueError, match="channels"):
        ssm._rows(torch.zeros(4, 9), "x", 8)


def test_norm64_against_differences():
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    for kind in ("rms", "layer"):
        for after in (False, True):
            a = [rnd(3, 12), 1 + 0.2 * rnd(12), rnd(12), rnd(3, 12)]
            d = rnd(3, 12)
            r = norm64(*a, 1e-4, kind, 3, after, d)
            for i, name in enumerate(("dx", "dw", "db", "dz")):
                v = rnd(*a[i].shape)
                f = []
                for e in (1e-5, -1e-5):
                    q = list(a)
                    q[i] = a[i] + e * v
                    f.append(float((norm64(*q, 1e-4, kind, 3, after)["out"] * d).sum()))
                assert abs((f[0] - f[1]) / 2e-5 - float((r[name] * v).sum())) < 1e-6


def _gfwd(lib, x=P, xr=64, g=P, gr=64, h0=None, f=None, seq=None, y=P, yr=64, B=2, L=4, C=64, form=1,
          dtype=1, ws=P, wsb=1 << 30):
    return lib.ssm_gated_scan_fwd(x, xr, g, gr, h0, f, seq, y, yr, B, L, C, form, dtype, ws, wsb, None)


def _gbwd(lib, x=P, xr=64, g=P, gr=64, d=P, dr=64, h0=None, f=None, seq=None, y=P, yr=64, dg=P,
          dgr=64, dh0=None, B=2, L=4, C=64, form=1, dtype=1, ws=P, wsb=1 << 30):
    return lib.ssm_gated_scan_bwd(x, xr, g, gr, d, dr, h0, f, seq, y, yr, dg, dgr, dh0, B, L, C, form,
                                  dtype, ws, wsb, None)


def _gstep(lib, x=P, xr=64, g=P, gr=64, state=P, idx=None, y=P, yr=64, B=2, L=4, C=64, n=4, form=1,
           dtype=1):
    return lib.ssm_gated_scan_step(x, xr, g, gr, state, idx, y, yr, B, L, C, n, form, dtype, None)


@pytest.mark.parametrize("call", [_gfwd, _gbwd, _gstep])
def test_gated_scan_refusals(lib, call):
    for status, how in ((1, dict(dtype=2)), (1, dict(form=2)), (1, dict(form=-1)), (1, dict(B=-1)),
                        (1, dict(L=-1)), (1, dict(C=0)), (2, dict(C=1 << 31, xr=1 << 31, yr=1 << 31)),
                        (2, dict(B=1 << 31)), (1, dict(x=None)), (1, dict(g=None)), (1, dict(y=None)),
                        (3, dict(x=ODD)), (3, dict(y=ODD)), (1, dict(xr=-1)), (1, dict(gr=-1)),
                        (1, dict(yr=63))):
        assert call(lib, **how) == status, how
        assert lib.ssm_last_error()
    assert call(lib, B=0, x=None, g=None, y=None) == 0


def test_gated_scan_workspace(lib):
    import ssm_sequence_models_amd as s
    # 256 blocks already (forward 128, or eight 128-token tiles): no cut; else segments of at least
    # four tiles, three floats a segment and channel; backward two floats a tile and channel more
    assert s.gated_scan_fwd_workspace_size(4, 8192, 4096) == 0
    assert s.gated_scan_bwd_workspace_size(4, 8192, 4096) == 4 * 64 * 2 * 4096 * 4
    assert s.gated_scan_fwd_workspace_size(2, 8192, 4096) == 0
    assert s.gated_scan_fwd_workspace_size(1, 1025, 64) == 2 * 3 * 64 * 4
    assert s.gated_scan_fwd_workspace_size(1, 1024, 64) == 0
    assert s.gated_scan_bwd_workspace_size(1, 1023, 64) == (2 * 3 + 8 * 2) * 64 * 4
    assert s.gated_scan_fwd_workspace_size(0, 5, 5) == 0
    assert _gfwd(lib, B=1, L=2000, ws=None) == 4
    assert _gfwd(lib, B=1, L=2000, wsb=16) == 4
    assert _gbwd(lib, ws=None) == 4
    assert _gbwd(lib, wsb=16) == 4
    assert _gbwd(lib, f=P, dh0=P) == 1
    assert _gstep(lib, n=0) == 1
    assert _gstep(lib, state=None) == 1


def test_scan_bwd_widest_rows(lib):
    """Rows beyond the matrix-core kernels' 32-bit offsets are laid out for the general ones (the
    same for both types), the widest row within them is not."""
    import ssm_sequence_models_amd as s
    size = lambda H, dt: s.scan_bwd_workspace_size(1, 128, H, 64, 1, 64, dt)  # noqa: E731
    assert size((1 << 17) + 1, torch.bfloat16) == size((1 << 17) + 1, torch.float32)
    assert size(1 << 17, torch.bfloat16) != size(1 << 17, torch.float32)


def test_gated_scan_binding_refusals():
    import ssm_sequence_models_amd as ssm
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        ssm.gated_scan_fwd(x, x)
    with pytest.raises(ValueError, match="form"):
        ssm.gated_scan_bwd(x, x, x, form="tanh")
    with pytest.raises(ValueError, match="batch, tokens, channels"):
        ssm.gated_scan_step(x[0], x[0], x[0])


def _sbwd(lib, x=P, dt=P, A=P, B=P, C=P, dy=P, h0=None, f=None, seq=None, dx=P, ddt=P, dA=P, dB=P,
          dC=P, dh0=None, b=2, L=100, H=4, hd=64, G=1, N=128, dtype=1, ws=P, wsb=1 << 40):
    return lib.ssm_scan_bwd(x, dt, A, B, C, dy, h0, f, seq, dx, ddt, dA, dB, dC, dh0, b, L, H, hd, G, N,
                            dtype, ws, wsb, None)


def test_scan_bwd_refusals(lib):
    for status, how in ((1, dict(dtype=5)), (1, dict(b=-1)), (1, dict(L=-1)), (1, dict(H=0)), (1, dict(G=3)),
                        (2, dict(N=6)), (2, dict(hd=512, N=128)), (2, dict(b=1 << 31)), (2, dict(L=1 << 40)),
                        (2, dict(b=1 << 25, L=1 << 25)), (1, dict(x=None)), (1, dict(dy=None)),
                        (1, dict(dA=None)), (1, dict(dx=None)), (1, dict(ddt=None)), (1, dict(dB=None)),
                        (3, dict(x=ODD)), (3, dict(h0=ctypes.c_void_p(264))), (1, dict(f=P, dh0=P)),
                        (4, dict(ws=None)), (4, dict(wsb=1000)), (4, dict(ws=ctypes.c_void_p(128)))):
        assert _sbwd(lib, **how) == status, how
        assert lib.ssm_last_error()


def test_scan_bwd_workspace(lib):
    import ssm_sequence_models_amd as s
    for dims in ((1, 64, 1, 4, 1, 4), (4, 8192, 64, 64, 1, 128), (1, 131072, 48, 64, 1, 128)):
        assert s.scan_bwd_workspace_size(*dims) > 0
    assert s.scan_bwd_workspace_size(0, 64, 1, 4, 1, 4) == 0
    assert s.scan_bwd_workspace_size(1, 64, 3, 4, 2, 4) == 0
    assert s.scan_bwd_workspace_size(1, 64, 1, 4, 1, 6) == 0


def test_scan_bwd_binding_refusals():
    import ssm_sequence_models_amd as ssm
    x, dt, A, B = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2), torch.zeros(2), torch.zeros(1, 4, 1, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        ssm.scan_bwd(x, dt, A, B, B, x)


def test_gated64_and_scan64_against_torch():
    """The plain forms' gradients against torch's differentiation of the plain forward."""
    from train_ref import gated64, scan_bwd64, scan_loss64
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    seq = torch.tensor([[0, 0, 1, 1, 1, 0, 0, 2, 2, 2, 2, 2]], dtype=torch.int32)
    i = dict(x=r(1, 12, 4, 3), dt=r(1, 12, 4).abs(), A=-r(4).abs(), Bm=r(1, 12, 2, 4), Cm=r(1, 12, 2, 4),
             dy=r(1, 12, 4, 3), h0=r(1, 4, 3, 4), dhT=r(1, 4, 3, 4), seq=seq)
    ref = scan_bwd64(**i)
    leaf = {k: v.clone().requires_grad_() if k not in ("dy", "dhT", "seq") else v for k, v in i.items()}
    scan_loss64(**leaf).backward()
    for name, k in (("dx", "x"), ("ddt", "dt"), ("dA", "A"), ("dB", "Bm"), ("dC", "Cm"), ("dh0", "h0")):
        assert torch.allclose(leaf[k].grad, ref[name], rtol=1e-10, atol=1e-12), name
    for form in ("log", "sigmoid"):
        x, gate, dy, h0, dhT = r(1, 12, 3), r(1, 12, 3) * 0.5, r(1, 12, 3), r(1, 3), r(1, 3)
        ref = gated64(x, gate, form, h0, seq, dy, dhT)
        xs, gs, hs = (v.clone().requires_grad_() for v in (x, gate, h0))
        h, loss = hs, 0.0
        for t in range(12):
            a = torch.exp(gs[:, t]) if form == "log" else torch.sigmoid(gs[:, t])
            u = xs[:, t] * (1.0 if form == "log" else 1 - a)
            start = t > 0 and int(seq[0, t]) != int(seq[0, t - 1])
            h = u if start else a * h + u
            loss = loss + (h * dy[:, t]).sum()
        (loss + (h * dhT).sum()).backward()
        for name, v in (("dx", xs), ("dgate", gs), ("dh0", hs)):
            assert torch.allclose(v.grad, ref[name], rtol=1e-10, atol=1e-12), (form, name)
