"""Plain 64-bit implementations of the training operators (norm, per-channel gated scan, the
scan's backward), written from their definitions row by row and token by token, on the CPU.
Each returns, beside a value, what its error bound needs: the sum of the magnitudes that the
value is made of."""
from __future__ import annotations

import torch

U = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def assert_bound(got, ref, bound, what):
    """|got - ref| <= bound element by element (all float64)."""
    g = got.detach().to("cpu").double()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert torch.isfinite(g).all(), f"{what}: non-finite values"
    over = (g - ref).abs() / bound.clamp_min(1e-300)
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 1.0, f"{what}: {int((over > 1).sum())} of {g.numel()} over the bound, worst {worst:.3g} times"


# ---------------------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------------------
def norm64(x, w, b, z, eps, kind, ngroups, after, dout=None):
    """dict of out and, with dout, dx, dz, dw, db; `*_mag`: the magnitudes behind each."""
    rows, C = x.shape
    m = C // ngroups
    x = x.double()
    w = torch.ones(C, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(C, dtype=torch.float64) if b is None else b.double()
    one = torch.ones_like(x)
    sg = one if z is None else torch.sigmoid(z.double())
    s = one if z is None else z.double() * sg
    ds = one if z is None else sg * (1 + z.double() * (1 - sg))
    before = z is not None and not after
    after = z is not None and after
    u = (x * s if before else x).view(rows, ngroups, m)
    mean = u.mean(-1, keepdim=True) if kind == "layer" else 0.0
    rstd = 1.0 / ((u - mean).square().mean(-1, keepdim=True) + eps).sqrt()
    n3 = (u - mean) * rstd
    # relative error of n: the rounding of u and of the mean against the deviation
    kappa = (u.abs().amax(-1, keepdim=True) * rstd).expand_as(n3).reshape(rows, C)
    n = n3.reshape(rows, C)
    pre = n * w + b
    gate = s if after else one
    zmag = 1.0 if z is None else 1.0 + z.double().abs()
    r = dict(out=pre * gate, out_mag=((n.abs() + kappa) * w.abs() + b.abs()) * gate.abs() * zmag)
    if dout is None:
        return r
    dout = dout.double()
    dp = dout * gate
    d3 = (dp * w).view(rows, ngroups, m)
    c1 = (d3 * n3).mean(-1, keepdim=True)
    c2 = d3.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(c1)
    du = ((d3 - n3 * c1 - c2) * rstd).reshape(rows, C)
    nk = n3.abs() + kappa.view(rows, ngroups, m)
    a1 = (d3.abs() * nk).mean(-1, keepdim=True)
    du_mag = ((d3.abs() + nk * a1 + nk * c1.abs() + d3.abs().mean(-1, keepdim=True)) * rstd).reshape(rows, C) * zmag
    r.update(dx=du * (s if before else 1.0), dx_mag=du_mag * (s.abs() if before else 1.0) * zmag)
    if before:
        r.update(dz=du * x * ds, dz_mag=du_mag * x.abs() * (sg * zmag * 2) * zmag)
    elif after:
        r.update(dz=dout * pre * ds, dz_mag=dout.abs() * ((n.abs() + kappa) * w.abs() + b.abs()) * (sg * zmag * 2) * zmag)
    nk2 = n.abs() + kappa
    r.update(dw=(dp * n).sum(0), dw_mag=(dp.abs() * nk2 * zmag).sum(0), db=dp.sum(0),
             db_mag=(dp.abs() * zmag).sum(0))
    return r
