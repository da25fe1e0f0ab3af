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


# ---------------------------------------------------------------------------------------
# per-channel gated recurrence
# ---------------------------------------------------------------------------------------
def starts_of(seq, B, L):
    """[B, L] bool: tokens that start a packed sequence (never token 0)."""
    m = torch.zeros(B, L, dtype=torch.bool)
    if seq is not None:
        m[:, 1:] = seq[:, 1:] != seq[:, :-1]
    return m


def gated64(x, gate, form, h0=None, seq=None, dy=None, dhT=None):
    """y, final and, with dy, dx, dgate, dh0 token by token; `*_err`: a bound of the fp32 error
    of each before its rounding to the output type, by the same recurrence: a token multiplies
    what it passes on and adds its own, each with k half-steps (k = 24 + 4 |gate|: the exp of a
    rounded argument, reciprocal, product and sum, and the joins of spans, whose products add
    fewer roundings than the tokens they span)."""
    B, L, C = x.shape
    x, g = x.double(), gate.double()
    log = form == "log"
    ag = torch.exp(g) if log else torch.sigmoid(g)
    i = torch.ones_like(g) if log else torch.sigmoid(-g)
    st = starts_of(seq, B, L)[..., None]
    a = ag.masked_fill(st, 0.0)
    u = i * x
    k = (24 + 4 * g.abs().clamp(max=200.0)) * U
    h = torch.zeros(B, C, dtype=torch.float64) if h0 is None else h0.double()
    mag, err = h.abs(), torch.zeros_like(h)
    hs, before, berr, bmag, es = (torch.empty_like(x) for _ in range(5))
    for t in range(L):
        s = st[:, t]
        before[:, t], berr[:, t], bmag[:, t] = (v.masked_fill(s, 0.0) for v in (h, err, mag))
        keep = a[:, t]
        # a start keeps nothing, whatever the state (also NaN or inf) was
        h = torch.where(s, torch.zeros_like(h), keep * h) + u[:, t]
        err = torch.where(s, torch.zeros_like(h), keep * err + k[:, t] * keep * mag) + k[:, t] * u[:, t].abs()
        mag = torch.where(s, torch.zeros_like(h), keep * mag) + u[:, t].abs()
        hs[:, t], es[:, t] = h, err + 1e-30
    r = dict(y=hs, y_err=es, final=h, final_err=err + 1e-30)
    if dy is None:
        return r
    dy = dy.double()
    E = torch.zeros(B, C, dtype=torch.float64) if dhT is None else dhT.double()
    Eerr, Emag = torch.zeros_like(E), E.abs()
    dx, dgate, dxe, dge = (torch.empty_like(x) for _ in range(4))
    for t in range(L - 1, -1, -1):
        kt = k[:, t]
        D, De, Dm = E + dy[:, t], Eerr + U * (Emag + dy[:, t].abs()), Emag + dy[:, t].abs()
        dx[:, t] = D * i[:, t]
        dxe[:, t] = i[:, t] * (De + kt * Dm) + 1e-30
        dl = D * a[:, t] * before[:, t]
        le = a[:, t] * (De * before[:, t].abs() + Dm * berr[:, t] + kt * Dm * bmag[:, t])
        if log:
            dgate[:, t], dge[:, t] = dl, le + 1e-30
        else:
            w = i[:, t] * ag[:, t] * x[:, t].abs()
            dgate[:, t] = i[:, t] * dl - D * x[:, t] * i[:, t] * ag[:, t]
            dge[:, t] = i[:, t] * (le + kt * a[:, t] * Dm * bmag[:, t]) + w * (De + kt * Dm) + 1e-30
        s = st[:, t]
        E = torch.where(s, torch.zeros_like(D), a[:, t] * D)
        Eerr = torch.where(s, torch.zeros_like(D), a[:, t] * De + kt * a[:, t] * Dm)
        Emag = torch.where(s, torch.zeros_like(D), a[:, t] * Dm)
    r.update(dx=dx, dx_err=dxe, dgate=dgate, dgate_err=dge, dh0=E, dh0_err=Eerr + 1e-30)
    return r


def check_err(got, ref, name, dtype):
    h = half_step(dtype)
    assert_bound(got, ref[name], h * ref[name].abs() + (1 + h) * ref[name + "_err"], name)


# ---------------------------------------------------------------------------------------
# the scan's backward
# ---------------------------------------------------------------------------------------
def _scan_tokens(x, dt, a, Bh, Ch, dy, h0, dhT):
    """States h_t, gradients g_t [B, L, H, P, N] and the gradient handed to h_{-1}, token by
    token (all float64; a [B, L, H] with 0 at the starts)."""
    B, L, H, P = x.shape
    N = Bh.shape[-1]
    h = h0
    hs, gs = (torch.empty(B, L, H, P, N, dtype=torch.float64) for _ in range(2))
    prev = torch.empty_like(hs)
    for t in range(L):
        prev[:, t] = h
        h = a[:, t, :, None, None] * h + (dt[:, t, :, None] * x[:, t])[..., None] * Bh[:, t, :, None, :]
        hs[:, t] = h
    g = dhT
    for t in range(L - 1, -1, -1):
        gs[:, t] = g + dy[:, t, :, :, None] * Ch[:, t, :, None, :]
        g = a[:, t, :, None, None] * gs[:, t]
    return hs, prev, gs, g


def scan_bwd64(x, dt, A, Bm, Cm, dy, h0=None, dhT=None, seq=None):
    """dx, ddt, dA, dB, dC, dh0 from the definition, token by token, and for each the magnitude
    its fp32 error scales with (`*_mag`).  The magnitudes come from the same recurrences over
    absolute values; q = dL/d log a is formed from sums over a 64-token chunk that cancel, so
    its magnitude is what the whole chunk adds up."""
    B, L, H, P = x.shape
    G, N = Bm.shape[2:]
    k = H // G
    x, dt, A, dy = x.double(), dt.double(), A.double(), dy.double()
    Bh, Ch = (v.double().repeat_interleave(k, 2) for v in (Bm, Cm))
    z = torch.zeros(B, H, P, N, dtype=torch.float64)
    h0 = z if h0 is None else h0.double()
    dhT = z if dhT is None else dhT.double()
    st = starts_of(seq, B, L)
    a = torch.exp(dt * A).masked_fill(st[..., None], 0.0)

    def grads(x, dt, Bh, Ch, dy, h0, dhT):
        hs, prev, gs, g = _scan_tokens(x, dt, a, Bh, Ch, dy, h0, dhT)
        gB = (gs * Bh[..., None, :]).sum(-1)
        q = a * (gs * prev).sum((-1, -2))
        group = lambda v: v.view(B, L, G, k, N).sum(3)  # noqa: E731
        r = dict(dx=dt[..., None] * gB, direct=(x * gB).sum(-1), q=q, dh0=g,
                 dB=group(((dt[..., None] * x)[..., None] * gs).sum(3)),
                 dC=group((dy[..., None] * hs).sum(3)))
        r["Y"] = (dy * (hs * Ch[..., None, :]).sum(-1)).sum(-1)
        r["through"] = q  # <g_t, a_t h_{t-1}> bounds what passes through the chunk
        return r
    r = grads(x, dt, Bh, Ch, dy, h0, dhT)
    m = grads(x.abs(), dt.abs(), Bh.abs(), Ch.abs(), dy.abs(), h0.abs(), dhT.abs())
    r["ddt"] = r["direct"] + A * r["q"]
    r["dA"] = (dt * r["q"]).sum((0, 1))
    each = m["Y"] + 2 * m["direct"] * dt.abs() + m["q"]
    qm = torch.empty_like(each)
    for t0 in range(0, L, 64):
        qm[:, t0:t0 + 64] = each[:, t0:t0 + 64].sum(1, keepdim=True)
    out = {n: r[n] for n in ("dx", "ddt", "dA", "dB", "dC", "dh0")}
    for n in ("dx", "dB", "dC", "dh0"):
        out[n + "_mag"] = m[n]
    out["ddt_mag"] = m["direct"] + A.abs() * qm
    out["dA_mag"] = (dt.abs() * qm).sum((0, 1))
    return out


def scan_loss64(x, dt, A, Bm, Cm, dy, h0, dhT, seq):
    """sum(y dy) + sum(final dfinal), differentiable by torch, token by token in float64."""
    B, L, H, P = x.shape
    k = H // Bm.shape[2]
    Bh, Ch = Bm.repeat_interleave(k, 2), Cm.repeat_interleave(k, 2)
    st = starts_of(seq, B, L)
    h, loss = h0, 0.0
    for t in range(L):
        a = torch.exp(dt[:, t] * A).masked_fill(st[:, t, None], 0.0)
        h = a[..., None, None] * h + (dt[:, t, :, None] * x[:, t])[..., None] * Bh[:, t, :, None, :]
        loss = loss + ((h * Ch[:, t, :, None, :]).sum(-1) * dy[:, t]).sum()
    return loss + (h * dhT).sum()
