"""Plain 64-bit implementations of the gated delta rule and of the queries' and keys' norm, token
by token and head by head on the CPU, with error bounds.

Bounds of the delta rule.  U = 2^-24.  A token's step h -> a h (I - b k k^T) does not lengthen any
row of h for gates <= 0 and 0 <= b |k|^2 <= 2, and neither does its transpose lengthen a gradient.
So an error made at one token reaches later outputs no larger than it was made, and an output's
error is at most the sum of the errors made before it.  The kernels make them by chunks of at most
64 tokens: sums over dstate, headdim and the chunk's tokens (twice: pairs and states), each of at
most n = dstate + headdim + 4 * 64 terms, and so at most n U times the sum of the magnitudes of
their terms.  That sum of magnitudes is what `*_mag` bounds by lengths of vectors (Cauchy-Schwarz),
their largest over the row.  Element by element: n U (chunks + 1) mag.  For the 2-norm roundings
count as independent, in random walk: 8 sqrt(n (chunks + 1)) U |mag|.  An output of dtype t adds
half a step of its own value."""
from __future__ import annotations

import torch

U = 2.0 ** -24


def delta64(q, k, v, beta, gate, scale, h0, seq, dy=None, dhT=None):
    """dict of y, final and, with dy, dq, dk, dv, dbeta, dgate, dh0, each with its `_mag`."""
    q, k, v, beta = q.double(), k.double(), v.double(), beta.double()
    B, L, H, P = v.shape
    G, N = k.shape[2:]
    rep = H // G
    a = torch.ones(B, L, H, dtype=torch.float64) if gate is None else torch.exp(gate.double())
    if seq is not None and L > 1:
        a[:, 1:][seq[:, 1:] != seq[:, :-1]] = 0.0
    kh, qh = k.repeat_interleave(rep, 2), q.repeat_interleave(rep, 2)
    h = torch.zeros(B, H, P, N, dtype=torch.float64) if h0 is None else h0.double()
    hs, es, y = [h], [], torch.zeros_like(v)
    for t in range(L):
        at, bt = a[:, t, :, None, None], beta[:, t, :, None]
        # a cut takes over nothing, whatever the state holds
        ah = torch.where(at == 0, torch.zeros_like(h), at * h)
        e = v[:, t] - (ah * kh[:, t, :, None, :]).sum(-1)
        h = ah + (bt * e)[..., None] * kh[:, t, :, None, :]
        y[:, t] = scale * (h * qh[:, t, :, None, :]).sum(-1)
        hs.append(h)
        es.append(e)
    length = lambda x: x.norm(dim=-1)  # noqa: E731
    # rows of the state, and what a token adds to them
    kn, qn = length(kh), length(qh)                                        # [B, L, H]
    rows = torch.stack([length(x) for x in hs], 1)                         # [B, L + 1, H, P]
    adds = torch.stack([e.abs() for e in es], 1) * (beta.abs() * kn)[..., None] if L else torch.zeros(B, 0, H, P)
    row = (rows.amax(1) + v.abs().amax(1) * (beta.abs() * kn).amax(1)[..., None] + adds.amax(1)) if L else rows[:, 0]
    r = dict(y=y, final=h, y_mag=(abs(scale) * qn)[..., None] * row[:, None],
             final_mag=row[..., None].expand_as(h))
    if dy is None:
        return r
    d = scale * dy.double()
    g = torch.zeros_like(h) if dhT is None else dhT.double()
    dq, dk = torch.zeros_like(qh), torch.zeros_like(kh)
    dv, dbeta, dgate = torch.zeros_like(v), torch.zeros_like(beta), torch.zeros_like(beta)
    gs = [g]
    for t in range(L - 1, -1, -1):
        at, bt, kt = a[:, t, :, None, None], beta[:, t, :, None], kh[:, t, :, None, :]
        g = g + d[:, t, ..., None] * qh[:, t, :, None, :]
        gs.append(g)
        ah = torch.where(at == 0, torch.zeros_like(g), at * hs[t])
        gk = (g * kt).sum(-1)
        de = bt * gk
        dah = g - de[..., None] * kt
        dq[:, t] = (hs[t + 1] * d[:, t, ..., None]).sum(2)
        dk[:, t] = (g * (bt * es[t])[..., None]).sum(2) - (ah * de[..., None]).sum(2)
        dv[:, t] = de
        dbeta[:, t] = (gk * es[t]).sum(-1)
        dgate[:, t] = (dah * ah).sum((-1, -2))
        g = torch.where(at == 0, torch.zeros_like(g), at * dah)
    gs.append(g)
    grow = (torch.stack([length(x) for x in gs], 1).amax(1)
            + d.abs().amax(1) * qn.amax(1)[..., None]) if L else rows[:, 0] * 0  # [B, H, P]
    hf, gf = row.norm(dim=-1), grow.norm(dim=-1)                           # whole states [B, H]
    dn = length(dy.double()) * abs(scale)                                  # [B, L, H]
    e_all = torch.stack([e.abs() for e in es], 1).amax(1).norm(dim=-1) if L else hf
    b_max = beta.abs().amax(1) if L else hf
    k_max = kn.amax(1) if L else hf
    vn = v.abs().amax(1).norm(dim=-1) if L else hf
    en = e_all + vn + hf * k_max                                           # errors e_t, [B, H]

    def groups(x):  # [B, L, H, N] -> sums over the heads of a key head
        return x.unflatten(2, (G, rep)).sum(3)

    per = lambda x: x[:, None].expand(B, L, H)  # noqa: E731
    q_mag = (dn * per(hf))[..., None].expand(B, L, H, N)
    k_mag = per(gf * b_max * (en + hf * k_max))[..., None].expand(B, L, H, N)
    r.update(dq=groups(dq), dq_mag=groups(q_mag), dk=groups(dk), dk_mag=groups(k_mag),
             dv=dv, dv_mag=(per(b_max * k_max))[..., None] * grow[:, None], dbeta=dbeta,
             dbeta_mag=per(gf * k_max * en), dgate=dgate,
             dgate_mag=per(gf * (hf + b_max * k_max * en)), dh0=g, dh0_mag=grow[..., None].expand_as(g))
    return r


def check_delta(got, ref, name, dtype, n, chunks):
    """The bounds above: element by element and by the 2-norm."""
    x, y, mag = got.detach().to("cpu").double(), ref[name], ref[name + "_mag"]
    assert x.shape == y.shape, (name, x.shape, y.shape)
    assert torch.isfinite(x).all(), f"{name}: non-finite values"
    if not y.numel():
        return
    half = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    err = (x - y).abs()
    own = half * y.abs() * (1 + half)
    bound = n * U * (chunks + 1) * mag * (1 + half) + own + torch.finfo(torch.float32).tiny
    worst = float((err / bound).max())
    assert worst <= 1.0, f"{name}: {int((err > bound).sum())} of {err.numel()} over the bound, worst {worst:.3g} times"
    most = 8 * (n * (chunks + 1)) ** 0.5 * U * mag.norm() + own.norm()
    assert float(err.norm()) <= float(most), f"{name}: error {float(err.norm()):.3g} by the 2-norm, bound {float(most):.3g}"


def qk_norm64(x, w, eps, kind, freq, pos, interleaved, dy=None):
    """out, out_mag and, with dy, dx, dx_mag, dw, dw_mag.  Errors in U of the magnitudes: the sum of
    D squares (D + 2), its root and reciprocal (3), two products and, turned, the angle's sine and
    cosine (4 with the argument's two roundings) and their two products (3)."""
    B, L, H, D = x.shape
    x = x.double()
    m = 1 if kind == "l2" else D
    s = (x * x).sum(-1, keepdim=True) / m + eps
    r = torch.where(s > 0, 1.0 / s.sqrt(), torch.zeros_like(s))
    n = x * r
    w1 = torch.ones(D, dtype=torch.float64) if w is None else w.double()

    def turn(v, back, sign=True):
        if freq is None:
            return v
        R = 2 * freq.shape[0]
        p = (torch.arange(L).expand(B, L) if pos is None else pos).double()
        ang = (p[..., None] * freq.double())[:, :, None]
        c, sn = torch.cos(ang), torch.sin(ang) * (-1.0 if back else 1.0)
        if not sign:
            c, sn = c.abs(), -sn.abs()  # a c - b sn = |a| |c| + |b| |sn|
        out = v.clone()
        a, b = (v[..., 0:R:2], v[..., 1:R:2]) if interleaved else (v[..., :R // 2], v[..., R // 2:R])
        first, second = a * c - b * sn, (a * sn if sign else a * sn.abs()) + b * c
        if interleaved:
            out[..., 0:R:2], out[..., 1:R:2] = first, second
        else:
            out[..., :R // 2], out[..., R // 2:R] = first, second
        return out

    y = n * w1
    out = dict(out=turn(y, False), out_mag=turn(y.abs(), False, sign=False))
    if dy is None:
        return out
    d, dmag = turn(dy.double(), True), turn(dy.double().abs(), True, sign=False)
    dw = (d * n).sum((0, 1, 2))
    dn, dnm = d * w1, dmag * w1.abs()
    c, cm = (dn * n).sum(-1, keepdim=True) / m, (dnm * n.abs()).sum(-1, keepdim=True) / m
    out.update(dx=r * (dn - n * c), dx_mag=r * (dnm + n.abs() * cm), dw=dw, dw_mag=(dmag * n.abs()).sum((0, 1, 2)))
    return out


def check_qk(got, ref, name, dtype, D, terms=0):
    """|got - ref| <= (2 D + 24 + terms) U mag and half a step of the type (D twice: the sum of squares
    and the backward's product; terms: additions over tokens and heads)."""
    x, y, mag = got.detach().to("cpu").double(), ref[name], ref[name + "_mag"]
    assert x.shape == y.shape, (name, x.shape, y.shape)
    assert torch.isfinite(x).all(), f"{name}: non-finite values"
    half = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    bound = (2 * D + 24 + terms) * U * mag * (1 + half) + half * y.abs() * (1 + half) + torch.finfo(torch.float32).tiny
    worst = float(((x - y).abs() / bound).max()) if y.numel() else 0.0
    assert worst <= 1.0, f"{name}: worst {worst:.3g} times the bound"
