"""The fp32 gradients of the scan's backward, ddt and dA, in 64 bits and the sizes that their errors
are compared with: norms, not sums of magnitudes, so that a wrong sum shows.

A gradient is a sum of products of random signs.  On the way to one value lie, one after the other,
at most K = 3 N + 2 P + 128 roundings to fp32 of partial sums (the contractions over dstate, whose
operands come in up to three parts, and over headdim; the tile's 16 rows and columns; the chunk's
tiles, the factors).  Each is off by at most 2^-24 of a partial sum that is no larger, in the mean
square, than the value's terms together, and their signs are random: 2^-24 sqrt(K) of it.  tol()
allows twice that.

dA sums dt q over the row.  What a chunk hands on enters the q of all its tokens alike, so a chunk's
tokens go by magnitude and only the chunks by squares.  On the matrix cores (`carried`) q holds one
more such term: the carried product f <G, S> of a chunk is that of the last of its range of 8 chunks
plus the sums U of the up to 7 chunks behind it minus the sums V of as many.  Each of these 14 has the
error above, 2^-24 sqrt(K) of a sum as large as q's, and random signs among them: sqrt(14) times that
in every token of the chunk, on top of q's own.  Chunks of one range share them (a chunk's are also in
those before it), so there the magnitudes go over the range of 1024 tokens, and the squares over the
ranges.
"""
from __future__ import annotations

import math

import torch

from train_ref import _scan_tokens, starts_of


def tol(P, N):
    return 2 * 2.0 ** -24 * math.sqrt(3 * N + 2 * P + 128)


def tol_dA(P, N, carried):
    return tol(P, N) * (1 + math.sqrt(14) if carried else 1)


def carried(i):
    """Whether the call runs on the bf16 matrix cores."""
    return i["x"].dtype == torch.bfloat16 and i["x"].shape[3] == 64 and i["Bm"].shape[3] in (64, 128)


def ddt_dA64(i, heads):
    """Per head of `heads`: ddt [B, L], dA, and the size that dA's error goes by."""
    x, dt, A, dy = (i[k].double() for k in ("x", "dt", "A", "dy"))
    B, L, H, P = x.shape
    k = H // i["Bm"].shape[2]
    N = i["Bm"].shape[3]
    st = starts_of(i["seq"], B, L)
    span = 1024 if carried(i) else 64
    out = []
    for h in heads:
        s = slice(h, h + 1)
        Bh, Ch = (i[n][:, :, h // k:h // k + 1].double() for n in ("Bm", "Cm"))
        a = torch.exp(dt[:, :, s] * A[s]).masked_fill(st[..., None], 0.0)
        z = torch.zeros(B, 1, P, N, dtype=torch.float64)
        h0, dhT = (z if i[n] is None else i[n][:, s].double() for n in ("h0", "dhT"))
        _, prev, gs, _ = _scan_tokens(x[:, :, s], dt[:, :, s], a, Bh, Ch, dy[:, :, s], h0, dhT)
        q = (a * (gs * prev).sum((-1, -2)))[..., 0]
        direct = (x[:, :, s] * (gs * Bh[..., None, :]).sum(-1)).sum(-1)[..., 0]
        dq = dt[:, :, h] * q
        by_span = torch.nn.functional.pad(dq.abs(), (0, -L % span)).view(B, -1, span).sum(-1)
        out.append((direct + A[h] * q, float(dq.sum()), float(by_span.norm())))
    return out


def errors(got_ddt, got_dA, ref, heads):
    """(largest ddt error of a head relative to its norm, largest dA error relative to its size)."""
    e = []
    for h, (ddt, dA, size) in zip(heads, ref):
        e.append((float((got_ddt[:, :, h].cpu().double() - ddt).norm() / ddt.norm()),
                  abs(float(got_dA[h]) - dA) / size))
    return max(x[0] for x in e), max(x[1] for x in e)
