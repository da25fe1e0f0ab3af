"""How far the delta rule's outputs are from those in 64 bits, by norms of a head's whole output, and the
bounds that those are compared with: relative to the output itself, so that a wrong term shows.

fp32 outputs.  A value is formed by a chain of contractions, over dstate (K h, twice in the backward, and the
pairs), headdim (the gradients of states and pairs) and a chunk's tokens (T, M, and the sums into the state and
out of it): at most C = 3 N + 3 P + 8 * 64 roundings of partial sums lie on a way to it.  Each is off by at most
2^-24 of a partial sum, in the mean square by half of that, and a partial sum is no larger, in the mean square,
than the value's terms together; their signs are random.  The terms are as large as the value but for what
cancels in e = v - a h k, by a factor of about 2 with keys of length 1.  So the 2-norm of the error is expected
below 2^-25 sqrt(C) * 2 = 2^-24 sqrt(C) of the output's, which is the bound.

bf16 outputs are such values rounded to bf16.  One differs from the rounded 64-bit value only if a border
between two bf16 numbers lies between the two values: for an error d and steps s >= 2^-8 |value| with probability
d / s.  Over an output of Gaussian values, whose d is the bound's b times their size in the mean square, the
share is below b 2^8 E[size / |value|], with the expectation cut off where d = s below 8; each difference is one
step, at most 2^-7 of the value.  So the 2-norm of the difference from the rounded 64-bit values is expected
below 2^-7 sqrt(8 * 2^8 b) of the output's; what differs at small values weighs less.
"""
from __future__ import annotations

import math

import torch

def bound(P, N, dtype):
    b = 2.0 ** -24 * math.sqrt(3 * N + 3 * P + 8 * 64)
    return b if dtype == torch.float32 else 2.0 ** -7 * math.sqrt(8 * 2 ** 8 * b)


def error(got, ref, dtype, heads_at):
    """The largest of the rows' and heads' errors by the 2-norm, relative to the output's (bf16: of values rounded
    to it)."""
    x, y = got.detach().cpu().double(), ref.double()
    if dtype != torch.float32:
        x, y = x.to(dtype).double(), y.to(dtype).double()
    x, y = (t.transpose(1, heads_at).flatten(2) for t in (x, y))
    return float(((x - y).norm(dim=2) / y.norm(dim=2)).max())
