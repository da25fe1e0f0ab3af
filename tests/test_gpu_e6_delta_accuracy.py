"""GPU accuracy of the gated delta rule by norms (delta_sharp.py), in rows uncut and cut into segments,
packed and not, with gates and states; and on the CPU that the bounds see what is wrong."""
import pytest
import torch

from delta_ref import delta64
from delta_sharp import bound, error
from test_gpu_e_delta import BF16, F32, STATE, _inputs, _run, _seq

CASES = [  # B, L, H, G, P, N, dtype, packed
    (1, 300, 2, 1, 64, 128, BF16, None), (2, 200, 4, 2, 32, 64, BF16, "random"), (1, 260, 2, 2, 130, 256, BF16, "edges"),
    (1, 2100, 1, 1, 64, 128, BF16, None), (1, 1030, 3, 3, 80, 64, BF16, "random"), (1, 1500, 2, 1, 64, 64, BF16, None),
    (2, 1100, 1, 1, 16, 200, BF16, "random"), (1, 300, 2, 1, 64, 128, F32, None), (2, 200, 4, 2, 40, 48, F32, "edges"),
    (1, 1100, 2, 1, 40, 48, F32, "random"), (1, 900, 1, 1, 32, 256, F32, None),
]
HEADS_AT = {"final": 1, "dh0": 1}


def _case(B, L, H, G, P, N, dtype, packed):
    return _inputs(B, L, H, G, P, N, dtype, seed=L + N), _seq(B, L, packed, 5)


def _reference(s, seq):
    return delta64(s["q"], s["k"], s["v"], s["beta"], s["gate"], 0.5, s["h0"], seq, s["dy"], s["dhT"])


def _errors(got, ref, dtype):
    return {n: error(got[n], ref[n], F32 if n in STATE else dtype, HEADS_AT.get(n, 2))
            for n in ("y", "final", "dq", "dk", "dv", "dbeta", "dgate", "dh0")}


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_errors_by_norms(case):
    s, seq = _case(*case)
    dtype = case[6]
    e = _errors(_run(s, 0.5, seq), _reference(s, seq), dtype)
    print(case, {n: f"{x:.1e}" for n, x in e.items()}, flush=True)
    for n, x in e.items():
        assert x <= bound(case[4], case[5], F32 if n in STATE else dtype), (n, e)


@pytest.mark.parametrize("case", [CASES[0], CASES[4], CASES[8]], ids=str)
def test_bounds_reject(case):
    """What is 0, one percent off, or formed from operands that are rounded to 8 bits is over the bounds; for
    fp32 outputs also from operands rounded to 16 bits."""
    s, seq = _case(*case)
    ref, dtype = _reference(s, seq), case[6]
    most = {n: bound(case[4], case[5], F32 if n in STATE else dtype) for n in ref if not n.endswith("_mag")}
    assert max(_errors(ref, ref, F32).values()) == 0.0
    for f in (0.0, 0.99):
        e = _errors({n: f * t for n, t in ref.items()}, ref, dtype)
        assert all(e[n] > 5 * most[n] for n in e), (f, e)
    r = torch.Generator().manual_seed(1)

    def rough(bits, names):
        off = {n: s[n].double() * (1 + 2.0 ** -bits * (2 * torch.rand(s[n].shape, generator=r) - 1)) for n in names}
        return _reference(dict(s, **off), seq)
    e = _errors(rough(9, ("v", "dy", "beta", "h0", "dhT")), ref, dtype)
    assert all(e[n] > 2 * most[n] for n in e), e
    e = _errors(rough(17, ("q", "k", "v", "dy")), ref, dtype)
    assert all(e[n] > 1.5 * most[n] for n in STATE), e
