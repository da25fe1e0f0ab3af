"""GPU test that no fp32 operand of the delta rule's products loses bits: sums that cancel down to the
last bit of a 21-bit number.  Without gates and with keys at right angles the chunk's inverse is the
identity, and all products are whole numbers (or halves) below 2^24: the outputs are exact."""
import pytest
import torch

from test_gpu_e_delta import BF16, F32, _run

pytestmark = pytest.mark.gpu
PARTS = (1024.0, 32.0, 1.0)  # the squares' sum, 2^20 + 2^10 + 1, needs three bf16 numbers
LESS = (1024.0, 32.0, 0.0)
WHOLE = sum(v * v for v in PARTS)
SHAPES = [(64, 128, BF16), (64, 64, BF16), (128, 256, BF16), (36, 44, BF16), (16, 16, F32)]
# three tokens of a chunk of 64, of the chunk's tiles alike and apart, and of a chunk of 32
WHERE = [(0, 1, 2), (5, 6, 9), (5, 20, 40), (15, 16, 63), (33, 34, 62), (1, 17, 30), (64, 80, 95), (97, 100, 126)]
ONE_CHUNK = {F32: 32, BF16: 64}


def _zeros(P, N, dtype, states=False):
    z = lambda *s: torch.zeros(*s, dtype=dtype)  # noqa: E731
    L = 130
    return dict(q=z(1, L, 1, N), k=z(1, L, 1, N), v=z(1, L, 1, P), beta=torch.ones(1, L, 1), gate=None,
                h0=torch.zeros(1, 1, P, N) if states else None, dy=z(1, L, 1, P),
                dhT=torch.zeros(1, 1, P, N) if states else None)


def _set(t, token, values, at):
    for v, i in zip(values, at):
        t[0, token, 0, i] = v


def _tokens(dtype):
    return [w for w in WHERE if len({t // ONE_CHUNK[dtype] for t in w}) == 1]


@pytest.mark.parametrize("P,N,dtype", SHAPES)
def test_forward_pairs(P, N, dtype):
    """y of c: (q_c.k_a) v_a + (q_c.k_b) v_b."""
    for a, b, c in _tokens(dtype):
        i = _zeros(P, N, dtype)
        _set(i["k"], a, PARTS, (0, 1, N - 1))
        _set(i["k"], b, LESS, (2, 3, N - 2))
        _set(i["q"], c, PARTS + PARTS, (0, 1, N - 1, 2, 3, N - 2))
        i["v"][0, a], i["v"][0, b] = 1.0, -1.0
        assert (_run(i, 1.0, None)["y"][0, c].float() == 1.0).all(), (a, b, c)


@pytest.mark.parametrize("P,N,dtype", SHAPES)
def test_forward_values(P, N, dtype):
    """What the tokens a and b write, 8 and 0 less what the state holds there, cancels in y of c."""
    for a, b, c in _tokens(dtype):
        i = _zeros(P, N, dtype, states=True)
        i["h0"][..., 0], i["h0"][..., N - 1] = WHOLE, WHOLE - 1.0
        i["k"][0, a, 0, 0] = i["k"][0, b, 0, N - 1] = 1.0
        i["q"][0, c, 0, 0], i["q"][0, c, 0, N - 1] = 1.0, -1.0
        i["v"][0, a] = 8.0
        got = _run(i, 1.0, None)
        assert (got["y"][0, c].float() == 8.0).all(), (a, b, c)
        assert (got["final"][..., 0] == 8.0).all() and (got["final"][..., N - 1] == 0.0).all(), (a, b, c)


@pytest.mark.parametrize("P,N,dtype", SHAPES)
def test_pairs_of_gradients(P, N, dtype):
    for a, b, c in _tokens(dtype):
        # dq of c: (dy_c.u_a) k_a + (dy_c.u_b) k_b
        i = _zeros(P, N, dtype)
        _set(i["k"], a, (1.0, 1.0), (0, N - 1))
        _set(i["k"], b, (1.0, -1.0), (0, N - 1))
        _set(i["v"], a, PARTS, (0, 1, P - 1))
        _set(i["v"], b, [-v for v in LESS], (0, 1, P - 1))
        _set(i["dy"], c, PARTS, (0, 1, P - 1))
        assert _run(i, 1.0, None)["dq"][0, c, 0, 0] == 1.0, ("dq", a, b, c)
        # dk of a: (dy_b.u_a) q_b + (dy_c.u_a) q_c
        i = _zeros(P, N, dtype)
        _set(i["v"], a, PARTS, (0, 1, P - 1))
        _set(i["dy"], b, PARTS, (0, 1, P - 1))
        _set(i["dy"], c, LESS, (0, 1, P - 1))
        i["q"][0, b], i["q"][0, c] = 1.0, -1.0
        assert (_run(i, 1.0, None)["dk"][0, a].float() == 1.0).all(), ("dk", a, b, c)


@pytest.mark.parametrize("P,N,dtype", SHAPES)
def test_pairs_of_errors(P, N, dtype):
    """The pairs of what tokens write and of its gradients, dz.e, into both keys."""
    for a, b, c in _tokens(dtype):
        # dk of a: -(dz_b.e_a) k_b - (dz_c.e_a) k_c, and half of it again from the queries at b and c
        i = _zeros(P, N, dtype)
        _set(i["v"], a, PARTS, (0, 1, P - 1))
        _set(i["k"], b, (1.0, 1.0), (0, N - 1))
        _set(i["k"], c, (1.0, -1.0), (0, N - 1))
        _set(i["q"], b, (0.5, 0.5), (0, N - 1))
        _set(i["q"], c, (0.5, -0.5), (0, N - 1))
        _set(i["dy"], b, PARTS, (0, 1, P - 1))
        _set(i["dy"], c, [-v for v in LESS], (0, 1, P - 1))
        assert _run(i, 1.0, None)["dk"][0, a, 0, 0] == -0.5, ("earlier", a, b, c)
        # dk of c: -(dz_c.e_a) k_a - (dz_c.e_b) k_b
        i = _zeros(P, N, dtype)
        _set(i["k"], a, (1.0, 1.0), (0, N - 1))
        _set(i["k"], b, (1.0, -1.0), (0, N - 1))
        _set(i["v"], a, PARTS, (0, 1, P - 1))
        _set(i["v"], b, [-v for v in LESS], (0, 1, P - 1))
        i["k"][0, c, 0, 2] = i["q"][0, c, 0, 2] = 1.0
        _set(i["dy"], c, PARTS, (0, 1, P - 1))
        assert _run(i, 1.0, None)["dk"][0, c, 0, 0] == -1.0, ("later", a, b, c)


@pytest.mark.parametrize("P,N,dtype", SHAPES)
def test_states(P, N, dtype):
    """The initial state into dq, the final state's gradient and what a token writes into dk."""
    for t in (0, 17, 31, 32, 63, 64, 100, 129):
        i = _zeros(P, N, dtype, states=True)
        for n in ("h0", "dhT"):
            i[n][:, :, 0], i[n][:, :, P - 1] = WHOLE, WHOLE - 1.0
        for n in ("v", "dy"):
            _set(i[n], t, (1.0, -1.0), (0, P - 1))
        got = _run(i, 1.0, None)
        assert (got["dq"][0, t].float() == 1.0).all() and (got["dk"][0, t].float() == 1.0).all(), ("dq, dk", t)
        i = _zeros(P, N, dtype, states=True)
        i["h0"][:, :, 0, 0], i["h0"][:, :, P - 1, 0] = WHOLE, WHOLE - 1.0
        i["dhT"][:, :, 0, 1:], i["dhT"][:, :, P - 1, 1:] = 1.0, -1.0
        i["k"][0, t, 0, 0] = 1.0
        assert (_run(i, 1.0, None)["dk"][0, t, 0, 1:].float() == -1.0).all(), ("dk", t)
