"""GPU test that gates and states that are not finite reach only what the formula has them reach: the
gate of a sequence's first token nothing at all, and no other sequence's states."""
import pytest
import torch

from test_gpu_e_delta import BF16, F32, GRADS, _inputs, _run

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf")]


def _two(B, L, at):
    seq = torch.zeros(B, L, dtype=torch.int32)
    seq[:, at:] = 1
    return seq


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", BAD + [-float("inf"), 1e30])
def test_gate_of_a_first_token_counts_for_nothing(bad, dtype):
    """Of the second and third sequence, of rows uncut and cut in segments: the same bits."""
    for B, L, H, starts in ((2, 260, 2, (70, 100)), (1, 2100, 1, (70, 1000))):
        s = _inputs(B, L, H, 1, 32, 64, dtype, seed=30)
        seq = _two(B, L, starts[0])
        seq[:, starts[1]:] = 2
        clean = _run(s, 1.0, seq)
        s = dict(s, gate=s["gate"].clone())
        s["gate"][0, list(starts)] = bad
        got = _run(s, 1.0, seq)
        for n in clean:
            assert torch.equal(got[n], clean[n]), (n, L)
        assert not got["dgate"][0, list(starts)].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("B,L,H,start", [(2, 260, 2, 70), (1, 2100, 1, 1000)])
def test_gate_stays_in_its_sequence(B, L, H, start, bad, dtype):
    """A gate within the first or the second sequence, in the chunk where they meet or away from it:
    other sequences' states, and their tokens in other chunks, have the same bits."""
    s = _inputs(B, L, H, 1, 32, 64, dtype, seed=31)
    seq = _two(B, L, start)
    Q = 64 if dtype == BF16 else 32
    lo, hi = start // Q * Q, -(-start // Q) * Q  # the chunk where the sequences meet
    clean = _run(s, 1.0, seq)
    for at in (start - 2, start - 50, start + 1, start + 40):
        t = dict(s, gate=s["gate"].clone())
        t["gate"][0, at, 0] = bad
        got = _run(t, 1.0, seq)
        for n, w in clean.items():
            assert torch.equal(got[n][1:], w[1:]), (n, at)
            g = got[n]
            if n == "final":
                assert at > start or torch.equal(g[0], w[0]), (n, at)
            elif n == "dh0":
                assert at < start or torch.equal(g[0], w[0]), (n, at)
            elif at < start:
                assert torch.equal(g[0, hi:], w[0, hi:]), (n, at)
            else:
                assert torch.equal(g[0, :lo], w[0, :lo]), (n, at)
        assert not torch.isfinite(got["final"][0, 0]).all() or at < start, at


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("B,L,H,start", [(2, 260, 2, 70), (1, 2100, 1, 1000)])
def test_states_stay_in_their_sequences(B, L, H, start, bad, dtype):
    s = _inputs(B, L, H, 1, 32, 64, dtype, seed=32)
    seq = _two(B, L, start)
    Q = 64 if dtype == BF16 else 32
    lo, hi = start // Q * Q, -(-start // Q) * Q
    clean = _run(s, 1.0, seq)
    for name in ("h0", "dhT"):
        t = dict(s, **{name: s[name].clone()})
        t[name][0, 0, 3, 5] = bad
        got = _run(t, 1.0, seq)
        assert torch.equal(got["y"][0, hi:], clean["y"][0, hi:]) and torch.equal(got["final"], clean["final"]), name
        if name == "h0":  # every gradient of its sequence's tokens may see it, no other one
            for n in GRADS[:-1]:
                assert torch.equal(got[n][0, hi:], clean[n][0, hi:]), n
        else:
            assert torch.equal(got["y"], clean["y"]) and torch.equal(got["dh0"], clean["dh0"])
            for n in GRADS[:-1]:
                assert torch.equal(got[n][0, :lo], clean[n][0, :lo]), n
