"""GPU tests that a NaN or infinity of one packed sequence stays within the chunks (of 128 tokens at
most) that the sequence has tokens in: all other tokens keep the bits that they have without it."""
import pytest
import torch

from test_gpu_c_scan_bwd import BF16, F32, _inputs, _run

pytestmark = pytest.mark.gpu
CUTS = (200, 420)  # starts inside chunks 1 and 3 of 128 tokens, 3 and 6 of 64
NAMES = ("dx", "ddt", "dB", "dC")


def _rows(got):
    dx, ddt, _, dB, dC, dh0 = got
    return dict(dx=dx, ddt=ddt, dB=dB, dC=dC), dh0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("B,H,G,P,N,dtype", [(1, 2, 1, 64, 128, BF16), (1, 4, 2, 64, 64, BF16),
                                             (2, 48, 1, 64, 64, BF16), (1, 2, 1, 32, 64, BF16),
                                             (1, 2, 1, 16, 16, F32), (1, 2, 2, 24, 8, F32)])
def test_bad_sequence(B, H, G, P, N, dtype, bad):
    L = 1400
    i = _inputs(B, L, H, G, P, N, dtype, True, seed=31 + N)
    ids = torch.zeros(B, L, dtype=torch.int32)
    for c in CUTS:
        ids[:, c:] += 1
    i["seq"] = ids
    clean, clean_h = _rows(_run(i))
    # the middle sequence, its last token among the bad ones; then what comes in from both ends
    cases = [(k, slice(CUTS[0] + 3, CUTS[1], 9), 128, 512) for k in ("x", "Bm", "Cm", "dy")]
    cases += [(k, slice(CUTS[0], CUTS[0] + 1), 128, 512) for k in ("dy", "Cm")]
    cases += [(k, slice(CUTS[1] - 1, CUTS[1]), 128, 512) for k in ("x", "Bm")]
    cases += [("h0", slice(None), 0, 256), ("dhT", slice(None), 384, L)]
    for key, where, lo, hi in cases:
        j = dict(i)
        j[key] = i[key].clone()
        j[key][:, where] = bad
        got, got_h = _rows(_run(j))
        torch.cuda.synchronize()
        for name in NAMES:
            for k in (slice(0, lo), slice(hi, L)):
                assert torch.equal(got[name][:, k], clean[name][:, k]), (key, name, k)
        if key != "h0":
            assert torch.equal(got_h, clean_h), key


@pytest.mark.parametrize("P,N,dtype", [(64, 128, BF16), (16, 16, F32)])
def test_start_on_a_chunk_edge(P, N, dtype):
    """A start on the first token of a chunk: nothing of the sequence before it has a token there, nor
    of it in the chunk before."""
    L = 600
    i = _inputs(1, L, 2, 1, P, N, dtype, True, seed=3)
    ids = torch.zeros(1, L, dtype=torch.int32)
    ids[:, 256:] = 1
    i["seq"] = ids
    clean, clean_h = _rows(_run(i))
    for key, t, keep in (("x", 255, slice(256, L)), ("Bm", 255, slice(256, L)), ("dy", 256, slice(0, 256)),
                         ("Cm", 256, slice(0, 256))):
        j = dict(i)
        j[key] = i[key].clone()
        j[key][:, t] = float("nan")
        got, got_h = _rows(_run(j))
        torch.cuda.synchronize()
        for name in NAMES:
            assert torch.equal(got[name][:, keep], clean[name][:, keep]), (key, name)
        assert torch.equal(got_h, clean_h)
