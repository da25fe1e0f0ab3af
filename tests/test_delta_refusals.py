"""Refusals of the gated delta rule and of the queries' and keys' norm, on the CPU: status codes of the
C entry points for arguments that fail their host-side checks (no call reaches a launch), the Python
layer's own, workspace sizes, and the 64-bit plain forms against autograd."""
import ctypes

import pytest
import torch

from delta_ref import delta64, qk_norm64

P = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(257)
FOUR = ctypes.c_void_p(260)
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    import ssm_sequence_models_amd as s
    return s._lib


def _lead(a):
    return [a.get("q", P), a.get("q_row", 64), a.get("k", P), a.get("k_row", 64), a.get("v", P), a.get("v_row", 128),
            a.get("beta", P), a.get("gate"), F(a.get("scale", 1.0))]


def _sizes(a):
    return [a.get("b", 2), a.get("L", 70), a.get("H", 4), a.get("P", 32), a.get("G", 2), a.get("N", 32)]


def _fwd(lib, **a):
    return lib.ssm_delta_scan_fwd(*_lead(a), a.get("h0"), a.get("hT"), a.get("seq"), a.get("y", P), a.get("y_row", 128),
                                  *_sizes(a), a.get("dtype", 1), a.get("ws", P), a.get("wsb", 1 << 40), None)


def _bwd(lib, **a):
    return lib.ssm_delta_scan_bwd(*_lead(a), a.get("dy", P), a.get("dy_row", 128), a.get("h0"), a.get("dhT"), a.get("seq"),
                                  a.get("dq", P), a.get("dq_row", 64), a.get("dk", P), a.get("dk_row", 64),
                                  a.get("dv", P), a.get("dv_row", 128), a.get("dbeta", P), a.get("dgate"), a.get("dh0"),
                                  *_sizes(a), a.get("dtype", 1), a.get("ws", P), a.get("wsb", 1 << 40), None)


def _step(lib, **a):
    return lib.ssm_delta_scan_step(*_lead(a), a.get("state", P), a.get("idx"), a.get("y", P), a.get("y_row", 128),
                                   *_sizes(a), a.get("slots", 3), a.get("dtype", 1), None)


COMMON = ((1, dict(dtype=7)), (1, dict(b=-1)), (1, dict(L=-1)), (1, dict(H=0)), (1, dict(P=0)), (1, dict(G=0)),
          (1, dict(N=0)), (1, dict(G=3)), (2, dict(N=30)), (2, dict(N=260)), (2, dict(P=65537)),
          (1, dict(scale=float("nan"))), (1, dict(scale=float("inf"))), (2, dict(b=1 << 31)), (2, dict(L=1 << 31)),
          (2, dict(b=1 << 20, H=1 << 12, G=1)), (2, dict(b=1 << 15, L=1 << 20, H=64)), (1, dict(q=None)), (1, dict(k=None)),
          (1, dict(v=None)), (1, dict(beta=None)), (3, dict(q=ODD)), (3, dict(k=ODD)), (3, dict(v=ODD)), (3, dict(beta=ODD)),
          (3, dict(gate=ODD)), (1, dict(q_row=-1)), (1, dict(k_row=-64)), (1, dict(v_row=-1)))


@pytest.mark.parametrize("call,more", [
    (_fwd, ((1, dict(y=None)), (3, dict(y=ODD)), (1, dict(y_row=127)), (3, dict(h0=FOUR)), (3, dict(hT=FOUR)), (3, dict(seq=ODD)),
            (4, dict(ws=None)), (4, dict(wsb=100)), (4, dict(ws=FOUR)))),
    (_bwd, ((1, dict(dy=None)), (1, dict(dq=None)), (1, dict(dk=None)), (1, dict(dv=None)), (1, dict(dbeta=None)),
            (3, dict(dgate=ODD)), (1, dict(dq_row=63)), (1, dict(dk_row=63)), (1, dict(dv_row=127)), (1, dict(dy_row=-1)),
            (3, dict(dhT=FOUR)), (3, dict(dh0=FOUR)), (1, dict(dhT=P, dh0=P)), (4, dict(ws=None)), (4, dict(wsb=100)), (4, dict(ws=FOUR)))),
    (_step, ((1, dict(state=None)), (3, dict(state=FOUR)), (3, dict(idx=ODD)), (1, dict(slots=0)), (1, dict(y=None)), (1, dict(y_row=127))))])
def test_delta_refusals(lib, call, more):
    for status, how in COMMON + more:
        assert call(lib, **how) == status, how
        assert lib.ssm_last_error()


def test_delta_nothing_to_do(lib):
    none = dict(q=None, k=None, v=None, beta=None, y=None, dy=None, dq=None, dk=None, dv=None, dbeta=None, ws=None, state=None)
    assert _step(lib, L=0, **none) == 0 and _step(lib, b=0, **none) == 0
    assert _fwd(lib, b=0, **none) == 0 and _bwd(lib, b=0, **none) == 0


def test_delta_workspace_sizes():
    import ssm_sequence_models_amd as s
    f, b = s.delta_scan_fwd_workspace_size, s.delta_scan_bwd_workspace_size
    for size in (f, b):
        assert size(0, 64, 4, 64, 2, 64) == 0 and size(2, 0, 4, 64, 2, 64) == 0
        assert size(2, 64, 4, 64, 3, 64) == 0 and size(2, 64, 4, 64, 2, 62) == 0
        assert size(1 << 20, 1 << 20, 1 << 12, 64, 1, 64) == 0 and size(1 << 62, 1, 4, 64, 2, 64) == 0
        assert 0 < size(2, 64, 4, 64, 2, 64) <= size(2, 65, 4, 64, 2, 64) <= size(2, 128, 4, 64, 2, 64)
        assert size(1, 100, 2, 16, 1, 16, torch.float32) > 0


def _qk(lib, bwd, **a):
    lead = [a.get("q", P), a.get("q_row", 128), a.get("k", P), a.get("k_row", 64), a.get("wq"), a.get("wk"), a.get("freq"), a.get("pos")]
    tail = [a.get("b", 2), a.get("L", 5), a.get("HQ", 4), a.get("HK", 2), a.get("D", 32), a.get("R", 0), 0, F(a.get("eps", 1e-6)),
            a.get("kind", 0), a.get("dtype", 1), None]
    if not bwd:
        return lib.ssm_qk_norm_fwd(*lead, a.get("qo", P), a.get("qo_row", 128), a.get("ko", P), a.get("ko_row", 64), *tail)
    return lib.ssm_qk_norm_bwd(*lead, a.get("dqo", P), a.get("dqo_row", 128), a.get("dko", P), a.get("dko_row", 64), a.get("qo", P),
                               a.get("qo_row", 128), a.get("ko", P), a.get("ko_row", 64), a.get("dwq"), a.get("dwk"), a.get("ws"),
                               a.get("wsb", 0), *tail)


@pytest.mark.parametrize("bwd", [False, True])
def test_qk_norm_refusals(lib, bwd):
    for status, how in ((1, dict(dtype=5)), (1, dict(kind=2)), (1, dict(b=-1)), (1, dict(L=-1)), (1, dict(HQ=0)), (1, dict(HK=0)),
                        (1, dict(D=0)), (2, dict(D=257)), (1, dict(R=-2)), (1, dict(R=3, freq=P)), (1, dict(R=34, freq=P)),
                        (1, dict(R=8)), (1, dict(eps=-1.0)), (1, dict(eps=float("nan"))), (2, dict(b=1 << 31)),
                        (2, dict(b=1 << 16, L=1 << 16)), (2, dict(HQ=1 << 24)), (1, dict(q=None)), (1, dict(k=None)), (3, dict(q=ODD)),
                        (3, dict(wq=ODD)), (3, dict(freq=ODD, R=8)), (3, dict(pos=ODD)), (1, dict(qo=None)), (1, dict(ko=None)),
                        (1, dict(q_row=-1)), (1, dict(qo_row=127)), (1, dict(ko_row=63))):
        assert _qk(lib, bwd, **how) == status, how
        assert lib.ssm_last_error()
    if bwd:
        assert _qk(lib, True, dqo=None) == 1 and _qk(lib, True, dko_row=-1) == 1
        assert _qk(lib, True, dwq=P) == 4 and _qk(lib, True, dwk=P, ws=P, wsb=64) == 4
    assert _qk(lib, bwd, b=0, q=None, k=None, qo=None, ko=None, dqo=None, dko=None) == 0


def test_qk_norm_workspace_size():
    import ssm_sequence_models_amd as s
    f = s.qk_norm_bwd_workspace_size
    assert f(0, 5, 64) == 0 and f(2, 0, 64) == 0 and f(2, 5, 257) == 0 and f(1 << 62, 2, 64) == 0
    assert f(2, 5, 64) == 10 * 2 * 64 * 4 and f(4, 8192, 128) == 1024 * 2 * 128 * 4


def test_python_refusals(monkeypatch):
    import ssm_sequence_models_amd as s
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU tensor"):
        s.delta_scan_fwd(z(1, 2, 1, 8), z(1, 2, 1, 8), z(1, 2, 2, 4), z(1, 2, 2))
    with pytest.raises(ValueError, match="GPU tensor"):
        s.qk_norm_fwd(z(1, 2, 1, 8), z(1, 2, 1, 8))
    real = s._need

    def need(t, name, *a, **k):  # every other check, on tensors of the CPU
        if t is not None:
            class On:
                is_cuda = True
                def __getattr__(self, n):
                    return getattr(t, n)
            real(On(), name, *a, **k)
    monkeypatch.setattr(s, "_need", need)
    ok = dict(q=z(1, 2, 1, 8), k=z(1, 2, 1, 8), v=z(1, 2, 2, 4), beta=z(1, 2, 2))
    for how, text in ((dict(q=z(1, 2, 8)), "must be"), (dict(q=z(1, 2, 1, 12)), "shape"), (dict(v=z(1, 2, 3, 4), q=z(1, 2, 2, 8), k=z(1, 2, 2, 8)), "multiple"),
                      (dict(beta=z(1, 2, 1)), "shape"), (dict(gate=z(2, 2, 2)), "shape"), (dict(k=z(1, 2, 1, 16)[..., ::2]), "side by side"),
                      (dict(k=z(1, 2, 1, 8).bfloat16()), "must be"), (dict(initial_state=z(1, 2, 4, 4)), "shape"),
                      (dict(seq_idx=z(1, 3, dtype=torch.int32)), "shape"), (dict(y=z(1, 2, 2, 5)), "shape"),
                      (dict(q=z(2, 5, 1, 8)[:, :2], k=z(2, 2, 1, 8), v=z(2, 2, 2, 4), beta=z(2, 2, 2)), "one stride")):
        with pytest.raises((ValueError, TypeError), match=text):
            s.delta_scan_fwd(**{**ok, **how})
    with pytest.raises(ValueError, match="dgate given without gate"):
        s.delta_scan_bwd(**ok, dy=z(1, 2, 2, 4), dgate=z(1, 2, 2))
    with pytest.raises(ValueError, match="state must be"):
        s.delta_scan_step(**ok, state=z(3, 2, 4, 9))
    qk = dict(q=z(1, 2, 3, 8), k=z(1, 2, 1, 8))
    for how, text in ((dict(kind="layer"), "kind"), (dict(k=z(1, 2, 1, 9)), "shape"), (dict(q_weight=z(7)), "shape"),
                      (dict(inv_freq=z(5)), "pairs"), (dict(positions=z(1, 2, dtype=torch.int32)), "without inv_freq"),
                      (dict(inv_freq=z(2), positions=z(1, 3, dtype=torch.int32)), "shape"),
                      (dict(inv_freq=z(2), positions=z(1, 2, dtype=torch.int64)), "int32"), (dict(q_out=z(1, 2, 3, 9)), "shape")):
        with pytest.raises((ValueError, TypeError), match=text):
            s.qk_norm_fwd(**{**qk, **how})
    with pytest.raises(ValueError, match="without q_weight"):
        s.qk_norm_bwd(**qk, dq_out=z(1, 2, 3, 8), dk_out=z(1, 2, 1, 8), dq_weight=z(8))


def test_plain_delta_against_autograd():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    B, L, H, G, Pn, N = 2, 9, 4, 2, 3, 5
    p = dict(q=r(B, L, G, N), k=r(B, L, G, N) * 0.4, v=r(B, L, H, Pn), beta=torch.sigmoid(r(B, L, H)),
             gate=-r(B, L, H).abs(), h0=r(B, H, Pn, N))
    seq = torch.tensor([[0] * 4 + [1] * 5, [0] * 9], dtype=torch.int32)
    dy, dhT = r(B, L, H, Pn), r(B, H, Pn, N)
    for t in p.values():
        t.requires_grad_(True)
    h, ys = p["h0"], []
    for t in range(L):
        a = torch.exp(p["gate"][:, t])[..., None, None]
        if t:
            a = a * (seq[:, t] == seq[:, t - 1]).double()[:, None, None, None]
        kt, qt = (p[n][:, t].repeat_interleave(H // G, 1)[..., None] for n in ("k", "q"))
        h = a * h
        h = h + p["beta"][:, t, :, None, None] * (p["v"][:, t, :, :, None] - h @ kt) @ kt.mT
        ys.append((0.6 * h @ qt)[..., 0])
    ((torch.stack(ys, 1) * dy).sum() + (h * dhT).sum()).backward()
    d = {n: t.detach() for n, t in p.items()}
    ref = delta64(d["q"], d["k"], d["v"], d["beta"], d["gate"], 0.6, d["h0"], seq, dy, dhT)
    assert torch.allclose(ref["y"], torch.stack(ys, 1).detach(), atol=1e-12) and torch.allclose(ref["final"], h.detach(), atol=1e-12)
    for n in p:
        assert torch.allclose(ref["d" + n], p[n].grad, atol=1e-10), n


@pytest.mark.parametrize("kind,interleaved", [("l2", False), ("rms", True)])
def test_plain_qk_norm_against_autograd(kind, interleaved):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 3, 2, 8, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(8, generator=g, dtype=torch.float64, requires_grad=True)
    freq, dy = torch.tensor([1.0, 0.1, 0.01]), torch.randn(2, 3, 2, 8, generator=g, dtype=torch.float64)
    s = (x * x).sum(-1, keepdim=True) if kind == "l2" else (x * x).mean(-1, keepdim=True)
    m = x / (s + 1e-3).sqrt() * w
    ang = (torch.arange(3)[:, None].double() * freq.double())[None, :, None]
    i = torch.arange(3)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 3)
    c = torch.complex(m[..., a], m[..., b]) * torch.polar(torch.ones_like(ang), ang)
    y = torch.zeros_like(m)
    y = y.index_copy(3, a, c.real).index_copy(3, b, c.imag).index_copy(3, torch.tensor([6, 7]), m[..., 6:])
    (y * dy).sum().backward()
    ref = qk_norm64(x.detach(), w.detach(), 1e-3, kind, freq, None, interleaved, dy)
    assert torch.allclose(ref["out"], y.detach(), atol=1e-12)
    assert torch.allclose(ref["dx"], x.grad, atol=1e-12) and torch.allclose(ref["dw"], w.grad, atol=1e-12)
    assert bool((ref["out_mag"] >= ref["out"].abs() - 1e-12).all())
