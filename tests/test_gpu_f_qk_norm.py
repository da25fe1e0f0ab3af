"""GPU parity of ssm_qk_norm_fwd / _bwd against their formulas in 64 bits, and a layer that uses them
together with the conv, the gated delta rule and the output norm."""
import pytest
import torch

from delta_ref import U, check_delta, check_qk, delta64, qk_norm64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _cuda(t):
    return None if t is None else t.to("cuda")


def _inputs(B, L, HQ, HK, D, R, dtype, weights=True, seed=0, far=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = dict(q=(3 * r(B, L, HQ, D)).to(dtype), k=r(B, L, HK, D).to(dtype), wq=None, wk=None, freq=None, pos=None,
             dq=r(B, L, HQ, D).to(dtype), dk=r(B, L, HK, D).to(dtype))
    if weights:
        s["wq"], s["wk"] = 1 + 0.3 * r(D), 1 + 0.3 * r(D)
    if R:
        s["freq"] = 10000.0 ** (-torch.arange(R // 2, dtype=F32) / (R // 2))
        if far:
            s["pos"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, L), generator=g).to(torch.int32)
    return s


def _run(s, how):
    import ssm_sequence_models_amd as ssm
    c = {n: _cuda(t) for n, t in s.items()}
    args = dict(how, q_weight=c["wq"], k_weight=c["wk"], inv_freq=c["freq"], positions=c["pos"])
    q, k = ssm.qk_norm_fwd(c["q"], c["k"], **args)
    dq, dk, dwq, dwk = ssm.qk_norm_bwd(c["q"], c["k"], c["dq"], c["dk"], **args)
    torch.cuda.synchronize()
    return q, k, dq, dk, dwq, dwk


def _compare(s, kind="l2", eps=1e-6, interleaved=False):
    q, k, dq, dk, dwq, dwk = _run(s, dict(kind=kind, eps=eps, interleaved=interleaved))
    for x, w, dy, out, dx, dw in ((s["q"], s["wq"], s["dq"], q, dq, dwq), (s["k"], s["wk"], s["dk"], k, dk, dwk)):
        ref = qk_norm64(x, w, eps, kind, s["freq"], s["pos"], interleaved, dy)
        D = x.shape[3]
        check_qk(out, ref, "out", x.dtype, D)
        check_qk(dx, ref, "dx", x.dtype, D)
        if w is None:
            assert dw is None
        else:
            check_qk(dw, ref, "dw", F32, D, x[..., 0].numel())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,R", [(1, 0), (2, 2), (7, 4), (8, 8), (32, 32), (64, 0), (64, 24), (80, 40), (96, 96), (128, 64), (130, 18), (192, 192), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_widths(D, R, interleaved, dtype):
    _compare(_inputs(2, 5, 3, 2, D, R, dtype, seed=D), "rms" if D % 3 else "l2", interleaved=interleaved)


@pytest.mark.parametrize("B,L,HQ,HK", [(1, 1, 1, 1), (256, 1, 4, 4), (2, 2050, 3, 1), (1, 33, 24, 2), (3, 7, 1, 5)])
def test_sizes(B, L, HQ, HK):
    _compare(_inputs(B, L, HQ, HK, 64, 32, BF16, seed=L), "rms")
    _compare(_inputs(B, L, HQ, HK, 40, 40, F32, weights=L % 2 == 0, seed=L), "l2", interleaved=True)


def test_many_tokens():
    """More tokens than the blocks take at once."""
    _compare(_inputs(3, 9001, 1, 1, 16, 8, BF16, seed=3))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_positions(dtype):
    """Any int32 position: the angles are those of the product, not of its rounding."""
    s = _inputs(2, 40, 2, 2, 64, 64, dtype, seed=4, far=True)
    s["pos"][0, :4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, -1], dtype=torch.int32)
    _compare(s)


@pytest.mark.parametrize("kind", ["l2", "rms"])
def test_zero_heads_and_large_values(kind):
    s = _inputs(1, 6, 2, 2, 32, 16, F32, seed=5)
    s["q"][:, 1] = 0.0
    s["k"][:, 2] *= 1e15
    s["k"][:, 3] *= 1e-15
    _compare(s, kind, eps=0.0)
    q, k, dq, dk, _, _ = _run(s, dict(kind=kind, eps=0.0))
    assert not q[:, 1].any() and not dq[:, 1].any()


def test_nan_stays_in_its_head():
    s = _inputs(1, 9, 2, 2, 64, 32, BF16, weights=False, seed=6)
    clean = _run(s, {})
    s["q"][0, 4, 1, 3] = float("nan")
    got = _run(s, {})
    for a, b in zip(got[:4], clean[:4]):
        a, b = a.clone(), b.clone()
        a[0, 4, 1] = b[0, 4, 1] = 0
        assert torch.equal(a, b)
    assert torch.isnan(got[0][0, 4, 1]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,R,interleaved", [(64, 64, False), (80, 36, False), (48, 48, True)])
def test_strided_and_in_place(D, R, interleaved, dtype):
    """Channel ranges of a wider tensor at an odd offset, results in place of their inputs: the same
    bits as dense calls, nothing else touched."""
    import ssm_sequence_models_amd as ssm
    B, L, HQ, HK = 2, 21, 3, 2
    s = {n: _cuda(t) for n, t in _inputs(B, L, HQ, HK, D, R, dtype, seed=7).items()}
    how = dict(q_weight=s["wq"], k_weight=s["wk"], inv_freq=s["freq"], interleaved=interleaved, kind="rms")
    want = ssm.qk_norm_fwd(s["q"], s["k"], **how)
    wantg = ssm.qk_norm_bwd(s["q"], s["k"], s["dq"], s["dk"], **how)
    n = (HQ + HK) * D

    def wide(a, b):
        w = torch.full((B, L, n + 5), 9.0, device="cuda", dtype=dtype)[..., 1:]
        parts = w[..., :HQ * D].unflatten(-1, (HQ, D)), w[..., HQ * D:n].unflatten(-1, (HK, D))
        parts[0].copy_(a)
        parts[1].copy_(b)
        return w, parts

    w, (q, k) = wide(s["q"], s["k"])
    wd, (dq, dk) = wide(s["dq"], s["dk"])
    grads = ssm.qk_norm_bwd(q, k, dq, dk, dq=dq, dk=dk, **how)
    out = ssm.qk_norm_fwd(q, k, q_out=q, k_out=k, **how)
    for a, b in zip((*out, *grads), (*want, *wantg)):
        assert torch.equal(a, b)
    assert bool((w[..., n:] == 9.0).all()) and bool((wd[..., n:] == 9.0).all())


def test_positions_default():
    import ssm_sequence_models_amd as ssm
    s = {n: _cuda(t) for n, t in _inputs(3, 50, 2, 1, 32, 32, BF16, seed=8).items()}
    at = torch.arange(50, device="cuda", dtype=torch.int32).expand(3, 50).contiguous()
    a = ssm.qk_norm_fwd(s["q"], s["k"], inv_freq=s["freq"])
    b = ssm.qk_norm_fwd(s["q"], s["k"], inv_freq=s["freq"], positions=at)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_no_tokens():
    import ssm_sequence_models_amd as ssm
    z, w = torch.zeros(2, 0, 3, 8, device="cuda"), torch.ones(8, device="cuda")
    q, k = ssm.qk_norm_fwd(z, z)
    assert q.shape == z.shape and k.shape == z.shape
    _, _, dwq, dwk = ssm.qk_norm_bwd(z, z, z, z, q_weight=w, k_weight=w)
    assert not dwq.any() and not dwk.any()


def test_gradient_against_differences():
    s = _inputs(1, 3, 2, 1, 12, 8, F32, seed=9)
    got = _run(s, dict(kind="rms"))

    def loss(p):
        f = lambda x, w, d: float((qk_norm64(x, w, 1e-6, "rms", s["freq"], None, False)["out"] * d.double()).sum())  # noqa: E731
        return f(p["q"], p["wq"], s["dq"]) + f(p["k"], p["wk"], s["dk"])

    g = torch.Generator().manual_seed(10)
    for n, grad in (("q", got[2]), ("k", got[3]), ("wq", got[4]), ("wk", got[5])):
        d = torch.randn(s[n].shape, generator=g, dtype=torch.float64)
        up, down = (loss(dict(s, **{n: s[n].double() + f * 1e-5 * d})) for f in (1, -1))
        have = float((grad.cpu().double() * d).sum())
        size = float((grad.cpu().double().abs() * d.abs()).sum())
        assert abs(have - (up - down) / 2e-5) <= 1e-5 * size, n


def test_graph_replay_and_streams():
    import ssm_sequence_models_amd as ssm
    s = {n: _cuda(t) for n, t in _inputs(2, 600, 4, 2, 64, 32, BF16, seed=11).items()}
    how = dict(q_weight=s["wq"], k_weight=s["wk"], inv_freq=s["freq"])

    def work():
        return (*ssm.qk_norm_fwd(s["q"], s["k"], **how), *ssm.qk_norm_bwd(s["q"], s["k"], s["dq"], s["dk"], **how))

    want = work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for i in range(4):
        s["q"].normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, work())), i


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layer_training_step_and_decode(dtype):
    """A layer as it is used: conv over q | k | v, the heads' norm with positions, the gated delta
    rule, the gated output norm; its backward down to the conv's input; and single tokens on the
    pools.  Every stage against the 64-bit form of that stage on the stage's own inputs, and the
    decode against the prefill's next tokens."""
    import ssm_sequence_models_amd as ssm
    from train_ref import assert_bound, norm64
    B, L, H, G, P, N, K, R = 2, 75, 4, 2, 32, 32, 4, 16
    C = 2 * G * N + H * P
    g = torch.Generator().manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, w, bias = r(B, L, C).to(dtype), r(C, K) * 0.5, r(C) * 0.1
    beta, gate = torch.sigmoid(r(B, L, H)), -torch.rand(B, L, H, generator=g).cuda()
    z, wn, dout = r(B, L, H * P).to(dtype), 1 + 0.1 * r(H * P), r(B, L, H * P).to(dtype)
    wq, wk = 1 + 0.1 * r(N), 1 + 0.1 * r(N)
    freq = (100.0 ** (-torch.arange(R // 2, dtype=F32) / (R // 2))).cuda()
    pos = (torch.arange(L).expand(B, L) + 1000).to(torch.int32).cuda().contiguous()
    how = dict(q_weight=wq, k_weight=wk, inv_freq=freq, positions=pos)

    def split(t):
        return (t[..., :G * N].unflatten(-1, (G, N)), t[..., G * N:2 * G * N].unflatten(-1, (G, N)),
                t[..., 2 * G * N:].unflatten(-1, (H, P)))

    # forward
    c, conv_state = ssm.conv1d_fwd(x, w, bias, activation="silu")
    q0, k0, v = split(c)
    q, k = ssm.qk_norm_fwd(q0, k0, **how)
    y, state = ssm.delta_scan_fwd(q, k, v, beta, gate=gate, scale=N ** -0.5)
    out = ssm.norm_fwd(y.view(B, L, H * P), wn, z=z)
    # backward, the gradients of q, k and v straight into the conv's
    dy, dz, dwn, _ = ssm.norm_bwd(y.view(B, L, H * P), wn, dout, z=z)
    dc = torch.empty_like(c)
    dq0, dk0, dv = split(dc)
    dqn, dkn, _, dbeta, dgate, _ = ssm.delta_scan_bwd(q, k, v, beta, dy.view(B, L, H, P), gate=gate, scale=N ** -0.5, dv=dv)
    _, _, dwq, dwk = ssm.qk_norm_bwd(q0, k0, dqn, dkn, dq=dq0, dk=dk0, **how)
    dx, _, dw, db = ssm.conv1d_bwd(x, w, bias, dc, activation="silu")
    torch.cuda.synchronize()
    cpu = lambda t: t.detach().cpu()  # noqa: E731
    for x1, w1, o, do, dx1, dw1 in ((q0, wq, q, dqn, dq0, dwq), (k0, wk, k, dkn, dk0, dwk)):
        ref = qk_norm64(cpu(x1), cpu(w1), 1e-6, "l2", cpu(freq), cpu(pos), False, cpu(do))
        check_qk(o, ref, "out", dtype, N)
        check_qk(dx1, ref, "dx", dtype, N)
        check_qk(dw1, ref, "dw", F32, N, B * L * G)
    ref = delta64(*map(cpu, (q, k, v, beta, gate)), N ** -0.5, None, None, cpu(dy).view(B, L, H, P))
    for n, t in (("y", y), ("final", state), ("dq", dqn), ("dk", dkn), ("dv", dv), ("dbeta", dbeta), ("dgate", dgate)):
        check_delta(t, ref, n, F32 if n in ("final", "dbeta", "dgate") else dtype, N + P + 256, 3)
    ref = norm64(cpu(y).view(B * L, H * P), cpu(wn), None, cpu(z).view(B * L, -1), 1e-5, "rms", 1, False)
    half = 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2
    assert_bound(out.view(B * L, -1), ref["out"], (H * P + 40) * U * ref["out_mag"] + half * ref["out"].abs() + 1e-30, "out")
    assert dx.shape == x.shape and torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()

    # decode: three more tokens on the pools, against the row with them in it
    T = 3
    more = r(B, T, C).to(dtype)
    beta2, gate2 = torch.sigmoid(r(B, T, H)), -torch.rand(B, T, H, generator=g).cuda()
    pool = torch.zeros(4, C, K - 1, device="cuda", dtype=dtype)
    states = torch.zeros(4, H, P, N, device="cuda")
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    pool[slots.long()], states[slots.long()] = conv_state, state
    got = []
    for t in range(T):
        cs = ssm.conv1d_update(more[:, t, :, None].contiguous(), pool, w, bias, conv_state_indices=slots, activation="silu")
        qs, ks, vs = split(cs.transpose(1, 2).contiguous())
        at = torch.full((B, 1), 1000 + L + t, dtype=torch.int32, device="cuda")
        ssm.qk_norm_fwd(qs, ks, q_out=qs, k_out=ks, q_weight=wq, k_weight=wk, inv_freq=freq, positions=at)
        got.append(ssm.delta_scan_step(qs, ks, vs, beta2[:, t:t + 1].contiguous(), states, gate=gate2[:, t:t + 1].contiguous(),
                                       scale=N ** -0.5, state_indices=slots))
    c2, _ = ssm.conv1d_fwd(more, w, bias, initial_state=conv_state, activation="silu")
    q2, k2, v2 = split(c2)
    pos2 = (torch.arange(T).expand(B, T) + 1000 + L).to(torch.int32).cuda().contiguous()
    q2, k2 = ssm.qk_norm_fwd(q2, k2, **dict(how, positions=pos2))
    ref = delta64(*map(cpu, (q2, k2, v2, beta2, gate2)), N ** -0.5, cpu(state), None)
    check_delta(torch.cat(got, 1), ref, "y", dtype, N + P + 256, 3)
    check_delta(states[slots.long()], ref, "final", F32, N + P + 256, 3)
    assert not states[[1, 3]].any()
