"""GPU parity of ssm_scan_bwd against the definition in 64 bits, token by token.

Bounds: a value is a sum of products; with fp32 products and sums its error is below the
number of roundings on the way times half a step of the magnitudes it is made of.  On the way
lie at most: the contraction over dstate or headdim (N + P), the 64 tokens of a chunk, two
roundings a chunk along the row (chunks on both sides), the group's heads, and the factors
(exponentials of differences, each below 16 half-steps where it is not negligible; four of
them and the products): K = N + P + 64 + 2 chunks + heads + 128.  Outputs in bf16 add half a
step of bf16, and the operands that the bf16 matrix cores take in two parts each 2^-16 of the
magnitude (half a step of the second part of a value split in two), two such operands a term.
"""
import pytest
import torch

from train_ref import U, assert_bound, half_step, scan_bwd64, scan_loss64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("dx", "ddt", "dA", "dB", "dC", "dh0")


def _inputs(B, L, H, G, P, N, dtype, states, seed, A=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    i = dict(x=r(B, L, H, P).to(dtype), dt=torch.nn.functional.softplus(r(B, L, H) - 2.0),
             A=-torch.exp(torch.rand(H, generator=g) * 2.77) if A is None else A,
             Bm=r(B, L, G, N).to(dtype), Cm=r(B, L, G, N).to(dtype), dy=r(B, L, H, P).to(dtype),
             h0=None, dhT=None, seq=None)
    if states:
        i["h0"], i["dhT"] = r(B, H, P, N), r(B, H, P, N)
    return i


def _seq(B, L, kind, seed):
    if kind is None:
        return None
    if kind == "every":
        return torch.arange(L, dtype=torch.int32).expand(B, L).contiguous()
    ids = torch.zeros(B, L, dtype=torch.int32)
    if kind == "edges":  # starts on the edges of tiles and chunks and beside them
        for at in (1, 15, 16, 17, 63, 64, 65, 127, 128, 191, 193):
            if at < L:
                ids[:, at:] += 1
        return ids
    if kind == "back":   # ids that come back
        return ((torch.arange(L) // 7) % 2).to(torch.int32).expand(B, L).contiguous()
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(B, L, generator=g) < 3.0 / L).int().cumsum(1).to(torch.int32).contiguous()


def _run(i, **kw):
    import ssm_sequence_models_amd as ssm
    c = {k: None if v is None else v.cuda() for k, v in i.items()}
    return ssm.scan_bwd(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], c["dy"], initial_state=c["h0"],
                        dfinal_state=c["dhT"], seq_idx=c["seq"], **kw)


def _check(got, ref, i):
    B, L, H, P = i["x"].shape
    G, N = i["Bm"].shape[2:]
    K = N + P + 64 + 4 * (L // 64 + 1) + H // G + 128
    for name, t in zip(NAMES, got):
        own = name in ("dx", "dB", "dC") and i["x"].dtype == BF16
        h = half_step(BF16 if own else F32)
        k = K * U + (2 * 2.0 ** -16 if own else 0.0)
        if name == "dA":
            k += 2 * U  # its long sums are in double
        assert_bound(t, ref[name], h * ref[name].abs() + (1 + h) * k * ref[name + "_mag"] + 1e-30, name)


def _compare(i):
    got = _run(i)
    torch.cuda.synchronize()
    _check(got, scan_bwd64(**i), i)


SHAPES = [  # H, G, P, N
    (1, 1, 4, 4), (2, 1, 64, 128), (4, 2, 64, 64), (3, 3, 24, 16), (2, 1, 80, 32), (2, 2, 3, 8),
    (1, 1, 128, 128), (1, 1, 64, 256), (2, 1, 1, 4), (6, 2, 32, 64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shapes(shape, dtype):
    for L, states, kind in ((130, True, None), (70, False, "random")):
        i = _inputs(2, L, *shape, dtype, states, seed=L + sum(shape))
        i["seq"] = _seq(2, L, kind, 1)
        _compare(i)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 321])
@pytest.mark.parametrize("N", [64, 128])
def test_lengths(L, N):
    for dtype in (BF16, F32):
        _compare(_inputs(1, L, 2, 1, 64, N, dtype, True, seed=L))


@pytest.mark.parametrize("B,H,G,N", [(2, 48, 1, 64), (1, 95, 1, 64), (2, 50, 2, 128)])
def test_many_heads(B, H, G, N):
    """On both sides of the number of heads from which one block walks over a row's chunks."""
    _compare(_inputs(B, 200, H, G, 64, N, BF16, True, seed=B * H))


@pytest.mark.parametrize("kind", ["every", "edges", "back", "random"])
@pytest.mark.parametrize("dtype,P,N", [(BF16, 64, 128), (BF16, 64, 64), (F32, 16, 16)])
def test_packed(kind, dtype, P, N):
    for states in (True, False):
        i = _inputs(2, 200, 4, 2, P, N, dtype, states, seed=5)
        i["seq"] = _seq(2, 200, kind, 3)
        _compare(i)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decays(dtype):
    """Decays from none to instant, step sizes of zero and a large one in between, and a growing
    state: every factor is an exponential of a difference."""
    for A in ([-1e-4, -1.0], [-40.0, -2000.0], [-1e5, -1e9], [0.0, 0.02]):
        i = _inputs(1, 150, 2, 1, 64, 128, dtype, True, seed=7, A=torch.tensor(A))
        i["dt"][:, 40:50] = 0.0
        i["dt"][:, 100] = 30.0
        _compare(i)


def test_negative_steps():
    i = _inputs(1, 100, 2, 1, 64, 128, BF16, True, seed=8, A=torch.tensor([-0.3, -0.05]))
    i["dt"][:, ::3] *= -1.0
    _compare(i)


def test_many_heads_and_rows():
    """Groups of 1, 7 and 16 heads (heads that do not divide evenly over blocks), many rows."""
    for H, G, B in ((7, 1, 2), (16, 1, 1), (5, 5, 3), (34, 2, 1)):
        i = _inputs(B, 100, H, G, 64, 128, BF16, True, seed=H)
        i["seq"] = _seq(B, 100, "random", 3)
        _compare(i)


def test_long_row():
    """Few heads on one long ragged row (the row cut along its length)."""
    for N in (64, 128):
        i = _inputs(1, 2100, 1, 1, 64, N, BF16, True, seed=N)
        _compare(i)
        i["seq"] = _seq(1, 2100, "random", 4)
        _compare(i)


def test_empty():
    import ssm_sequence_models_amd as ssm
    i = _inputs(2, 0, 2, 1, 64, 128, BF16, True, seed=1)
    got = _run(i)
    assert torch.equal(got[5].cpu(), i["dhT"]) and float(got[2].abs().max()) == 0
    i["dhT"] = None
    assert float(_run(i)[5].abs().max()) == 0
    i = _inputs(0, 5, 2, 1, 64, 128, BF16, True, seed=1)
    assert float(_run(i)[2].abs().max()) == 0


def test_refused_alias():
    import ssm_sequence_models_amd as ssm
    i = _inputs(1, 5, 1, 1, 4, 4, F32, True, seed=1)
    d = i["dhT"].cuda()
    i["dhT"] = d
    with pytest.raises(ssm.SSMError):
        _run(i, dinitial_state=d)


def test_unaligned_inputs():
    """Tensors that start off the 16-byte grid take the general path: same results."""
    i = _inputs(1, 100, 2, 1, 64, 128, BF16, True, seed=11)
    want = scan_bwd64(**i)

    def off(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        v = buf[1:].view(t.shape)
        v.copy_(t)
        return v
    import ssm_sequence_models_amd as ssm
    for which in ("x", "Bm", "Cm", "dy", "dt"):
        c = {k: None if v is None else v.cuda() for k, v in i.items()}
        c[which] = off(i[which])
        _check(ssm.scan_bwd(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], c["dy"], initial_state=c["h0"],
                            dfinal_state=c["dhT"]), want, i)


def test_chunks_continue():
    """Truncated rows: the second call's dinitial_state as the first one's dfinal_state gives the
    whole row's gradients, dA adds up (cut off the 64-token grid)."""
    import ssm_sequence_models_amd as ssm
    i = _inputs(2, 200, 4, 1, 64, 128, BF16, True, seed=13)
    ref = scan_bwd64(**i)
    c = {k: None if v is None else v.cuda() for k, v in i.items()}
    cut = 90
    one = {k: c[k][:, :cut].contiguous() for k in ("x", "dt", "Bm", "Cm", "dy")}
    two = {k: c[k][:, cut:].contiguous() for k in ("x", "dt", "Bm", "Cm", "dy")}
    _, mid = ssm.scan_fwd(one["x"], one["dt"], c["A"], one["Bm"], one["Cm"], initial_state=c["h0"])
    b = ssm.scan_bwd(two["x"], two["dt"], c["A"], two["Bm"], two["Cm"], two["dy"], initial_state=mid,
                     dfinal_state=c["dhT"])
    a = ssm.scan_bwd(one["x"], one["dt"], c["A"], one["Bm"], one["Cm"], one["dy"],
                     initial_state=c["h0"], dfinal_state=b[5])
    got = [torch.cat([p, q], 1) for p, q in zip(a[:2], b[:2])] + [a[2] + b[2]]
    got += [torch.cat([a[3], b[3]], 1), torch.cat([a[4], b[4]], 1), a[5]]
    # the state handed over comes from the forward, whose operands are split in two parts:
    # 2^-16 of the magnitudes for every output that it reaches
    for name, t in zip(NAMES, got):
        own = name in ("dx", "dB", "dC")
        h = half_step(BF16 if own else F32)
        K = 128 + 64 + 64 + 16 + 4 + 128
        assert_bound(t, ref[name], h * ref[name].abs() + (1 + h) * (K * U + 4 * 2.0 ** -16) * ref[name + "_mag"] + 1e-30, name)


def test_initial_state_gradient_agrees():
    """dinitial_state is scan_bwd_initial_state's (both within their bounds of each other)."""
    import ssm_sequence_models_amd as ssm
    i = _inputs(2, 150, 2, 1, 64, 128, BF16, True, seed=17)
    got = _run(i)[5]
    c = {k: None if v is None else v.cuda() for k, v in i.items()}
    other = ssm.scan_bwd_initial_state(c["dt"], c["A"], c["Cm"], c["dy"], dfinal_state=c["dhT"])
    ref = scan_bwd64(**i)
    assert_bound(got, other.cpu().double(), (1024 * U + 4 * 2.0 ** -16) * ref["dh0_mag"] + 1e-30, "dh0")


def test_gradient_against_differences():
    """<gradient, v> against central differences of the 64-bit loss, and all of it against
    torch's differentiation of that loss."""
    i = _inputs(1, 30, 2, 1, 8, 8, F32, True, seed=19)
    i["seq"] = _seq(1, 30, "edges", 1)
    got = dict(zip(NAMES, _run(i)))
    ref = scan_bwd64(**i)
    args = {k: i[k].double() for k in ("x", "dt", "A", "Bm", "Cm", "h0")}
    leaf = {k: v.clone().requires_grad_() for k, v in args.items()}
    loss = scan_loss64(dy=i["dy"].double(), dhT=i["dhT"].double(), seq=i["seq"], **leaf)
    loss.backward()
    g = torch.Generator().manual_seed(3)
    for name, k in (("dx", "x"), ("ddt", "dt"), ("dA", "A"), ("dB", "Bm"), ("dC", "Cm"), ("dh0", "h0")):
        assert torch.allclose(leaf[k].grad, ref[name], rtol=1e-9, atol=1e-9), name
        v = torch.randn(args[k].shape, generator=g, dtype=torch.float64)
        f = []
        for e in (1e-5, -1e-5):
            q = dict(args)
            q[k] = args[k] + e * v
            f.append(float(scan_loss64(dy=i["dy"].double(), dhT=i["dhT"].double(), seq=i["seq"], **q)))
        dot = got[name].cpu().double() * v
        # third-order rest h^2 |f'''| / 6 below 1e-6 of these losses of order 100; fp32 gradients
        assert abs((f[0] - f[1]) / 2e-5 - float(dot.sum())) <= 1e-4 * (1 + float(dot.abs().sum())), name


def test_graph_replay_streams_and_repeat():
    """The same bits from run to run, on another stream, and from every replay of a captured
    graph with eager calls between the replays."""
    i = _inputs(2, 300, 6, 1, 64, 128, BF16, True, seed=23)
    i["seq"] = _seq(2, 300, "random", 2)
    i = {k: v.cuda() for k, v in i.items()}
    want = _run(i)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = _run(i)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _run(i)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        eager = _run(i)
        torch.cuda.synchronize()
        for a, b, c, d in zip(got, eager, other, want):
            assert torch.equal(a, d) and torch.equal(b, d) and torch.equal(c, d)


def test_layer_training_step():
    """One layer's training step as it is used: conv1d -> scan -> gated norm forward, then
    norm_bwd -> scan_bwd -> conv1d_bwd, against torch's differentiation of the same layer in 64
    bits.  fp32 activations, so that no intermediate is rounded to 16 bits: every stage is
    within 1e-5 of its own magnitudes, and the gradients are sums over a few hundred of them."""
    import ssm_sequence_models_amd as ssm
    g = torch.Generator().manual_seed(29)
    B, L, H, P, G, N, K = 2, 70, 2, 16, 1, 16, 4
    C = H * P + 2 * G * N
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = dict(xBC=r(B, L, C), w=0.5 * r(C, K), b=0.5 * r(C), dt=torch.nn.functional.softplus(r(B, L, H) - 2.0),
             A=-torch.exp(torch.rand(H, generator=g)), z=r(B, L, H * P), nw=1 + 0.1 * r(H * P))
    dout = r(B, L, H * P)
    c = {k: v.cuda() for k, v in t.items()}
    u, _ = ssm.conv1d_fwd(c["xBC"], c["w"], c["b"], activation="silu")
    x, Bm, Cm = (v.contiguous() for v in u.split([H * P, G * N, G * N], 2))
    x, Bm, Cm = x.view(B, L, H, P), Bm.view(B, L, G, N), Cm.view(B, L, G, N)
    y, _ = ssm.scan_fwd(x, c["dt"], c["A"], Bm, Cm)
    yf = y.view(B, L, H * P)
    out = ssm.norm_fwd(yf, c["nw"], z=c["z"])
    dy, dz, dnw, _ = ssm.norm_bwd(yf, c["nw"], dout.cuda(), z=c["z"])
    dx, ddt, dA, dB, dC, _ = ssm.scan_bwd(x, c["dt"], c["A"], Bm, Cm, dy.view(B, L, H, P))
    du = torch.cat([dx.view(B, L, H * P), dB.view(B, L, G * N), dC.view(B, L, G * N)], 2)
    dxBC, _, dw, db = ssm.conv1d_bwd(c["xBC"], c["w"], c["b"], du, activation="silu")

    leaf = {k: v.double().requires_grad_() for k, v in t.items()}
    pad = torch.nn.functional.pad(leaf["xBC"].transpose(1, 2), (K - 1, 0))
    zc = torch.nn.functional.conv1d(pad, leaf["w"][:, None], leaf["b"], groups=C).transpose(1, 2)
    uu = zc * torch.sigmoid(zc)
    xx, bb, cc = uu.split([H * P, G * N, G * N], 2)
    xx, bb, cc = xx.view(B, L, H, P), bb.view(B, L, G, N).repeat_interleave(H // G, 2), cc.view(B, L, G, N).repeat_interleave(H // G, 2)
    h, ys = torch.zeros(B, H, P, N, dtype=torch.float64), []
    for i in range(L):
        a = torch.exp(leaf["dt"][:, i] * leaf["A"])
        h = a[..., None, None] * h + (leaf["dt"][:, i, :, None] * xx[:, i])[..., None] * bb[:, i, :, None, :]
        ys.append((h * cc[:, i, :, None, :]).sum(-1))
    v = torch.stack(ys, 1).reshape(B, L, H * P) * leaf["z"] * torch.sigmoid(leaf["z"])
    want = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-5) * leaf["nw"]
    (want * dout.double()).sum().backward()
    for name, got, ref in (("out", out, want.detach()), ("dxBC", dxBC, leaf["xBC"].grad), ("dw", dw, leaf["w"].grad),
                           ("db", db, leaf["b"].grad), ("ddt", ddt, leaf["dt"].grad), ("dA", dA, leaf["A"].grad),
                           ("dz", dz, leaf["z"].grad), ("dnw", dnw, leaf["nw"].grad)):
        e = (got.cpu().double() - ref).norm() / ref.norm()
        assert float(e) < 1e-4, (name, float(e))
