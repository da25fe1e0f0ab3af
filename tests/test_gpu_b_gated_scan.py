"""GPU parity of ssm_gated_scan_fwd / _bwd / _step against the token-by-token form in 64 bits.
The bounds come with the reference: the fp32 error carried by the same recurrence, plus half a
step of the output's type."""
import pytest
import torch

from train_ref import check_err, gated64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
STATE = {"final", "dh0"}


def _cuda(t):
    return None if t is None else t.to("cuda")


def _inputs(B, L, C, form, dtype, states, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    gate = r(B, L, C) * 2 + 1 if form == "sigmoid" else -torch.rand(B, L, C, generator=g) ** 4 * 2
    h0, dhT = (r(B, C), r(B, C)) if states else (None, None)
    return r(B, L, C).to(dtype), gate.to(dtype), r(B, L, C).to(dtype), h0, dhT


def _seq(B, L, kind, seed):
    if kind is None:
        return None
    g = torch.Generator().manual_seed(seed)
    if kind == "every":          # each token its own sequence
        return torch.arange(L, dtype=torch.int32).expand(B, L).contiguous()
    if kind == "tiles":          # starts on the edges of 8, 128 and 512 tokens and beside them
        ids = torch.zeros(B, L, dtype=torch.int32)
        for at in (8, 16, 127, 128, 129, 256, 511, 512, 640, 1024):
            if at < L:
                ids[:, at:] += 1
        return ids
    if kind == "back":           # an id that comes back is a start too
        return ((torch.arange(L) // 5) % 2).to(torch.int32).expand(B, L).contiguous()
    ids = (torch.rand(B, L, generator=g) < 3.0 / L).int()
    return ids.cumsum(1).to(torch.int32).contiguous()


def _compare(x, gate, dy, h0, dhT, form, seq):
    import ssm_sequence_models_amd as ssm
    xg, gg, hg, sg = _cuda(x), _cuda(gate), _cuda(h0), _cuda(seq)
    y, final = ssm.gated_scan_fwd(xg, gg, form=form, initial_state=hg, seq_idx=sg)
    dx, dgate, dh0 = ssm.gated_scan_bwd(xg, gg, _cuda(dy), form=form, initial_state=hg,
                                        dfinal_state=_cuda(dhT), seq_idx=sg)
    torch.cuda.synchronize()
    ref = gated64(x, gate, form, h0, seq, dy, dhT)
    for name, t in (("y", y), ("final", final), ("dx", dx), ("dgate", dgate), ("dh0", dh0)):
        check_err(t, ref, name, F32 if name in STATE else x.dtype)


@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 127, 128, 129, 300])
@pytest.mark.parametrize("form", ["log", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lengths(L, form, dtype):
    for C, states in ((1, True), (65, False), (130, True)):
        x, gate, dy, h0, dhT = _inputs(2, L, C, form, dtype, states, seed=L + C)
        _compare(x, gate, dy, h0, dhT, form, None)


@pytest.mark.parametrize("kind", ["every", "tiles", "back", "random"])
@pytest.mark.parametrize("form", ["log", "sigmoid"])
def test_packed(kind, form):
    for L in (5, 260, 1300):
        x, gate, dy, h0, dhT = _inputs(2, L, 70, form, F32, True, seed=L)
        _compare(x, gate, dy, h0, dhT, form, _seq(2, L, kind, seed=L))


@pytest.mark.parametrize("L", [1023, 1025, 2600, 5000])
def test_cut_rows(L):
    """Few channels on long rows: rows cut into segments (from 1024 tokens on), ragged last tile
    and segment, with and without packed sequences."""
    for dtype, kind in ((F32, None), (BF16, "random"), (F32, "tiles")):
        x, gate, dy, h0, dhT = _inputs(1, L, 7, "sigmoid", dtype, True, seed=L)
        _compare(x, gate, dy, h0, dhT, "sigmoid", _seq(1, L, kind, seed=L))
    x, gate, dy, h0, dhT = _inputs(3, L, 64, "log", F32, False, seed=L)
    _compare(x, gate, dy, h0, dhT, "log", None)


def test_many_rows_uncut():
    """More rows than the GPU has units: one segment a row, several blocks a unit."""
    x, gate, dy, h0, dhT = _inputs(300, 140, 66, "sigmoid", BF16, True, seed=3)
    _compare(x, gate, dy, h0, dhT, "sigmoid", _seq(300, 140, "random", seed=3))


def test_extreme_gates():
    """Decays of exactly 0 and 1, far gates and infinite ones."""
    for form in ("log", "sigmoid"):
        x, gate, dy, h0, dhT = _inputs(1, 300, 64, form, F32, True, seed=9)
        far = [0.0, -1e4, -3e38] if form == "log" else [0.0, 100.0, -100.0, 3e38, -3e38]
        for j, v in enumerate(far):
            gate[:, 20 * j:20 * j + 9, ::2] = v
            gate[:, 150 + j] = v
        _compare(x, gate, dy, h0, dhT, form, None)
        inf = gate.clone()
        inf[:, 200, ::3] = -float("inf")
        import ssm_sequence_models_amd as ssm
        y, _ = ssm.gated_scan_fwd(x.cuda(), inf.cuda(), form=form)
        far = gate.clone()
        far[:, 200, ::3] = -1e30
        want, _ = ssm.gated_scan_fwd(x.cuda(), far.cuda(), form=form)
        assert torch.equal(y, want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("L", [300, 2600])
def test_other_sequences_stay_finite(bad, L):
    """NaN or infinity in one packed sequence (inputs, gates, gradients, initial state) leaves
    the others' outputs as they are without it."""
    import ssm_sequence_models_amd as ssm
    x, gate, dy, h0, dhT = _inputs(1, L, 70, "sigmoid", F32, True, seed=4)
    ids = torch.zeros(1, L, dtype=torch.int32)
    a, b = L // 3, 2 * L // 3
    ids[:, a:b] = 1
    ids[:, b:] = 2

    def both():
        args = (x.cuda(), gate.cuda())
        y, f = ssm.gated_scan_fwd(*args, initial_state=h0.cuda(), seq_idx=ids.cuda())
        return y, f, *ssm.gated_scan_bwd(*args, dy.cuda(), initial_state=h0.cuda(),
                                         dfinal_state=dhT.cuda(), seq_idx=ids.cuda())
    clean = both()
    for t in (x, gate, dy):
        t[:, a + 3:b - 1:7] = bad
    got = both()
    h0[:] = bad
    x[:, :a] = bad
    got0 = both()
    torch.cuda.synchronize()
    for o, k in ((got, slice(0, a)), (got, slice(b, L)), (got0, slice(b, L))):
        for i in (0, 2, 3):
            assert torch.equal(o[i][:, k], clean[i][:, k])
        assert torch.equal(o[1], clean[1])
    assert torch.equal(got[4], clean[4])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_and_in_place(dtype):
    """x and gate as channel ranges of one projection, gradients into ranges of another, and the
    final state in place of the initial one (also on cut rows)."""
    import ssm_sequence_models_amd as ssm
    for L in (77, 2000):
        B, C = 2, 37
        x, gate, dy, h0, dhT = _inputs(B, L, C, "sigmoid", dtype, True, seed=L)
        wide = torch.full((B, L, 2 * C + 5), 9.0, dtype=dtype)
        wide[..., :C], wide[..., C:2 * C] = x, gate
        wide = wide.cuda()
        out = torch.full((B, L, 2 * C + 5), 5.0, dtype=dtype, device="cuda")
        yw = torch.full((B, L, C + 3), 5.0, dtype=dtype, device="cuda")
        state = h0.cuda()
        y, final = ssm.gated_scan_fwd(wide[..., :C], wide[..., C:2 * C], initial_state=state,
                                      final_state=state, y=yw[..., 3:])
        dx, dgate, dh0 = ssm.gated_scan_bwd(wide[..., :C], wide[..., C:2 * C], dy.cuda(),
                                            initial_state=h0.cuda(), dfinal_state=dhT.cuda(),
                                            dx=out[..., :C], dgate=out[..., C:2 * C])
        torch.cuda.synchronize()
        ref = gated64(x, gate, "sigmoid", h0, None, dy, dhT)
        for name, t in (("y", y), ("final", state), ("dx", dx), ("dgate", dgate), ("dh0", dh0)):
            check_err(t, ref, name, F32 if name in STATE else dtype)
        assert (out[..., 2 * C:] == 5.0).all() and (yw[..., :3] == 5.0).all()


def test_no_tokens():
    import ssm_sequence_models_amd as ssm
    x = torch.empty(2, 0, 5, device="cuda")
    h = torch.randn(2, 5, device="cuda")
    assert torch.equal(ssm.gated_scan_fwd(x, x, initial_state=h)[1], h)
    assert float(ssm.gated_scan_fwd(x, x)[1].abs().max()) == 0
    assert torch.equal(ssm.gated_scan_bwd(x, x, x, dfinal_state=h)[2], h)
    assert float(ssm.gated_scan_bwd(x, x, x)[2].abs().max()) == 0
    e = torch.empty(0, 3, 5, device="cuda")
    assert ssm.gated_scan_fwd(e, e)[0].shape == (0, 3, 5)


def test_refused_alias():
    import ssm_sequence_models_amd as ssm
    x = torch.zeros(1, 4, 8, device="cuda")
    h = torch.zeros(1, 8, device="cuda")
    with pytest.raises(ssm.SSMError):
        ssm.gated_scan_bwd(x, x, x, dfinal_state=h, dinitial_state=h)


def test_chunks_continue():
    """State passing: two calls joined by the state are the whole row, both ways."""
    import ssm_sequence_models_amd as ssm
    x, gate, dy, h0, dhT = _inputs(2, 700, 66, "sigmoid", F32, True, seed=8)
    ref = gated64(x, gate, "sigmoid", h0, None, dy, dhT)
    xg, gg, dg = x.cuda(), gate.cuda(), dy.cuda()
    cut = 333
    c = lambda t: t.contiguous()  # noqa: E731
    ya, mid = ssm.gated_scan_fwd(c(xg[:, :cut]), c(gg[:, :cut]), initial_state=h0.cuda())
    yb, fin = ssm.gated_scan_fwd(c(xg[:, cut:]), c(gg[:, cut:]), initial_state=mid)
    bb = ssm.gated_scan_bwd(c(xg[:, cut:]), c(gg[:, cut:]), c(dg[:, cut:]), initial_state=mid,
                            dfinal_state=dhT.cuda())
    ba = ssm.gated_scan_bwd(c(xg[:, :cut]), c(gg[:, :cut]), c(dg[:, :cut]), initial_state=h0.cuda(),
                            dfinal_state=bb[2])
    for name, t in (("y", torch.cat([ya, yb], 1)), ("final", fin), ("dx", torch.cat([ba[0], bb[0]], 1)),
                    ("dgate", torch.cat([ba[1], bb[1]], 1)), ("dh0", ba[2])):
        check_err(t, ref, name, F32)


def test_rows_far_apart():
    """A row stride from 2^26 elements on (beyond the lanes' 32-bit offsets), offsets past 2^32
    bytes: the outputs of the packed input.  Both round the same sums once, and fp32 sums of the
    same terms differ by 1e-5 of them at most, so they are a step of bf16 apart at most."""
    import ssm_sequence_models_amd as ssm
    L, C, row = 140, 66, 1 << 26
    x, gate, dy, _, _ = _inputs(1, L, C, "sigmoid", BF16, False, seed=9)
    wide = torch.empty(L * row, dtype=BF16, device="cuda").as_strided((1, L, C), (L * row, row, 1))
    wide.copy_(x)
    x, gate, dy = x.cuda(), gate.cuda(), dy.cuda()
    want = ssm.gated_scan_fwd(x, gate, form="sigmoid")
    got = ssm.gated_scan_fwd(wide, gate, form="sigmoid")
    want += ssm.gated_scan_bwd(x, gate, dy, form="sigmoid")
    got += ssm.gated_scan_bwd(wide, gate, dy, form="sigmoid")
    for a, b in zip(want, got):
        step = 2 * torch.finfo(a.dtype).eps / 2 if a.dtype == BF16 else 0.0
        assert torch.allclose(a.double(), b.double(), rtol=1.01 * step + 1e-5, atol=1e-5)


@pytest.mark.parametrize("C", [1, 7, 64, 300])
@pytest.mark.parametrize("form", ["log", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step(C, form, dtype):
    """Decode on a pool: the tokens' own rows, untouched other slots, rows outside the pool."""
    import ssm_sequence_models_amd as ssm
    for T in (1, 3):
        B, n = 6, 9
        x, gate, _, _, _ = _inputs(B, T, C, form, dtype, False, seed=C + T)
        pool = torch.randn(n, C, generator=torch.Generator().manual_seed(1))
        slots = torch.tensor([4, -1, 0, 8, 9, 2], dtype=torch.int32)
        pg = pool.cuda()
        y = ssm.gated_scan_step(x.cuda(), gate.cuda(), pg, form=form, state_indices=slots.cuda())
        torch.cuda.synchronize()
        on = [b for b in range(B) if 0 <= int(slots[b]) < n]
        at = slots[on].long()
        ref = gated64(x[on], gate[on], form, pool[at])
        check_err(y[on], ref, "y", dtype)
        check_err(pg[at.cuda()], ref, "final", F32)
        assert float(y[[1, 4]].abs().max()) == 0
        keep = [s for s in range(n) if s not in at.tolist()]
        assert torch.equal(pg[keep].cpu(), pool[keep])


def test_step_continues_prefill():
    """A prefill's final state in the pool, then token by token, is the whole row; without
    indices row b uses slot b; strided inputs."""
    import ssm_sequence_models_amd as ssm
    x, gate, _, h0, _ = _inputs(3, 140, 40, "sigmoid", F32, True, seed=12)
    ref = gated64(x, gate, "sigmoid", h0)
    wide = torch.cat([x, gate], 2).cuda()
    y, pool = ssm.gated_scan_fwd(wide[:, :130, :40].contiguous(), wide[:, :130, 40:].contiguous(),
                                 initial_state=h0.cuda())
    ys = [y]
    for t in range(130, 140):
        ys.append(ssm.gated_scan_step(wide[:, t:t + 1, :40], wide[:, t:t + 1, 40:], pool))
    check_err(torch.cat(ys, 1), ref, "y", F32)
    check_err(pool, ref, "final", F32)


def test_gradient_against_differences():
    """<gradient, v> against central differences of the 64-bit loss (h = 1e-4: the third-order
    rest is below 1e-6 of these losses of order 10)."""
    import ssm_sequence_models_amd as ssm
    for form in ("log", "sigmoid"):
        x, gate, dy, h0, dhT = _inputs(1, 40, 6, form, F32, True, seed=5)
        seq = _seq(1, 40, "random", 2)
        dx, dgate, dh0 = ssm.gated_scan_bwd(x.cuda(), gate.cuda(), dy.cuda(), form=form,
                                            initial_state=h0.cuda(), dfinal_state=dhT.cuda(),
                                            seq_idx=seq.cuda())
        g = torch.Generator().manual_seed(6)
        for i, (t, grad) in enumerate(((x, dx), (gate, dgate), (h0, dh0))):
            v = torch.randn(t.shape, generator=g, dtype=torch.float64)
            f = []
            for e in (1e-4, -1e-4):
                q = [x.double(), gate.double(), h0.double()]
                q[i] = q[i] + e * v
                r = gated64(q[0], q[1], form, q[2], seq)
                f.append(float((r["y"] * dy.double()).sum() + (r["final"] * dhT.double()).sum()))
            dot = (grad.cpu().double() * v)
            assert abs((f[0] - f[1]) / 2e-4 - float(dot.sum())) <= 1e-5 * float(dot.abs().sum()) + 1e-4


def test_graph_replay_and_streams():
    """The same bits on another stream and from every replay of a captured graph, with eager
    calls between the replays."""
    import ssm_sequence_models_amd as ssm
    x, gate, dy, h0, dhT = (_cuda(t) for t in _inputs(2, 3000, 40, "sigmoid", BF16, True, seed=2))
    seq = _seq(2, 3000, "random", 1).cuda()

    def both():
        y, f = ssm.gated_scan_fwd(x, gate, initial_state=h0, seq_idx=seq)
        return y, f, *ssm.gated_scan_bwd(x, gate, dy, initial_state=h0, dfinal_state=dhT, seq_idx=seq)
    want = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = both()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        eager = both()
        torch.cuda.synchronize()
        for a, b, c, d in zip(got, eager, other, want):
            assert torch.equal(a, d) and torch.equal(b, d) and torch.equal(c, d)
