"""GPU parity of ssm_delta_scan_fwd / _bwd / _step against the token-by-token form in 64 bits; the
bounds come with the reference."""
import pytest
import torch

from delta_ref import check_delta, delta64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
STATE = {"final", "dh0", "dbeta", "dgate"}
GRADS = ("dq", "dk", "dv", "dbeta", "dgate", "dh0")


def _cuda(t):
    return None if t is None else t.to("cuda")


def _inputs(B, L, H, G, P, N, dtype, states=True, gate=True, seed=0, keys="normal"):
    """Keys of length 1 (within the rounding of their type), as the recurrence takes them."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda t: (0.99 * torch.nn.functional.normalize(t, dim=-1)).to(dtype)  # noqa: E731
    k = r(B, L, G, N)
    if keys == "one":  # the same key all along
        k = k[:, :1].expand(B, L, G, N)
    elif keys == "near":  # what a SiLU leaves
        k = torch.nn.functional.silu(k + 0.5)
    return dict(q=unit(r(B, L, G, N)), k=unit(k), v=r(B, L, H, P).to(dtype),
                beta=torch.rand(B, L, H, generator=g) * (1.0 if keys == "normal" else 2.0),
                gate=-torch.rand(B, L, H, generator=g) ** 4 * 3 if gate else None,
                h0=r(B, H, P, N) if states else None, dy=r(B, L, H, P).to(dtype),
                dhT=r(B, H, P, N) if states else None)


def _seq(B, L, kind, seed=0):
    if kind is None:
        return None
    if kind == "every":
        return torch.arange(L, dtype=torch.int32).expand(B, L).contiguous()
    if kind == "edges":  # starts on the edges of chunks and beside them
        ids = torch.zeros(B, L, dtype=torch.int32)
        for at in (1, 31, 32, 33, 63, 64, 65, 96, 128, 191):
            if at < L:
                ids[:, at:] += 1
        return ids
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(B, L, generator=g) < 3.0 / L).int().cumsum(1).to(torch.int32).contiguous()


def _run(s, scale, seq, **more):
    import ssm_sequence_models_amd as ssm
    c = {n: _cuda(t) for n, t in s.items()}
    seq = _cuda(seq)
    y, final = ssm.delta_scan_fwd(c["q"], c["k"], c["v"], c["beta"], gate=c["gate"], scale=scale,
                                  initial_state=c["h0"], seq_idx=seq)
    got = dict(zip(GRADS, ssm.delta_scan_bwd(c["q"], c["k"], c["v"], c["beta"], c["dy"], gate=c["gate"],
                                             scale=scale, initial_state=c["h0"], dfinal_state=c["dhT"],
                                             seq_idx=seq)))
    torch.cuda.synchronize()
    return dict(y=y, final=final, **got)


def _compare(s, scale=0.25, seq=None):
    got = _run(s, scale, seq)
    ref = delta64(s["q"], s["k"], s["v"], s["beta"], s["gate"], scale, s["h0"], seq, s["dy"], s["dhT"])
    L, P, N = s["v"].shape[1], s["v"].shape[3], s["k"].shape[3]
    for name, t in got.items():
        if t is None:
            assert name == "dgate" and s["gate"] is None
            continue
        check_delta(t, ref, name, F32 if name in STATE else s["v"].dtype, N + P + 256, -(-L // 32))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 63, 64, 65, 129])
def test_lengths(L, dtype):
    _compare(_inputs(2, L, 2, 1, 16, 32, dtype, states=L % 2 == 1, seed=L))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("P,N", [(1, 4), (7, 12), (16, 64), (40, 48), (64, 68), (64, 128), (80, 100), (128, 128), (24, 132), (130, 256)])
def test_widths(P, N, dtype):
    _compare(_inputs(1, 70, 2, 2, P, N, dtype, seed=P + N))


@pytest.mark.parametrize("B,H,G", [(3, 4, 4), (1, 6, 2), (2, 8, 1), (1, 5, 5)])
def test_heads(B, H, G):
    _compare(_inputs(B, 100, H, G, 32, 64, BF16, seed=H))
    _compare(_inputs(B, 50, H, G, 16, 32, F32, seed=H))


@pytest.mark.parametrize("dtype,H,G", [(BF16, 128, 32), (BF16, 96, 16), (F32, 64, 16)])
def test_many_heads_of_a_key_head(dtype, H, G):
    """Enough heads that a block forms a key head's products for several: the bits of heads with keys of
    their own, and the 64-bit form in two rows."""
    B, L, P, N = 16, 150, 8, 16
    s = _inputs(B, L, H, G, P, N, dtype, seed=H)
    seq = _seq(B, L, "random")
    got = _run(s, 0.5, seq)
    own = _run(dict(s, **{n: s[n].repeat_interleave(H // G, 2) for n in ("q", "k")}), 0.5, seq)
    for n in ("y", "final", "dv", "dbeta", "dgate", "dh0"):
        assert torch.equal(got[n], own[n]), n
    two = {n: None if t is None else t[:2].contiguous() for n, t in s.items()}
    ref = delta64(two["q"], two["k"], two["v"], two["beta"], two["gate"], 0.5, two["h0"], seq[:2], two["dy"], two["dhT"])
    for n, t in got.items():
        check_delta(t[:2], ref, n, F32 if n in STATE else dtype, N + P + 256, -(-L // 32))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["every", "edges", "random"])
def test_packed(kind, dtype):
    _compare(_inputs(2, 200, 2, 1, 32, 64, dtype, seed=1), seq=_seq(2, 200, kind))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_without_gate(dtype):
    _compare(_inputs(2, 150, 4, 2, 32, 64, dtype, gate=False, seed=2))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keys", ["one", "near"])
def test_keys_alike(keys, dtype):
    """beta up to 2 on the same or nearly the same key: the pairs' matrix has powers as large as
    binomials, its inverse has not."""
    _compare(_inputs(1, 150, 2, 1, 32, 64, dtype, seed=3, keys=keys))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_extreme_gates(dtype):
    s = _inputs(1, 140, 3, 1, 16, 32, dtype, seed=4)
    s["gate"][:, :, 0] = 0.0                 # nothing decays
    s["gate"][:, 10::7, 1] = -1e30           # tokens that forget everything, as a reset does
    s["gate"][:, 3::11, 1] = -float("inf")
    s["gate"][:, :, 2] = -40.0               # only the token itself
    s["beta"][:, ::3] = 0.0                  # tokens that write nothing
    s["beta"][:, 1::3] = 1.0
    _compare(s)


def test_scaled_gradients():
    """The gradients are linear in dy and dfinal_state, however small or large those are."""
    s = _inputs(1, 130, 2, 1, 64, 64, BF16, seed=5)
    one = _run(s, 0.5, None)
    for f in (2.0 ** -60, 2.0 ** 40):
        more = _run(dict(s, dy=(s["dy"].double() * f).to(BF16), dhT=s["dhT"] * f), 0.5, None)
        for n in GRADS:
            assert torch.equal(more[n].double(), one[n].double() * f), n


def test_long_row():
    _compare(_inputs(1, 1500, 2, 1, 64, 64, BF16, seed=6), seq=_seq(1, 1500, "random"))


@pytest.mark.parametrize("dtype,B,L,H,G,P,N", [(BF16, 1, 2100, 1, 1, 64, 128), (BF16, 1, 1030, 3, 3, 80, 64), (F32, 1, 1100, 2, 1, 40, 48),
                                               (BF16, 2, 1100, 1, 1, 16, 200), (F32, 1, 900, 1, 1, 32, 256)])
def test_cut_rows(dtype, B, L, H, G, P, N):
    """Few heads: rows in segments side by side, joined through what each makes of the state before it."""
    _compare(_inputs(B, L, H, G, P, N, dtype, seed=L), scale=1.0)
    s = _inputs(B, L, H, G, P, N, dtype, gate=False, states=False, seed=L + 1)
    seq = torch.zeros(B, L, dtype=torch.int32)
    seq[:, L // 3:] = 1
    seq[0, L // 2 + 1:] = 2
    _compare(s, scale=1.0, seq=seq)


def test_cut_rows_stay_apart():
    """A NaN in the first of two sequences leaves the segments behind its end as they are, and in the
    second those before its start."""
    s = _inputs(1, 2100, 1, 1, 64, 64, BF16, seed=18)
    seq = torch.zeros(1, 2100, dtype=torch.int32)
    seq[:, 1000:] = 1
    clean = _run(s, 1.0, seq)
    for name, at in (("v", 300), ("k", 999), ("dy", 1500), ("q", 1001)):
        bad = dict(s, **{name: s[name].clone()})
        bad[name].view(1, 2100, -1)[0, at, 0] = float("nan")
        got = _run(bad, 1.0, seq)
        for n, t in got.items():
            if n == "final":
                assert at >= 1000 or torch.equal(t, clean[n]), (name, n)
            elif n == "dh0":
                assert at < 1000 or torch.equal(t, clean[n]), (name, n)
            elif at < 1000:
                assert torch.equal(t[:, 1024:], clean[n][:, 1024:]), (name, n)
            else:
                assert torch.equal(t[:, :960], clean[n][:, :960]), (name, n)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_repeat_is_equal(dtype):
    s = _inputs(2, 300, 4, 1, 64, 128, dtype, seed=7)
    a, b = _run(s, 1.0, _seq(2, 300, "random")), _run(s, 1.0, _seq(2, 300, "random"))
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_tokens_and_outputs(dtype):
    """Queries, keys and values as channel ranges of one tensor at an odd offset, gradients into the
    ranges of another, the final state in place of the initial one: the same bits as dense."""
    import ssm_sequence_models_amd as ssm
    B, L, H, G, P, N = 2, 77, 4, 2, 24, 36
    s = {n: _cuda(t) for n, t in _inputs(B, L, H, G, P, N, dtype, seed=8).items()}
    how = dict(gate=s["gate"], scale=0.3)
    y, final = ssm.delta_scan_fwd(s["q"], s["k"], s["v"], s["beta"], initial_state=s["h0"], **how)
    grads = ssm.delta_scan_bwd(s["q"], s["k"], s["v"], s["beta"], s["dy"], initial_state=s["h0"],
                               dfinal_state=s["dhT"], **how)
    width = 2 * G * N + H * P

    def ranges(fill):
        wide = torch.full((B, L, width + 3), 5.0, device="cuda", dtype=dtype)[..., 1:]
        parts = (wide[..., :G * N].unflatten(-1, (G, N)), wide[..., G * N:2 * G * N].unflatten(-1, (G, N)),
                 wide[..., 2 * G * N:width].unflatten(-1, (H, P)))
        if fill:
            for p, t in zip(parts, (s["q"], s["k"], s["v"])):
                p.copy_(t)
        return wide, parts

    _, (q, k, v) = ranges(True)
    _, (_, _, dy) = ranges(False)
    dy.copy_(s["dy"])
    state = s["h0"].clone()
    wide_y, (_, _, y2) = ranges(False)
    ssm.delta_scan_fwd(q, k, v, s["beta"], initial_state=state, final_state=state, y=y2, **how)
    assert torch.equal(y2, y) and torch.equal(state, final)
    assert bool((wide_y[..., :2 * G * N] == 5.0).all()) and bool((wide_y[..., width:] == 5.0).all())
    wide, (dq, dk, dv) = ranges(False)
    g2 = ssm.delta_scan_bwd(q, k, v, s["beta"], dy, initial_state=s["h0"], dfinal_state=s["dhT"], dq=dq,
                            dk=dk, dv=dv, **how)
    for n, a, b in zip(GRADS, grads, g2):
        assert torch.equal(a, b), n
    assert bool((wide[..., width:] == 5.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_token_for_all(dtype):
    """A token that stands for all of a row (stride 0), with lengths that end inside a chunk: the same
    bits as its copies, in every operand and in all of them."""
    import ssm_sequence_models_amd as ssm
    s = {n: _cuda(t) for n, t in _inputs(1, 77, 4, 2, 32, 32, dtype, seed=18).items()}
    names = ("q", "k", "v", "dy")
    for which in (*((n,) for n in names), ("q", "dy"), names):
        one = {n: s[n][:, :1].expand_as(s[n]) if n in which else s[n] for n in names}

        def run(c):
            how = dict(gate=s["gate"], initial_state=s["h0"])
            return (*ssm.delta_scan_fwd(c["q"], c["k"], c["v"], s["beta"], **how),
                    *ssm.delta_scan_bwd(c["q"], c["k"], c["v"], s["beta"], c["dy"], dfinal_state=s["dhT"], **how))
        assert one[which[0]].stride(1) == 0
        for a, b in zip(run(one), run({n: t.contiguous() for n, t in one.items()})):
            assert torch.equal(a, b), which


def test_no_tokens():
    import ssm_sequence_models_amd as ssm
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    h = torch.randn(2, 4, 8, 16, device="cuda")
    y, final = ssm.delta_scan_fwd(z(2, 0, 2, 16), z(2, 0, 2, 16), z(2, 0, 4, 8), z(2, 0, 4), initial_state=h)
    assert y.shape == (2, 0, 4, 8) and torch.equal(final, h)
    _, final = ssm.delta_scan_fwd(z(2, 0, 2, 16), z(2, 0, 2, 16), z(2, 0, 4, 8), z(2, 0, 4))
    assert not final.any()
    out = ssm.delta_scan_bwd(z(2, 0, 2, 16), z(2, 0, 2, 16), z(2, 0, 4, 8), z(2, 0, 4), z(2, 0, 4, 8), dfinal_state=h)
    assert torch.equal(out[5], h)
    y, final = ssm.delta_scan_fwd(z(0, 3, 2, 16), z(0, 3, 2, 16), z(0, 3, 4, 8), z(0, 3, 4))
    assert y.numel() == 0 and final.numel() == 0
    pool = h.clone()
    y = ssm.delta_scan_step(z(2, 0, 2, 16), z(2, 0, 2, 16), z(2, 0, 4, 8), z(2, 0, 4), pool)
    assert y.numel() == 0 and torch.equal(pool, h)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_chunks_continue(dtype):
    """A row in two calls, the state handed on and its gradient handed back, against the whole row."""
    import ssm_sequence_models_amd as ssm
    s = _inputs(2, 201, 2, 1, 32, 64, dtype, seed=9)
    ref = delta64(s["q"], s["k"], s["v"], s["beta"], s["gate"], 1.0, s["h0"], None, s["dy"], s["dhT"])
    c = {n: _cuda(t) for n, t in s.items()}
    for at in (1, 64, 90):
        a = {n: t[:, :at].contiguous() for n, t in c.items() if n not in ("h0", "dhT")}
        b = {n: t[:, at:].contiguous() for n, t in c.items() if n not in ("h0", "dhT")}
        args = lambda p: (p["q"], p["k"], p["v"], p["beta"])  # noqa: E731
        ya, mid = ssm.delta_scan_fwd(*args(a), gate=a["gate"], initial_state=c["h0"])
        yb, final = ssm.delta_scan_fwd(*args(b), gate=b["gate"], initial_state=mid)
        gb = ssm.delta_scan_bwd(*args(b), b["dy"], gate=b["gate"], initial_state=mid, dfinal_state=c["dhT"])
        ga = ssm.delta_scan_bwd(*args(a), a["dy"], gate=a["gate"], initial_state=c["h0"], dfinal_state=gb[5])
        got = dict(y=torch.cat([ya, yb], 1), final=final, dh0=ga[5])
        for i, n in enumerate(GRADS[:5]):
            got[n] = torch.cat([ga[i], gb[i]], 1)
        for n, t in got.items():
            check_delta(t, ref, n, F32 if n in STATE else dtype, 32 + 64 + 256, 10)


def test_gradient_against_differences():
    """Along random directions of every input, against central differences of the 64-bit forward."""
    s = _inputs(1, 70, 2, 1, 8, 16, F32, seed=10)
    seq = _seq(1, 70, "edges")
    got = _run(s, 0.7, seq)

    def loss(p):
        r = delta64(p["q"], p["k"], p["v"], p["beta"], p["gate"], 0.7, p["h0"], seq)
        return float((r["y"] * s["dy"].double()).sum() + (r["final"] * s["dhT"].double()).sum())

    g = torch.Generator().manual_seed(11)
    for n, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("beta", "dbeta"), ("gate", "dgate"), ("h0", "dh0")):
        d = torch.randn(s[n].shape, generator=g, dtype=torch.float64)
        eps = 1e-5
        up, down = (loss(dict(s, **{n: s[n].double() + f * d})) for f in (eps, -eps))
        want = (up - down) / (2 * eps)
        have = float((got[grad].cpu().double() * d).sum())
        # second order of the difference, and the fp32 gradient's own 352 U of its terms
        size = float((got[grad].cpu().double().abs() * d.abs()).sum())
        assert abs(have - want) <= 1e-5 * size + 1e-6 * abs(want), (n, have, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n_new", [1, 3])
@pytest.mark.parametrize("P,N", [(1, 4), (33, 36), (64, 64), (128, 128), (24, 200)])
def test_step(P, N, n_new, dtype):
    import ssm_sequence_models_amd as ssm
    B, H, G, slots = 5, 4, 2, 9
    s = _inputs(B, n_new, H, G, P, N, dtype, seed=12)
    pool = torch.randn(slots, H, P, N, generator=torch.Generator().manual_seed(13))
    idx = torch.tensor([7, 0, -1, 3, slots], dtype=torch.int32)
    got_pool = _cuda(pool)
    c = {n: _cuda(t) for n, t in s.items()}
    y = ssm.delta_scan_step(c["q"], c["k"], c["v"], c["beta"], got_pool, gate=c["gate"], scale=0.5,
                            state_indices=_cuda(idx))
    torch.cuda.synchronize()
    on = [0, 1, 3]
    ref = delta64(*(s[n][on] for n in ("q", "k", "v", "beta", "gate")), 0.5, pool[idx[on].long()], None)
    check_delta(y[on], ref, "y", dtype, N + P + 256, 1)
    check_delta(got_pool[idx[on].long().cuda()], ref, "final", F32, N + P + 256, 1)
    assert not y[[2, 4]].any()
    off = [i for i in range(slots) if i not in (7, 0, 3)]
    assert torch.equal(got_pool[off].cpu(), pool[off])


def test_step_continues_prefill():
    """Row slots without indices; a prefill and single tokens make the whole row."""
    import ssm_sequence_models_amd as ssm
    s = _inputs(3, 68, 2, 1, 32, 64, BF16, seed=14)
    c = {n: _cuda(t) for n, t in s.items()}
    cut = lambda a, b: [c[n][:, a:b].contiguous() for n in ("q", "k", "v", "beta")]  # noqa: E731
    y, pool = ssm.delta_scan_fwd(*cut(0, 64), gate=c["gate"][:, :64].contiguous(), initial_state=c["h0"])
    ys = [y]
    for t in range(64, 68):
        ys.append(ssm.delta_scan_step(*cut(t, t + 1), pool, gate=c["gate"][:, t:t + 1].contiguous()))
    ref = delta64(*(s[n] for n in ("q", "k", "v", "beta", "gate")), 1.0, s["h0"], None)
    check_delta(torch.cat(ys, 1), ref, "y", BF16, 32 + 64 + 256, 7)
    check_delta(pool, ref, "final", F32, 32 + 64 + 256, 7)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_sequences_stay_finite(bad, dtype):
    """A value that is not finite stays in the chunks (64 tokens in bf16, 32 in fp32) that its
    sequence has tokens in, forward in those from its own on: rows, and other sequences' tokens in
    other chunks, do not see it."""
    import ssm_sequence_models_amd as ssm
    B, L, H = 2, 260, 2
    seq = torch.zeros(B, L, dtype=torch.int32)
    seq[:, 70:] = 1
    for name, at in (("k", 66), ("v", 66), ("q", 66), ("v", 69), ("k", 100), ("dy", 66), ("beta", 66)):
        s = _inputs(B, L, H, 1, 32, 64, dtype, seed=15)
        clean = _run(s, 1.0, seq)
        s = dict(s, **{name: s[name].clone()})
        s[name].view(B, L, -1)[0, at, 0] = bad
        got = _run(s, 1.0, seq)
        Q = 64 if dtype == BF16 else 32
        lo, hi = at // Q * Q, at // Q * Q + Q  # its chunk
        for n, t in got.items():
            w = clean[n]
            assert torch.equal(t[1], w[1]), (name, at, n)
            if n in ("final", "dh0"):
                if at < 70 and n == "final":
                    assert torch.isfinite(t).all(), (name, at, n)
                if at >= 70 and n == "dh0":
                    assert torch.isfinite(t).all(), (name, at, n)
                continue
            if at < 70:   # sequence 0: tokens behind the chunk belong to sequence 1
                assert torch.equal(t[0, max(hi, 70):], w[0, max(hi, 70):]), (name, at, n)
            else:         # sequence 1: tokens of the chunks before its first
                assert torch.equal(t[0, :70 // Q * Q], w[0, :70 // Q * Q]), (name, at, n)
            if n == "y":  # forward: nothing reaches back over a chunk either
                assert torch.equal(t[0, :lo], w[0, :lo]), (name, at, n)


def test_rows_far_apart():
    """Token rows 2^26 elements apart: offsets pass 32 bits."""
    import ssm_sequence_models_amd as ssm
    L, H, P, N, row = 66, 1, 16, 16, 1 << 26
    s = _inputs(1, L, H, 1, P, N, BF16, seed=16)
    c = {n: _cuda(t) for n, t in s.items()}
    y, final = ssm.delta_scan_fwd(c["q"], c["k"], c["v"], c["beta"], gate=c["gate"], initial_state=c["h0"])
    far = torch.empty((L - 1) * row + 3 * 16, device="cuda", dtype=BF16)
    parts = [far[16 * i:].as_strided((1, L, 1, 16), (row, row, 16, 1)) for i in range(3)]
    for p, n in zip(parts, ("q", "k", "v")):
        p.copy_(c[n])
    y2, final2 = ssm.delta_scan_fwd(*parts, c["beta"], gate=c["gate"], initial_state=c["h0"])
    assert torch.equal(y, y2) and torch.equal(final, final2)


def test_step_slots_far_apart():
    """A slot behind 2^31 elements of the pool: the bits of a pool of its own."""
    import ssm_sequence_models_amd as ssm
    H, P, N, slots = 32, 128, 128, 4100
    c = {n: _cuda(t) for n, t in _inputs(2, 1, H, 16, P, N, BF16, seed=19).items()}
    small = c["h0"].clone()
    pool = torch.empty(slots, H, P, N, device="cuda")
    at = torch.tensor([slots - 1, 3], dtype=torch.int32, device="cuda")
    pool[slots - 1], pool[3] = small[0], small[1]
    args = (c["q"], c["k"], c["v"], c["beta"])
    y = ssm.delta_scan_step(*args, pool, gate=c["gate"], state_indices=at)
    assert torch.equal(y, ssm.delta_scan_step(*args, small, gate=c["gate"]))
    assert torch.equal(pool[slots - 1], small[0]) and torch.equal(pool[3], small[1])


def test_graph_replay_and_streams():
    """Captured forward, backward and step, replayed with eager work between, equal eager calls; and
    the same on a stream of its own."""
    import ssm_sequence_models_amd as ssm
    s = _inputs(2, 150, 4, 2, 64, 64, BF16, seed=17)
    c = {n: _cuda(t) for n, t in s.items()}
    pool = torch.randn(2, 4, 64, 64, device="cuda")
    tok = {n: c[n][:, :1].contiguous() for n in ("q", "k", "v", "beta", "gate")}

    def work(pool):
        y, final = ssm.delta_scan_fwd(c["q"], c["k"], c["v"], c["beta"], gate=c["gate"], initial_state=c["h0"])
        g = ssm.delta_scan_bwd(c["q"], c["k"], c["v"], c["beta"], c["dy"], gate=c["gate"],
                               initial_state=c["h0"], dfinal_state=final)
        t = ssm.delta_scan_step(tok["q"], tok["k"], tok["v"], tok["beta"], pool, gate=tok["gate"])
        return (y, final, *g, t)

    p0, p1 = pool.clone(), pool.clone()
    want = [t.clone() for t in work(p0)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = work(p1)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(p0, p1)
    graph = torch.cuda.CUDAGraph()
    p2 = pool.clone()
    with torch.cuda.graph(graph):
        held = work(p2)
    p0.copy_(pool)
    for i in range(4):
        p2.copy_(p0)
        graph.replay()
        torch.cuda.synchronize()
        eager = work(p0)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i
        assert torch.equal(p0, p2)
