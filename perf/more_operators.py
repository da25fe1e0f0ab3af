"""The operators of a layer that overwrites its state along keys, as measured cases.

  delta_scan_fwd   the gated delta rule over long rows, from an initial to a final state:
                   e_t = v_t - a_t h_{t-1} k_t,  h_t = a_t h_{t-1} + beta_t e_t k_t^T,
                   y_t = scale h_t q_t,  a_t = exp(gate_t); the state h is [headdim, dstate]
  delta_scan_bwd   its backward: dq, dk, dv, dbeta, dgate and the gradient of the initial state
  delta_scan_step  its decode form on a state pool
  qk_norm_fwd      the norm of every head of the queries and keys (l2 or rms, with weights), and
                   the rotation of its first channels by the token's position, in one pass
  qk_norm_bwd      its backward: dq, dk and the sums over the tokens for the weights

With `own` false `run` computes the plain form of an operator in elementary torch operations
(32 bits; 64 for sums of log decays, for sums of products that cancel, for the long sums of the
weights' gradients and for the rotation's angles); with `own` true it calls the framework's entry
points.  `exact` is the definition in 64 bits: the delta rule token by token, the norm head by
head.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64  # tokens per chunk of the delta rule's plain form, a power of two
EPS = 1e-6
DEV = "cuda"


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def _delta(name, op, B, L, H, G, P, N, dtype, states, packed):
    return dict(name=name, op=op, B=B, L=L, H=H, G=G, P=P, N=N, dtype=dtype, states=states,
                packed=packed)


def _qk(name, op, B, L, HQ, HK, D, R, kind, weights, interleaved, dtype):
    return dict(name=name, op=op, B=B, L=L, HQ=HQ, HK=HK, D=D, R=R, kind=kind, weights=weights,
                interleaved=interleaved, dtype=dtype)


def listed():
    return [
        # two small fp32 heads, the shape that gradient checks run at: latency
        _delta("delta_fwd tiny f32", "delta_scan_fwd", 1, 64, 2, 1, 16, 16, "f32", True, 0),
        # a layer's prefill on packed 8K rows with state passing, two value heads a key head
        _delta("delta_fwd layer packed", "delta_scan_fwd", 4, 8192, 32, 16, 128, 128, "bf16", True, 4),
        # one long ragged row with few heads: a document read by a small model
        _delta("delta_fwd long row", "delta_scan_fwd", 1, 32845, 8, 8, 64, 128, "bf16", True, 0),
        # a small training step in fp32 with odd sizes
        _delta("delta_bwd odd f32", "delta_scan_bwd", 2, 515, 6, 3, 40, 48, "f32", True, 2),
        # the layer's backward
        _delta("delta_bwd layer packed", "delta_scan_bwd", 4, 8192, 32, 16, 128, 128, "bf16", True, 4),
        # truncated back-propagation through one long ragged row, the smaller state
        _delta("delta_bwd long row n64", "delta_scan_bwd", 1, 16421, 16, 8, 64, 64, "bf16", True, 0),
        # decode: one new token for each of 256 requests in a pool of 512 slots
        _delta("delta_step decode", "delta_scan_step", 256, 1, 32, 16, 128, 128, "bf16", True, 0),
        # four draft tokens for each of a few requests
        _delta("delta_step drafts", "delta_scan_step", 8, 4, 16, 16, 64, 128, "bf16", True, 0),
        # decode: the queries and keys of 256 new tokens, unit norm, no positions
        _qk("qk_norm_fwd decode", "qk_norm_fwd", 256, 1, 16, 16, 128, 0, "l2", False, False, "bf16"),
        # the layer's prefill, weights and half of the channels rotated
        _qk("qk_norm_fwd layer", "qk_norm_fwd", 4, 8192, 16, 16, 128, 64, "rms", True, False, "bf16"),
        # the layer's backward
        _qk("qk_norm_bwd layer", "qk_norm_bwd", 4, 8192, 16, 16, 128, 64, "rms", True, False, "bf16"),
        # few keys, neighbouring channels as pairs, odd sizes, fp32
        _qk("qk_norm_bwd odd f32", "qk_norm_bwd", 3, 1027, 6, 2, 80, 32, "l2", True, True, "f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_scan_fwd", "delta_scan_fwd", "delta_scan_bwd", "delta_scan_bwd",
                     "delta_scan_step", "qk_norm_fwd", "qk_norm_bwd"])
    if op == "delta_scan_step":
        P, N, G = rng.choice([32, 64, 80, 128]), rng.choice([16, 64, 128, 256]), rng.choice([1, 2, 8, 16])
        H = G * rng.choice([1, 2, 4])
        B = max(1, min(_log_int(rng, 1, 512), 256 * 32 * 128 * 128 // (H * P * N)))
        return dict(op=op, B=B, L=_log_int(rng, 1, 8), H=H, G=G, P=P, N=N,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), states=True, packed=0)
    if op.startswith("delta"):
        # most layers have heads of 64 or 128 in bf16; any other sizes and fp32 at moderate sizes
        if rng.random() < 0.6:
            dtype, P, N, cap = "bf16", rng.choice([64, 128]), rng.choice([64, 128]), 32768 * 32 * 128 * 128
        else:
            dtype = rng.choice(["bf16", "f32"])
            P, N, cap = rng.choice([16, 24, 40, 64, 128, 256]), rng.choice([16, 32, 48, 80, 128, 192, 256]), 2048 * 16 * 128 * 128
        G = rng.choice([1, 2, 4, 8, 16])
        H = G * rng.choice([1, 1, 2, 4])
        L = _log_int(rng, 1, 32768)
        B = _log_int(rng, 1, 8)
        while B > 1 and B * L * H * P * N > cap:
            B -= 1
        L = max(1, min(L, cap // (B * H * P * N)))
        return dict(op=op, B=B, L=L, H=H, G=G, P=P, N=N, dtype=dtype, states=rng.random() < 0.6,
                    packed=rng.choice([0, 0, 2, 5]))
    D = rng.choice([32, 64, 64, 80, 96, 128, 128, 192, 256])
    HK = rng.choice([1, 2, 4, 8, 16])
    HQ = HK * rng.choice([1, 1, 2, 4])
    B = _log_int(rng, 1, 8)
    L = max(1, min(_log_int(rng, 1, 32768), 32768 * 32 * 128 // (B * (HQ + HK) * D)))
    return dict(op=op, B=B, L=L, HQ=HQ, HK=HK, D=D, R=rng.choice([0, D // 2, D]),
                kind=rng.choice(["l2", "rms"]), weights=rng.random() < 0.5,
                interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]))


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _packed(case, g):
    """seq_idx of rows that hold `packed` sequences cut at random places."""
    B, L, n = case["B"], case["L"], case["packed"]
    if not n or L <= n:
        return None
    cuts = torch.rand(B, L, device=DEV, generator=g)
    cuts[:, 0] = -1.0
    ids = torch.zeros(B, L, device=DEV, dtype=torch.int32)
    ids.scatter_(1, cuts.topk(n - 1, dim=1).indices, 1)
    return ids.cumsum(1).to(torch.int32).contiguous()


def _prepare_delta(case, g):
    B, L, H, G, P, N = (case[k] for k in "BLHGPN")
    dt_ = DTYPES[case["dtype"]]
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    silu = torch.nn.functional.silu

    def unit(t):  # the conv's activations of a head, normed
        return torch.nn.functional.normalize(silu(t), dim=-1).to(dt_)

    # the values are a channel range of the conv's output, beside the raw queries and keys
    wide = torch.empty(B, L, 2 * G * N + H * P, device=DEV, dtype=dt_)
    wide[..., 2 * G * N:] = silu(rnd(B, L, H * P))
    rate = torch.exp(torch.rand(H, device=DEV, generator=g) * math.log(16.0))
    s = dict(case=case, q=unit(rnd(B, L, G, N)), k=unit(rnd(B, L, G, N)),
             v=wide[..., 2 * G * N:].view(B, L, H, P), beta=torch.sigmoid(rnd(B, L, H)),
             gate=-rate * torch.nn.functional.softplus(rnd(B, L, H) - 4.0),
             scale=N ** -0.5, h0=None, dhT=None, dy=None, seq=None)
    if case["op"] == "delta_scan_step":
        s["pool"] = 0.1 * rnd(2 * B, H, P, N)
        s["slots"] = torch.randperm(2 * B, device=DEV, generator=g)[:B].to(torch.int32)
        return s
    if case["states"]:
        s["h0"] = 0.1 * rnd(B, H, P, N)
    if case["op"] == "delta_scan_bwd":
        s["dy"] = rnd(B, L, H, P).to(dt_)
        if case["states"]:
            s["dhT"] = 0.1 * rnd(B, H, P, N)
    s["seq"] = _packed(case, g)
    return s


def _prepare_qk(case, g):
    B, L, HQ, HK, D, R = (case[k] for k in ("B", "L", "HQ", "HK", "D", "R"))
    dt_ = DTYPES[case["dtype"]]
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    # queries and keys are channel ranges of a projection's output (q | k | v)
    wide = torch.empty(B, L, (HQ + 2 * HK) * D, device=DEV, dtype=dt_)
    wide[..., :(HQ + HK) * D] = rnd(B, L, (HQ + HK) * D)
    s = dict(case=case, q=wide[..., :HQ * D].view(B, L, HQ, D),
             k=wide[..., HQ * D:(HQ + HK) * D].view(B, L, HK, D), wq=None, wk=None, freq=None, pos=None)
    if case["weights"]:
        s["wq"], s["wk"] = 1.0 + 0.1 * rnd(D), 1.0 + 0.1 * rnd(D)
    if R:
        s["freq"] = 10000.0 ** (-torch.arange(R // 2, device=DEV, dtype=torch.float32) / (R // 2))
        # each row continues a request somewhere in a long context
        s["pos"] = (torch.randint(0, 131072, (B, 1), device=DEV, generator=g)
                    + torch.arange(L, device=DEV)).to(torch.int32)
    if case["op"] == "qk_norm_bwd":
        s["dq"], s["dk"] = rnd(B, L, HQ, D).to(dt_), rnd(B, L, HK, D).to(dt_)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (_prepare_delta if case["op"].startswith("delta") else _prepare_qk)(case, g)


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------
def _chunks(v, pad):
    """[b, L, heads, d] -> [b, nc, heads, CHUNK, d] in 32 bits, zeros past the row."""
    v = torch.nn.functional.pad(v.float(), (0, 0, 0, 0, 0, pad))
    return v.unflatten(1, (-1, CHUNK)).transpose(2, 3).contiguous()


def _unit_lower_inverse(low):
    """(I + low)^-1 of a strictly lower triangular `low` [..., Q, Q], by blocks: the inverse of
    [[A, 0], [C, D]] is [[A', 0], [-D' C A', D']]."""
    Q = low.shape[-1]
    inv = torch.eye(Q, device=low.device).expand_as(low).clone()
    n = 1
    while n < Q:
        blocks = inv.unflatten(-1, (Q // (2 * n), 2 * n)).unflatten(-3, (Q // (2 * n), 2 * n))
        lows = low.unflatten(-1, (Q // (2 * n), 2 * n)).unflatten(-3, (Q // (2 * n), 2 * n))
        at = torch.arange(Q // (2 * n), device=low.device)
        diag = blocks[..., at, :, at, :]                       # [pairs, ..., 2n, 2n]
        c = lows[..., at, :, at, :][..., n:, :n]
        diag[..., n:, :n] = -(diag[..., n:, n:] @ c @ diag[..., :n, :n])
        blocks[..., at, :, at, :] = diag
        n *= 2
    return inv


def _delta_chunks(s):
    """What both directions need of every chunk, with the state at its start."""
    q, k, v = s["q"], s["k"], s["v"]
    b, L, H, P = v.shape
    G, N = k.shape[2:]
    Q = CHUNK
    nc = -(-L // Q)
    pad = nc * Q - L
    dev = v.device
    E = torch.nn.functional.pad(s["gate"].double(), (0, 0, 0, pad)).cumsum(1)  # [b, nc Q, H]
    E = E.view(b, nc, Q, H).transpose(2, 3)                    # [b, nc, H, Q]
    R = torch.zeros(b, nc * Q, device=dev, dtype=torch.int32)  # sequences begun so far
    if s["seq"] is not None:
        R[:, 1:L] = (s["seq"][:, 1:] != s["seq"][:, :-1]).int()
        R = R.cumsum(1, dtype=torch.int32)
        R[:, L:] = R[:, L - 1:L]
    R = R.view(b, nc, 1, Q)
    Eend, Rend = E[..., -1:], R[..., -1:]
    Eprev = torch.cat([torch.zeros_like(Eend[:, :1]), Eend[:, :-1]], 1)
    Rprev = torch.cat([torch.zeros_like(Rend[:, :1]), Rend[:, :-1]], 1)

    def factor(Et, Rt, Es, Rs, keep=None):  # product of the decays from s (exclusive) to t
        d = torch.where(Rt == Rs, Et - Es, -math.inf)
        if keep is not None:
            d = torch.where(keep, d, -math.inf)
        return d.exp().float()

    tril = torch.ones(Q, Q, device=dev, dtype=torch.bool).tril()
    lam = factor(E[..., :, None], R[..., :, None], E[..., None, :], R[..., None, :], tril)
    to_end = factor(Eend, Rend, E, R)[..., None]               # [b, nc, H, Q, 1]
    start = factor(E, R, Eprev, Rprev)[..., None]
    through = factor(Eend, Rend, Eprev, Rprev)[..., None]      # [b, nc, H, 1, 1]
    kc, qc = _chunks(k, pad), _chunks(q, pad) * s["scale"]
    rep = H // G
    kk = (kc @ kc.mT).repeat_interleave(rep, 2)
    M = lam * (qc @ kc.mT).repeat_interleave(rep, 2)
    kh, qh = kc.repeat_interleave(rep, 2), qc.repeat_interleave(rep, 2)
    vc, beta = _chunks(v, pad), _chunks(s["beta"][..., None], pad)
    lo = lam * kk * tril.tril(-1)
    T = _unit_lower_inverse(lo * beta.mT)
    # over a chunk the state's rows go through phi, and gain what its own tokens bring
    ke = kh * (beta * to_end)
    own_e = T @ vc
    W = T @ (kh * start)
    gain = own_e.mT @ ke                                       # [b, nc, H, P, N]
    phi = through * torch.eye(N, device=dev) - W.mT @ ke
    h = s["h0"] if s["h0"] is not None else torch.zeros(b, H, P, N, device=dev)
    S = torch.empty(b, nc, H, P, N, device=dev)
    for c in range(nc):
        S[:, c] = h
        h = h @ phi[:, c] + gain[:, c]
    e = own_e - W @ S.mT
    return dict(lam=lam, tril=tril, to_end=to_end, start=start, through=through, kh=kh, qh=qh, vc=vc,
                beta=beta, lo=lo, M=M, T=T, phi=phi, S=S, e=e, u=beta * e, final=h, pad=pad)


def _tokens(v, L):
    """[b, nc, heads, CHUNK, d] -> [b, L, heads, d]."""
    return v.transpose(2, 3).flatten(1, 2)[:, :L]


def _plain_delta_fwd(s):
    c = _delta_chunks(s)
    y = c["start"] * (c["qh"] @ c["S"].mT) + c["M"] @ c["u"]
    return dict(y=_tokens(y, s["v"].shape[1]).to(s["v"].dtype).contiguous(), final=c["final"])


def _plain_delta_bwd(s):
    c = _delta_chunks(s)
    lam, tril, to_end, start, through, kh, qh, beta, lo, M, T, phi, S, e, u = (
        c[n] for n in ("lam", "tril", "to_end", "start", "through", "kh", "qh", "beta", "lo", "M", "T", "phi",
                       "S", "e", "u"))
    b, L, H, P = s["v"].shape
    G, N = s["k"].shape[2:]
    nc = S.shape[1]
    dyc = _chunks(s["dy"], c["pad"])
    # the gradient of the state after each chunk
    du_in = M.mT @ dyc
    dz_in = T.mT @ (beta * du_in)
    gain = (start * dyc).mT @ qh - (start * dz_in).mT @ kh
    g = s["dhT"] if s["dhT"] is not None else torch.zeros(b, H, P, N, device=S.device)
    D = torch.empty_like(S)
    for i in range(nc - 1, -1, -1):
        D[:, i] = g
        g = g @ phi[:, i].mT + gain[:, i]
    kd = to_end * (kh @ D.mT)
    du = du_in + kd
    dz = T.mT @ (beta * du)
    dm = dyc @ u.mT
    db = -(dz @ e.mT)
    dml, dbl = dm * lam, db * lam * tril.tril(-1) * beta.mT
    q_out = start * (dyc @ S)                                  # through the state before the chunk
    k_out = -start * (dz @ S)
    k_end = to_end * (u @ D)                                   # through the gradient after it
    dq = q_out + dml @ kh
    dk = k_out + k_end + dml.mT @ qh + dbl.mT @ kh + dbl @ kh
    dbeta = (du * e).sum(-1) + (db * lo).sum(-2)
    # log decays: every product that spans token t carries its decay once
    w = (dm * M + db * lo * beta.mT).double() * tril.tril(-1)
    from_start = ((q_out * qh).sum(-1) + (k_out * kh).sum(-1)).double()
    end = (kd * u).sum(-1).double()
    dE = w.sum(-1) - w.sum(-2) + from_start - end
    dE[..., -1] += end.sum(-1) + through.double()[..., 0, 0] * (S * D).sum((-1, -2)).double()
    dgate = _tokens(dE.flip(-1).cumsum(-1).flip(-1)[..., None].float(), L)[..., 0].contiguous()
    if s["seq"] is not None:                                   # a start takes nothing over
        dgate[:, 1:].masked_fill_((s["seq"][:, 1:] != s["seq"][:, :-1])[..., None], 0.0)
    t = s["v"].dtype

    def heads(x):  # the heads of a key head share it
        return _tokens(x.unflatten(2, (G, -1)).sum(3), L).to(t).contiguous()

    return dict(dq=heads(dq * s["scale"]), dk=heads(dk), dv=_tokens(dz, L).to(t).contiguous(),
                dbeta=_tokens(dbeta[..., None], L)[..., 0].contiguous(), dgate=dgate, dh0=g)


def _plain_delta_step(s):
    slots = s["slots"].long()
    h = s["pool"][slots]
    H, G = s["v"].shape[2], s["k"].shape[2]
    a = torch.exp(s["gate"])[..., None, None]
    ys = []
    for t in range(s["v"].shape[1]):
        k = s["k"][:, t].float().repeat_interleave(H // G, 1)[..., None]
        q = s["q"][:, t].float().repeat_interleave(H // G, 1)[..., None]
        h = a[:, t] * h
        e = s["v"][:, t].float()[..., None] - h @ k
        h = h + (s["beta"][:, t, :, None, None] * e) * k.mT
        ys.append((h @ q)[..., 0] * s["scale"])
    s["pool"][slots] = h
    return dict(y=torch.stack(ys, 1).to(s["v"].dtype), pool=s["pool"])


def _angles(s):
    """cos, sin [B, L, 1, R/2] of the rotation."""
    a = s["pos"].double()[..., None, None] * s["freq"].double()
    return a.cos().float(), a.sin().float()


def _turn(x, cos, sin, interleaved):
    """Pairs of x's first R channels turned by the angles; the rest as it is."""
    R = 2 * cos.shape[-1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _unit(x, kind):
    sq = x * x
    r = torch.rsqrt((sq.sum(-1, keepdim=True) if kind == "l2" else sq.mean(-1, keepdim=True)) + EPS)
    return x * r, r


def _plain_qk_fwd(s):
    case = s["case"]
    rot = _angles(s) if case["R"] else None

    def one(x, w):
        n = _unit(x.float(), case["kind"])[0]
        n = n if w is None else n * w
        return (n if rot is None else _turn(n, *rot, case["interleaved"])).to(x.dtype)

    return dict(q=one(s["q"], s["wq"]), k=one(s["k"], s["wk"]))


def _plain_qk_bwd(s):
    case = s["case"]
    if case["R"]:
        cos, sin = _angles(s)

    def one(x, w, dy):
        n, r = _unit(x.float(), case["kind"])
        d = dy.float()
        if case["R"]:
            d = _turn(d, cos, -sin, case["interleaved"])
        dw = None if w is None else (d * n).sum((0, 1, 2), dtype=torch.float64).float()
        d = d if w is None else d * w
        dn = (d * n).sum(-1, keepdim=True) if case["kind"] == "l2" else (d * n).mean(-1, keepdim=True)
        return (r * (d - n * dn)).to(x.dtype), dw

    dq, dwq = one(s["q"], s["wq"], s["dq"])
    dk, dwk = one(s["k"], s["wk"], s["dk"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def run(state):
    s = state
    case = s["case"]
    op = case["op"]
    if not own:
        return {"delta_scan_fwd": _plain_delta_fwd, "delta_scan_bwd": _plain_delta_bwd,
                "delta_scan_step": _plain_delta_step, "qk_norm_fwd": _plain_qk_fwd,
                "qk_norm_bwd": _plain_qk_bwd}[op](s)
    import ssm_sequence_models_amd as ssm
    if op == "delta_scan_fwd":
        y, final = ssm.delta_scan_fwd(s["q"], s["k"], s["v"], s["beta"], gate=s["gate"], scale=s["scale"],
                                      initial_state=s["h0"], seq_idx=s["seq"])
        return dict(y=y, final=final)
    if op == "delta_scan_bwd":
        dq, dk, dv, dbeta, dgate, dh0 = ssm.delta_scan_bwd(
            s["q"], s["k"], s["v"], s["beta"], s["dy"], gate=s["gate"], scale=s["scale"],
            initial_state=s["h0"], dfinal_state=s["dhT"], seq_idx=s["seq"])
        return dict(dq=dq, dk=dk, dv=dv, dbeta=dbeta, dgate=dgate, dh0=dh0)
    if op == "delta_scan_step":
        y = ssm.delta_scan_step(s["q"], s["k"], s["v"], s["beta"], s["pool"], gate=s["gate"],
                                scale=s["scale"], state_indices=s["slots"])
        return dict(y=y, pool=s["pool"])
    how = dict(q_weight=s["wq"], k_weight=s["wk"], eps=EPS, kind=case["kind"], inv_freq=s["freq"],
               positions=s["pos"], interleaved=case["interleaved"])
    if op == "qk_norm_fwd":
        q, k = ssm.qk_norm_fwd(s["q"], s["k"], **how)
        return dict(q=q, k=k)
    dq, dk, dwq, dwk = ssm.qk_norm_bwd(s["q"], s["k"], s["dq"], s["dk"], **how)
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("delta"):
        B, L, H, G, P, N = (case[k] for k in "BLHGPN")
        keys, values, state = B * L * G * N * es, B * L * H * P * es, B * H * P * N * 4
        rates, ids = B * L * H * 4, B * L * 4 if case["packed"] else 0
        if case["op"] == "delta_scan_bwd":
            # eight products of P x N a token and head: h k and u k^T again, dy q^T, dh k, dz k^T,
            # and dy h, u dh, dz h for dq and dk
            return dict(bytes=4 * keys + 3 * values + 4 * rates + (3 if case["states"] else 1) * state + ids,
                        flops=16.0 * B * L * H * P * N)
        # three: h k, u k^T, h q
        return dict(bytes=2 * keys + 2 * values + 2 * rates + (2 if case["states"] else 1) * state + ids,
                    flops=6.0 * B * L * H * P * N)
    n = case["B"] * case["L"] * (case["HQ"] + case["HK"]) * case["D"]
    bwd = case["op"] == "qk_norm_bwd"
    w = 8 * case["D"] * (2 if bwd else 1) if case["weights"] else 0
    p = case["B"] * case["L"] * 4 + case["R"] * 2 if case["R"] else 0
    return dict(bytes=n * es * (3 if bwd else 2) + w + p, flops=n * (14.0 if bwd else 6.0))


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _exact_delta(s):
    """Token by token: forward as defined (states kept at every SEG-th token and recomputed in
    between), backward from the derivative of one token's step."""
    case = s["case"]
    q, k, v, beta = s["q"].double(), s["k"].double(), s["v"].double(), s["beta"].double()
    b, L, H, P = v.shape
    G, N = k.shape[2:]
    rep = H // G
    dev = v.device
    a = torch.exp(s["gate"].double())
    if s["seq"] is not None:
        begins = torch.zeros(b, L, dtype=torch.bool, device=dev)
        begins[:, 1:] = s["seq"][:, 1:] != s["seq"][:, :-1]
        a = a.masked_fill(begins[..., None], 0.0)
    step = case["op"] == "delta_scan_step"
    if step:
        pool, at = s["pool"].double(), s["slots"].long()
        h = pool[at]
    else:
        h = s["h0"].double() if s["h0"] is not None else torch.zeros(b, H, P, N, device=dev, dtype=torch.float64)

    def col(x, t):  # a key head's vector for each of its heads, as a column
        return x[:, t].repeat_interleave(rep, 1).unsqueeze(-1)

    def token(h, t):
        kt = col(k, t)
        ah = a[:, t, :, None, None] * h
        e = v[:, t].unsqueeze(-1) - ah @ kt
        return torch.baddbmm(ah.flatten(0, 1), (beta[:, t, :, None, None] * e).flatten(0, 1),
                             kt.mT.contiguous().flatten(0, 1)).view_as(h), e

    bwd = case["op"] == "delta_scan_bwd"
    SEG = 64
    kept, y = [], None if bwd else torch.empty_like(v)
    for t in range(L):
        if bwd and t % SEG == 0:
            kept.append(h)
        h, _ = token(h, t)
        if not bwd:
            y[:, t] = (h @ col(q, t))[..., 0] * s["scale"]
    if step:
        pool[at] = h
        return dict(y=y, pool=pool)
    if not bwd:
        return dict(y=y, final=h)
    dy = s["dy"].double() * s["scale"]
    g = s["dhT"].double() if s["dhT"] is not None else torch.zeros_like(h)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dv, dbeta, dgate = torch.empty_like(v), torch.empty_like(beta), torch.empty_like(beta)
    for c in range(len(kept) - 1, -1, -1):
        t0, t1 = c * SEG, min(L, c * SEG + SEG)
        hs, es = [kept[c]], []
        for t in range(t0, t1):
            h, e = token(hs[-1], t)
            hs.append(h)
            es.append(e)
        for t in range(t1 - 1, t0 - 1, -1):
            before, after, e = hs[t - t0], hs[t - t0 + 1], es[t - t0]
            kt, qt, d = col(k, t), col(q, t), dy[:, t].unsqueeze(-1)
            bt, at = beta[:, t, :, None, None], a[:, t, :, None, None]
            g = g + d * qt.mT                                  # the gradient of h_t
            gk = g @ kt
            de = bt * gk                                       # of e_t
            ah = at * before
            dah = g - de * kt.mT                               # of a_t h_{t-1}
            dq[:, t] = (after.mT @ d)[..., 0].unflatten(1, (G, rep)).sum(2)
            dk[:, t] = (g.mT @ (bt * e) - ah.mT @ de)[..., 0].unflatten(1, (G, rep)).sum(2)
            dv[:, t] = de[..., 0]
            dbeta[:, t] = (gk * e)[..., 0].sum(-1)
            dgate[:, t] = (dah * ah).sum((-1, -2))
            g = at * dah
    return dict(dq=dq, dk=dk, dv=dv, dbeta=dbeta, dgate=dgate, dh0=g)


def _exact_qk(s):
    """Every head as defined; the rotation as a product of complex numbers, the backward from the
    Jacobian of x -> x / |x|."""
    case = s["case"]
    D, R = case["D"], case["R"]
    turn = None
    if R:
        ang = (s["pos"].double().unsqueeze(-1) * s["freq"].double()).unsqueeze(2)
        turn = torch.polar(torch.ones_like(ang), ang)

    def rotate(x, z):
        if z is None:
            return x
        y = x.clone()
        i = torch.arange(R // 2, device=x.device)
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
        c = torch.complex(x[..., first], x[..., second]) * z
        y[..., first], y[..., second] = c.real, c.imag
        return y

    def one(x, w, dy):
        x = x.double()
        n = 1 if case["kind"] == "l2" else D
        dev = (x.pow(2).sum(-1, keepdim=True) / n + EPS).sqrt()
        w = torch.ones(D, device=x.device, dtype=torch.float64) if w is None else w.double()
        if dy is None:
            return rotate(x / dev * w, turn)
        d = rotate(dy.double(), None if turn is None else turn.conj())
        dn = d * w
        return dn / dev - x * (dn * x).sum(-1, keepdim=True) / (n * dev ** 3), (d * x / dev).sum((0, 1, 2))

    if case["op"] == "qk_norm_fwd":
        return dict(q=one(s["q"], s["wq"], None), k=one(s["k"], s["wk"], None))
    (dq, dwq), (dk, dwk) = one(s["q"], s["wq"], s["dq"]), one(s["k"], s["wk"], s["dk"])
    if not case["weights"]:
        dwq = dwk = None
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_delta if case["op"].startswith("delta") else _exact_qk)(s)
