"""The norm as the last step of the layer's own paths (conv_scan_fwd, decode_step with `norm`):
bit for bit what norm_fwd gives on their y, whose parity has tests of its own, with every gate
order, groups and bias; a prefill continued by decode steps, against the 64-bit norm; a captured
decode step, replayed."""
import pytest
import torch

from gpu_util import TOL_ABS, TOL_REL
from test_gpu_9b_decode_step import _bits, _case
from test_gpu_a_norm import _check
from train_ref import half_step, norm64

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _norm(rows, C, seed, gate, bias, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    how = dict(weight=1.0 + 0.25 * torch.randn(C, generator=g))
    if bias:
        how["bias"] = 0.5 * torch.randn(C, generator=g)
    if gate != "none":
        how["z"] = (2.0 * torch.randn(*rows, C, generator=g)).to(dtype)
        how["norm_before_gate"] = gate == "after"
    return how


def _cuda(how):
    return {k: v.to("cuda") if isinstance(v, torch.Tensor) else v for k, v in how.items()}


@pytest.mark.parametrize("gate,kind,groups,bias,L", [("before", "rms", 1, False, 1),
                                                     ("after", "layer", 2, True, 3),
                                                     ("none", "rms", 4, False, 1)])
def test_decode_step(gate, kind, groups, bias, L):
    import ssm_sequence_models_amd as ssm
    H, P, N, G = 4, 64, 64, 1
    c = _case(6, 9, H, P, N, G, 4, 4, L, 11)
    d = _cuda(c)
    how = dict(_cuda(_norm((6, L), H * P, 5, gate, bias)), kind=kind, ngroups=groups)

    def step(pool, spool, **more):
        return ssm.decode_step(d["x"], pool, d["w"], d["b"], d["dt"], d["A"], spool, H, P, G, N,
                               conv_state_indices=d["idx"], cache_seqlens=d["seqlens"], **more)
    pool, spool = d["pool"].clone(), d["spool"].clone()
    y = step(pool, spool)
    want = ssm.norm_fwd(y.reshape(6, L, H * P), **how)
    pool2, spool2 = d["pool"].clone(), d["spool"].clone()
    y2 = torch.empty_like(y)
    got = step(pool2, spool2, y=y2, norm=how)
    assert got.shape == (6, L, H * P)
    assert torch.equal(_bits(y2), _bits(y)) and torch.equal(_bits(got), _bits(want))
    assert torch.equal(_bits(pool2), _bits(pool)) and torch.equal(_bits(spool2), _bits(spool))
    # a refused norm leaves the pools as they were
    pool3, spool3 = d["pool"].clone(), d["spool"].clone()
    with pytest.raises(ValueError):
        step(pool3, spool3, norm=dict(how, ngroups=3))
    assert torch.equal(_bits(pool3), _bits(d["pool"])) and torch.equal(_bits(spool3), _bits(d["spool"]))


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_prefill_then_decode(dtype):
    """conv_scan_fwd with norm over a prompt, then decode_step with norm, token by token, on the
    states it left: the rows of one prefill of everything, normed."""
    import ssm_sequence_models_amd as ssm
    B, L, T, H, P, G, N, K = 2, 70, 3, 2, 64, 1, 64, 4
    C = H * P + 2 * G * N
    g = torch.Generator().manual_seed(3)
    xBC = torch.randn(B, L + T, C, generator=g).to(dtype).cuda()
    w, b = (torch.rand(C, K, generator=g) - 0.5).cuda(), (torch.rand(C, generator=g) - 0.5).cuda()
    dt = torch.nn.functional.softplus(torch.randn(B, L + T, H, generator=g) - 2.0).cuda()
    A = -torch.exp(torch.rand(H, generator=g) * 2.0).cuda()
    host = _norm((B, L + T), H * P, 8, "before", False, dtype)
    how = _cuda(host)
    y, _, _ = ssm.conv_scan_fwd(xBC, w, b, dt, A, H, P, G, N)
    out, conv_state, state = ssm.conv_scan_fwd(
        xBC[:, :L].contiguous(), w, b, dt[:, :L].contiguous(), A, H, P, G, N,
        norm=dict(how, z=how["z"][:, :L].contiguous()))
    ref = norm64(y[:, :L].reshape(-1, H * P).cpu(), host["weight"], None,
                 host["z"][:, :L].reshape(-1, H * P), 1e-5, "rms", 1, False)
    _check(out.view(-1, H * P), ref, "out", dtype)
    for t in range(L, L + T):
        yt = torch.empty(B, 1, H, P, dtype=dtype, device="cuda")
        z = how["z"][:, t:t + 1]  # rows at a stride
        got = ssm.decode_step(xBC[:, t].unsqueeze(-1).contiguous(), conv_state, w, b,
                              dt[:, t:t + 1].contiguous(), A, state, H, P, G, N, y=yt,
                              norm=dict(how, z=z))
        ref = norm64(yt.view(B, H * P).cpu(), host["weight"], None, host["z"][:, t], 1e-5, "rms",
                     1, False)
        _check(got.view(B, H * P), ref, "out", dtype)
        # the prefill's own y of that token: both round to the type (half a step each), from fp32
        # values that are within the scan tests' tolerances of the exact ones
        assert torch.allclose(yt[:, 0].double(), y[:, t].double(), atol=2 * TOL_ABS,
                              rtol=2 * (TOL_REL + half_step(dtype)))


def test_captured_decode_step():
    import ssm_sequence_models_amd as ssm
    H, P, N, G = 4, 64, 64, 1
    d = _cuda(_case(6, 9, H, P, N, G, 4, 4, 1, 12))
    how = _cuda(_norm((6, 1), H * P, 6, "before", False))
    pool, spool = d["pool"].clone(), d["spool"].clone()
    y, co = torch.empty(6, 1, H, P, dtype=BF16, device="cuda"), torch.empty_like(d["x"])
    out = torch.empty(6, 1, H * P, dtype=BF16, device="cuda")

    def step(pool, spool, out):
        ssm.decode_step(d["x"], pool, d["w"], d["b"], d["dt"], d["A"], spool, H, P, G, N,
                        conv_state_indices=d["idx"], cache_seqlens=d["seqlens"], conv_out=co, y=y,
                        norm=dict(how, out=out))
    eager, epool, espool = torch.empty_like(out), pool.clone(), spool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pool, spool, out)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        step(epool, espool, eager)
        torch.cuda.synchronize()
        assert torch.equal(_bits(out), _bits(eager)) and torch.equal(_bits(spool), _bits(espool))
