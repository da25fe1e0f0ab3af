"""GPU calls of more blocks than one dimension of a launch takes: 2^32 threads and more."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_qk_norm_of_many_tokens():
    import ssm_sequence_models_amd as ssm
    n = (1 << 27) + 9
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k = (torch.randn(1, n, 1, 1, device="cuda", dtype=BF16, generator=g) for _ in range(2))
    a, b = ssm.qk_norm_fwd(q, k, eps=0.0)
    assert torch.equal(a, torch.sign(q)) and torch.equal(b, torch.sign(k))
    w = torch.full((1,), 2.0, device="cuda")
    _, _, dw, _ = ssm.qk_norm_bwd(q, k, a, b, q_weight=w, k_weight=w, eps=0.0)
    # n d is 1 or 1 - 2^-24 (x^2 and its root are exact, 1 / x and x (1 / x) rounded once each), and 0 for x = 0; a
    # lane's sums of them, up to 4096, round to whole numbers, the blocks' (to 2^17) are exact, so are those in 64 bits:
    # the number of tokens, rounded once
    assert dw.item() == torch.tensor(int((q != 0).sum())).float().item()


def test_step_of_many_rows():
    """All but three rows skipped, whose outputs are 0."""
    import ssm_sequence_models_amd as ssm
    B, H, slots = 1 << 16, 1024, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    q, k, v, beta = r(B, 1, 1, 4).to(BF16), r(B, 1, 1, 4).to(BF16), r(B, 1, H, 1).to(BF16), torch.rand(B, 1, H, device="cuda")
    pool = r(slots, H, 1, 4)
    at = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, 40000, B - 1], device="cuda")
    at[rows] = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    few = pool.clone()
    want = ssm.delta_scan_step(q[rows], k[rows], v[rows], beta[rows], few, state_indices=at[rows])
    y = ssm.delta_scan_step(q, k, v, beta, pool, state_indices=at)
    assert torch.equal(y[rows], want) and torch.equal(pool, few)
    y[rows] = 0
    assert not y.any()
