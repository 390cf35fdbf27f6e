"""The operators around the layer on arrays of more than 2^31 elements: copies of one
small problem, whose results have the small call's bits wherever they lie.
Needs an MI355X.
"""
import pytest
import torch

from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def normal(*shape, dtype=torch.bfloat16, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def copies(v, n):
    return v.repeat(n, *[1] * (v.dim() - 1))


def test_recurrence_over_many_sequences():
    B, T, D, n = 2, 4096, 2048, 130
    x, ga, gi, dy = (normal(B, T, D, seed=i) for i in range(4))
    lam = normal(D, dtype=torch.float32, seed=5) - 4
    h0, last = normal(B, D, dtype=torch.float32, seed=6), normal(B, D, dtype=torch.float32, seed=7)
    lengths = torch.tensor([T, 3001], dtype=torch.int32, device="cuda")
    small = mesa.lru_fwd(x, ga, gi, lam, h0=h0, lengths=lengths, return_state=True)
    small.update(mesa.lru_bwd(x, ga, gi, lam, dy, h0=h0, lengths=lengths, d_hfinal=last, state_grads=True))
    assert n * B * T * D > 2 ** 31
    x, ga, gi, dy, h0, last, lengths = (copies(v, n) for v in (x, ga, gi, dy, h0, last, lengths))
    ws = torch.empty(mesa.lru_workspace_bytes(n * B, T, D), dtype=torch.uint8, device="cuda")
    big = mesa.lru_fwd(x, ga, gi, lam, h0=h0, lengths=lengths, return_state=True, workspace=ws)
    big.update(mesa.lru_bwd(x, ga, gi, lam, dy, h0=h0, lengths=lengths, d_hfinal=last, state_grads=True, workspace=ws,
                            states_in_workspace=True))
    torch.cuda.synchronize()
    for k in ("y", "h_final", "dx", "dga", "dgi", "dh0"):
        for i in (0, n // 2, n - 1):
            assert torch.equal(big[k][i * B:(i + 1) * B], small[k]), (k, i)


def test_recurrence_over_one_long_sequence():
    """Gates that leave at most exp(-8 softplus(1) / 2) = 0.0053 of a state a token: a call on the last tokens alone
    agrees from its 60th on but for two roundings to bf16 and fp32 noise."""
    T, D, tail = 1_100_000, 2048, 700
    assert T * D > 2 ** 31
    x, ga, gi = normal(1, T, D, seed=1), normal(1, T, D, seed=2).abs_(), normal(1, T, D, seed=3)
    lam = torch.ones(D, device="cuda")
    y = mesa.lru_fwd(x, ga, gi, lam)["y"]
    end = mesa.lru_fwd(*(v[:, -tail:].contiguous() for v in (x, ga, gi)), lam)["y"]
    torch.cuda.synchronize()
    got, want = y[:, 60 - tail:].float(), end[:, 60:].float()
    assert ((got - want).abs() <= (2 * 2.0 ** -8 + 1e-5) * want.abs() + 1e-6).all()
    assert (want.abs() > 0.1).float().mean() > 0.3


def test_norm_over_many_rows():
    R, D, n = 4096, 2048, 257
    x, res, dy, dres = (normal(R, D, seed=i) for i in range(4))
    w = 1 + 0.1 * normal(D, dtype=torch.float32, seed=5)
    assert n * R * D > 2 ** 31
    for group in (None, 128):
        small = mesa.rmsnorm(x, w, residual=res, quant_group=group)
        big = mesa.rmsnorm(copies(x, n), w, residual=copies(res, n), quant_group=group)
        torch.cuda.synchronize()
        for k in small:
            for i in (0, n // 2, n - 1):
                assert torch.equal(big[k][i * R:(i + 1) * R].view(torch.uint8), small[k].view(torch.uint8)), (group, k, i)
        del big
    small = mesa.rmsnorm_bwd(res, w, dy, d_residual=dres)
    big = mesa.rmsnorm_bwd(copies(res, n), w, copies(dy, n), d_residual=copies(dres, n))
    torch.cuda.synchronize()
    for i in (0, n // 2, n - 1):
        assert torch.equal(big["ds"][i * R:(i + 1) * R], small["ds"]), i


def test_preprocessing_gradient_over_many_sequences():
    B, H, T, d, W, n = 1, 16, 2048, 128, 4, 520
    q, k = normal(B, H, T, d, seed=1), normal(B, H, T, d, seed=2)
    dq, dk = normal(B, H, T, d, dtype=torch.float32, seed=3), normal(B, H, T, d, dtype=torch.float32, seed=4)
    w_q, w_k = normal(H, d, W, dtype=torch.float32, seed=5), normal(H, d, W, dtype=torch.float32, seed=6)
    assert n * B * H * T * d > 2 ** 31
    one = mesa.qk_preprocess_bwd(*(copies(v, 8) for v in (q, k)), w_q, w_k, *(copies(v, 8) for v in (dq, dk)))
    big = mesa.qk_preprocess_bwd(*(copies(v, n) for v in (q, k)), w_q, w_k, *(copies(v, n) for v in (dq, dk)))
    torch.cuda.synchronize()
    for name in ("dq_raw", "dk_raw"):
        for i in (0, n // 2, n - 1):
            assert torch.equal(big[name][i], one[name][0]), (name, i)
