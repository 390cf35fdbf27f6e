"""Arrays of more than 2^31 elements: every copy of a small problem, the sums over all of them, and
a carry along one long sequence that decays slowly.  Needs an MI355X.
"""
import pytest
import torch

from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def normal(*shape, dtype=torch.bfloat16, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def copies(v, n):
    return v.repeat(n, *[1] * (v.dim() - 1))


def all_equal(big, small, n, what):
    """Each of the n copies, byte for byte."""
    big, small = big.view(torch.uint8), small.view(torch.uint8)
    for i, part in enumerate(big.chunk(n)):
        assert torch.equal(part, small), (what, i)


def test_recurrence_sums_and_copies():
    """dlam: the same partial sums n times, added in 64 bits: n times the small call's but for the roundings of both."""
    B, T, D, n = 2, 4096, 2048, 130
    x, ga, gi, dy = (normal(B, T, D, seed=i) for i in range(4))
    lam = normal(D, dtype=torch.float32, seed=5) - 4
    h0, last = normal(B, D, dtype=torch.float32, seed=6), normal(B, D, dtype=torch.float32, seed=7)
    lengths = torch.tensor([T, 3001], dtype=torch.int32, device="cuda")

    def run(x, ga, gi, dy, h0, last, lengths):
        r = mesa.lru_fwd(x, ga, gi, lam, h0=h0, lengths=lengths, return_state=True)
        r.update(mesa.lru_bwd(x, ga, gi, lam, dy, h0=h0, lengths=lengths, d_hfinal=last, state_grads=True))
        torch.cuda.synchronize()
        return r

    args = (x, ga, gi, dy, h0, last, lengths)
    small = run(*args)
    big = run(*(copies(v, n) for v in args))
    for k in ("y", "h_final", "dx", "dga", "dgi", "dh0"):
        all_equal(big[k], small[k], n, k)
    want = n * small["dlam"].double()
    assert ((big["dlam"].double() - want).abs() <= 3 * E * want.abs()).all()


def test_norm_sums_and_copies():
    """dw against 64-bit sums, with the bound of one lane's 64 rows in fp32 and each term's own error
    (test_gpu_norm.py: (depth / 2 + 12) e with depth 138)."""
    R, D, n = 4096, 2048, 257
    x, res, dy, dres = (normal(R, D, seed=i) for i in range(4))
    w = 1 + 0.1 * normal(D, dtype=torch.float32, seed=5)
    for group in (None, 0, 128):
        small = mesa.rmsnorm(x, w, residual=res, quant_group=group)
        big = mesa.rmsnorm(copies(x, n), w, residual=copies(res, n), quant_group=group)
        torch.cuda.synchronize()
        for k in small:
            all_equal(big[k], small[k], n, (group, k))
        del big
    small = mesa.rmsnorm_bwd(res, w, dy, d_residual=dres)
    big = mesa.rmsnorm_bwd(copies(res, n), w, copies(dy, n), d_residual=copies(dres, n))
    torch.cuda.synchronize()
    all_equal(big["ds"], small["ds"], n, "ds")
    s = res.double()
    terms = dy.double() * s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-6)
    bound = (64 + 0.5 * 138 + 12) * E * terms.abs().sum(0)
    assert ((small["dw"].double() - terms.sum(0)).abs() <= bound).all()
    assert ((big["dw"].double() - n * terms.sum(0)).abs() <= n * bound).all()


def test_preprocessing_sums_and_copies():
    """Both calls walk alike, so their partial sums are equal and the 64-bit sums multiples of one another."""
    B, H, T, d, W, n, few = 1, 16, 2048, 128, 4, 520, 8
    q, k = normal(B, H, T, d, seed=1), normal(B, H, T, d, seed=2)
    dq, dk = normal(B, H, T, d, dtype=torch.float32, seed=3), normal(B, H, T, d, dtype=torch.float32, seed=4)
    w = normal(H, d, W, dtype=torch.float32, seed=5), normal(H, d, W, dtype=torch.float32, seed=6)
    one = mesa.qk_preprocess_bwd(copies(q, few), copies(k, few), *w, copies(dq, few), copies(dk, few))
    big = mesa.qk_preprocess_bwd(copies(q, n), copies(k, n), *w, copies(dq, n), copies(dk, n))
    torch.cuda.synchronize()
    for name in ("dq_raw", "dk_raw"):
        all_equal(big[name], one[name][:1], n, name)
    for name in ("dw_q", "dw_k"):
        want = one[name].double() * (n / few)
        assert ((big[name].double() - want).abs() <= 3 * E * want.abs()).all(), name


def test_slow_decay_along_one_long_sequence():
    """1.1 M tokens that forget over 100 to 100 000 tokens, forward and backward, in one call and in two that hand the
    state and its gradient on.

    With r = -log(a) of a channel's slowest token, an error of 4 e of the largest state (or adjoint) a token adds up over
    1/r tokens to 4 e / r of it, in either call (b: both); to that come two roundings to bf16.  A carry that is lost or
    taken from another tile is off by the order of the state itself: b is below 0.025 of the largest one where a state
    lasts for 32768 tokens (256 tiles forward, 512 backward), below 0.15 everywhere."""
    T, D, cut, c = 1_100_000, 2048, 524_287, 8.0
    assert T * D > 2 ** 31
    x, ga, gi, dy = (normal(1, T, D, seed=i) for i in range(4))
    ga.clamp_(-0.5, 0.5)
    rate = torch.logspace(-5, -2, D, dtype=torch.float64, device="cuda")
    lam = torch.log(torch.expm1(rate / c)).float()      # r = rate sigmoid(ga)
    b = 2 * 4 * E / (rate * torch.sigmoid(torch.tensor(-0.5, device="cuda").double()))
    halves = [[v[:, :cut] for v in (x, ga, gi, dy)], [v[:, cut:] for v in (x, ga, gi, dy)]]
    y = mesa.lru_fwd(x, ga, gi, lam, c=c)["y"]
    g = mesa.lru_bwd(x, ga, gi, lam, dy, c=c, state_grads=True)
    first = mesa.lru_fwd(*halves[0][:3], lam, c=c, return_state=True)
    second = mesa.lru_fwd(*halves[1][:3], lam, c=c, h0=first["h_final"])
    g2 = mesa.lru_bwd(*halves[1][:3], lam, halves[1][3], c=c, h0=first["h_final"], state_grads=True)
    g1 = mesa.lru_bwd(*halves[0][:3], lam, halves[0][3], c=c, d_hfinal=g2["dh0"], state_grads=True)
    torch.cuda.synchronize()
    chunks = [(h, t, min(t + 32768, hi)) for h, lo, hi in ((0, 0, cut), (1, cut, T)) for t in range(lo, hi, 32768)]

    def gates(t, u):
        sr, si = torch.sigmoid(ga[0, t:u].float()), torch.sigmoid(gi[0, t:u].float())
        r = rate.float() * sr
        return sr, si, r, torch.sqrt(-torch.expm1(-2 * r))

    hmax, gmax = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
    for _, t, u in chunks:
        _, si, _, m = gates(t, u)
        hmax = torch.maximum(hmax, y[0, t:u].float().abs().amax(0))
        gmax = torch.maximum(gmax, (g["dx"][0, t:u].float() / (m * si)).abs().amax(0))
    assert hmax.min() > 0.5 and gmax.min() > 0.5
    eh, eg = b.float() * hmax, b.float() * gmax
    assert (b < 0.15).all() and (b[rate < 6e-5] < 0.13).all() and (b[rate > 6e-5] < 0.025).all()
    half = 2 * 2.0 ** -8
    for h, t, u in chunks:
        lo = (0, cut)[h]
        part, grads = (first, second)[h], (g1, g2)[h]
        sr, si, r, m = gates(t, u)
        xv = x[0, t:u].float().abs()
        bounds = {"dx": m * si * eg, "dgi": m * si * xv * (1 - si) * eg,
                  "dga": r * (1 - sr) * (eg * (si * xv / m + hmax) + gmax * eh)}
        got, want = y[0, t:u].float(), part["y"][0, t - lo:u - lo].float()
        assert ((got - want).abs() <= half * want.abs() + eh).all(), ("y", t)
        for k, bound in bounds.items():
            got, want = g[k][0, t:u].float(), grads[k][0, t - lo:u - lo].float()
            assert ((got - want).abs() <= half * want.abs() + bound + 1e-30).all(), (k, t)
    assert ((g["dh0"] - g1["dh0"]).abs() <= eg).all()
