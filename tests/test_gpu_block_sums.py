"""Sums over rows, tokens and sequences of the operators around the layer: their error does not grow
with the number of terms.  Equal rows make a sum in fp32 lose in one direction: S + t with S = n t is
rounded the same way for all S between two powers of two, by up to n e t (e = 2^-24), a relative
error of order n e at the end of a chain of n; 64-bit sums of short fp32 ones keep the short ones'.
Needs an MI355X.
"""
import numpy as np
import pytest
import torch

from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def normal(*shape, dtype=torch.float32, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def copies(v, n):
    return v.expand(n, *v.shape[1:]).contiguous()


@pytest.mark.parametrize("R,D,dtype,res", [(1 << 24, 16, "bf16", "bf16"), (1 << 22, 300, "bf16", "f32"),
                                           (1 << 20, 2500, "bf16", "bf16"), (1 << 18, 9000, "bf16", "bf16")])
def test_norm_weight_gradient_over_many_equal_rows(R, D, dtype, res):
    """dw = R dy n.  n = s r is off by (depth / 2 + 4) e with the row sum's depth min(D, 128) + 10; a lane adds at most
    64 rows in fp32, the rest is 64-bit: in all (64 + depth / 2 + 8) e."""
    t = {"bf16": torch.bfloat16, "f32": torch.float32}
    s, dy, w = normal(1, D, dtype=t[res], seed=1), normal(1, D, dtype=t[dtype], seed=2), 1 + 0.1 * normal(D, seed=3)
    dw = mesa.rmsnorm_bwd(copies(s, R), w, copies(dy, R), eps=1e-5)["dw"].double()
    sd = s[0].double()
    want = R * dy[0].double() * sd / torch.sqrt(sd.square().mean() + 1e-5)
    bound = (64 + 0.5 * (min(D, 128) + 10) + 8) * E * want.abs()
    assert ((dw - want).abs() <= bound).all(), float(((dw - want).abs() / want.abs()).max() / E)


@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("R,D", [(600_001, 5), (1_048_577, 16), (540_675, 130), (270_337, 301), (131_073, 1001), (131_071, 2048),
                                 (32_769, 2501), (65_537, 4104), (33_793, 9001), (65_535, 8200)])
def test_norm_weight_gradient_over_several_runs_of_rows(R, D, dtype, res):
    """Random rows in numbers that leave a last run short, full, or to some groups of a workgroup only, in every row
    group and at every end of a row; the bound as above, of the terms' magnitudes."""
    t = {"bf16": torch.bfloat16, "f32": torch.float32}
    s, dy, w = normal(R, D, dtype=t[res], seed=1), normal(R, D, dtype=t[dtype], seed=2), 1 + 0.1 * normal(D, seed=3)
    dres = normal(R, D, dtype=t[res], seed=4)
    got = mesa.rmsnorm_bwd(s, w, dy, d_residual=dres, eps=1e-5)
    want, size = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    depth = 0.5 * (min(D, 128) + 10)
    for i in range(0, R, 1 << 15):
        sd, d = s[i:i + (1 << 15)].double(), dy[i:i + (1 << 15)].double()
        r = 1 / torch.sqrt(sd.square().mean(1, keepdim=True) + 1e-5)
        n, g = sd * r, d * w.double()
        want += (d * n).sum(0)
        size += (d * n).abs().sum(0)
        ds = r * (g - n * (g * n).mean(1, keepdim=True)) + dres[i:i + (1 << 15)].double()
        mag = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
        half = 2.0 ** -8 if res == "bf16" else E
        assert ((got["ds"][i:i + (1 << 15)].double() - ds).abs() <= (3 * depth + 12) * E * mag + (half + 2 * E) * ds.abs()).all(), i
    assert ((got["dw"].double() - want).abs() <= (64 + depth + 8) * E * size).all()


@pytest.mark.parametrize("T,n", [(6, 1 << 18), (30, 1 << 17), (64, 1 << 16), (200, 1 << 14)])
def test_decay_parameter_gradient_over_many_equal_sequences(T, n):
    """Copies of one sequence: a power of two times its gradient, bit for bit."""
    D = 8
    x, ga, gi, dy = (normal(1, T, D, seed=i) for i in range(4))
    lam = normal(D, seed=5) - 5
    one = mesa.lru_bwd(x, ga, gi, lam, dy)["dlam"]
    many = mesa.lru_bwd(*(copies(v, n) for v in (x, ga, gi)), lam, copies(dy, n))["dlam"]
    torch.cuda.synchronize()
    assert one.abs().min() > 0 and torch.equal(many, one * n), float(((many / (one * n)) - 1).abs().max() / E)


def test_decay_parameter_gradient_over_a_long_sequence():
    """Equal tokens from the state that they keep (h = u / (1 - a), g alike): every token's v is the same but for its
    state's and adjoint's rounding.  2^21 tokens, a = 0.5 .. 0.9.

    v = -log(a) g ((a^2 / m) s_i x - a h).  With w = -2 log(a) <= 2, |ga|, |gi| <= 1 and m >= 0.4, the gates, a, m and the
    quotient are off by at most 60 e; h and g sum at most 1 / (1 - a) = 10 tokens' worth of such errors; the two terms of
    the difference add in magnitude.  A tile adds 64 tokens with 14 roundings."""
    T, D = 1 << 21, 8
    gen = np.random.default_rng(4)
    a = np.linspace(0.5, 0.9, D)
    ga, gi, x, dy = (gen.uniform(-1, 1, D).astype(np.float32) for _ in range(4))
    sr, si = 1 / (1 + np.exp(-ga.astype(np.float64))), 1 / (1 + np.exp(-gi.astype(np.float64)))
    lam = np.log(np.expm1(-np.log(a) / (8 * sr))).astype(np.float32)
    w = 16 * np.log1p(np.exp(lam.astype(np.float64))) * sr
    a, m = np.exp(-w / 2), np.sqrt(-np.expm1(-w))
    u = m * si * x
    h, g = u / (1 - a), dy / (1 - a)
    slope = 1 / (1 + np.exp(-lam.astype(np.float64))) / np.log1p(np.exp(lam.astype(np.float64)))
    want = T * 0.5 * w * g * (a * a / m * si * x - a * h) * slope
    size = T * 0.5 * w * np.abs(g) * (a * a / m * np.abs(si * x) + a * np.abs(h)) * slope
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    rows = [dev(v)[None, None].expand(1, T, D).contiguous() for v in (x, ga, gi)]
    got = mesa.lru_bwd(*rows, dev(lam), dev(dy)[None, None].expand(1, T, D).contiguous(), h0=dev(h.astype(np.float32))[None],
                       d_hfinal=dev((a * g).astype(np.float32))[None])["dlam"].cpu().numpy()
    # the initial state and the last adjoint are rounded too: 10 e and a few tokens of 2^21
    assert (np.abs(got - want) <= (2 * 60 * 10 + 14) * E * size).all(), (np.abs(got - want) / size / E).max()


@pytest.mark.parametrize("d", [16, 64, 128])
def test_tap_gradient_over_many_equal_sequences(d):
    """Copies of one token and its history: a power of two times its gradient, bit for bit."""
    H, W, n = 1, 4, (1 << 15) * 16 // d
    q, k, qh, kh = (normal(1, H, r, d, seed=i) for i, r in enumerate((1, 1, W - 1, W - 1)))
    dq, dk = normal(1, H, 1, d, seed=4), normal(1, H, 1, d, seed=5)
    w = normal(H, d, W, seed=6), normal(H, d, W, seed=7)
    one = mesa.qk_preprocess_bwd(q, k, *w, dq, dk, q_hist=qh, k_hist=kh)
    many = mesa.qk_preprocess_bwd(copies(q, n), copies(k, n), *w, copies(dq, n), copies(dk, n), q_hist=copies(qh, n),
                                  k_hist=copies(kh, n))
    torch.cuda.synchronize()
    for key in ("dw_q", "dw_k"):
        assert torch.equal(many[key], one[key] * n), (key, float(((many[key] / (one[key] * n)) - 1).abs().max() / E))


@pytest.mark.parametrize("d,T", [(16, 1 << 22), (128, 1 << 19)])
def test_tap_gradient_over_many_equal_tokens(d, T):
    """dw[j][i] = T e[j] x[j] for equal rows (history alike).  e = (d - o <o, d>) / n is off by some 60 e of its terms'
    magnitudes (5 of the convolution, as much again of the norm's, a tree of 5 levels, quotients); a lane adds at most 29
    tokens in fp32."""
    H, W = 1, 4
    q, dq = normal(1, H, 1, d, seed=1), normal(1, H, 1, d, seed=2)
    w = normal(H, d, W, seed=3)
    rows = lambda v, n: v.expand(1, H, n, d).contiguous()  # noqa: E731
    r = mesa.qk_preprocess_bwd(rows(q, T), rows(q, T), w, w, rows(dq, T), rows(dq, T), q_hist=rows(q, W - 1),
                               k_hist=rows(q, W - 1))
    x, g, s = q[0, 0, 0].double(), dq[0, 0, 0].double(), w[0].double().sum(-1)
    y = s * x
    n = y.norm()
    o = y / n
    e, size = (g - o * (o * g).sum()) / n, (g.abs() + o.abs() * (o * g).abs().sum()) / n
    # (the taps' sum cancels: the convolution's error counts against their magnitudes)
    spread = float((w[0].double().abs().sum(-1) * x.abs()).norm() / n)
    for key in ("dw_q", "dw_k"):
        got = r[key][0].double()
        bound = (60 * spread + 29 + 4) * E * T * size * x.abs()
        assert ((got - (T * e * x)[:, None]).abs() <= bound[:, None]).all(), key
