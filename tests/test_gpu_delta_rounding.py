"""Gated delta rule on the GPU: results in bf16 are rounded once, from numbers of fp32's precision.

x = 1 + 2^-8 + 2^-18 lies 2^-18 above the middle between two neighbours of bf16, 1 and 1 + 2^-7, and
rounds to the upper one.  Its first bf16 part is 1 + 2^-7 and its second -2^-8 (the rest needs a third),
so the sum of two is the middle itself, which rounds to 1.  In every case here all products and sums are
x times small powers of two or sums of few of them, exact in fp32, so the results are the oracle's,
rounded, bit for bit.  Needs an MI355X.
"""
import numpy as np
import pytest
import torch

from delta_helpers import to_dev
from oracle.delta_oracle import delta_backward, delta_forward
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu

X = 1 + 2.0 ** -8 + 2.0 ** -18
NAMES = ("q", "k", "v", "gamma", "beta")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def zeros(B, H, Hk, T, dk, dv):
    return dict(q=np.zeros((B, Hk, T, dk)), k=np.zeros((B, Hk, T, dk)), v=np.zeros((B, H, T, dv)),
                d_o=np.zeros((B, H, T, dv)), gamma=np.ones((B, H, T)), beta=np.zeros((B, H, T)), s0=None, d_sfinal=None,
                lengths=None)


def powers(rng, *shape):
    return rng.choice([-1.0, 1.0], shape) * 2.0 ** rng.integers(-3, 4, shape)


def rounded(want):
    one = torch.from_numpy(want).float()
    assert bool((one.double() == torch.from_numpy(want)).all())  # (so the oracle's numbers are exact)
    return one.to(torch.bfloat16)


def check_forward(a):
    t = to_dev(a, torch.bfloat16)
    got = mesa.delta_fwd(*(t[n] for n in NAMES), s0=t["s0"])["o"]
    want = delta_forward(*(a[n] for n in NAMES), s0=a["s0"])["o"]
    assert torch.equal(got.cpu(), rounded(want))
    return want


def check_backward(a):
    t = to_dev(a, torch.bfloat16)
    got = mesa.delta_bwd(*(t[n] for n in NAMES), t["d_o"], s0=t["s0"])
    want = delta_backward(*(a[n] for n in NAMES), a["d_o"], s0=a["s0"])
    for n in ("dq", "dk", "dv"):
        assert torch.equal(got[n].cpu(), rounded(want[n])), n
    return want


@pytest.mark.parametrize("dk,dv", [(32, 16), (64, 80), (128, 64)])
@pytest.mark.parametrize("T", [1, 100, 1300])
def test_what_queries_read_of_a_state(T, dk, dv):
    """beta = 0 and gamma = 1: o_t is a column of s0.  1300 tokens go in segments."""
    rng = np.random.default_rng([T, dk])
    a = zeros(1, 2, 2, T, dk, dv)
    a["k"][..., 0] = 1.0
    a["q"][:, :, np.arange(T), np.arange(T) % dk] = 1.0
    a["v"][:] = powers(rng, 1, 2, T, dv)
    a["s0"] = X * powers(rng, 1, 2, dv, dk)
    check_forward(a)


@pytest.mark.parametrize("dk,dv", [(32, 16), (64, 80), (128, 64)])
def test_what_queries_read_of_earlier_tokens(dk, dv):
    """Orthonormal keys: a query that is token j's key reads beta_j v_j, from its own chunk and at dk = 128 from the one before."""
    rng = np.random.default_rng(dk)
    a = zeros(1, 2, 2, dk, dk, dv)
    at = np.arange(dk)
    a["k"][:, :, at, at] = 1.0
    a["q"][:, :, at, np.where(at < 20, at, at - 20)] = 1.0
    a["v"][:] = powers(rng, 1, 2, dk, dv)
    a["beta"][:] = X / 2 ** rng.integers(0, 3, (1, 2, dk))
    check_forward(a)


@pytest.mark.parametrize("dk", [32, 64, 128])
def test_products_of_queries_and_keys(dk):
    """q.k = x, of three products."""
    rng = np.random.default_rng(dk)
    a = zeros(1, 2, 2, 64, dk, 32)
    a["k"][..., :3] = 1.0
    a["q"][..., :3] = 1.0, 2.0 ** -8, 2.0 ** -18
    a["v"][:] = powers(rng, 1, 2, 64, 32)
    a["beta"][:, :, 0] = 1.0
    check_forward(a)


@pytest.mark.parametrize("Hk", [1, 2])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("second", [1, 17, 63, 70])
@pytest.mark.parametrize("strength", [0.0, 1.0])
def test_gradients_of_pairs(strength, second, dk, Hk):
    """Two tokens on one key, the first with beta = x; the second, with 1 or nothing written, alone has a query and a
    gradient (at 70 in the chunk behind: what the first leaves is in the state)."""
    a = zeros(1, 2, Hk, 71, dk, 16)
    a["k"][..., 0] = 1.0
    a["q"][:, :, second, :2] = 1.0
    a["v"][:, 0, 0, 3], a["v"][:, 1, 0, 3] = 1.0, -0.125
    a["beta"][:, :, 0], a["beta"][:, :, second] = X, strength
    a["d_o"][:, :, second, 3] = 1.0
    want = check_backward(a)
    assert np.abs(want["dk"][:, :, 0, 1]).max() >= 7 / 8
    assert np.abs(want["dk"][:, :, second, 0]).max() >= 7 / 4 if strength else np.abs(want["dq"][:, :, second, 0]).max() >= 7 / 8
