"""Gated delta rule on the GPU: the gradient at small forget factors, down to 0, against the fp64 oracle.

The bound is delta_helpers' for dgamma, on dgamma itself: 20 stages of 2^-23 of the sizes of the two terms
whose difference it is, in the 2-norm over a head and 16 times that number by number.  Needs an MI355X.
"""
import numpy as np
import pytest
import torch

from delta_helpers import draw, e32, to_dev
from oracle.delta_oracle import delta_backward
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "gamma", "beta")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# 0, the smallest subnormal and normal numbers of fp32 and others between, both sides of 2^-64
SMALL = [0.0, 2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 2.0 ** -125, 2.0 ** -100, 2.0 ** -64, 2.0 ** -65, 1.25 * 2.0 ** -64,
         2.0 ** -40, 2.0 ** -20, 2.0 ** -10]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def check(a, dt, layout="heads", walks=1):
    a["gamma"] = a["gamma"].astype(np.float32).astype(np.float64)
    t = to_dev(a, dt, layout)
    r = mesa.delta_bwd(*(t[n] for n in NAMES), t["d_o"], s0=t["s0"], lengths=t["lengths"], d_sfinal=t["d_sfinal"])
    want = delta_backward(*(a[n] for n in NAMES), a["d_o"], s0=a["s0"], lengths=a["lengths"], d_sfinal=a["d_sfinal"])
    off = np.abs(r["dgamma"].double().cpu().numpy() - want["dgamma"])
    size = want["dgamma_sizes"] + np.abs(want["dgamma"])
    e, norm = e32(a, 20 * walks), np.linalg.norm(size, axis=-1)
    assert np.isfinite(off).all()
    assert np.all(np.linalg.norm(off, axis=-1) <= e * norm), np.max(np.linalg.norm(off, axis=-1) / np.maximum(norm, 1e-300))
    assert np.all(off <= 16 * e * np.maximum(size, norm[..., None] / np.sqrt(size.shape[-1])))
    return want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(32, 16), (64, 80), (128, 128)])
@pytest.mark.parametrize("value", SMALL)
def test_one_value(value, dk, dv, dtype):
    """At the ends of tiles and chunks and between, in one head alone too."""
    a = draw(2, 2, 2, 150, dk, dv, DTYPES[dtype], seed=4)
    at = [0, 15, 16, 50, 63, 64, 127, 149]
    a["gamma"][0, :, at] = value
    a["gamma"][1, 1, 70] = value
    want = check(a, DTYPES[dtype])
    assert np.median(np.abs(want["dgamma"][0][:, at])) > 0.05


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_neighbours(dtype):
    """Small factors side by side: a gradient that reaches over one of them is that much smaller."""
    a = draw(1, 4, 2, 130, 64, 48, DTYPES[dtype], seed=5)
    for h, pair in enumerate([(0.0, 0.0), (0.0, 2.0 ** -70), (2.0 ** -100, 2.0 ** -100), (2.0 ** -30, 2.0 ** -66)]):
        for i in (1, 31, 62, 63, 100):
            a["gamma"][0, h, i:i + 2] = pair
    check(a, DTYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_all_of_a_chunk(dtype):
    a = draw(1, 3, 1, 200, 128, 64, DTYPES[dtype], seed=6)
    a["gamma"][0, 0, 64:128] = 0.0
    a["gamma"][0, 1] = 0.0
    a["gamma"][0, 2, 60:] = 2.0 ** -80
    check(a, DTYPES[dtype], "tokens")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_and_segments(dtype):
    """Zeros at the last valid token and behind it, in walks of several segments."""
    a = draw(3, 1, 1, 1300, 64, 64, DTYPES[dtype], seed=7, gates="slow", lengths=[1300, 700, 65])
    rng = np.random.default_rng(7)
    a["gamma"][rng.random(a["gamma"].shape) < 0.01] = 0.0
    for b, n in enumerate((1300, 700, 65)):
        a["gamma"][b, :, n - 1:n + 1] = 0.0
    check(a, DTYPES[dtype], walks=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_states_and_nothing_written(dtype):
    """Without s0 the first token's factor acts on nothing; where beta = 0 the states before are what it acts on."""
    a = draw(1, 2, 2, 100, 64, 64, DTYPES[dtype], seed=8, s0=False)
    a["gamma"][:, :, [0, 40, 41]] = 0.0
    a["beta"][:, :, 40] = 0.0
    want = check(a, DTYPES[dtype])
    assert not want["dgamma"][:, :, 0].any()


def test_against_differences_of_the_forward():
    """At gamma = 0, where the loss is defined on one side: its difference to a small factor."""
    a = draw(1, 2, 2, 70, 32, 32, torch.float32, seed=9)
    a["gamma"][:, :, [20, 66]] = 0.0
    t = to_dev(a, torch.float32)
    g = mesa.delta_bwd(*(t[n] for n in NAMES), t["d_o"], s0=t["s0"], d_sfinal=t["d_sfinal"])["dgamma"]

    def loss(gamma):
        r = mesa.delta_fwd(t["q"], t["k"], t["v"], gamma, t["beta"], s0=t["s0"], return_state=True)
        return ((r["o"].double() * t["d_o"].double()).sum((2, 3)) + (r["s_final"].double() * t["d_sfinal"].double()).sum((2, 3)))
    step = 2.0 ** -5
    for i in (20, 66):
        up = t["gamma"].clone()
        up[:, :, i] = step
        num = (loss(up) - loss(t["gamma"])) / step
        # the loss is of first degree in one token's factor; o and s_final are 2^-20 of their norms off, and there
        # are 70 x 32 and 32 x 32 of them
        bound = 2.0 ** -20 * (np.linalg.norm(a["d_o"]) * 32 ** 0.5 * 3 + np.linalg.norm(a["d_sfinal"]) * 8) / step
        assert bool(((num - g[:, :, i].double()).abs() <= bound).all()), (num, g[:, :, i], bound)
        assert bool((g[:, :, i].abs() > 4 * bound).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,at", [(1, 0), (50, 20), (130, 64), (130, 127), (1300, 700)])
@pytest.mark.parametrize("value", [float("nan"), -0.5])
def test_a_factor_that_is_none(value, T, at, dtype):
    """A NaN, or a number below 0, is not taken for a factor that forgets everything: as in the definition a NaN's state is
    NaN from its token on, and its gradients are before it and behind it.  Other heads are as without it."""
    a = draw(1, 2, 1, T, 64, 48, DTYPES[dtype], seed=10)
    t = to_dev(a, DTYPES[dtype])
    want = mesa.delta_fwd(*(t[n] for n in NAMES), s0=t["s0"], return_state=True)
    t["gamma"][0, 1, at] = value
    ws = torch.empty(mesa.delta_workspace_bytes(*(t[n] for n in NAMES), keep_states=True), device="cuda", dtype=torch.uint8)
    r = mesa.delta_fwd(*(t[n] for n in NAMES), s0=t["s0"], return_state=True, keep_states=True, workspace=ws)
    assert bool(r["o"][0, 1, at:].isnan().all()) and bool(r["s_final"][0, 1].isnan().all())
    first = at // 64 * 64
    assert torch.equal(r["o"][0, 1, :first], want["o"][0, 1, :first])
    for n in ("o", "s_final"):
        assert torch.equal(r[n][0, 0], want[n][0, 0])
    for kept in (False, True):
        g = mesa.delta_bwd(*(t[n] for n in NAMES), t["d_o"], s0=t["s0"], d_sfinal=t["d_sfinal"], state_grads=True,
                           workspace=ws if kept else None, states_in_workspace=kept)
        assert bool(g["ds0"][0, 1].isnan().all()) and bool(g["dv"][0, 1, :at].isnan().all())
        assert bool(g["dgamma"][0, 1, at:].isnan().all()) and bool(g["dbeta"][0, 1, at:].isnan().all())
        assert bool(g["dq"][0, 0, at:].isnan().all())  # (shared by both heads)
        assert bool(g["dv"][0, 0].isfinite().all()) and bool(g["dgamma"][0, 0].isfinite().all())
