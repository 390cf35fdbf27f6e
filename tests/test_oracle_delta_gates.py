"""The oracle's gradient at forget factors of 0 (CPU only)."""
import numpy as np
import torch

from delta_helpers import draw
from oracle.delta_oracle import delta_backward, delta_forward

FIVE = ("q", "k", "v", "gamma", "beta")


def test_gradient_at_a_factor_of_zero():
    """The loss is of first degree in one token's factor, so any difference gives its gradient, at 0 too, where it is not 0."""
    a = draw(1, 2, 1, 12, 32, 16, torch.float32)
    a["gamma"][:, :, [0, 5, 11]] = 0.0

    def loss(x):
        f = delta_forward(*(x[n] for n in FIVE), s0=x["s0"])
        return np.sum(f["o"] * x["d_o"], (2, 3)) + np.sum(f["s_final"] * x["d_sfinal"], (2, 3))

    g = delta_backward(*(a[n] for n in FIVE), a["d_o"], s0=a["s0"], d_sfinal=a["d_sfinal"])["dgamma"]
    for i in (0, 5, 11):
        for step in (1.0, 0.25, -0.5):
            b = {**a, "gamma": a["gamma"].copy()}
            b["gamma"][:, :, i] = step
            assert np.allclose((loss(b) - loss(a)) / step, g[:, :, i], rtol=1e-11, atol=1e-11)
        assert np.abs(g[:, :, i]).min() > 0.05
