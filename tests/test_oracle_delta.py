"""The fp64 oracle of the gated delta rule, pinned to what does not share its code (CPU only)."""
import numpy as np
import pytest
import torch

from delta_helpers import draw
from oracle.delta_oracle import clip, delta_backward, delta_forward

FIVE = ("q", "k", "v", "gamma", "beta")


def test_orthonormal_keys_are_a_table():
    """gamma = beta = 1 and orthonormal keys: S k_j = v_j for every key so far; a key met again takes its new value."""
    d, rng = 16, np.random.default_rng(0)
    basis = np.linalg.qr(rng.standard_normal((d, d)))[0]
    order = np.concatenate([np.arange(d), [3, 7]])
    v = rng.standard_normal((1, 1, d + 2, 5))
    k = basis[order][None, None]
    one = np.ones((1, 1, d + 2))
    S = delta_forward(k, k, v, one, one)["s_final"][0, 0]
    want = v[0, 0, :d].copy()
    want[3], want[7] = v[0, 0, d], v[0, 0, d + 1]
    assert np.allclose(S @ basis.T, want.T, atol=1e-13)


def test_one_step_of_gradient_descent():
    """S_t is gamma S_{t-1} after one step of size beta on |S k - v|^2 / 2."""
    a = draw(1, 2, 2, 3, 32, 16, torch.float32)
    f = delta_forward(*(a[n] for n in FIVE), s0=a["s0"])
    for h in range(2):
        S = a["gamma"][0, h, 2] * f["states"][2][0, h]
        k, v = a["k"][0, h, 2], a["v"][0, h, 2]
        step = np.outer(S @ k - v, k)
        assert np.allclose(f["s_final"][0, h], S - a["beta"][0, h, 2] * step, atol=1e-13)


def test_transition_matrices():
    """Unrolled: S_T = sum_j beta_j v_j k_j^T prod_{i>j} gamma_i (I - beta_i k_i k_i^T) + S_0 prod."""
    a = draw(1, 1, 1, 12, 32, 16, torch.float32)
    maps = [a["gamma"][0, 0, t] * (np.eye(32) - a["beta"][0, 0, t] * np.outer(a["k"][0, 0, t], a["k"][0, 0, t]))
            for t in range(12)]
    S = a["s0"][0, 0]
    for m in maps:
        S = S @ m
    for j in range(12):
        x = a["beta"][0, 0, j] * np.outer(a["v"][0, 0, j], a["k"][0, 0, j])
        for m in maps[j + 1:]:
            x = x @ m
        S = S + x
    assert np.allclose(S, delta_forward(*(a[n] for n in FIVE), s0=a["s0"])["s_final"][0, 0], atol=1e-13)


def test_lengths_and_parts():
    a = draw(3, 2, 1, 20, 32, 16, torch.float32, lengths=[20, 0, 7])
    f = delta_forward(*(a[n] for n in FIVE), s0=a["s0"], lengths=a["lengths"])
    assert np.array_equal(f["s_final"][1], a["s0"][1]) and not f["o"][1].any() and not f["o"][2, :, 7:].any()
    for b, n in enumerate(a["lengths"]):
        g = delta_forward(*(a[x][b:b + 1, :, :n] for x in FIVE), s0=a["s0"][b:b + 1])
        assert np.array_equal(g["s_final"][0], f["s_final"][b]) and np.array_equal(g["o"][0], f["o"][b, :, :n])


@pytest.mark.parametrize("H,Hk,lengths", [(2, 2, None), (4, 2, [13, 6]), (3, 1, [13, 0])])
def test_gradients_against_differences(H, Hk, lengths):
    a = draw(2, H, Hk, 13, 32, 16, torch.float32, lengths=lengths)

    def loss(x):
        f = delta_forward(*(x[n] for n in FIVE), s0=x["s0"], lengths=x["lengths"])
        return np.sum(f["o"] * x["d_o"]) + np.sum(f["s_final"] * x["d_sfinal"])

    g = delta_backward(*(a[n] for n in FIVE), a["d_o"], s0=a["s0"], lengths=a["lengths"], d_sfinal=a["d_sfinal"])
    rng = np.random.default_rng(1)
    for n in FIVE + ("s0",):
        d = rng.standard_normal(a[n].shape)
        step = 1e-5
        numeric = (loss({**a, n: a[n] + step * d}) - loss({**a, n: a[n] - step * d})) / (2 * step)
        # a cubic's worth of curvature times step^2, and 2^-53 of the loss over the step
        assert abs(numeric - np.sum(g["d" + n] * d)) <= 1e-7 * (1 + np.linalg.norm(g["d" + n]) * np.linalg.norm(d)), n


def test_clip():
    g = [np.array([3.0]), np.array([[0.0, 4.0]])]
    r = clip(g, 2.5, eps=0.0)
    assert r["norm"] == 5.0 and r["scale"] == 0.5 and np.array_equal(r["grads"][1], [[0.0, 2.0]])
    assert clip(g, 6.0)["scale"] == 1.0
