"""Pins of the oracle of the operators around the Mesa layer (CPU only).

Closed forms, torch's fp64 automatic differentiation of the formulas, and
differences of the forward; none shares code with the oracle.  The planted
slips at the end show that each pin constrains the arithmetic.
"""
import os
import types

import numpy as np
import pytest
import torch

from oracle import block_oracle as real

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "oracle", "block_oracle.py")


def draw_lru(seed=0, B=3, T=9, D=5):
    rng = np.random.default_rng(seed)
    x, ga, gi, dy = (rng.standard_normal((B, T, D)) for _ in range(4))
    lam = rng.uniform(-6, 1, D)
    return dict(x=x, ga=ga, gi=gi, lam=lam, dy=dy, h0=rng.standard_normal((B, D)),
                d_hfinal=rng.standard_normal((B, D)), lengths=np.array([T, 4, 0]))


def torch_lru(x, ga, gi, lam, h0, lengths, c):
    """The recurrence written on the decay's logarithm, in torch, for automatic differentiation."""
    la = -c * torch.nn.functional.softplus(lam) * torch.sigmoid(ga)
    u = torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(gi) * x
    h, y = h0, []
    for t in range(x.shape[1]):
        live = torch.from_numpy(t < np.asarray(lengths))[:, None]
        h = torch.where(live, torch.exp(la[:, t]) * h + u[:, t], h)
        y.append(torch.where(live, h, torch.zeros_like(h)))
    return torch.stack(y, 1), h


def check_lru_forward(O):
    d = draw_lru()
    out = O.lru_forward(d["x"], d["ga"], d["gi"], d["lam"], c=3.0, h0=d["h0"], lengths=d["lengths"])
    t = {k: torch.from_numpy(v) for k, v in d.items()}
    y, h = torch_lru(t["x"], t["ga"], t["gi"], t["lam"], t["h0"], d["lengths"], 3.0)
    assert np.abs(out["y"] - y.numpy()).max() < 1e-13
    assert np.abs(out["h_final"] - h.numpy()).max() < 1e-13
    # constant gates: h_t is a geometric sum
    a = 0.5
    lam = np.log(np.expm1(-np.log(a) * 2 / 1.0))  # softplus(lam) sigmoid(0) = log 2
    one = np.ones((1, 6, 1))
    y = O.lru_forward(one, 0 * one, 0 * one, np.array([lam]), c=1.0)["y"][0, :, 0]
    want = 0.5 * np.sqrt(0.75) * (1 - a ** np.arange(1, 7)) / (1 - a)
    assert np.abs(y - want).max() < 1e-14


def check_lru_backward(O):
    d = draw_lru(1)
    r = O.lru_backward(d["x"], d["ga"], d["gi"], d["lam"], d["dy"], c=3.0, h0=d["h0"], lengths=d["lengths"],
                       d_hfinal=d["d_hfinal"])
    t = {k: torch.from_numpy(v).requires_grad_(k in ("x", "ga", "gi", "lam", "h0")) for k, v in d.items() if k != "lengths"}
    y, h = torch_lru(t["x"], t["ga"], t["gi"], t["lam"], t["h0"], d["lengths"], 3.0)
    L = (y * t["dy"]).sum() + (h * t["d_hfinal"]).sum()
    g = torch.autograd.grad(L, [t[k] for k in ("x", "ga", "gi", "lam", "h0")])
    for key, v in zip(("dx", "dga", "dgi", "dlam", "dh0"), g):
        assert np.abs(r[key] - v.numpy()).max() < 1e-12, key
    # and against differences of the oracle's own forward
    for key in ("x", "ga", "gi", "lam", "h0"):
        base = {k: d[k] for k in ("x", "ga", "gi", "lam", "h0", "lengths")}
        e = np.random.default_rng(7).standard_normal(d[key].shape)
        up, dn = (O.lru_forward(**dict(base, c=3.0, **{key: d[key] + s * 1e-5 * e})) for s in (1, -1))
        num = ((up["y"] - dn["y"]) * d["dy"]).sum() + ((up["h_final"] - dn["h_final"]) * d["d_hfinal"]).sum()
        num /= 2e-5
        assert abs(num - (r["d" + key] * e).sum()) < 1e-8 * (1 + abs(num)), key


def check_lru_step(O):
    d = draw_lru(2, T=1)
    h = O.lru_step(d["x"][:, 0], d["ga"][:, 0], d["gi"][:, 0], d["lam"], d["h0"], c=3.0)
    assert np.abs(h - O.lru_forward(d["x"], d["ga"], d["gi"], d["lam"], c=3.0, h0=d["h0"])["h_final"]).max() == 0


def check_saturated_gates(O):
    """A closed recurrence gate keeps the state exactly (a = 1, m = 0), gradients finite."""
    x, z = np.ones((1, 2, 1)), np.zeros((1, 2, 1))
    far = np.full((1, 2, 1), -800.0)
    o = O.lru_forward(x, far, z, np.zeros(1), h0=np.array([[3.0]]))
    assert np.array_equal(o["y"], np.full((1, 2, 1), 3.0))
    r = O.lru_backward(x, far, z, np.zeros(1), x)
    assert all(np.isfinite(v).all() for v in r.values()) and np.array_equal(r["dh0"], [[2.0]])


def check_rmsnorm(O):
    rng = np.random.default_rng(3)
    x, res, w = rng.standard_normal((4, 300)), rng.standard_normal((4, 300)), rng.uniform(0.5, 2, 300)
    t = torch.from_numpy
    o = O.rmsnorm(x, w, residual=res, eps=0.3)
    want = torch.nn.functional.rms_norm(t(x + res), (300,), t(w), 0.3).numpy()
    assert np.abs(o["y"] - want).max() < 1e-13 and np.array_equal(o["residual"], x + res)
    for group in (0, 128):
        o = O.rmsnorm(x, w, residual=res, eps=0.3, group=group)
        n = 1 if group == 0 else 3
        assert o["scale"].shape == (4, n)
        for i in range(n):
            part = slice(None) if group == 0 else slice(128 * i, 128 * i + 128)
            assert np.abs(o["scale"][:, i] - np.abs(want[:, part]).max(1) / 448).max() < 1e-15
            ref = t(want[:, part] / o["scale"][:, i:i + 1]).to(torch.float8_e4m3fn).double().numpy()
            assert np.array_equal(o["q"][:, part], ref)
    z = O.rmsnorm(np.zeros((1, 8)), w[:8], group=0)
    assert np.array_equal(z["q"], np.zeros((1, 8))) and z["scale"][0, 0] == 2.0 ** -100 / 448


def check_e4m3(O):
    """Every bf16 value of magnitude 2^-12 .. 448 (ties and the subnormal range among them) against torch's rounding."""
    bits = np.arange(0x3980, 0x43E1, dtype=np.uint32)
    v = (bits << 16).view(np.float32)
    v = np.concatenate([[0.0], v, -v]).astype(np.float64)
    assert np.array_equal(O.e4m3_round(v), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def check_rmsnorm_backward(O):
    rng = np.random.default_rng(4)
    s, w, dy, dres = rng.standard_normal((5, 7)), rng.uniform(0.5, 2, 7), rng.standard_normal((5, 7)), rng.standard_normal((5, 7))
    r = O.rmsnorm_backward(s, w, dy, d_residual=dres, eps=0.2)
    ts, tw = torch.from_numpy(s).requires_grad_(), torch.from_numpy(w).requires_grad_()
    y = torch.nn.functional.rms_norm(ts, (7,), tw, 0.2)
    gs, gw = torch.autograd.grad((y * torch.from_numpy(dy)).sum() + (ts * torch.from_numpy(dres)).sum(), [ts, tw])
    assert np.abs(r["ds"] - gs.numpy()).max() < 1e-13 and np.abs(r["dw"] - gw.numpy()).max() < 1e-13


def check_prep_backward(O):
    for W, T, eps in ((1, 5, 1e-6), (4, 6, 1e-6), (4, 2, 1e-6), (3, 6, 1.5)):
        rng = np.random.default_rng(W + T)
        B, H, d = 2, 3, 4
        x, w = rng.standard_normal((B, H, T, d)), rng.uniform(-0.5, 0.5, (H, d, W))
        hist, do, dho = rng.standard_normal((B, H, W - 1, d)), rng.standard_normal((B, H, T, d)), rng.standard_normal((B, H, W - 1, d))
        r = O.qk_preprocess_backward(x, w, do, hist, dho, eps=eps)
        tx, tw, th = (torch.from_numpy(v).requires_grad_() for v in (x, w, hist))
        seq = torch.cat([th, tx], 2)
        y = sum(tw[None, :, None, :, i] * seq[:, :, W - 1 - i:W - 1 - i + T] for i in range(W))
        n = y.norm(dim=-1, keepdim=True)
        if eps > 1:
            assert (n < eps).any() and (n > eps).any()  # both branches of the normalisation
        out = y / torch.where(n > eps, n, torch.full_like(n, eps))
        L = (out * torch.from_numpy(do)).sum() + (seq[:, :, T:] * torch.from_numpy(dho)).sum()
        g = torch.autograd.grad(L, [tx, tw, th], allow_unused=True)
        for key, v in zip(("dx", "dw", "dhist"), g):
            assert r[key].size == 0 or np.abs(r[key] - v.numpy()).max() < 1e-13, (W, T, key)


CHECKS = [check_lru_forward, check_lru_backward, check_lru_step, check_saturated_gates, check_rmsnorm, check_e4m3,
          check_rmsnorm_backward, check_prep_backward]


@pytest.mark.parametrize("check", CHECKS, ids=lambda c: c.__name__[6:])
def test_oracle(check):
    check(real)


MUTATIONS = {
    "input_scale_without_decay": ("np.sqrt(-np.expm1(-w))", "np.sqrt(-np.expm1(-w / 2))"),
    "decay_squared": ("np.exp(-0.5 * w)", "np.exp(-w)"),
    "rows_behind_the_length_change_the_state": ("live = t < n", "live = t <= n"),
    "output_before_update": ("y[live, t] = h[live]", "y[live, t] = prev[live, t]"),
    "adjoint_not_decayed": ("after[L] = a[L, t] * g", "after[L] = g"),
    "decay_gradient_current_state": ("a[L, t] * prev[L, t])", "a[L, t] * (a[L, t] * prev[L, t] + m[L, t] * si[L, t] * x[L, t]))"),
    "decay_gradient_without_input_scale": ("(ratio * si[L, t] * x[L, t] - ", "(0 * ratio * si[L, t] * x[L, t] - "),
    "gate_gradient_slope": ("v * sr1[L, t]", "v * (1.0 - sr1[L, t])"),
    "input_gate_gradient_slope": ("si[L, t] * si1[L, t]", "si1[L, t]"),
    "lam_gradient_slope": ("dloglam * _sigmoid(lam) / _softplus(lam)", "dloglam / _softplus(lam)"),
    "norm_eps_outside_root": ("np.sqrt((s * s).mean(1, keepdims=True) + eps)\n    out",
                              "(np.sqrt((s * s).mean(1, keepdims=True)) + eps)\n    out"),
    "norm_scale_by_rows_only": ("np.abs(y[:, i * g:(i + 1) * g]).max(1)", "np.abs(y).max(1)"),
    "e4m3_subnormal_step": ("np.maximum(ex - 1, -6)", "np.maximum(ex - 1, -7)"),
    "e4m3_two_mantissa_bits": ("- 3.0)", "- 2.0)"),
    "norm_gradient_projection": ("(g * xhat).mean(1", "g.mean(1"),
    "norm_weight_gradient": ("(dy * xhat).sum(0)", "(dy * s).sum(0)"),
    "norm_residual_gradient_dropped": ("ds = ds + _f64(d_residual)", "pass"),
    "prep_gradient_below_eps": ("np.where(n > eps, ", "np.where(n > 0, "),
    "prep_gradient_taps_reversed": ("dseq[:, :, t + W - 1 - i] += w", "dseq[:, :, t + i] += w"),
    "prep_gradient_history": ("dseq[:, :, T:] += ", "dseq[:, :, :W - 1] += "),
    "prep_weight_gradient_rows": ('"bhj,bhij->hji", dy, rows', '"bhj,bhij->hji", dy, rows[:, :, ::-1]'),
}


@pytest.mark.parametrize("name", sorted(MUTATIONS))
def test_planted_slip_is_caught(name):
    old, new = MUTATIONS[name]
    src = open(SRC).read()
    assert src.count(old) >= 1, name
    mod = types.ModuleType("block_oracle_" + name)
    mod.__dict__["__name__"] = mod.__name__
    exec(compile(src.replace(old, new), SRC, "exec"), mod.__dict__)
    caught = 0
    for check in CHECKS:
        try:
            check(mod)
        except AssertionError:
            caught += 1
    assert caught, f"no pin notices {name}"
