"""Plausible slips, planted in a copy of the gated delta rule's oracle, are caught by its pins (CPU only).

Each edits the oracle's source text, loads it as a module of its own and runs the checks of
``test_oracle_delta`` and ``test_oracle_delta_gates`` on it; one at least has to fail.
"""
import os
import types

import pytest

import test_oracle_delta as pins
import test_oracle_delta_gates as gates

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "oracle", "delta_oracle.py")

SLIPS = {
    "no_decay": ("S[b] *= gamma[b, :, t, None, None]", "pass"),
    "decay_behind_the_write": ("            S[b] *= gamma[b, :, t, None, None]\n            w[b, :, t] = v[b, :, t] -",
                               "            w[b, :, t] = v[b, :, t] -"),
    "value_alone_is_written": ("w[b, :, t] = v[b, :, t] - np.einsum", "w[b, :, t] = v[b, :, t] - 0.0 * np.einsum"),
    "residual_sign": ("w[b, :, t] = v[b, :, t] - np.einsum", "w[b, :, t] = v[b, :, t] + np.einsum"),
    "residual_of_the_query": ('np.einsum("hij,hj->hi", S[b], k[b, :, t])', 'np.einsum("hij,hj->hi", S[b], q[b, :, t])'),
    "no_write_strength": ("S[b] += (beta[b, :, t, None] * w", "S[b] += (w"),
    "output_before_the_write": ("            S[b] += (beta[b, :, t, None] * w[b, :, t])[:, :, None] * k[b, :, t, None, :]\n"
                                '            o[b, :, t] = np.einsum("hij,hj->hi", S[b], q[b, :, t])',
                                '            o[b, :, t] = np.einsum("hij,hj->hi", S[b], q[b, :, t])\n'
                                "            S[b] += (beta[b, :, t, None] * w[b, :, t])[:, :, None] * k[b, :, t, None, :]"),
    "lengths_ignored": ("return np.arange(T)[None, :] < n[:, None]", "return np.arange(T)[None, :] < T + 0 * n[:, None]"),
    "length_one_more": ("return np.arange(T)[None, :] < n[:, None]", "return np.arange(T)[None, :] <= n[:, None]"),
    "start_state_ignored": ("if s0 is None else _f64(s0).copy()", "if True else None"),
    "shared_heads_in_turn": ("np.repeat(_f64(q), R, axis=1), np.repeat(_f64(k), R, axis=1)",
                             "np.tile(_f64(q), (1, R, 1, 1)), np.tile(_f64(k), (1, R, 1, 1))"),
    "shared_gradients_of_the_first_head": ("g[n].reshape(B, Hk, H // Hk, T, -1).sum(2)", "g[n].reshape(B, Hk, H // Hk, T, -1)[:, :, 0]"),
    "dq_of_the_state_before": ('np.einsum("hij,hi->hj", after, do)', 'np.einsum("hij,hi->hj", before, do)'),
    "last_state_has_no_gradient": ("if d_sfinal is None else _f64(d_sfinal).copy()", "if True else None"),
    "dbeta_of_the_value": ("np.sum(nk * w, -1)", "np.sum(nk * v[b, :, t], -1)"),
    "dv_without_strength": ('g["dv"][b, :, t] = dw', 'g["dv"][b, :, t] = nk'),
    "dk_through_the_write_alone": ('                                - ga * np.einsum("hij,hi->hj", before, dw))', "                                )"),
    "dk_residual_without_decay": ('- ga * np.einsum("hij,hi->hj", before, dw)', '- np.einsum("hij,hi->hj", before, dw)'),
    "dgamma_through_the_carry_alone": ("np.sum(M * before, (-2, -1))", "np.sum(N[b] * before, (-2, -1))"),
    "dgamma_of_the_state_after": ("np.sum(M * before, (-2, -1))", "np.sum(M * after, (-2, -1))"),
    "dgamma_at_the_logarithm": ("np.sum(M * before, (-2, -1))", "gamma[b, :, t] * np.sum(M * before, (-2, -1))"),
    "dgamma_zero_at_zero": ("np.sum(M * before, (-2, -1))", "(gamma[b, :, t] != 0) * np.sum(M * before, (-2, -1))"),
    "adjoint_without_decay": ("N[b] = ga[..., None] * M", "N[b] = M"),
    "adjoint_without_the_residual": ("N[b] = ga[..., None] * M", "N[b] = ga[..., None] * N[b]"),
    "norm_not_rooted": ("math.sqrt(sum(", "(lambda x: x)(sum("),
    "norm_of_sizes": ("np.sum(_f64(g) ** 2)", "np.sum(np.abs(_f64(g)))"),
    "scale_above_one": ("scale = 1.0 if ratio >= 1.0 else ratio", "scale = ratio"),
    "outputs_not_scaled": ("[_f64(g) * scale for g in grads]", "[_f64(g) for g in grads]"),
}


def checks():
    yield pins.test_orthonormal_keys_are_a_table, ()
    yield pins.test_one_step_of_gradient_descent, ()
    yield pins.test_transition_matrices, ()
    yield pins.test_lengths_and_parts, ()
    for args in ((2, 2, None), (4, 2, [13, 6]), (3, 1, [13, 0])):
        yield pins.test_gradients_against_differences, args
    yield pins.test_clip, ()
    yield gates.test_gradient_at_a_factor_of_zero, ()


def caught(source, monkeypatch):
    """The checks that fail on an oracle of this source."""
    m = types.ModuleType("planted")
    exec(compile(source, "planted", "exec"), m.__dict__)
    for module in (pins, gates):
        for name in ("delta_forward", "delta_backward", "clip"):
            if hasattr(module, name):
                monkeypatch.setattr(module, name, getattr(m, name))
    failed = []
    for check, args in checks():
        try:
            check(*args)
        except AssertionError:
            failed.append(check.__name__)
    return failed


def test_the_oracle_itself_passes(monkeypatch):
    with open(SRC) as f:
        assert not caught(f.read(), monkeypatch)


@pytest.mark.parametrize("name", sorted(SLIPS))
def test_planted_slip_is_caught(name, monkeypatch):
    old, new = SLIPS[name]
    with open(SRC) as f:
        source = f.read()
    assert source.count(old) == 1, old
    assert caught(source.replace(old, new), monkeypatch)
