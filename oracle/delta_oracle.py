"""fp64 CPU oracle of the gated delta rule and of gradient clipping.

MesaNet page, technical summary: the rule that takes one step a token on the
objective which the Mesa layer solves.  Plain NumPy, token by token, sharing no
code with the HIP path.
"""
from __future__ import annotations

import math

import numpy as np


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def _live(lengths, B, T):
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    return np.arange(T)[None, :] < n[:, None]


def _per_head(q, k, H):
    R = H // q.shape[1]
    return np.repeat(_f64(q), R, axis=1), np.repeat(_f64(k), R, axis=1)


def delta_forward(q, k, v, gamma, beta, *, s0=None, lengths=None):
    """w_t = v_t - gamma_t S_{t-1} k_t, S_t = gamma_t S_{t-1} + beta_t w_t k_t^T, o_t = S_t q_t.

    q, k [B, Hk, T, dk]; v [B, H, T, dv]; gamma, beta [B, H, T]; s0 [B, H, dv, dk] or
    None; lengths [B] or None.  Returns dict(o [B, H, T, dv], 0 behind a length,
    s_final, states: S_{t-1} for each t [T][B, H, dv, dk], w [B, H, T, dv]).
    """
    v, gamma, beta = _f64(v), _f64(gamma), _f64(beta)
    B, H, T, dv = v.shape
    q, k = _per_head(q, k, H)
    live = _live(lengths, B, T)
    S = np.zeros((B, H, dv, k.shape[-1])) if s0 is None else _f64(s0).copy()
    o, w, states = np.zeros_like(v), np.zeros_like(v), []
    for t in range(T):
        states.append(S.copy())
        for b in np.flatnonzero(live[:, t]):
            S[b] *= gamma[b, :, t, None, None]
            w[b, :, t] = v[b, :, t] - np.einsum("hij,hj->hi", S[b], k[b, :, t])
            S[b] += (beta[b, :, t, None] * w[b, :, t])[:, :, None] * k[b, :, t, None, :]
            o[b, :, t] = np.einsum("hij,hj->hi", S[b], q[b, :, t])
    return dict(o=o, s_final=S, states=states, w=w)


def delta_backward(q, k, v, gamma, beta, d_o, *, s0=None, lengths=None, d_sfinal=None):
    """Gradients of L = sum <d_o_t, o_t> + <d_sfinal, s_final>, by the chain rule through each
    token's three statements, backwards: dict(dq, dk, dv, dgamma, dbeta, ds0) and
    dgamma_sizes, the sizes of the two terms whose difference dgamma is: |<N, S>| + |dw . S k|."""
    f = delta_forward(q, k, v, gamma, beta, s0=s0, lengths=lengths)
    Hk = np.shape(q)[1]
    v, gamma, beta, d_o = _f64(v), _f64(gamma), _f64(beta), _f64(d_o)
    B, H, T, dv = v.shape
    q, k = _per_head(q, k, H)
    live = _live(lengths, B, T)
    g = {n: np.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dgamma", gamma), ("dbeta", beta))}
    N = np.zeros((B, H, dv, k.shape[-1])) if d_sfinal is None else _f64(d_sfinal).copy()
    sizes = np.zeros_like(gamma)
    for t in range(T - 1, -1, -1):
        for b in np.flatnonzero(live[:, t]):
            before, w, kt, qt, do = f["states"][t][b], f["w"][b, :, t], k[b, :, t], q[b, :, t], d_o[b, :, t]
            ga, be = gamma[b, :, t, None], beta[b, :, t, None]
            after = ga[..., None] * before + (be * w)[:, :, None] * kt[:, None, :]
            g["dq"][b, :, t] = np.einsum("hij,hi->hj", after, do)
            N[b] += do[:, :, None] * qt[:, None, :]
            nk = np.einsum("hij,hj->hi", N[b], kt)
            g["dbeta"][b, :, t] = np.sum(nk * w, -1)
            dw = be * nk
            g["dv"][b, :, t] = dw
            g["dk"][b, :, t] = (np.einsum("hij,hi->hj", N[b], be * w)
                                - ga * np.einsum("hij,hi->hj", before, dw))
            M = N[b] - dw[:, :, None] * kt[:, None, :]
            g["dgamma"][b, :, t] = np.sum(M * before, (-2, -1))
            sizes[b, :, t] = (np.abs(np.sum(N[b] * before, (-2, -1)))
                              + np.abs(np.sum(dw * np.einsum("hij,hj->hi", before, kt), -1)))
            N[b] = ga[..., None] * M
    for n in ("dq", "dk"):
        g[n] = g[n].reshape(B, Hk, H // Hk, T, -1).sum(2)
    g["ds0"], g["dgamma_sizes"] = N, sizes
    return g


def clip(grads, max_norm, eps=1e-6):
    """dict(norm, scale, grads): the 2-norm of all arrays together, min(1, max_norm / (norm + eps)), the scaled arrays."""
    norm = math.sqrt(sum(float(np.sum(_f64(g) ** 2)) for g in grads))
    ratio = max_norm / (norm + eps)
    scale = 1.0 if ratio >= 1.0 else ratio
    return dict(norm=norm, scale=scale, grads=[_f64(g) * scale for g in grads])
