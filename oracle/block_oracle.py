"""fp64 CPU oracle for the operators around the Mesa layer.

The gated linear recurrence that alternates with the Mesa layer in the
Hawk-Mesa hybrid (MesaNet page, "architecture" section), the RMS norm with
the residual addition in front of either, and the gradient of the query/key
preprocessing.  Plain NumPy, token by token, sharing no code with the HIP path.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0, e) / (1.0 + e)


def _softplus(z):
    return np.maximum(z, 0.0) + np.log1p(np.exp(-np.abs(z)))


def lru_gates(x, ga, gi, lam, c):
    """w = -2 log a, decay a, input scale m = sqrt(1 - a^2), and the two sigmoids."""
    sr, si = _sigmoid(_f64(ga)), _sigmoid(_f64(gi))
    w = 2.0 * c * _softplus(_f64(lam)) * sr
    return w, np.exp(-0.5 * w), np.sqrt(-np.expm1(-w)), sr, si


def lru_forward(x, ga, gi, lam, *, c: float = 8.0, h0=None, lengths=None):
    """h_t = a_t h_{t-1} + m_t sigmoid(gi_t) x_t, a_t = exp(-c softplus(lam) sigmoid(ga_t)),
    m_t = sqrt(1 - a_t^2); y_t = h_t for t < length, 0 behind it.

    x, ga, gi [B, T, D]; lam [D]; h0 [B, D] or None; lengths [B] or None.
    Returns dict(y [B, T, D], h_final [B, D]: the state after the last valid
    token, prev [B, T, D]: the state before each token).
    """
    x = _f64(x)
    B, T, D = x.shape
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    _, a, m, _, si = lru_gates(x, ga, gi, lam, c)
    h = np.zeros((B, D)) if h0 is None else _f64(h0).copy()
    y, prev = np.zeros((B, T, D)), np.zeros((B, T, D))
    for t in range(T):
        prev[:, t] = h
        live = t < n
        h[live] = a[live, t] * h[live] + m[live, t] * si[live, t] * x[live, t]
        y[live, t] = h[live]
    return dict(y=y, h_final=h, prev=prev)


def lru_backward(x, ga, gi, lam, dy, *, c: float = 8.0, h0=None, lengths=None, d_hfinal=None):
    """Gradients of L = sum <dy_t, y_t> + <d_hfinal, h_final> of lru_forward.

    With g_t = dy_t + a_{t+1} g_{t+1} (d_hfinal behind the last valid token):
        dx = g m si,  dgi = g m x si (1 - si),
        v = (w/2) g ((a^2 / m) si x - a h_{t-1})     (= dL / d log w),
        dga = v (1 - sr),  dlam = sum v sigmoid(lam) / softplus(lam),  dh0 = a_0 g_0.
    """
    x, dy, lam = _f64(x), _f64(dy), _f64(lam)
    B, T, D = x.shape
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    w, a, m, _, si = lru_gates(x, ga, gi, lam, c)
    sr1, si1 = _sigmoid(-_f64(ga)), _sigmoid(-_f64(gi))   # 1 - sigmoid, without the cancellation
    prev = lru_forward(x, ga, gi, lam, c=c, h0=h0, lengths=lengths)["prev"]
    out = {k: np.zeros((B, T, D)) for k in ("dx", "dga", "dgi")}
    dloglam = np.zeros(D)
    after = np.zeros((B, D)) if d_hfinal is None else _f64(d_hfinal).copy()
    for t in range(T - 1, -1, -1):
        L = np.nonzero(t < n)[0]
        if L.size == 0:
            continue
        g = after[L] + dy[L, t]
        ratio = np.divide(a[L, t] ** 2, m[L, t], out=np.zeros_like(g), where=m[L, t] > 0)
        v = 0.5 * w[L, t] * g * (ratio * si[L, t] * x[L, t] - a[L, t] * prev[L, t])
        out["dx"][L, t] = g * m[L, t] * si[L, t]
        out["dgi"][L, t] = g * m[L, t] * x[L, t] * si[L, t] * si1[L, t]
        out["dga"][L, t] = v * sr1[L, t]
        dloglam += v.sum(0)
        after[L] = a[L, t] * g
    out["dlam"] = dloglam * _sigmoid(lam) / _softplus(lam)
    out["dh0"] = after
    return out


def lru_step(x, ga, gi, lam, h, *, c: float = 8.0):
    """One token: x, ga, gi, h [N, D] -> the new state (also the output)."""
    _, a, m, _, si = lru_gates(x, ga, gi, lam, c)
    return a * _f64(h) + m * si * _f64(x)


E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100


def e4m3_round(v):
    """v rounded to the nearest e4m3 value (4 exponent bits of bias 7, 3 mantissa
    bits, no infinities, largest 448), ties to the even mantissa."""
    v = _f64(v)
    a = np.abs(v)
    _, ex = np.frexp(np.where(a > 0, a, 1.0))            # a = f 2^ex, f in [0.5, 1)
    step = np.exp2(np.maximum(ex - 1, -6) - 3.0)         # spacing of the binade, 2^-9 below 2^-6
    return np.copysign(np.minimum(np.rint(a / step) * step, E4M3_MAX), v)


def rmsnorm(x, w, *, residual=None, eps: float = 1e-6, group=None):
    """s = x + residual; y = w s / sqrt(mean(s^2) + eps) per row; with group the
    e4m3 values of y / scale, scale = max|y| / 448 over the row (group 0) or over
    each `group` consecutive channels (max|y| at least 2^-100).

    Returns dict(residual [R, D] = s, y [R, D], and with group: q [R, D] values
    after the rounding, scale [R, groups])."""
    s = _f64(x) + (0.0 if residual is None else _f64(residual))
    R, D = s.shape
    y = _f64(w) * s / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    out = dict(residual=s, y=y)
    if group is not None:
        g = group or D
        n = -(-D // g)
        scale = np.stack([np.maximum(np.abs(y[:, i * g:(i + 1) * g]).max(1), AMAX_FLOOR) for i in range(n)], 1) / E4M3_MAX
        out["scale"] = scale
        out["q"] = e4m3_round(y / np.repeat(scale, g, axis=1)[:, :D])
    return out


def rmsnorm_backward(s, w, dy, *, d_residual=None, eps: float = 1e-6):
    """Gradients of y = w s / sqrt(mean(s^2) + eps) at s (plus d_residual, what
    reaches s along the residual stream) and at w (summed over rows)."""
    s, w, dy = _f64(s), _f64(w), _f64(dy)
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    xhat, g = s * rstd, dy * w
    ds = rstd * (g - xhat * (g * xhat).mean(1, keepdims=True))
    if d_residual is not None:
        ds = ds + _f64(d_residual)
    return dict(ds=ds, dw=(dy * xhat).sum(0))


def qk_preprocess_backward(x, w, d_out, hist=None, d_hist_out=None, eps: float = 1e-6):
    """Gradients of qk_preprocess (y_t = sum_i w[.., i] x_{t-i}, out = y / max(||y||, eps))
    of one of queries or keys, for L = <d_out, out> + <d_hist_out, hist_out>.

    With n = ||y||: dy = (d - out <out, d>) / n where n > eps, else d / eps;
    dx_s = sum_i w[.., i] dy_{s+i} (s runs over history rows too), plus
    d_hist_out on the last W-1 raw rows; dw[h, j, i] = sum_{b,t} dy_t[j] x_{t-i}[j].
    Returns dict(dx [B, H, T, d], dw [H, d, W], dhist [B, H, W-1, d])."""
    x, w, d_out = _f64(x), _f64(w), _f64(d_out)
    B, H, T, d = x.shape
    W = w.shape[-1]
    seq = np.concatenate([np.zeros((B, H, W - 1, d)) if hist is None else _f64(hist), x], axis=2)
    dseq, dw = np.zeros_like(seq), np.zeros_like(w)
    if d_hist_out is not None:
        dseq[:, :, T:] += _f64(d_hist_out)
    for t in range(T):
        rows = seq[:, :, t:t + W][:, :, ::-1]                       # row i: token t - i
        y = np.einsum("hji,bhij->bhj", w, rows)
        n = np.sqrt((y * y).sum(-1, keepdims=True))
        o = y / np.maximum(n, eps)
        dot = np.where(n > eps, (o * d_out[:, :, t]).sum(-1, keepdims=True), 0.0)
        dy = (d_out[:, :, t] - o * dot) / np.maximum(n, eps)
        dw += np.einsum("bhj,bhij->hji", dy, rows)
        for i in range(W):
            dseq[:, :, t + W - 1 - i] += w[None, :, :, i] * dy
    return dict(dx=dseq[:, :, W - 1:], dw=dw, dhist=dseq[:, :, :W - 1])
