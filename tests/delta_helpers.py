"""Inputs of the gated delta rule's tests, and how far results may be from the fp64 oracle.

The bounds are derived from the arithmetic, before any run.  With unit keys and
0 <= beta <= 1 a token's map S -> gamma S (I - beta k k^T) does not lengthen S, so
an error of the state is not amplified by later tokens, and errors of different
chunks add like independent ones.  Every product that a state or an fp32 result
depends on has operands that are exact or in three bf16 parts (residual 2^-24,
and the dropped products of a second and a third part 2 * 2^-24: at most 2^-22 of
a product, 2^-23 in the 2-norm of many) and sums in fp32.  From an input to a
result run at most 12 such stages forward (k.k, the inverse's two products, K M,
c K M, T P, beta, tail, K^T U, c M, Q M, A U) and 20 backward, each adding at most
2^-23 of the 2-norm of what it acts on; a state remembers min(chunks, 1 / (64 (1 -
gamma))) + 1 chunks, whose errors add by squares.  So, in the 2-norm over a head,
    e32 = stages * 2^-23 * sqrt(remembered),
2.0e-6 for one chunk forward.  A plane that is lost (2^-16 of a product at most,
about 2^-18 in the norm, in every stage) is about ten times that.  Numbers are
compared one by one with 16 times e32 of their row's or head's root mean square:
a row's 64 and more products spread by less than that.  A bf16 result adds half a
step of its value, 2^-8, and operands of two parts (2^-16, 2^-15 for both).
"""
import numpy as np
import torch

from oracle.delta_oracle import delta_backward, delta_forward

NAMES = ("q", "k", "v", "gamma", "beta", "d_o", "s0", "d_sfinal")
ROWS = ("q", "k", "v", "d_o")
GATES = {"usual": (2.0, 6.0), "slow": (4.0, 9.0), "fast": (-3.0, 3.0)}


def round_to(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).double().numpy()


def draw(B, H, Hk, T, dk, dv, dtype, seed=0, gates="usual", s0=True, lengths=None, beta=(0.0, 1.0)):
    """float64 arrays that hold values of the given type (gates and states: fp32)."""
    rng = np.random.default_rng([seed, B, H, Hk, T, dk, dv])
    f32 = torch.float32

    def unit(*shape):
        x = rng.standard_normal(shape)
        return round_to(x / np.linalg.norm(x, axis=-1, keepdims=True), dtype)

    a = dict(q=unit(B, Hk, T, dk), k=unit(B, Hk, T, dk), v=round_to(rng.standard_normal((B, H, T, dv)), dtype),
             d_o=round_to(rng.standard_normal((B, H, T, dv)), dtype),
             gamma=round_to(1 / (1 + np.exp(-rng.uniform(*GATES[gates], (B, H, T)))), f32),
             beta=round_to(rng.uniform(*beta, (B, H, T)), f32), s0=None, d_sfinal=None,
             lengths=None if lengths is None else np.asarray(lengths, dtype=np.int32))
    if s0:
        a["s0"] = round_to(rng.standard_normal((B, H, dv, dk)) * 2 / np.sqrt(dk), f32)
        a["d_sfinal"] = round_to(rng.standard_normal((B, H, dv, dk)), f32)
    return a


def to_dev(a, dtype, layout="heads", poison=True):
    """Device tensors: rows [B, heads, T, d] dense, as [B, T, heads, d] ("tokens"), or slices of wider rows ("slices")."""
    t = {"lengths": None if a["lengths"] is None else torch.from_numpy(a["lengths"]).cuda()}
    for n in NAMES:
        if a[n] is None:
            t[n] = None
            continue
        x = torch.from_numpy(a[n].astype(np.float32)).cuda().to(dtype if n in ROWS else torch.float32)
        if poison and a["lengths"] is not None and n not in ("s0", "d_sfinal"):
            for b, stop in enumerate(a["lengths"]):  # rows behind a length may hold anything
                x[b, :, max(int(stop), 0):] = float("nan") if n in ("q", "gamma", "d_o") else float("inf")
        if n not in ("s0", "d_sfinal"):
            if layout == "tokens":
                x = x.transpose(1, 2).contiguous().transpose(1, 2)
            elif layout == "slices":
                y = x.transpose(1, 2)
                wide = torch.full(y.shape[:2] + (y.shape[2] + 1,) + y.shape[3:], float("nan"), dtype=x.dtype, device="cuda")
                wide[:, :, 1:] = y
                x = wide[:, :, 1:].transpose(1, 2)
        t[n] = x
    return t


def remembered(a):
    T = a["v"].shape[2]
    n = -(-T // 64)
    if n == 0:
        return 1.0
    return min(n, 1 / (64 * max(1 - float(a["gamma"].mean()), 1e-6))) + 1


def e32(a, stages):
    return stages * 2.0 ** -23 * np.sqrt(remembered(a))


def close(got, want, e, dtype, what, rows=True):
    """Per head in the 2-norm, and number by number."""
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    half = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24
    flat = (got - want).reshape(got.shape[0] * got.shape[1], -1) if want.ndim > 2 else (got - want)[None]
    ref = want.reshape(flat.shape)
    assert np.isfinite(flat).all(), what
    low = 2.0 ** -15 if dtype is torch.bfloat16 else 0.0
    norm = np.linalg.norm(ref, axis=-1)
    off = np.linalg.norm(flat, axis=-1)
    worst = float(np.max(off / np.maximum(norm, 1e-30) * (norm > 0), initial=0.0))
    assert np.all(off <= (e + half + low) * norm), (what, worst, e)
    if want.ndim > 2 and rows:
        rms = np.sqrt(np.mean(want ** 2, axis=-1, keepdims=True))
    else:
        rms = np.zeros(want.shape[:-1] + (1,))
    axes = tuple(range(2, want.ndim)) if want.ndim > 2 else None
    head = np.sqrt(np.mean(want ** 2, axis=axes, keepdims=True))
    bound = half * np.abs(want) + 16 * (e + low) * np.maximum(rms, head)
    bad = np.abs(got - want) > bound
    assert not bad.any(), (what, float(np.max(np.abs(got - want) / np.maximum(bound, 1e-300))), e)
    return worst


def check_forward(r, a, dtype, walks=1):
    """walks: 2 where a walk goes in segments.  A segment's start is its map times the start before it:
    each of the map's columns is a walk of its own, whose errors meet the start in no fixed direction."""
    want = delta_forward(*(a[n] for n in NAMES[:5]), s0=a["s0"], lengths=a["lengths"])
    e = e32(a, 12 * walks)
    close(r["o"], want["o"], e, dtype, "o")
    if "s_final" in r:
        close(r["s_final"], want["s_final"], e, torch.float32, "s_final")
    behind(r, a, ("o",))
    return want


def behind(r, a, names):
    if a["lengths"] is not None:
        for b, stop in enumerate(np.clip(a["lengths"], 0, a["v"].shape[2])):
            for n in names:
                assert not r[n][b, :, int(stop):].any(), (n, b)


def check_backward(r, a, dtype, walks=1):
    want = delta_backward(*(a[n] for n in NAMES[:6]), s0=a["s0"], lengths=a["lengths"], d_sfinal=a["d_sfinal"])
    e = e32(a, 20 * walks)
    for n in ("dq", "dk", "dv"):
        close(r[n], want[n], e, dtype, n)
    close(r["dbeta"], want["dbeta"], e, torch.float32, "dbeta")
    # a difference <N, S> - dw . S k, each term with the bound's error, formed at log gamma and
    # divided: with keys that repeat the terms cancel (S lies along k, which I - k k^T removes)
    off = (r["dgamma"].double().cpu().numpy() - want["dgamma"]) * a["gamma"]
    size = want["dgamma_sizes"] * a["gamma"] + np.abs(want["dgamma"] * a["gamma"])
    assert np.isfinite(off).all()
    norm = np.linalg.norm(size, axis=-1)
    assert np.all(np.linalg.norm(off, axis=-1) <= e * norm), ("dgamma", np.linalg.norm(off, axis=-1) / norm, e)
    assert np.all(np.abs(off) <= 16 * e * np.maximum(size, norm[..., None] / np.sqrt(size.shape[-1])))
    if "ds0" in r:
        close(r["ds0"], want["ds0"], e, torch.float32, "ds0")
    behind(r, a, ("dq", "dk", "dv", "dgamma", "dbeta"))
    return want
