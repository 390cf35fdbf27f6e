"""Gradient of the query/key preprocessing on the GPU against the fp64 oracle.

Bounds, element by element, with e = 2^-24: the convolution's sum of W products
is off by at most (W + 1) e of its magnitudes; the norm's relative error rn is
that error's norm over n, plus a tree of at most 20 roundings, plus 3 e for the
reciprocal square root; the rest follows the formula term by term, each product
or sum adding e of its magnitude.  bf16 outputs add half a step, 2^-8.
Needs an MI355X.
"""
import numpy as np
import pytest
import torch

from oracle.block_oracle import qk_preprocess_backward
from test_regression_sequence_amd import mesa
from test_regression_sequence_amd.inputs import CONFIGS, make_preprocess_inputs, small_fwd

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def to_dev(a, dtype):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t.float()


def rounded(a, dtype):
    a = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    return (a.to(torch.bfloat16) if dtype == "bf16" else a).float().numpy()


def grads_in(cfg, W, seed=21):
    rng = np.random.default_rng([cfg.seed, seed])
    shp, hshp = (cfg.B, cfg.H, cfg.T, cfg.d), (cfg.B, cfg.H, W - 1, cfg.d)
    g = {"d" + n: rng.standard_normal(shp).astype(np.float32) for n in "qk"}
    g.update({"h" + n: rounded(rng.standard_normal(hshp), cfg.dtype) for n in "qk"})
    return g


def run(x, g, dtype, hist, dhist, eps=1e-6, **kw):
    return mesa.qk_preprocess_bwd(
        to_dev(x["q"], dtype), to_dev(x["k"], dtype), torch.from_numpy(x["wq"]).cuda(), torch.from_numpy(x["wk"]).cuda(),
        torch.from_numpy(g["dq"]).cuda(), torch.from_numpy(g["dk"]).cuda(),
        q_hist=to_dev(x["hq"], dtype) if hist else None, k_hist=to_dev(x["hk"], dtype) if hist else None,
        d_q_hist_out=to_dev(g["hq"], dtype) if dhist else None, d_k_hist_out=to_dev(g["hk"], dtype) if dhist else None,
        eps=eps, history_grads=True, **kw)


def bounds(x, w, d, hist, eps, dhist):
    """Error bounds of e, dx (history rows first) and dw, before any rounding to bf16."""
    B, H, T, D = x.shape
    W = w.shape[-1]
    seq = np.concatenate([np.zeros((B, H, W - 1, D)) if hist is None else hist, x], 2).astype(np.float64)
    rows = [seq[:, :, W - 1 - i:W - 1 - i + T] for i in range(W)]
    taps = [w[None, :, None, :, i].astype(np.float64) for i in range(W)]
    y = sum(t * r for t, r in zip(taps, rows))
    ey = (W + 1) * E * sum(np.abs(t * r) for t, r in zip(taps, rows))
    nrm = np.linalg.norm(y, axis=-1, keepdims=True)
    n = np.maximum(nrm, eps)
    rn = np.linalg.norm(ey, axis=-1, keepdims=True) / n + 23 * E
    o, en, a = np.abs(y) / n, ey / n, np.abs(d)
    dot = (o * a).sum(-1, keepdims=True)
    edot = (en * a).sum(-1, keepdims=True) + dot * (rn + 24 * E)
    ee = (a * (rn + 2 * E) + o * edot + en * dot + o * dot * (2 * rn + 6 * E)) / n
    e = (a + o * dot) / n
    dx, ex = np.zeros_like(seq), np.zeros_like(seq)
    for i in range(W):
        ex[:, :, W - 1 - i:W - 1 - i + T] += np.abs(taps[i]) * (ee + (W + 2) * E * e)
    if dhist is not None:
        ex[:, :, T:] += 2 * E * np.abs(dhist)
    dw = np.stack([((ee + (B * T + 4) * E * e) * np.abs(r)).sum((0, 2)) for r in rows], -1)
    return ex[:, :, W - 1:], ex[:, :, :W - 1], dw


def close(got, want, bound, dtype, what):
    got = got.float().cpu().numpy().astype(np.float64)
    tol = bound + (2.0 ** -8 if dtype == "bf16" else E) * np.abs(want) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.nanmax(np.abs(got - want) / tol)))


def check(x, g, r, dtype, hist, dhist, eps=1e-6, sl=None):
    for n in "qk":
        h = x["h" + n] if hist else None
        dh = g["h" + n] if dhist else None
        ref = qk_preprocess_backward(x[n], x["w" + n], g["d" + n], h, dh, eps=eps)
        bx, bh, bw = bounds(x[n], x["w" + n], g["d" + n].astype(np.float64), h, eps, dh)
        close(r[f"d{n}_raw"], ref["dx"], bx, dtype, n + " raw")
        close(r["dw_" + n], ref["dw"], bw, "f32", n + " taps")
        close(r[f"d{n}_hist"], ref["dhist"], bh, dtype, n + " history")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,T,W", [(128, 300, 4), (128, 77, 2), (64, 600, 3), (64, 5, 4), (64, 1, 4), (128, 2, 4),
                                   (16, 40, 1), (16, 2100, 4), (128, 64, 3), (64, 129, 2)])
@pytest.mark.parametrize("hist,dhist", [(False, False), (True, True), (True, False), (False, True)])
def test_matches_oracle(dtype, d, T, W, hist, dhist):
    cfg = small_fwd(B=2, H=3, T=T, d=d, dtype=dtype)
    x = make_preprocess_inputs(cfg, window=W)
    g = grads_in(cfg, W)
    r = run(x, g, dtype, hist, dhist)
    torch.cuda.synchronize()
    check(x, g, r, dtype, hist, dhist)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_below_eps_and_rows_of_zeros(dtype):
    """Rows whose norm is below eps are only scaled; a row of zeros has a finite gradient."""
    cfg = small_fwd(B=1, H=2, T=40, d=64, dtype=dtype)
    x = make_preprocess_inputs(cfg, window=3)
    for n in "qk":
        x[n][:, :, 10:20] = 0
        x[n][:, :, 25:30] *= np.float32(2.0 ** -8)
    g = grads_in(cfg, 3)
    r = run(x, g, dtype, True, False, eps=0.25)
    torch.cuda.synchronize()
    check(x, g, r, dtype, True, False, eps=0.25)


def test_split_sequence_hands_its_history_gradient_back():
    """Gradients of a sequence in one call equal those of its two halves, the second half's
    history gradient entering the first: within the bound of either (fp32)."""
    cfg = small_fwd(B=2, H=2, T=150, d=128, dtype="f32")
    x = make_preprocess_inputs(cfg, window=4)
    g = grads_in(cfg, 4)
    cut = 71
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    w = dev(x["wq"]), dev(x["wk"])
    second = mesa.qk_preprocess_bwd(dev(x["q"][:, :, cut:]), dev(x["k"][:, :, cut:]), *w, dev(g["dq"][:, :, cut:]),
                                    dev(g["dk"][:, :, cut:]), q_hist=dev(x["q"][:, :, cut - 3:cut]),
                                    k_hist=dev(x["k"][:, :, cut - 3:cut]), history_grads=True)
    first = mesa.qk_preprocess_bwd(dev(x["q"][:, :, :cut]), dev(x["k"][:, :, :cut]), *w, dev(g["dq"][:, :, :cut]),
                                   dev(g["dk"][:, :, :cut]), q_hist=dev(x["hq"]), k_hist=dev(x["hk"]),
                                   d_q_hist_out=second["dq_hist"], d_k_hist_out=second["dk_hist"], history_grads=True)
    torch.cuda.synchronize()
    joined = {}
    for n in "qk":
        joined[f"d{n}_raw"] = torch.cat([first[f"d{n}_raw"], second[f"d{n}_raw"]], 2)
        joined[f"d{n}_hist"] = first[f"d{n}_hist"]
        joined["dw_" + n] = first["dw_" + n] + second["dw_" + n]
    check(x, g, joined, "f32", True, False)


def test_empty_sequence_passes_history_gradients_through():
    cfg = small_fwd(B=1, H=2, T=0, d=64, dtype="bf16")
    x = make_preprocess_inputs(cfg, window=4)
    g = grads_in(cfg, 4)
    r = run(x, g, "bf16", True, True)
    torch.cuda.synchronize()
    for n in "qk":
        assert np.array_equal(r[f"d{n}_hist"].float().cpu().numpy(), g["h" + n])
        assert (r["dw_" + n] == 0).all()
    r = run(x, g, "bf16", True, False)
    torch.cuda.synchronize()
    assert (r["dq_hist"] == 0).all() and (r["dk_hist"] == 0).all()


def test_repeated_calls_are_bitwise_equal():
    cfg = small_fwd(B=3, H=4, T=1300, d=128, dtype="bf16")
    x = make_preprocess_inputs(cfg, window=4)
    g = grads_in(cfg, 4)
    first = None
    for _ in range(3):
        r = run(x, g, "bf16", True, True)
        torch.cuda.synchronize()
        first = first or r
        for key in r:
            assert torch.equal(r[key], first[key]), key


def test_gradients_match_differences():
    """Central differences of the GPU forward in fp32 (step 2^-7: truncation of order 2^-14,
    rounding of L of order 2^-24 sqrt(n) / step)."""
    cfg = small_fwd(B=1, H=2, T=30, d=64, dtype="f32")
    x = make_preprocess_inputs(cfg, window=4)
    g = grads_in(cfg, 4)
    r = run(x, g, "f32", True, True)
    dev = {k: torch.from_numpy(v).cuda() for k, v in x.items() if isinstance(v, np.ndarray)}
    gd = {k: torch.from_numpy(v).cuda().double() for k, v in g.items()}

    def loss(**kw):
        u = dict(dev, **kw)
        f = mesa.qk_preprocess(u["q"], u["k"], u["wq"], u["wk"], q_hist=u["hq"], k_hist=u["hk"], return_history=True)
        return float(sum((f[n].double() * gd["d" + n]).sum() + (f[n + "_hist"].double() * gd["h" + n]).sum() for n in "qk"))

    gen = torch.Generator(device="cuda").manual_seed(1)
    step = 2.0 ** -7
    for key, gk in (("q", "dq_raw"), ("k", "dk_raw"), ("wq", "dw_q"), ("wk", "dw_k"), ("hq", "dq_hist"), ("hk", "dk_hist")):
        e = torch.randn(dev[key].shape, generator=gen, device="cuda")
        num = (loss(**{key: dev[key] + step * e}) - loss(**{key: dev[key] - step * e})) / (2 * step)
        ana = float((r[gk].double() * e.double()).sum())
        assert abs(num - ana) <= 5e-3 * float(r[gk].double().norm()) + 2e-3, (key, num, ana)


def test_lm_workload_sampled_slices():
    """The layer workload's shape (B=8, H=16, T=4096, d=128, bf16), raw gradients on sampled slices."""
    cfg = CONFIGS[3]
    x = make_preprocess_inputs(cfg, window=4)
    rng = np.random.default_rng(5)
    shp = (cfg.B, cfg.H, cfg.T, cfg.d)
    g = {"d" + n: rng.standard_normal(shp, dtype=np.float32) for n in "qk"}
    r = mesa.qk_preprocess_bwd(to_dev(x["q"], "bf16"), to_dev(x["k"], "bf16"), torch.from_numpy(x["wq"]).cuda(),
                               torch.from_numpy(x["wk"]).cuda(), torch.from_numpy(g["dq"]).cuda(),
                               torch.from_numpy(g["dk"]).cuda())
    torch.cuda.synchronize()
    for b, h in ((0, 0), (7, 15), (3, 8)):
        for n in "qk":
            s = (slice(b, b + 1), slice(h, h + 1))
            w = x["w" + n][h:h + 1]
            ref = qk_preprocess_backward(x[n][s], w, g["d" + n][s])
            bx, _, _ = bounds(x[n][s], w, g["d" + n][s].astype(np.float64), None, 1e-6, None)
            close(r[f"d{n}_raw"][s], ref["dx"], bx, "bf16", n)
    h = 5  # one head's taps, summed over the batch
    ref = qk_preprocess_backward(x["q"][:, h:h + 1], x["wq"][h:h + 1], g["dq"][:, h:h + 1])
    _, _, bw = bounds(x["q"][:, h:h + 1], x["wq"][h:h + 1], g["dq"][:, h:h + 1].astype(np.float64), None, 1e-6, None)
    close(r["dw_q"][h:h + 1], ref["dw"], bw, "f32", "taps")
