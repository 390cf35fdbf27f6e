"""Residual addition and RMS norm, and its gradient, on the GPU against the fp64 oracle.

Bounds, element by element, with e = 2^-24 (half a step of fp32): a row's sum of
D terms is formed by lanes that add at most 128 terms each and a tree of 10 more
levels, so its relative error is at most DEPTH e with DEPTH = min(D, 128) + 10
for terms of one sign (else DEPTH e of the sum of magnitudes); the root halves
it; each further product or quotient adds e or 2 e.  bf16 outputs add half a
step, 2^-8 of the value; e4m3 outputs half a step of theirs, 2^-4 of the value
or 2^-10 (of the scaled value) in the subnormal range.  Needs an MI355X.
"""
import numpy as np
import pytest
import torch

from oracle.block_oracle import rmsnorm, rmsnorm_backward
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def depth(D):
    return min(D, 128) + 10


def half(t):
    return 2.0 ** -8 if t == "bf16" else E


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def draw(R, D, dtype, res, seed=0):
    rng = np.random.default_rng([seed, R, D])
    f = lambda t, s=1.0: torch.from_numpy((s * rng.standard_normal((R, D))).astype(np.float32)).to(TORCH[t])  # noqa: E731
    d = dict(x=f(dtype), residual=f(res, 2.0), dy=f(dtype), d_residual=f(res))
    d["w"] = torch.from_numpy(rng.uniform(0.5, 1.5, D).astype(np.float32))
    return d, {k: v.cuda() for k, v in d.items()}


def close(got, want, bound, what):
    got = host(got)
    bad = ~(np.abs(got - want) <= bound + 1e-37)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           float(np.nanmax(np.abs(got - want) / (bound + 1e-37))))


def check_forward(d, r, dtype, res, group, eps, residual=True):
    ref = rmsnorm(host(d["x"]), host(d["w"]), residual=host(d["residual"]) if residual else None, eps=eps, group=group)
    D = ref["y"].shape[1]
    rel = (0.5 * depth(D) + 8) * E
    if group is None:
        close(r["y"], ref["y"], (rel + half(dtype)) * np.abs(ref["y"]), "y")
    else:
        g = group or D
        close(r["scale"], ref["scale"], (rel + 2 * E) * ref["scale"], "scale")
        v = ref["y"] / np.repeat(ref["scale"], g, axis=1)[:, :D]
        close(r["y"], v, np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) * (1 + 1e-5) + (2 * rel + 8 * E) * np.abs(v), "codes")
        # what the codes and scales stand for lies on the oracle's rounding, but for values next to a tie
        off = host(r["y"]) != ref["q"]
        near = np.abs(np.abs(host(r["y"]) + ref["q"]) / 2 - np.abs(v)) <= (2 * rel + 8 * E) * np.abs(v) + 1e-30
        assert near[off].all(), int((off & ~near).sum())
    if "residual" in r:
        s = ref["residual"]
        close(r["residual"], s, (half(res) + 2 * E) * np.abs(s), "residual")


SIZES = [(1, 1), (3, 7), (5, 16), (2, 64), (9, 100), (4, 128), (33, 129), (2, 255), (7, 256), (3, 1001), (65, 2048),
         (2, 2056), (3, 5000), (2, 8192), (2, 12001), (2, 16384), (4500, 40), (2100, 515)]


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("R,D", SIZES)
def test_forward_matches_the_oracle(R, D, dtype, res):
    d, t = draw(R, D, dtype, res)
    for group in (None, 0, 128):
        r = mesa.rmsnorm(t["x"], t["w"], residual=t["residual"], eps=1e-5, quant_group=group)
        torch.cuda.synchronize()
        check_forward(d, r, dtype, res, group, 1e-5)
    r = mesa.rmsnorm(t["x"], t["w"], eps=0.5)  # without a residual
    torch.cuda.synchronize()
    assert set(r) == {"y"}
    check_forward(d, r, dtype, dtype, None, 0.5, residual=False)


def check_backward(d, g, dtype, res, with_res):
    s, w, dy = host(d["residual"]), host(d["w"]), host(d["dy"])
    R, D = s.shape
    dres = host(d["d_residual"]) if with_res else None
    ref = rmsnorm_backward(s, w, dy, d_residual=dres, eps=1e-5)
    rstd = 1 / np.sqrt((s * s).mean(1, keepdims=True) + 1e-5)
    n, gg = np.abs(s * rstd), np.abs(dy * w)
    size = rstd * (gg + n * (gg * n).mean(1, keepdims=True))
    bound = (1.5 * depth(D) + 12) * E * size + 2 * E * np.abs(ref["ds"])
    close(g["ds"], ref["ds"], bound + half(res) * np.abs(ref["ds"]), "ds")
    if dtype != res:
        close(g["dx"], ref["ds"], bound + half(dtype) * np.abs(ref["ds"]), "dx")
    # at most R additions deep over the rows
    close(g["dw"], ref["dw"], (R + 0.5 * depth(D) + 12) * E * (np.abs(dy) * n).sum(0), "dw")


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("R,D", SIZES)
def test_backward_matches_the_oracle(R, D, dtype, res):
    d, t = draw(R, D, dtype, res, seed=1)
    for with_res in (True, False):
        g = mesa.rmsnorm_bwd(t["residual"], t["w"], t["dy"], d_residual=t["d_residual"] if with_res else None, eps=1e-5)
        torch.cuda.synchronize()
        check_backward(d, g, dtype, res, with_res)


def test_rows_of_zeros_and_extremes():
    """A row of zeros (finite scale, codes 0), tiny and huge rows, and one row with NaN that leaves the others alone."""
    D = 300
    x = torch.randn(6, D, generator=torch.Generator().manual_seed(3))
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e15
    x[3, 5] = float("nan")
    x[4, 1:] = 0
    w = torch.ones(D)
    for group in (None, 0, 128):
        r = mesa.rmsnorm(x.cuda(), w.cuda(), eps=1e-6, quant_group=group)
        torch.cuda.synchronize()
        ok = [0, 1, 2, 4, 5]
        check_forward(dict(x=x[ok], w=w), {k: v[ok] for k, v in r.items()}, "f32", "f32", group, 1e-6, residual=False)
    assert (r["y"][0].float() == 0).all() and torch.isfinite(r["scale"][0]).all()


def test_in_place_residual():
    """out["residual"] may be the residual, and the backward's ds may be d_residual: same values as apart."""
    for dtype, res in TYPES:
        # (2561, 4101: a row's last vector and its neighbour lie in different waves)
        for D in (3, 96, 1001, 2561, 4096, 4101, 12000, 12295):
            d, t = draw(5, D, dtype, res, seed=4)
            a = mesa.rmsnorm(t["x"], t["w"], residual=t["residual"], quant_group=128)
            b_res = t["residual"].clone()
            b = mesa.rmsnorm(t["x"], t["w"], residual=b_res, quant_group=128, out={"residual": b_res})
            ga = mesa.rmsnorm_bwd(t["residual"], t["w"], t["dy"], d_residual=t["d_residual"])
            buf = t["d_residual"].clone()
            gb = mesa.rmsnorm_bwd(t["residual"], t["w"], t["dy"], d_residual=buf, out={"ds": buf})
            torch.cuda.synchronize()
            assert b["residual"] is b_res and gb["ds"] is buf
            for p, q in ((a, b), (ga, gb)):
                for key in p:
                    assert torch.equal(p[key].view(torch.uint8), q[key].view(torch.uint8)), (dtype, res, D, key)


def test_no_rows():
    w = torch.ones(40, device="cuda")
    x = torch.empty((0, 40), device="cuda")
    r = mesa.rmsnorm(x, w, residual=x, quant_group=0)
    assert r["y"].shape == (0, 40) and r["scale"].shape == (0, 1) and r["residual"].shape == (0, 40)
    dw = torch.full((40,), 3.0, device="cuda")
    g = mesa.rmsnorm_bwd(x, w, x, out={"dw": dw})
    torch.cuda.synchronize()
    assert g["ds"].shape == (0, 40) and (dw == 0).all()


def test_repeated_calls_are_bitwise_equal():
    _, t = draw(3001, 1500, "bf16", "bf16", seed=5)
    first = None
    for _ in range(3):
        r = mesa.rmsnorm_bwd(t["residual"], t["w"], t["dy"], d_residual=t["d_residual"])
        torch.cuda.synchronize()
        first = first or r
        for key in r:
            assert torch.equal(r[key], first[key]), key


def test_gradients_match_differences():
    """Central differences of the GPU forward (fp32): with a step of 2^-6 the truncation is
    of order 2^-12 of the gradient and the rounding of L below 2^-24 sqrt(n) |dy y| / step."""
    R, D = 6, 200
    d, t = draw(R, D, "f32", "f32", seed=6)
    x0 = torch.zeros_like(t["x"])
    g = mesa.rmsnorm_bwd(t["residual"], t["w"], t["dy"], d_residual=t["d_residual"])

    def loss(s, w):
        r = mesa.rmsnorm(x0, w, residual=s)
        return float((r["y"].double() * t["dy"].double()).sum() + (r["residual"].double() * t["d_residual"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(1)
    step = 2.0 ** -6
    for which, gk in ((0, "ds"), (1, "dw")):
        base = [t["residual"], t["w"]]
        e = torch.randn(base[which].shape, generator=gen, device="cuda")
        vals = []
        for sign in (1, -1):
            a = list(base)
            a[which] = base[which] + sign * step * e
            vals.append(loss(*a))
        num, ana = (vals[0] - vals[1]) / (2 * step), float((g[gk].double() * e.double()).sum())
        assert abs(num - ana) <= 3e-3 * float(g[gk].double().norm()) + 1e-3, (gk, num, ana)


def test_stream_over_the_rows():
    """out["residual"] may be x where the types are equal, and without a residual the stream is x itself."""
    for dtype in ("f32", "bf16"):
        for D in (5, 130, 2048, 2561, 4101, 9000, 12295):
            d, t = draw(7, D, dtype, dtype, seed=6)
            want = mesa.rmsnorm(t["x"], t["w"], residual=t["residual"])
            x = t["x"].clone()
            got = mesa.rmsnorm(x, t["w"], residual=t["residual"], out={"residual": x})
            alone = mesa.rmsnorm(t["x"], t["w"], return_residual=True)
            torch.cuda.synchronize()
            assert got["residual"] is x and torch.equal(x, want["residual"]) and torch.equal(got["y"], want["y"])
            assert torch.equal(alone["residual"], t["x"])


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("D", [2, 5, 9, 10, 11, 12, 13, 14, 15, 134, 518, 1001, 2051, 4109, 12006])
def test_rows_that_end_within_a_vector(D, dtype, res):
    """Every remainder of D by 8 against the oracle, and nothing written behind the last row."""
    R, mark = 3, 77
    d, t = draw(R, D, dtype, res, seed=5)
    for group in (None, 0, 128):
        y_type = TORCH[dtype] if group is None else torch.float8_e4m3fn
        y, stream = torch.empty(R * D + 16, dtype=y_type, device="cuda"), torch.empty(R * D + 16, dtype=TORCH[res], device="cuda")
        y.view(torch.uint8).fill_(mark)
        stream.view(torch.uint8).fill_(mark)
        r = mesa.rmsnorm(t["x"], t["w"], residual=t["residual"], eps=1e-5, quant_group=group,
                         out={"y": y[:R * D].view(R, D), "residual": stream[:R * D].view(R, D)})
        torch.cuda.synchronize()
        check_forward(d, r, dtype, res, group, 1e-5)
        assert (y.view(torch.uint8)[R * D * y.element_size():] == mark).all()
        assert (stream.view(torch.uint8)[R * D * stream.element_size():] == mark).all()
    ds = torch.empty(R * D + 16, dtype=TORCH[res], device="cuda")
    ds.view(torch.uint8).fill_(mark)
    g = mesa.rmsnorm_bwd(t["residual"], t["w"], t["dy"], d_residual=t["d_residual"], eps=1e-5,
                         out={"ds": ds[:R * D].view(R, D)})
    torch.cuda.synchronize()
    check_backward(d, g, dtype, res, True)
    assert (ds.view(torch.uint8)[R * D * ds.element_size():] == mark).all()
