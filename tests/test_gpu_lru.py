"""Gated linear recurrence on the GPU against the fp64 oracle, element by element.

The bounds come from the arithmetic, before any run: with e = 2^-24 (half a
step of fp32, relative) and the hardware's exp2, reciprocal and square roots
good to one unit in the last place (2 e),
    sigmoid(z):  (2 |z| + 6) e    (z log2(e) is two roundings of the exponent),
    rate:        8 e,    w = rate sigmoid:  es + 9 e,
    a = exp(-w/2): (w/2) (ew + 3 e) + 2 e,
    1 - a^2:     ew + 9 e below w = 1/4 (series), else (2 ea + 2 e) / (1 - a^2),
    m: half of it + 4 e,   u = m sigmoid(gi) x:  em + es + 3 e,
and an error E_t of the state follows E_t = a_t E_{t-1} + ea a_t |h_{t-1}| +
eu |u_t| + 2 e |h_t|; products over several tokens (a split of the sequence)
only reorder these terms, which the factor SLACK covers.  bf16 outputs add
half a step, 2^-8 of the value.  Needs an MI355X.
"""
import numpy as np
import pytest
import torch

from oracle.block_oracle import lru_backward, lru_forward, lru_gates, lru_step
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
SLACK = 2.0  # fused or separate roundings of one product chain: at most one more each
C = 8.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16)


def draw(B, T, D, dtype, seed=0, ragged=False, h0=True, lam=(-9.0, -3.0), scale=1.0):
    rng = np.random.default_rng([seed, B, T, D])
    d = {k: rng.standard_normal((B, T, D)).astype(np.float32) * np.float32(scale if k != "dy" else 1) for k in ("x", "ga", "gi", "dy")}
    if dtype == "bf16":
        d = {k: bf16(v).float().numpy() for k, v in d.items()}
    d["lam"] = rng.uniform(*lam, D).astype(np.float32)
    d["h0"] = rng.standard_normal((B, D)).astype(np.float32) if h0 else None
    d["d_hfinal"] = rng.standard_normal((B, D)).astype(np.float32) if h0 else None
    d["lengths"] = None
    if ragged:
        n = rng.integers(0, T + 1, B)
        n[0] = T
        if B > 1:
            n[1] = 0
        d["lengths"] = n.astype(np.int32)
    return d


def to_dev(d, dtype, poison=True):
    t = {}
    for k, v in d.items():
        if v is None:
            t[k] = None
            continue
        v = torch.from_numpy(v.copy()).cuda()
        if k in ("x", "ga", "gi", "dy") and dtype == "bf16":
            v = v.to(torch.bfloat16)
        t[k] = v
    if poison and d["lengths"] is not None:  # rows behind a length may hold anything
        for b, n in enumerate(d["lengths"]):
            for k, bad in (("x", float("nan")), ("ga", float("inf")), ("gi", float("nan")), ("dy", float("-inf"))):
                t[k][b, n:] = bad
    return t


def unit_errors(d):
    """Per element: w, a, m, u and the relative errors of a, m, sigma_i, u and their like."""
    w, a, m, sr, si = lru_gates(d["x"], d["ga"], d["gi"], d["lam"], C)
    es = lambda z: (2 * np.abs(z) + 6) * E  # noqa: E731
    esr, esi = es(d["ga"].astype(np.float64)), es(d["gi"].astype(np.float64))
    ew = esr + 9 * E
    ea = 0.5 * w * (ew + 3 * E) + 2 * E
    m2 = np.maximum(m * m, 1e-300)
    em = 0.5 * np.where(w < 0.26, np.maximum(ew + 9 * E, (w > 0.24) * (2 * ea + 2 * E) / m2), (2 * ea + 2 * E) / m2) + 4 * E
    x = d["x"].astype(np.float64)
    off = lambda z: 1 / (1 + np.exp(np.minimum(z.astype(np.float64), 700)))  # noqa: E731  1 - sigmoid
    return dict(w=w, a=a, m=m, sr1=off(d["ga"]), si=si, si1=off(d["gi"]), u=m * si * x, x=x, ea=ea, em=em, esr=esr, esi=esi, ew=ew,
                eu=em + esi + 3 * E)


def state_bound(d, q, ref):
    B, T, D = q["a"].shape
    n = np.full(B, T) if d["lengths"] is None else d["lengths"]
    err, out = np.zeros((B, D)), np.zeros((B, T, D))
    before = np.zeros((B, T, D))
    for t in range(T):
        before[:, t] = err
        h1 = np.abs(ref["prev"][:, t])
        h = np.abs(ref["y"][:, t])
        new = q["a"][:, t] * err + q["ea"][:, t] * q["a"][:, t] * h1 + q["eu"][:, t] * np.abs(q["u"][:, t]) + 2 * E * h
        live = (t < n)[:, None]
        err = np.where(live, new, err)
        out[:, t] = np.where(live, err, 0)
    return out, before, err


def within(got, want, bound, dtype, what):
    got = got.float().cpu().numpy().astype(np.float64)
    tol = SLACK * bound + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0) + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           float(np.nanmax(np.abs(got - want) / tol)))


def run_fwd(d, t, **kw):
    return mesa.lru_fwd(t["x"], t["ga"], t["gi"], t["lam"], c=C, h0=t["h0"], lengths=t["lengths"], return_state=True, **kw)


def check_forward(d, r, dtype):
    ref = lru_forward(d["x"], d["ga"], d["gi"], d["lam"], c=C, h0=d["h0"], lengths=d["lengths"])
    q = unit_errors(d)
    by, _, bh = state_bound(d, q, ref)
    within(r["y"], ref["y"], by, dtype, "y")
    within(r["h_final"], ref["h_final"], bh, "f32", "h_final")
    return ref, q


def check_backward(d, r, dtype):
    args = (d["x"], d["ga"], d["gi"], d["lam"])
    kw = dict(c=C, h0=d["h0"], lengths=d["lengths"])
    ref, fwd = lru_backward(*args, d["dy"], d_hfinal=d["d_hfinal"], **kw), lru_forward(*args, **kw)
    q = unit_errors(d)
    _, eh, _ = state_bound(d, q, fwd)
    B, T, D = q["a"].shape
    n = np.full(B, T) if d["lengths"] is None else d["lengths"]
    g = np.zeros((B, D)) if d["d_hfinal"] is None else d["d_hfinal"].astype(np.float64)
    eg, G, EG = np.zeros((B, D)), np.zeros((B, T, D)), np.zeros((B, T, D))
    for t in range(T - 1, -1, -1):
        live = (t < n)[:, None]
        now = g + d["dy"][:, t].astype(np.float64)
        enow = eg + 2 * E * np.abs(now)
        G[:, t], EG[:, t] = np.where(live, now, 0), np.where(live, enow, 0)
        g = np.where(live, q["a"][:, t] * now, g)
        eg = np.where(live, q["a"][:, t] * (enow + q["ea"][:, t] * np.abs(now)), eg)
    aG, h1 = np.abs(G), np.abs(fwd["prev"])
    dxg, dgig = q["m"] * q["si"], np.abs(q["u"]) * q["si1"]
    within(r["dx"], ref["dx"], EG * dxg + aG * dxg * q["eu"], dtype, "dx")
    within(r["dgi"], ref["dgi"], EG * dgig + aG * dgig * (q["eu"] + 2 * q["esi"] + 3 * E), dtype, "dgi")
    with np.errstate(divide="ignore", invalid="ignore"):
        vu = np.where(q["m"] > 0, 0.5 * q["w"] * q["a"] ** 2 / q["m"] * q["si"] * np.abs(q["x"]), 0)
    va = 0.5 * q["w"] * q["a"]
    ev = vu * (q["ew"] + 2 * q["ea"] + q["em"] + q["esi"] + 6 * E) + va * h1 * (q["ew"] + q["ea"] + 4 * E) + va * eh
    size = vu + va * h1
    bv = EG * size + aG * ev + 2 * E * aG * size
    within(r["dga"], ref["dga"], (bv + aG * size * (2 * q["esr"] + 3 * E)) * q["sr1"], dtype, "dga")
    # the sum over tokens: at most T + B additions deep
    lam = d["lam"].astype(np.float64)
    slope = (1 / (1 + np.exp(-lam))) / np.log1p(np.exp(lam))
    within(r["dlam"], ref["dlam"], (bv.sum((0, 1)) + (T + B + 8) * E * (aG * size).sum((0, 1))) * slope, "f32", "dlam")
    if "dh0" in r:
        within(r["dh0"], ref["dh0"], eg, "f32", "dh0")


SIZES = [  # B, T, D, ragged
    (1, 1, 2, False), (2, 1, 64, False), (3, 2, 7, True), (2, 150, 3, True), (1, 130, 2, False), (1, 63, 256, False), (2, 64, 128, False), (3, 65, 100, True),
    (2, 127, 260, False), (1, 128, 512, False), (2, 129, 1001, True), (5, 200, 36, True), (1, 1000, 68, False),
    (4, 300, 516, True), (1, 2500, 33, False), (2, 1111, 320, True),
    (3, 47, 65, True), (2, 48, 66, False), (2, 49, 127, False), (1, 95, 130, False), (3, 96, 64, True), (2, 97, 2, False),
    (7, 2, 100, True), (5, 7, 64, True), (9, 8, 130, True), (3, 9, 65, False), (5, 15, 192, True), (3, 16, 33, False),
    (4, 17, 128, True), (3, 31, 66, True), (2, 32, 1001, True), (3, 33, 64, True), (20, 5, 2048, True), (6, 30, 257, True),
    (1, 16384, 5, False), (1, 16385, 66, False), (2, 32769, 6, True), (1, 40000, 3, False), (1, 70001, 2, False),
    (1, 1023, 63, False), (2, 1025, 129, True), (1, 2048, 64, False), (3, 2049, 70, True),
    (1, 767, 63, False), (2, 769, 129, True), (1, 1535, 64, False), (3, 1537, 70, True), (40, 100, 200, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D,ragged", SIZES)
def test_forward_and_backward_match_the_oracle(dtype, B, T, D, ragged):
    d = draw(B, T, D, dtype, ragged=ragged, h0=(B + T) % 2 == 0)
    t = to_dev(d, dtype)
    ws = torch.empty(mesa.lru_workspace_bytes(B, T, D, dtype=t["x"].dtype), device="cuda", dtype=torch.uint8)
    r = run_fwd(d, t, workspace=ws)
    kw = dict(c=C, h0=t["h0"], lengths=t["lengths"], d_hfinal=t["d_hfinal"], state_grads=True)
    g = mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], workspace=ws, states_in_workspace=True, **kw)
    alone = mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], **kw)
    torch.cuda.synchronize()
    check_forward(d, r, dtype)
    check_backward(d, g, dtype)
    for key in g:  # states taken over or formed again: the same values
        assert torch.equal(g[key], alone[key]), key


@pytest.mark.parametrize("lam,scale", [((-30.0, -12.0), 1.0), ((0.0, 6.0), 1.0), ((-6.0, 2.0), 12.0)])
def test_decays_from_none_to_complete(lam, scale):
    """Rates so small that a rounds to 1, so large that it underflows, and gates deep in saturation."""
    d = draw(2, 150, 65, "f32", lam=lam, scale=scale, seed=3)
    t = to_dev(d, "f32")
    r = run_fwd(d, t)
    g = mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], c=C, h0=t["h0"], d_hfinal=t["d_hfinal"], state_grads=True)
    torch.cuda.synchronize()
    check_forward(d, r, "f32")
    check_backward(d, g, "f32")


def test_infinite_gate_logits_keep_or_open():
    """ga = -inf: a = 1, the state passes unchanged and no input enters; gi = -inf: no input; all gradients finite."""
    d = draw(1, 70, 8, "f32", seed=4)
    d["ga"][:, ::3] = -np.inf
    d["gi"][:, 1::3] = -np.inf
    d["ga"][:, 2::3] = np.inf
    t = to_dev(d, "f32")
    r = run_fwd(d, t)
    g = mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], c=C, h0=t["h0"], d_hfinal=t["d_hfinal"], state_grads=True)
    torch.cuda.synchronize()
    fin = {k: (np.clip(v, -200, 200) if k in ("ga", "gi") else v) for k, v in d.items()}  # the same gates to 1e-87
    ref = lru_forward(fin["x"], fin["ga"], fin["gi"], fin["lam"], c=C, h0=fin["h0"])
    assert np.abs(r["y"].cpu().numpy() - ref["y"]).max() <= 1e-5
    y = r["y"]
    assert torch.equal(y[:, 3], y[:, 2])
    gr = lru_backward(fin["x"], fin["ga"], fin["gi"], fin["lam"], fin["dy"], c=C, h0=fin["h0"], d_hfinal=fin["d_hfinal"])
    for key in g:
        assert torch.isfinite(g[key]).all(), key
        assert np.abs(g[key].cpu().numpy() - gr[key]).max() <= 1e-4 * max(1, np.abs(gr[key]).max()), key


def test_all_lengths_zero_and_out_of_range():
    d = draw(3, 130, 66, "f32", seed=5)
    t = to_dev(d, "f32")
    for lens, clamped in (([0, 0, 0], [0, 0, 0]), ([-5, 131, 2 ** 31 - 1], [0, 130, 130])):
        t["lengths"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        d["lengths"] = np.array(clamped, dtype=np.int32)
        r = run_fwd(d, t)
        g = mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], c=C, h0=t["h0"], lengths=t["lengths"],
                         d_hfinal=t["d_hfinal"], state_grads=True)
        torch.cuda.synchronize()
        check_forward(d, r, "f32")
        check_backward(d, g, "f32")


def test_empty_sequence():
    d = draw(2, 0, 40, "f32", seed=6)
    t = to_dev(d, "f32")
    r = run_fwd(d, t)
    g = mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], c=C, h0=t["h0"], d_hfinal=t["d_hfinal"], state_grads=True)
    torch.cuda.synchronize()
    assert r["y"].shape == (2, 0, 40) and torch.equal(r["h_final"], t["h0"])
    assert torch.equal(g["dh0"], t["d_hfinal"]) and torch.equal(g["dlam"], torch.zeros(40, device="cuda"))
    r = mesa.lru_fwd(t["x"], t["ga"], t["gi"], t["lam"], return_state=True)
    assert torch.equal(r["h_final"], torch.zeros(2, 40, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 72, 33 * 8])
def test_slices_of_one_projection(dtype, D):
    """x, ga, gi as thirds of one tensor, the gradients as thirds of another: equal to dense tensors, gaps untouched."""
    B, T = 2, 150
    d = draw(B, T, D, dtype, seed=7)
    t = to_dev(d, dtype)
    wide = torch.cat([t["x"], t["ga"], t["gi"], torch.full_like(t["x"], float("nan"))], 2)
    sl = [wide[..., i * D:(i + 1) * D] for i in range(3)]
    kw = dict(c=C, h0=t["h0"])
    a = mesa.lru_fwd(t["x"], t["ga"], t["gi"], t["lam"], return_state=True, **kw)
    b = mesa.lru_fwd(*sl, t["lam"], return_state=True, **kw)
    grads = torch.full_like(wide, 7.0)
    out = {k: grads[..., i * D:(i + 1) * D] for i, k in enumerate(("dx", "dga", "dgi"))}
    ga = mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], d_hfinal=t["d_hfinal"], state_grads=True, **kw)
    gb = mesa.lru_bwd(*sl, t["lam"], t["dy"], d_hfinal=t["d_hfinal"], state_grads=True, out=out, **kw)
    torch.cuda.synchronize()
    for p, q in ((a, b), (ga, gb)):
        for key in p:
            assert torch.equal(p[key], q[key]), key
    assert (grads[..., 3 * D:] == 7.0).all()
    h1, h2 = t["h0"].clone(), t["h0"].clone()
    s1 = mesa.lru_step(t["x"][:, 0].contiguous(), t["ga"][:, 0].contiguous(), t["gi"][:, 0].contiguous(), t["lam"], h1, c=C)
    row = wide[:, 0].contiguous()
    s2 = mesa.lru_step(*[row[:, i * D:(i + 1) * D] for i in range(3)], t["lam"], h2, c=C)
    torch.cuda.synchronize()
    assert torch.equal(h1, h2) and torch.equal(s1["y"], s2["y"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", [(1, 2), (1, 3), (1, 2048), (3, 1001), (5, 4), (2, 5), (70, 6), (3, 7), (2, 9), (300, 15), (65, 4099), (256, 130), (17, 4096)])
def test_step_matches_the_oracle(dtype, N, D):
    d = draw(N, 1, D, dtype, seed=8)
    t = to_dev(d, dtype)
    h = t["h0"].clone()
    r = mesa.lru_step(t["x"][:, 0].contiguous(), t["ga"][:, 0].contiguous(), t["gi"][:, 0].contiguous(), t["lam"], h, c=C)
    torch.cuda.synchronize()
    ref = lru_step(d["x"][:, 0], d["ga"][:, 0], d["gi"][:, 0], d["lam"], d["h0"], c=C)
    q = unit_errors(d)
    bound = q["ea"][:, 0] * q["a"][:, 0] * np.abs(d["h0"]) + q["eu"][:, 0] * np.abs(q["u"][:, 0]) + 2 * E * np.abs(ref)
    within(h, ref, bound, "f32", "h")
    within(r["y"], ref, bound, dtype, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_split_sequence_and_steps_continue_it(dtype):
    """A sequence in one call, in two calls joined by the state, and its last tokens as single steps."""
    B, T, D, cut = 2, 333, 200, 190
    d = draw(B, T, D, dtype, seed=9)
    t = to_dev(d, dtype)
    whole = run_fwd(d, t)
    part = lambda k, a, b: t[k][:, a:b].contiguous()  # noqa: E731
    a = mesa.lru_fwd(part("x", 0, cut), part("ga", 0, cut), part("gi", 0, cut), t["lam"], c=C, h0=t["h0"], return_state=True)
    b = mesa.lru_fwd(part("x", cut, T), part("ga", cut, T), part("gi", cut, T), t["lam"], c=C, h0=a["h_final"],
                     return_state=True, out={"h_final": a["h_final"]})
    torch.cuda.synchronize()
    ref = lru_forward(d["x"], d["ga"], d["gi"], d["lam"], c=C, h0=d["h0"])
    q = unit_errors(d)
    by, _, bh = state_bound(d, q, ref)
    within(torch.cat([a["y"], b["y"]], 1), ref["y"], by, dtype, "split y")
    within(b["h_final"], ref["h_final"], bh, "f32", "split h_final")
    h = mesa.lru_fwd(part("x", 0, T - 5), part("ga", 0, T - 5), part("gi", 0, T - 5), t["lam"], c=C, h0=t["h0"],
                     return_state=True)["h_final"]
    for s in range(T - 5, T):
        r = mesa.lru_step(part("x", s, s + 1)[:, 0], part("ga", s, s + 1)[:, 0], part("gi", s, s + 1)[:, 0], t["lam"], h, c=C)
        torch.cuda.synchronize()
        within(r["y"], ref["y"][:, s], by[:, s], dtype, "step y")
    within(h, ref["h_final"], bh, "f32", "step state")
    within(whole["h_final"], ref["h_final"], bh, "f32", "whole")


def test_repeated_calls_are_bitwise_equal():
    d = draw(2, 3000, 300, "bf16", seed=10, ragged=True)
    t = to_dev(d, "bf16")
    first = None
    for _ in range(4):
        r = run_fwd(d, t)
        r.update(mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], c=C, h0=t["h0"], lengths=t["lengths"],
                              d_hfinal=t["d_hfinal"], state_grads=True))
        torch.cuda.synchronize()
        if first is None:
            first = r
        for key in r:
            assert torch.equal(r[key], first[key]), key


def test_final_state_over_the_initial_one():
    """h_final may be h0 itself, with many tiles reading it and one writing it."""
    d = draw(2, 6000, 256, "bf16", seed=13, ragged=True)
    t = to_dev(d, "bf16")
    want = run_fwd(d, t)
    for _ in range(5):
        state = t["h0"].clone()
        r = mesa.lru_fwd(t["x"], t["ga"], t["gi"], t["lam"], c=C, h0=state, lengths=t["lengths"], return_state=True,
                         out={"h_final": state})
        torch.cuda.synchronize()
        assert r["h_final"] is state
        assert torch.equal(state, want["h_final"]) and torch.equal(r["y"], want["y"])


def test_closed_gates_are_exact():
    """ga = -inf from a zero state: outputs, and the gradients of x, ga, gi and lam, are 0; dh0 is the sum of dy."""
    t = {k: torch.randn(2, 150, 64, generator=torch.Generator().manual_seed(i)).cuda() for i, k in enumerate(("x", "gi", "dy"))}
    ga, lam = torch.full_like(t["x"], -float("inf")), torch.zeros(64, device="cuda")
    r = mesa.lru_fwd(t["x"], ga, t["gi"], lam, return_state=True)
    g = mesa.lru_bwd(t["x"], ga, t["gi"], lam, torch.ones_like(t["dy"]), state_grads=True)
    torch.cuda.synchronize()
    assert not r["y"].any() and not r["h_final"].any()
    for key in ("dx", "dga", "dgi", "dlam"):
        assert not g[key].any(), key
    assert (g["dh0"] == 150).all()


def test_initial_gradient_over_the_final_one():
    """dh0 may be d_hfinal itself, with many tiles reading it and one writing it."""
    d = draw(2, 6000, 129, "bf16", seed=14, ragged=True)
    t = to_dev(d, "bf16")
    kw = dict(c=C, h0=t["h0"], lengths=t["lengths"], state_grads=True)
    last = torch.randn(2, 129, generator=torch.Generator().manual_seed(3)).cuda()
    want = mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], d_hfinal=last, **kw)
    for _ in range(5):
        both = last.clone()
        g = mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], d_hfinal=both, out={"dh0": both}, **kw)
        torch.cuda.synchronize()
        assert g["dh0"] is both
        for key in want:
            assert torch.equal(g[key], want[key]), key


def test_decay_parameters_beyond_every_use():
    """Where softplus(lam) is 0 in fp32 the state stays and no gradient reaches the inputs; where exp(-c softplus(lam)
    sigmoid(ga)) is 0, or far below a half step, every token starts anew, y = sigmoid(gi) x; infinities included,
    nothing is NaN."""
    lam = torch.tensor([-float("inf"), -1e30, -200.0, 200.0, 1e30, float("inf")]).cuda()
    gen = torch.Generator().manual_seed(5)
    x, ga, gi, dy = (torch.randn(2, 300, 6, generator=gen).cuda() for _ in range(4))
    h0 = torch.randn(2, 6, generator=gen).cuda()
    for c in (8.0, 1e38):
        r = mesa.lru_fwd(x, ga, gi, lam, c=c, h0=h0, return_state=True)
        g = mesa.lru_bwd(x, ga, gi, lam, dy, c=c, h0=h0, state_grads=True)
        state = h0.clone()
        y1 = mesa.lru_step(*(v[:, 0].contiguous() for v in (x, ga, gi)), lam, state, c=c)["y"]
        torch.cuda.synchronize()
        for v in (r, g):
            assert all(torch.isfinite(e).all() for e in v.values())
        assert torch.equal(r["y"][..., :3], h0[:, None, :3].expand(-1, 300, -1))
        assert torch.equal(y1[:, :3], h0[:, :3]) and torch.equal(state[:, :3], h0[:, :3])
        assert not any(g[k][..., :3].any() for k in ("dx", "dga", "dgi"))
        si, xd = torch.sigmoid(gi.double()), x.double()
        want = {"y": si * xd, "dx": si * dy.double(), "dgi": dy.double() * xd * si * (1 - si)}
        for k, w in want.items():
            got = (r if k == "y" else g)[k].double()[..., 3:]
            assert ((got - w[..., 3:]).abs() <= 16 * E * w[..., 3:].abs()).all(), k
        assert ((y1.double() - want["y"][:, 0])[:, 3:].abs() <= 16 * E * want["y"][:, 0, 3:].abs()).all()
        # lam = 200 with c = 8: over these gates (above -4.6, so sigmoid(ga) > 0.01) -log a > 16, a < 1.2e-7 and
        # -log(a) a < 1.9e-6, which bounds dga / (|g| (|h| + |x|)) with factors below 5 each; elsewhere a is 0
        assert ga.min() > -4.6 and (g["dga"][..., 3].abs() < 1e-4).all() and (g["dh0"][:, 3].abs() < 1e-6).all()
        assert not g["dga"][..., 4:].any() and not g["dh0"][:, 4:].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_wherever_rows_start_in_a_cache_line(dtype):
    """Tensors 16 bytes behind a cache line, and rows of a wider tensor, against aligned ones."""
    d = draw(3, 700, 192, dtype, seed=15, ragged=True)
    t = to_dev(d, dtype)
    want = run_fwd(d, t)
    kw = dict(c=C, h0=t["h0"], lengths=t["lengths"])
    grads = mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], **kw)
    step = 16 // t["x"].element_size()
    shape, n = t["x"].shape, t["x"].numel()

    def behind(v):
        buf = torch.empty(n + step, dtype=v.dtype, device="cuda")[step:].view(shape)
        return buf.copy_(v)

    def wider(v):
        return torch.cat([v, v[..., :step]], -1)[..., :192]

    for move in (behind, wider):
        x, ga, gi = (move(t[k]) for k in ("x", "ga", "gi"))
        r = mesa.lru_fwd(x, ga, gi, t["lam"], return_state=True, **kw)
        g = mesa.lru_bwd(x, ga, gi, t["lam"], t["dy"], **kw)
        torch.cuda.synchronize()
        assert torch.equal(r["y"], want["y"]) and torch.equal(r["h_final"], want["h_final"])
        for k in grads:
            assert torch.equal(g[k], grads[k]), (move.__name__, k)


def test_causality():
    """Inputs behind token t change nothing up to it, bit for bit."""
    d = draw(1, 700, 96, "f32", seed=11)
    t = to_dev(d, "f32")
    a = run_fwd(d, t)
    for k in ("x", "ga", "gi"):
        t[k][:, 401:] = 3.0
    b = run_fwd(d, t)
    torch.cuda.synchronize()
    assert torch.equal(a["y"][:, :401], b["y"][:, :401]) and not torch.equal(a["y"][:, 401], b["y"][:, 401])


def test_gradients_match_differences():
    """Central differences of the GPU forward (fp32) along random directions.  The step
    d = 2^-7 leaves a truncation of order d^2 and a rounding of order 2^-24 |L| / d; with
    L a sum of some 2e4 terms of order 1 the latter is below 1e-3 of the gradient's length."""
    B, T, D = 2, 90, 64
    d = draw(B, T, D, "f32", seed=12, lam=(-5.0, -2.0))
    t = to_dev(d, "f32")
    g = mesa.lru_bwd(t["x"], t["ga"], t["gi"], t["lam"], t["dy"], c=C, h0=t["h0"], d_hfinal=t["d_hfinal"], state_grads=True)

    def loss(**kw):
        u = dict(t, **kw)
        r = mesa.lru_fwd(u["x"], u["ga"], u["gi"], u["lam"], c=C, h0=u["h0"], return_state=True)
        return float((r["y"].double() * t["dy"].double()).sum() + (r["h_final"].double() * t["d_hfinal"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(1)
    step = 2.0 ** -7
    for key, gk in (("x", "dx"), ("ga", "dga"), ("gi", "dgi"), ("lam", "dlam"), ("h0", "dh0")):
        e = torch.randn(t[key].shape, generator=gen, device="cuda")
        num = (loss(**{key: t[key] + step * e}) - loss(**{key: t[key] - step * e})) / (2 * step)
        ana = float((g[gk].double() * e.double()).sum())
        size = float(g[gk].double().norm())
        assert abs(num - ana) <= 5e-3 * size + 1e-3, (key, num, ana, size)
