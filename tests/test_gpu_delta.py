"""Gated delta rule on the GPU against the fp64 oracle, forward, backward and step (bounds:
delta_helpers).  Needs an MI355X."""
import numpy as np
import pytest
import torch

from delta_helpers import check_backward, check_forward, close, draw, e32, to_dev
from oracle.delta_oracle import delta_forward
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def args(t):
    return t["q"], t["k"], t["v"], t["gamma"], t["beta"]


def forward(t, **kw):
    return mesa.delta_fwd(*args(t), s0=t["s0"], lengths=t["lengths"], return_state=True, **kw)


def backward(t, **kw):
    return mesa.delta_bwd(*args(t), t["d_o"], s0=t["s0"], lengths=t["lengths"], d_sfinal=t["d_sfinal"],
                          state_grads=True, **kw)


# one token, ends of a tile, of an inner step and of a chunk, and behind them; several chunks
LENGTHS = [1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 65, 128, 130, 200]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(T, dtype):
    dt = DTYPES[dtype]
    a = draw(2, 2, 2, T, 64, 64, dt, seed=T, s0=T % 2 == 1)
    t = to_dev(a, dt)
    check_forward(forward(t), a, dt)
    check_backward(backward(t), a, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(32, 16), (32, 32), (32, 80), (64, 16), (64, 96), (64, 256), (128, 128), (128, 48), (128, 208)])
def test_sizes(dk, dv, dtype):
    dt = DTYPES[dtype]
    a = draw(1, 3, 3, 100, dk, dv, dt, seed=dk + dv)
    t = to_dev(a, dt)
    check_forward(forward(t), a, dt)
    check_backward(backward(t), a, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["heads", "tokens", "slices"])
@pytest.mark.parametrize("H,Hk", [(4, 4), (4, 2), (6, 2), (5, 1)])
def test_layouts_and_shared_heads(H, Hk, layout, dtype):
    dt = DTYPES[dtype]
    a = draw(2, H, Hk, 90, 64, 48, dt, seed=H, lengths=[70, 90])
    t = to_dev(a, dt, layout)
    r = forward(t)
    assert layout == "slices" or r["o"].stride() == t["v"].stride()
    check_forward(r, a, dt)
    check_backward(backward(t), a, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gates", ["slow", "fast"])
def test_gates_and_lengths_over_several_chunks(gates, dtype):
    dt = DTYPES[dtype]
    a = draw(5, 2, 1, 300, 128, 64, dt, gates=gates, lengths=[300, 0, 1, 64, 257])
    t = to_dev(a, dt)
    check_forward(forward(t), a, dt)
    check_backward(backward(t), a, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_states_that_the_forward_leaves(dtype):
    dt = DTYPES[dtype]
    a = draw(2, 4, 2, 150, 64, 80, dt, lengths=[150, 99])
    t = to_dev(a, dt)
    ws = torch.empty(mesa.delta_workspace_bytes(*args(t), keep_states=True), device="cuda", dtype=torch.uint8)
    r = forward(t, workspace=ws, keep_states=True)
    check_forward(r, a, dt)
    plain = forward(t)
    assert all(torch.equal(r[n], plain[n]) for n in r)
    g = backward(t, workspace=ws, states_in_workspace=True)
    check_backward(g, a, dt)
    again = backward(t)
    assert all(torch.equal(g[n], again[n]) for n in g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_sequence_in_parts(dtype):
    """Two calls and single tokens, each on the last one's state, against one call's definition."""
    dt = DTYPES[dtype]
    a = draw(2, 4, 2, 140, 128, 64, dt)
    t = to_dev(a, dt)
    want = delta_forward(*(a[n] for n in ("q", "k", "v", "gamma", "beta")), s0=a["s0"])
    e = e32(a, 24)
    outs, state = [], t["s0"].clone()
    for lo, hi in ((0, 77), (77, 135)):
        r = mesa.delta_fwd(*(t[n][:, :, lo:hi] for n in ("q", "k", "v", "gamma", "beta")), s0=state, return_state=True,
                           out={"s_final": state})
        outs.append(r["o"])
    for i in range(135, 140):
        outs.append(mesa.delta_step(*(t[n][:, :, i] for n in ("q", "k", "v", "gamma", "beta")), state)["o"][:, :, None])
    close(torch.cat(outs, 2), want["o"], e, dt, "o")
    close(state, want["s_final"], e, torch.float32, "s_final")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,Hk,dk,dv", [(1, 1, 1, 128, 128), (3, 4, 2, 64, 128), (5, 3, 3, 32, 16), (2, 2, 1, 128, 208),
                                          (2, 6, 2, 32, 240), (7, 2, 2, 64, 1024)])
def test_step(N, H, Hk, dk, dv, dtype):
    dt = DTYPES[dtype]
    a = draw(N, H, Hk, 1, dk, dv, dt)
    t = to_dev(a, dt)
    want = delta_forward(*(a[n] for n in ("q", "k", "v", "gamma", "beta")), s0=a["s0"])
    for wide in (False, True):
        x = {n: t[n][:, :, 0] for n in ("q", "k", "v", "gamma", "beta")}
        if wide:  # slices of wider rows
            x = {n: torch.cat([v, v, v], 1)[:, v.shape[1]:2 * v.shape[1]] for n, v in x.items()}
        s = t["s0"].clone()
        r = mesa.delta_step(*x.values(), s)
        # two dots of dk products in fp32, added in pairs of lanes: 2^-24 (8 + log2) of the sum of their sizes
        e = 16 * 2.0 ** -24 * np.sqrt(dk)
        close(r["o"][:, :, None], want["o"], e, dt, "o")
        close(s, want["s_final"], e, torch.float32, "state")


def test_repeated_and_opposite_keys():
    """Equal keys, beta = 1 and no forgetting: each value replaces the last one; the inverse is bidiagonal
    where a series in its powers would reach 10^18."""
    B, H, T, d = 1, 1, 128, 64
    a = draw(B, H, H, T, d, d, torch.float32, s0=False)
    a["k"][:] = a["k"][:, :, :1]
    a["k"][:, :, 1::2] *= -1.0
    a["q"][:] = a["k"][:, :, :1]
    a["gamma"][:], a["beta"][:] = 1.0, 1.0
    t = to_dev(a, torch.float32)
    r = forward(t)
    # |k|^2 of fp32 unit vectors is 1 to 2^-23 or so, and an output is one product with it
    sign = np.where(np.arange(T) % 2, -1.0, 1.0)[None, None, :, None]
    got = r["o"].double().cpu().numpy()
    assert np.abs(got - sign * a["v"]).max() <= 64 * 2.0 ** -23 * np.abs(a["v"]).max()
    check_backward(mesa.delta_bwd(*args(t), t["d_o"]), a, torch.float32)


def test_no_tokens():
    a = draw(2, 2, 1, 0, 64, 48, torch.float32)
    t = to_dev(a, torch.float32)
    r = forward(t)
    assert r["o"].shape == (2, 2, 0, 48) and torch.equal(r["s_final"], t["s0"])
    g = backward(t)
    assert torch.equal(g["ds0"], t["d_sfinal"])
    r = mesa.delta_fwd(*args(t), return_state=True)
    assert not r["s_final"].any()


def test_zero_gates():
    """beta = 0 writes nothing and has a gradient; gamma = 0 forgets everything."""
    a = draw(2, 2, 2, 100, 64, 64, torch.float32)
    a["beta"][:, :, ::3] = 0.0
    a["gamma"][:, :, 50] = 0.0
    t = to_dev(a, torch.float32)
    check_forward(forward(t), a, torch.float32)
    a["gamma"][:, :, 50] = 0.5
    t = to_dev(a, torch.float32)
    check_backward(backward(t), a, torch.float32)


def test_backward_of_a_gate_that_forgets_everything():
    """gamma = 0: the gradient at log gamma is 0 there, and so dgamma is written; all others are as defined."""
    a = draw(2, 2, 2, 150, 64, 64, torch.float32, seed=3)
    a["gamma"][:, :, [0, 50, 64, 149]] = 0.0
    t = to_dev(a, torch.float32)
    r = backward(t)
    assert not r["dgamma"][:, :, [0, 50, 64, 149]].any()
    check_backward(r, a, torch.float32)


def segmented(t):
    """Whether walks of these inputs go in segments: they have maps then, which as many heads as fill the card have not."""
    big = {n: t[n][:1].expand(512, *t[n].shape[1:]) for n in ("q", "k", "v", "gamma", "beta")}
    return mesa.delta_workspace_bytes(*args(t)) * 512 > t["q"].shape[0] * (mesa.delta_workspace_bytes(*args(big)) + 512 * 8192)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,T,dk,dv", [(1, 1, 1024, 64, 64), (2, 1, 1601, 128, 48), (1, 1, 2100, 32, 80), (3, 3, 1500, 128, 128)])
def test_segments(H, Hk, T, dk, dv, dtype):
    """Few heads and many chunks: lengths that end in each segment, at its ends, before the first and behind the last."""
    dt = DTYPES[dtype]
    a = draw(4, H, Hk, T, dk, dv, dt, gates="slow", lengths=[T + 5, 0, 513, T // 2])
    t = to_dev(a, dt, "tokens")
    assert segmented(t)
    ws = torch.empty(mesa.delta_workspace_bytes(*args(t), keep_states=True), device="cuda", dtype=torch.uint8)
    ws.fill_(0xFF)
    r = forward(t, workspace=ws, keep_states=True)
    check_forward(r, a, dt, walks=2)
    g = backward(t, workspace=ws, states_in_workspace=True)
    check_backward(g, a, dt, walks=2)
    again = backward(t, workspace=ws, states_in_workspace=True)
    alone = backward(t)
    assert all(torch.equal(g[n], again[n]) and torch.equal(g[n], alone[n]) for n in g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_segments_without_states(dtype):
    dt = DTYPES[dtype]
    a = draw(1, 2, 2, 1300, 64, 64, dt, gates="slow", s0=False)
    t = to_dev(a, dt)
    assert segmented(t)
    check_forward(mesa.delta_fwd(*args(t)), a, dt, walks=2)
    check_backward(mesa.delta_bwd(*args(t), t["d_o"]), a, dt, walks=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_segments_in_place(dtype):
    """s_final over s0 and ds0 over d_sfinal where most segments have no chunk and so end at once, beside
    the one that starts from what they overwrite."""
    dt = DTYPES[dtype]
    B = 32
    a = draw(B, 1, 1, 1100, 64, 64, dt, gates="slow", lengths=[1 + 7 * b for b in range(B)])
    t = to_dev(a, dt)
    assert segmented(t)
    s, ds = t["s0"].clone(), t["d_sfinal"].clone()
    r = mesa.delta_fwd(*args(t), s0=s, lengths=t["lengths"], return_state=True, out={"s_final": s})
    check_forward(r, a, dt, walks=2)
    g = mesa.delta_bwd(*args(t), t["d_o"], s0=t["s0"], lengths=t["lengths"], d_sfinal=ds, state_grads=True, out={"ds0": ds})
    check_backward(g, a, dt, walks=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_strengths_up_to_two(dtype):
    """1 - beta between -1 and 1 does not lengthen a state either; no forgetting."""
    dt = DTYPES[dtype]
    a = draw(2, 2, 2, 200, 64, 64, dt, beta=(0.0, 2.0))
    a["gamma"][:] = 1.0
    t = to_dev(a, dt)
    check_forward(forward(t), a, dt)
    check_backward(backward(t), a, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [150, 1300])
def test_powers_of_two_pass_through(T, dtype):
    """The rule is linear in (v, s0), its gradients in (d_o, d_sfinal): powers of two change exponents alone."""
    dt = DTYPES[dtype]
    t = to_dev(draw(2, 2, 1, T, 64, 48, dt, gates="slow"), dt)
    k, m = 2.0 ** 30, 2.0 ** -25
    u = dict(t, v=t["v"] * k, s0=t["s0"] * k, d_o=t["d_o"] * m, d_sfinal=t["d_sfinal"] * m)
    f, f2, g, g2 = forward(t), forward(u), backward(t), backward(u)
    for n in f:
        assert torch.equal(f[n] * k, f2[n]), n
    for n, by in (("dq", k * m), ("dk", k * m), ("dv", m), ("dgamma", k * m), ("dbeta", k * m), ("ds0", m)):
        assert torch.equal(g[n] * by, g2[n]), n
