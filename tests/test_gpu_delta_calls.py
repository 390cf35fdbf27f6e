"""How the gated delta rule and clipping are called: on several streams at once, captured and replayed,
with shared workspaces, from slices and broadcast inputs, together as a block's training step, and
refused calls.  Needs an MI355X.
"""
import math

import numpy as np
import pytest
import torch

from delta_helpers import check_backward, check_forward, draw, to_dev
from oracle import block_oracle
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


BF16, F32 = torch.bfloat16, torch.float32
INPUTS = ("q", "k", "v", "gamma", "beta")


def inputs(seed, B, H, Hk, T, dk, dv, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dtype)  # noqa: E731
    return dict(q=unit(normal(B, Hk, T, dk)), k=unit(normal(B, Hk, T, dk)), v=normal(B, H, T, dv).to(dtype),
                gamma=torch.sigmoid(4 + normal(B, H, T)), beta=torch.sigmoid(normal(B, H, T)),
                d_o=normal(B, H, T, dv).to(dtype), s0=normal(B, H, dv, dk) / 8, d_sfinal=normal(B, H, dv, dk))


def workspace(a, fill=None):
    ws = torch.empty(mesa.delta_workspace_bytes(*(a[n] for n in INPUTS), keep_states=True), device="cuda", dtype=torch.uint8)
    return ws if fill is None else ws.fill_(fill)


def train(a, ws=None, stream=None, out=None):
    args = [a[n] for n in INPUTS]
    r = mesa.delta_fwd(*args, s0=a["s0"], return_state=True, keep_states=ws is not None, workspace=ws, stream=stream, out=out)
    r.update(mesa.delta_bwd(*args, a["d_o"], s0=a["s0"], d_sfinal=a["d_sfinal"], state_grads=True, workspace=ws,
                            states_in_workspace=ws is not None, stream=stream, out=out))
    return r


def equal(p, q, what=""):
    for key in p:
        assert torch.equal(p[key].reshape(-1).view(torch.uint8), q[key].reshape(-1).view(torch.uint8)), (what, key)


def test_calls_on_streams_at_once_match_calls_alone():
    cases = [inputs(1, 2, 4, 4, 700, 128, 128), inputs(2, 1, 2, 1, 1500, 64, 96, F32), inputs(3, 1, 2, 2, 1100, 32, 48)]
    grads = [torch.randn(n, device="cuda") for n in (300000, 7, 65537)]
    alone = [train(a) for a in cases]
    clipped = mesa.grad_clip(grads, 1.0, out=[torch.empty_like(g) for g in grads])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for rep in range(4):
        rs = [train(a, None, s) for a, s in zip(cases, streams)]
        with torch.cuda.stream(streams[3]):
            outs = [torch.empty_like(g) for g in grads]
        c = mesa.grad_clip(grads, 1.0, out=outs, stream=streams[3])
        torch.cuda.synchronize()
        for r, want in zip(rs, alone):
            equal(want, r, rep)
        assert torch.equal(c["norm"], clipped["norm"]) and all(map(torch.equal, c["grads"], clipped["grads"]))


def test_results_allocated_for_a_side_stream_are_not_reused_early():
    a = inputs(5, 2, 8, 8, 2000, 128, 128)
    want = mesa.delta_fwd(*(a[n] for n in INPUTS))["o"]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        mesa.delta_fwd(*(a[n] for n in INPUTS), stream=s)  # dropped while it runs
        mine = torch.zeros_like(want)
        torch.cuda.synchronize()
        assert not mine.any()
    r = mesa.delta_fwd(*(a[n] for n in INPUTS), stream=s)
    torch.cuda.synchronize()
    assert torch.equal(r["o"], want)


@pytest.mark.parametrize("which", ["train", "segments", "shared f32", "step", "clip"])
def test_replays_in_a_graph(which):
    """Captured once, replayed with new inputs and eager work of the same operators between the replays."""
    if which in ("train", "segments", "shared f32"):
        sizes = {"train": (2, 4, 4, 300, 128, 128), "segments": (1, 1, 1, 1400, 64, 64), "shared f32": (2, 4, 2, 150, 32, 80, F32)}
        make = lambda s: inputs(s, *sizes[which])  # noqa: E731
        ws, other = workspace(make(0)), workspace(make(0))
        call = lambda a, stream=None, out=None: train(a, ws if out else other, stream, out)  # noqa: E731
    elif which == "step":
        make = lambda s: {n: v[:, :, 0].contiguous() if n in INPUTS else v for n, v in inputs(s, 9, 4, 2, 1, 64, 96).items()}  # noqa: E731

        def call(a, stream=None, out=None):
            state = out["state"] if out else a["s0"].clone()
            if out:
                state.copy_(a["s0"])
            r = mesa.delta_step(*(a[n] for n in INPUTS), state, stream=stream, out=out)
            return dict(r, state=state)
    else:
        def make(s):
            g = torch.Generator(device="cuda").manual_seed(s)
            return {str(n): torch.randn(n, generator=g, device="cuda").to(BF16 if n % 2 else F32) for n in (100, 7, 50001, 1 << 18)}
        cws = torch.empty(mesa.lib().mesa_grad_clip_workspace_bytes(), device="cuda", dtype=torch.uint8)

        def call(a, stream=None, out=None):
            outs = [out[n] if out else torch.empty_like(v) for n, v in a.items()]
            r = mesa.grad_clip(list(a.values()), 3.0, out=outs, workspace=cws if out else None, stream=stream)
            if out:
                out["norm"].copy_(r["norm"])
            return dict(zip(a, outs), norm=r["norm"])

    srcs = [make(11), make(12)]
    refs = [call(a) for a in srcs]
    cap = {k: v.clone() for k, v in srcs[0].items()}
    out = {k: v.clone() for k, v in refs[0].items()}
    call(cap, None, out)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        call(cap, s, out)
    torch.cuda.synchronize()
    for rep, i in enumerate([0, 0, 1, 0, 1, 1]):
        for k in cap:
            cap[k].copy_(srcs[i][k])
        for v in out.values():
            v.view(-1).view(torch.uint8).fill_(0xAB)
        eager = call(srcs[1 - i])
        graph.replay()
        torch.cuda.synchronize()
        equal(refs[i], out, rep)
        equal(refs[1 - i], eager, rep)


def test_two_graphs_share_a_workspace():
    """Forward and backward captured apart, with one workspace that other sizes use in between;
    the backward is replayed twice on the states of one forward."""
    a, b = inputs(21, 1, 2, 2, 1200, 64, 64), inputs(22, 3, 4, 2, 200, 128, 48)
    ws = max(workspace(a), workspace(b), key=lambda t: t.numel())
    want = [{k: v.clone() for k, v in train(x, ws).items()} for x in (a, b)]
    torch.cuda.synchronize()
    graphs = []
    for x in (a, b):
        args, out = [x[n] for n in INPUTS], {}
        f, w, s = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(f, stream=s):
            out.update(mesa.delta_fwd(*args, s0=x["s0"], return_state=True, keep_states=True, workspace=ws, stream=s))
        with torch.cuda.graph(w, stream=s):
            out.update(mesa.delta_bwd(*args, x["d_o"], s0=x["s0"], d_sfinal=x["d_sfinal"], state_grads=True, workspace=ws,
                                      states_in_workspace=True, stream=s))
        graphs.append((f, w, out))
    for rep in range(3):
        for (f, w, out), ref in zip(graphs, want):
            f.replay()
            w.replay()
            for key in ("dq", "dk", "dv", "dgamma", "dbeta", "ds0"):
                out[key].fill_(float("nan"))
            w.replay()
            torch.cuda.synchronize()
            equal(ref, out, rep)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_any_workspace_and_equal_inputs_give_bitwise_equal_results(dtype):
    a = inputs(31, 2, 4, 2, 333, 64, 80, dtype)
    want = train(a)
    for fill in (0x00, 0xFF, 0x7F):
        equal(want, train(a, workspace(a, fill)), fill)
    for _ in range(3):
        equal(want, train(a))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_broadcast_inputs_and_outputs_in_one_wider_tensor(dtype):
    """One gate for all heads, one sequence for all of a batch: strides of 0 are read as they are.  Outputs are
    slices of one tensor, whose other elements stay as they were."""
    B, H, T, d = 3, 4, 140, 64
    a = inputs(41, B, H, H, T, d, d, dtype)
    for n in ("gamma", "beta"):
        a[n] = a[n][:, :1].expand(B, H, T)
    for n in ("q", "v", "d_o"):
        a[n] = a[n][:1].expand(B, H, T, d)
    dense = {n: t.contiguous() for n, t in a.items()}
    want = train(dense)
    equal(want, train(a))
    wide = torch.full((B, T, 3 * H * d + 32), 7.0, device="cuda", dtype=dtype)
    flat = torch.full((B, T, 3, H), 7.0, device="cuda")
    part = lambda i: wide[..., 16 + i * H * d:16 + (i + 1) * H * d].view(B, T, H, d).transpose(1, 2)  # noqa: E731
    out = {n: part(i) for i, n in enumerate(("dq", "dk", "dv"))}
    out.update(dgamma=flat[:, :, 0].transpose(1, 2), dbeta=flat[:, :, 2].transpose(1, 2))
    wide_o = torch.full((B, T, 2, H, d), 7.0, device="cuda", dtype=dtype)
    out["o"] = wide_o[:, :, 1].transpose(1, 2)
    equal(want, train(a, out=out))
    assert bool((wide[..., :16] == 7).all()) and bool((wide[..., -16:] == 7).all())
    assert bool((flat[:, :, 1] == 7).all()) and bool((wide_o[:, :, 0] == 7).all())


def test_states_in_place():
    """s_final over s0, ds0 over d_sfinal."""
    a = inputs(51, 2, 2, 1, 1100, 64, 48)
    want = train(a)
    b = {n: t.clone() for n, t in a.items()}
    args = [b[n] for n in INPUTS]
    g = mesa.delta_bwd(*args, b["d_o"], s0=b["s0"], d_sfinal=b["d_sfinal"], state_grads=True, out={"ds0": b["d_sfinal"]})
    f = mesa.delta_fwd(*args, s0=b["s0"], return_state=True, out={"s_final": b["s0"]})
    equal({**f, **g}, want)
    assert f["s_final"] is b["s0"] and g["ds0"] is b["d_sfinal"]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_what_is_not_finite_stays_in_its_head(dtype):
    a = inputs(61, 2, 4, 4, 300, 64, 64, dtype)
    want = train(a)
    for n, at, value in (("k", (0, 1, 100, 3), math.nan), ("v", (0, 1, 70, 5), math.inf), ("beta", (0, 1, 250), math.nan),
                         ("d_o", (0, 1, 299, 0), math.nan), ("gamma", (0, 1, 0), math.nan)):
        b = {m: t.clone() for m, t in a.items()}
        b[n][at] = value
        r = train(b)
        for key in want:
            x, y = r[key].clone(), want[key].clone()
            x[0, 1], y[0, 1] = 0, 0
            assert torch.equal(x, y), (n, key)
        if n in ("k", "v", "beta"):  # and before its 64 tokens nothing forward has changed
            first = at[2] // 64 * 64
            assert torch.equal(r["o"][0, 1, :first], want["o"][0, 1, :first]), n


def test_one_token_whose_unused_stride_is_anything():
    a = inputs(71, 2, 3, 3, 1, 64, 64)
    want = train(a)
    odd = dict(a)
    for n in ("q", "k", "v", "d_o"):
        x = a[n]
        odd[n] = x.as_strided(x.shape, (x.stride(0), x.stride(1), (1 << 33) + 5, 1))
    equal(want, train(odd))
    step = mesa.delta_step(*(odd[n][:, :, 0] for n in INPUTS), a["s0"].clone())
    assert step["o"].shape == (2, 3, 64)


def test_run_together_as_a_training_step():
    """Preprocessing -> gated delta rule -> norm, back again through all three, and the clipping of every gradient:
    each stage against its oracle on the GPU's own inputs of that stage, the whole chain against differences, and
    the decode step behind it."""
    g = torch.Generator(device="cuda").manual_seed(81)
    B, H, Hk, T, d, dv, W = 2, 4, 2, 130, 64, 48, 4

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    x = dict(q=normal(B, Hk, T, d), k=normal(B, Hk, T, d), wq=normal(Hk, d, W) / 2, wk=normal(Hk, d, W) / 2,
             v=normal(B, H, T, dv), gamma=0.9 + 0.08 * torch.rand((B, H, T), generator=g, device="cuda"),
             beta=0.2 + 0.6 * torch.rand((B, H, T), generator=g, device="cuda"), w=1 + 0.1 * normal(dv))
    dy = normal(B * H * T, dv)

    def forward(x, **kw):
        pre = mesa.qk_preprocess(x["q"], x["k"], x["wq"], x["wk"])
        f = mesa.delta_fwd(pre["q"], pre["k"], x["v"], x["gamma"], x["beta"], return_state=True, **kw)
        return pre, f, mesa.rmsnorm(f["o"].view(-1, dv), x["w"])["y"]

    shapes = mesa.qk_preprocess(x["q"], x["k"], x["wq"], x["wk"])
    assert shapes["q"].dtype is F32
    ws = torch.empty(mesa.delta_workspace_bytes(shapes["q"], shapes["k"], x["v"], x["gamma"], x["beta"], keep_states=True),
                     device="cuda", dtype=torch.uint8)
    pre, f, y = forward(x, keep_states=True, workspace=ws)
    n = mesa.rmsnorm_bwd(f["o"].view(-1, dv), x["w"], dy)
    d_o = n["ds"].view(B, H, T, dv)
    args = (pre["q"], pre["k"], x["v"], x["gamma"], x["beta"])
    r = mesa.delta_bwd(*args, d_o, workspace=ws, states_in_workspace=True)
    p = mesa.qk_preprocess_bwd(x["q"], x["k"], x["wq"], x["wk"], r["dq"], r["dk"])
    grads = dict(q=p["dq_raw"], k=p["dk_raw"], wq=p["dw_q"], wk=p["dw_k"], v=r["dv"], gamma=r["dgamma"], beta=r["dbeta"], w=n["dw"])

    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    a = dict(zip(INPUTS, map(host, args)), d_o=host(d_o), s0=None, d_sfinal=None, lengths=None)
    check_forward(f, a, F32)
    check_backward(r, a, F32)
    for m, key in (("q", "dq"), ("k", "dk")):
        ref = block_oracle.qk_preprocess_backward(host(x[m]), host(x["w" + m]), host(r[key]))
        assert np.linalg.norm(host(grads[m]) - ref["dx"]) <= 2e-5 * np.linalg.norm(ref["dx"])

    loss = lambda x: float((forward(x)[2].double() * dy.double()).sum())  # noqa: E731
    step = 2.0 ** -7
    for m in x:
        size = 0.1 if m in ("gamma", "beta") else 1.0   # (gates stay between 0 and 1)
        e = normal(*x[m].shape).clamp(-2, 2) * size
        num = (loss({**x, m: x[m] + step * e}) - loss({**x, m: x[m] - step * e})) / (2 * step)
        ana = float((grads[m].double() * e.double()).sum())
        # truncation step^2 = 2^-14 of a third derivative; y's errors of 2^-22 over sqrt(numbers) and the step
        bound = 5e-3 * size * float(grads[m].double().norm()) + 2.0 ** -15 * math.sqrt(dy.numel())
        assert abs(num - ana) <= bound, (m, num, ana, bound)

    every = list(grads.values())
    kept = [t.double().clone() for t in every]
    norm = math.sqrt(sum(float(t.square().sum()) for t in kept))
    c = mesa.grad_clip(every, 1.0)
    assert abs(float(c["norm"]) - norm) <= 2.0 ** -23 * norm
    for t, k in zip(every, kept):
        assert bool(((t.double() - k / (norm + 1e-6)).abs() <= 2.0 ** -21 * k.abs() / norm).all())

    longer = {m: torch.cat([x[m], x[m][:, :, :1]], 2) if m in ("q", "k", "v", "gamma", "beta") else x[m] for m in x}
    whole = forward(longer)
    now = [t[:, :, -1] for t in (whole[0]["q"], whole[0]["k"], longer["v"], longer["gamma"], longer["beta"])]
    state = f["s_final"].clone()
    o = mesa.delta_step(*now, state)["o"]
    assert float((o - whole[1]["o"][:, :, -1]).norm()) <= 1e-5 * float(o.norm())
    assert float((state - whole[1]["s_final"]).norm()) <= 1e-5 * float(state.norm())


def test_binding_refuses_what_the_kernels_cannot_take():
    a = inputs(91, 2, 4, 2, 20, 64, 48)
    args = [a[n] for n in INPUTS]

    def bad(fn, *p, **kw):
        with pytest.raises(mesa.MesaError):
            fn(*p, **kw)

    def swap(i, t):
        return args[:i] + [t] + args[i + 1:]

    for fn in (mesa.delta_fwd, lambda *p, **kw: mesa.delta_bwd(*p, a["d_o"], **kw)):
        bad(fn, *swap(0, a["q"].cpu()))
        bad(fn, *[t.half() if t.dtype is BF16 else t for t in args])
        bad(fn, *swap(2, a["v"].float()))
        bad(fn, *swap(1, a["k"][:, :, :10]))
        bad(fn, *swap(2, a["v"][0]))
        bad(fn, *swap(2, a["v"][:, :3]))                                   # 3 heads on 2 of keys
        bad(fn, *swap(0, a["q"].transpose(2, 3).contiguous().transpose(2, 3)))
        bad(fn, *swap(3, a["gamma"].bfloat16()))
        bad(fn, *swap(4, a["beta"][:, :1]))
        bad(fn, *swap(2, torch.cat([a["v"], a["v"]], 3)[..., 4:52]))       # rows at 8 bytes
        bad(fn, *swap(2, a["v"][..., :40]))
        bad(fn, *[t[..., :48] if i < 2 else t for i, t in enumerate(args)])
        bad(fn, *args, s0=a["s0"].double())
        bad(fn, *args, s0=a["s0"][:1])
        bad(fn, *args, lengths=torch.ones(2, device="cuda", dtype=torch.int64))
        bad(fn, *args, workspace=torch.empty(64, device="cuda", dtype=torch.uint8))
        bad(fn, *args, workspace=torch.empty(1 << 24, dtype=torch.uint8))
    bad(mesa.delta_fwd, *args, keep_states=True)
    bad(mesa.delta_fwd, *args, out={"o": torch.empty(2, 4, 20, 48, device="cuda")})
    bad(mesa.delta_fwd, *args, out={"o": a["v"]})
    bad(mesa.delta_fwd, *args, out={"o": torch.empty(1, 4, 20, 48, device="cuda", dtype=BF16).expand(2, 4, 20, 48)})
    bad(mesa.delta_bwd, *args, a["d_o"], states_in_workspace=True)
    bad(mesa.delta_bwd, *args, a["d_o"].float())
    bad(mesa.delta_bwd, *args, a["d_o"], d_sfinal=a["s0"].bfloat16())
    bad(mesa.delta_bwd, *args, a["d_o"], out={"dq": a["q"]})
    bad(mesa.delta_bwd, *args, a["d_o"], out={"dv": a["d_o"]})
    one = [t[:, :, 0] for t in args]
    bad(mesa.delta_step, *args, a["s0"])
    bad(mesa.delta_step, *one, a["s0"].double())
    bad(mesa.delta_step, *one, a["s0"][..., :32])
    bad(mesa.delta_step, one[0], one[1][:, :1], *one[2:], a["s0"])
    bad(mesa.delta_step, *one, a["s0"], out={"o": torch.empty(2, 4, 96, device="cuda", dtype=BF16)[..., ::2]})
