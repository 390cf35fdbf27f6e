"""How the operators around the layer are called: on several streams at once, captured
and replayed, with shared workspaces, together as a block, and refused calls.
Needs an MI355X.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle, mesa_backward
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def lru_inputs(seed, B, T, D, dtype=torch.bfloat16):
    g = gen(seed)
    return dict(x=normal(g, B, T, D, dtype=dtype), ga=normal(g, B, T, D, dtype=dtype), gi=normal(g, B, T, D, dtype=dtype),
                lam=-6 + 3 * torch.rand(D, generator=g, device="cuda"), dy=normal(g, B, T, D, dtype=dtype),
                h0=normal(g, B, D, dtype=torch.float32))


def train(a, ws, stream=None, out=None):
    args = (a["x"], a["ga"], a["gi"], a["lam"])
    r = mesa.lru_fwd(*args, h0=a["h0"], return_state=True, workspace=ws, stream=stream, out=out)
    r.update(mesa.lru_bwd(*args, a["dy"], h0=a["h0"], state_grads=True, workspace=ws, states_in_workspace=True,
                          stream=stream, out=out))
    return r


def norm_train(a, stream=None, out=None, ws=None):
    r = mesa.rmsnorm(a["x"], a["w"], residual=a["res"], quant_group=128, stream=stream, out=out)
    r.update(mesa.rmsnorm_bwd(r["residual"], a["w"], a["dy"], d_residual=a["res"], stream=stream, out=out, workspace=ws))
    return r


def norm_inputs(seed, R, D):
    g = gen(seed)
    return dict(x=normal(g, R, D), res=normal(g, R, D), dy=normal(g, R, D), w=1 + 0.1 * normal(g, D, dtype=torch.float32))


def prep_inputs(seed, B, H, T, d, W):
    g = gen(seed)
    return dict(q=normal(g, B, H, T, d), k=normal(g, B, H, T, d), wq=normal(g, H, d, W, dtype=torch.float32),
                wk=normal(g, H, d, W, dtype=torch.float32), dq=normal(g, B, H, T, d, dtype=torch.float32),
                dk=normal(g, B, H, T, d, dtype=torch.float32))


def prep_bwd(a, stream=None, out=None, ws=None):
    return mesa.qk_preprocess_bwd(a["q"], a["k"], a["wq"], a["wk"], a["dq"], a["dk"], stream=stream, out=out, workspace=ws)


def equal(p, q, what=""):
    for key in p:
        assert torch.equal(p[key].view(torch.uint8), q[key].view(torch.uint8)), (what, key)


def test_calls_on_streams_at_once_match_calls_alone():
    """Two recurrences (whose tiles wait for one another), a norm and a preprocessing gradient on
    four streams without waiting between them, workspaces and results allocated by the calls."""
    a, b = lru_inputs(1, 2, 3000, 900), lru_inputs(2, 3, 1500, 1001, torch.float32)
    n, p = norm_inputs(3, 5000, 1030), prep_inputs(4, 2, 4, 900, 128, 4)
    sizes = [mesa.lru_workspace_bytes(*v["x"].shape, dtype=v["x"].dtype) for v in (a, b)]

    def ws(i):
        return torch.empty(sizes[i], device="cuda", dtype=torch.uint8)

    alone = [train(a, ws(0)), train(b, ws(1)), norm_train(n), prep_bwd(p)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for rep in range(3):
        w0, w1 = ws(0), ws(1)
        torch.cuda.synchronize()
        got = []
        for _ in range(3):
            got = [train(a, w0, streams[0]), train(b, w1, streams[1]), norm_train(n, streams[2]), prep_bwd(p, streams[3])]
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(alone, got)):
            equal(x, y, (rep, i))


def test_results_allocated_for_a_side_stream_are_not_reused_early():
    """A call on a side stream allocates there: dropping its results at once and allocating on the
    current stream must not hand their memory out while the side stream still writes it."""
    a = lru_inputs(5, 1, 8000, 1024)
    want = mesa.lru_fwd(a["x"], a["ga"], a["gi"], a["lam"])["y"]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        mesa.lru_fwd(a["x"], a["ga"], a["gi"], a["lam"], stream=s)  # dropped while it runs
        mine = torch.zeros_like(want)
        torch.cuda.synchronize()
        assert not mine.any()
    r = mesa.lru_fwd(a["x"], a["ga"], a["gi"], a["lam"], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(r["y"], want)


@pytest.mark.parametrize("which", ["lru", "norm", "prep", "step"])
def test_replays_in_a_graph(which):
    """Captured once, replayed with new inputs and eager work of the same operators between the replays."""
    if which == "lru":
        make = lambda s: lru_inputs(s, 2, 1300, 520)  # noqa: E731
        ws = torch.empty(mesa.lru_workspace_bytes(2, 1300, 520), device="cuda", dtype=torch.uint8)
        other_ws = torch.empty_like(ws)
        call = lambda a, stream=None, out=None: train(a, ws if out else other_ws, stream, out)  # noqa: E731
    elif which == "norm":
        make = lambda s: norm_inputs(s, 700, 2050)  # noqa: E731
        nws = torch.empty(mesa.rmsnorm_bwd_workspace_bytes(700, 2050), device="cuda", dtype=torch.uint8)
        call = lambda a, stream=None, out=None: norm_train(a, stream, out, nws if out else None)  # noqa: E731
    elif which == "prep":
        make = lambda s: prep_inputs(s, 2, 3, 500, 64, 4)  # noqa: E731
        pws = torch.empty(mesa.qk_preprocess_bwd_workspace_bytes(2, 3, 500, 64, 4), device="cuda", dtype=torch.uint8)
        call = lambda a, stream=None, out=None: prep_bwd(a, stream, out, pws if out else None)  # noqa: E731
    else:
        make = lambda s: {k: v[:, 0].contiguous() if v.dim() == 3 else v for k, v in lru_inputs(s, 9, 1, 777).items()}  # noqa: E731

        def call(a, stream=None, out=None):
            h = out["h"] if out else a["h0"].clone()
            if out:
                h.copy_(a["h0"])
            r = mesa.lru_step(a["x"], a["ga"], a["gi"], a["lam"], h, stream=stream, out=out)
            return dict(r, h=h)

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
            v.view(torch.uint8).fill_(0xAB)
        eager = call(srcs[1 - i])
        graph.replay()
        torch.cuda.synchronize()
        equal(refs[i], out, rep)
        equal(refs[1 - i], eager, rep)


def test_two_graphs_share_a_workspace():
    """Forward and backward captured apart, with one workspace that other sizes use in between;
    the backward is replayed twice on the states of one forward."""
    a, b = lru_inputs(21, 1, 2000, 300), lru_inputs(22, 2, 700, 260)
    ws = torch.empty(max(mesa.lru_workspace_bytes(1, 2000, 300), mesa.lru_workspace_bytes(2, 700, 260)),
                     device="cuda", dtype=torch.uint8)
    ra, rb = train(a, ws), train(b, ws)
    ra, rb = ({k: v.clone() for k, v in r.items()} for r in (ra, rb))
    torch.cuda.synchronize()
    graphs = []
    for inp in (a, b):
        out = {}
        args = (inp["x"], inp["ga"], inp["gi"], inp["lam"])
        f, w, s = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(f, stream=s):
            out.update(mesa.lru_fwd(*args, h0=inp["h0"], return_state=True, workspace=ws, stream=s))
        with torch.cuda.graph(w, stream=s):
            out.update(mesa.lru_bwd(*args, inp["dy"], h0=inp["h0"], state_grads=True, workspace=ws,
                                    states_in_workspace=True, stream=s))
        graphs.append((f, w, out))
    for rep in range(3):
        for (f, w, out), ref in zip(graphs, (ra, rb)):
            f.replay()
            w.replay()
            for key in ("dx", "dga", "dgi", "dlam", "dh0"):
                out[key].fill_(float("nan"))
            w.replay()
            torch.cuda.synchronize()
            equal(ref, out, rep)


def test_run_together_as_a_training_block():
    """norm -> projections -> preprocessing -> Mesa layer, and norm -> projections -> recurrence, on one
    residual stream, forward and backward, in fp32 where the operator has it, against the oracles of
    every stage on the GPU's own inputs of that stage; and the whole chain's gradient at the block's
    input against differences of the recurrence half."""
    g = gen(31)
    B, T, D, H, d = 1, 130, 256, 4, 64
    f32 = torch.float32
    x, res = normal(g, B * T, D, dtype=f32), normal(g, B * T, D, dtype=f32)
    w = 1 + 0.1 * normal(g, D, dtype=f32)
    P = normal(g, 3, D, D, dtype=f32) / 16
    lam = -6 + 3 * torch.rand(D, generator=g, device="cuda")
    dy = normal(g, B, T, D, dtype=f32)

    def forward(xx):
        n = mesa.rmsnorm(xx, w, residual=res)
        wide = torch.cat([n["y"] @ P[i] for i in range(3)], 1).view(B, T, 3 * D)
        part = [wide[..., i * D:(i + 1) * D] for i in range(3)]
        ws = torch.empty(mesa.lru_workspace_bytes(B, T, D, dtype=f32), device="cuda", dtype=torch.uint8)
        return n, part, ws, mesa.lru_fwd(*part, lam, workspace=ws)

    n, part, ws, f = forward(x)
    dwide = torch.empty((B, T, 3 * D), device="cuda")
    grads = mesa.lru_bwd(*part, lam, dy, workspace=ws, states_in_workspace=True,
                         out={k: dwide[..., i * D:(i + 1) * D] for i, k in enumerate(("dx", "dga", "dgi"))})
    dn = sum(dwide.view(B * T, 3 * D)[:, i * D:(i + 1) * D] @ P[i].T for i in range(3))
    back = mesa.rmsnorm_bwd(n["residual"], w, dn)
    e = normal(g, B * T, D, dtype=f32)
    step = 2.0 ** -7
    num = sum(s * float((forward(x + s * step * e)[3]["y"].double() * dy.double()).sum()) for s in (1, -1)) / (2 * step)
    ana = float((back["ds"].double() * e.double()).sum())
    # truncation of order step^2 = 2^-14 of the third derivative, rounding 2^-24 |L| / step
    assert abs(num - ana) <= 5e-3 * float(back["ds"].double().norm()) + 1e-3, (num, ana)
    h = lambda t: t.cpu().numpy()  # noqa: E731
    ref = block_oracle.lru_backward(*[h(t) for t in part], h(lam), h(dy))
    for key in ("dx", "dga", "dgi", "dlam"):
        assert np.abs(h(grads[key]) - ref[key]).max() <= 2e-5 * max(1.0, np.abs(ref[key]).max()), key

    # the Mesa half: the preprocessing's gradient takes the layer's dq and dk as they come
    bf = torch.bfloat16
    raw = [normal(g, B, H, T, d) for _ in range(2)]
    taps = [normal(g, H, d, 4, dtype=f32) / 2 for _ in range(2)]
    pre = mesa.qk_preprocess(*raw, *taps)
    v = normal(g, B, H, T, d)
    gamma, beta = torch.rand((B, H, T), generator=g, device="cuda") * 0.1 + 0.9, torch.rand((B, H, T), generator=g, device="cuda")
    ml = 0.25 + torch.rand((H, d), generator=g, device="cuda")
    kw = dict(chunk=64, max_steps=10)
    fw = mesa.fwd_chunked(pre["q"], pre["k"], v, gamma, beta, ml, return_x=True, **kw)
    do = normal(g, B, H, T, d, dtype=f32)
    bw = mesa.bwd_chunked(pre["q"], pre["k"], v, gamma, beta, ml, fw["x"], do, **kw)
    r = mesa.qk_preprocess_bwd(*raw, *taps, bw["dq"], bw["dk"])
    torch.cuda.synchronize()
    hf = lambda t: t.float().cpu().numpy()  # noqa: E731
    layer = mesa_backward(hf(pre["q"]), hf(pre["k"]), hf(v), hf(gamma), hf(beta), hf(ml), hf(do), max_steps=10, tol=0.0, chunk=64)
    for i, (name, key) in enumerate((("q", "dq"), ("k", "dk"))):
        # the layer's own bf16 products carry up to 2e-2 relative (its smoke check's bar); the preprocessing adds half a step
        ref = block_oracle.qk_preprocess_backward(hf(raw[i]), hf(taps[i]), layer[key])["dx"]
        got = hf(r[f"d{name}_raw"])
        assert np.linalg.norm(got - ref) <= 3e-2 * np.linalg.norm(ref), name
    assert bf is r["dq_raw"].dtype


def test_binding_refuses_what_the_kernels_cannot_take():
    a = lru_inputs(41, 2, 20, 64)
    args = [a["x"], a["ga"], a["gi"], a["lam"]]

    def bad(fn, *p, **kw):
        with pytest.raises(mesa.MesaError):
            fn(*p, **kw)

    bad(mesa.lru_fwd, a["x"].cpu(), *args[1:])
    bad(mesa.lru_fwd, a["x"].half(), a["ga"].half(), a["gi"].half(), a["lam"])
    bad(mesa.lru_fwd, a["x"], a["ga"].float(), a["gi"], a["lam"])
    bad(mesa.lru_fwd, a["x"], a["ga"][:, :10], a["gi"], a["lam"])
    bad(mesa.lru_fwd, a["x"][0], a["ga"][0], a["gi"][0], a["lam"])
    bad(mesa.lru_fwd, *[t.transpose(1, 2).contiguous().transpose(1, 2) for t in args[:3]], a["lam"])
    bad(mesa.lru_fwd, a["x"][:1].expand(2, 20, 64), *args[1:])
    bad(mesa.lru_fwd, a["x"], a["ga"], torch.cat([a["gi"], a["gi"]], 2)[..., :64], a["lam"])   # another token stride
    wide = torch.cat([a["x"], a["ga"], a["gi"], a["x"]], 2)
    bad(mesa.lru_fwd, *[wide[..., 4 + 64 * i:68 + 64 * i] for i in range(3)], a["lam"])         # 8-byte aligned slices
    bad(mesa.lru_fwd, *args, c=0.0)
    bad(mesa.lru_fwd, *args, lengths=torch.ones(2, device="cuda", dtype=torch.int64))
    bad(mesa.lru_fwd, *args, h0=torch.zeros(2, 65, device="cuda"))
    bad(mesa.lru_fwd, *args, workspace=torch.empty(64, device="cuda", dtype=torch.uint8))
    bad(mesa.lru_fwd, *args, out={"y": torch.empty(2, 20, 64, device="cuda")})
    bad(mesa.lru_bwd, *args, a["dy"].float())
    bad(mesa.lru_bwd, *args, a["dy"], states_in_workspace=True)
    bad(mesa.lru_bwd, *args, a["dy"], out={"dx": torch.empty(2, 20, 128, device="cuda", dtype=torch.bfloat16)[..., :64]})
    bad(mesa.lru_step, a["x"][:, 0], a["ga"][:, 0], a["gi"][:, 0], a["lam"], a["h0"].double())
    x = a["x"][0].contiguous()
    w = torch.ones(64, device="cuda")
    bad(mesa.rmsnorm, x.T, w)
    bad(mesa.rmsnorm, x, w.bfloat16())
    bad(mesa.rmsnorm, x, w, quant_group=64)
    bad(mesa.rmsnorm, x, w, quant_group=-1)
    bad(mesa.rmsnorm, x, w, eps=0.0)
    bad(mesa.rmsnorm, x.float(), w, residual=x)
    bad(mesa.rmsnorm, x, w, residual=x[:5])
    bad(mesa.rmsnorm_bwd, x, w, x[:5])
    bad(mesa.rmsnorm_bwd, x, w, x, d_residual=x.float())
    p = prep_inputs(42, 1, 2, 9, 64, 4)
    bad(mesa.qk_preprocess_bwd, p["q"], p["k"], p["wq"], p["wk"], p["dq"].bfloat16(), p["dk"])
    bad(mesa.qk_preprocess_bwd, p["q"], p["k"], p["wq"], p["wk"], p["dq"], p["dk"], q_hist=p["q"][:, :, :2].contiguous())
    bad(mesa.qk_preprocess_bwd, p["q"], p["k"], p["wq"], p["wk"], p["dq"], p["dk"], out={"dq_raw": p["q"]})
    with pytest.raises(mesa.MesaError):
        mesa.lru_fwd(*args, workspace=torch.empty(1 << 20, dtype=torch.uint8))
