"""Cases of the operators that a block around the Mesa layer is built from.

Five kinds of call, each on what a user's program has in hand:

* ``step``   one new token of the gated linear recurrence (the layer that
             alternates with the Mesa layer in the Hawk-Mesa hybrid),
* ``scan``   the same recurrence over whole sequences,
* ``train``  the recurrence forward and its backward pass, one after the other,
* ``norm``   residual addition and RMS norm, with an 8-bit or a plain output,
* ``norm_bwd`` the gradient of that,
* ``prep_bwd`` the gradient of the query/key preprocessing (causal depthwise
             convolution, then L2 norm) that stands before the Mesa layer.

Where ``own`` is false, ``run`` computes them from elementary torch operations
in 32 bits; where it is true, it calls the library.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0
GROUP = 128          # channels that share a scale in the grouped 8-bit output
AMAX_FLOOR = 2.0 ** -100
DECAY = 8.0          # c of the recurrence
EPS = 1e-6


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # 256 sequences decoding at the width of the decode workload (16 heads of 128)
        dict(name="step-256", kind="step", N=256, D=2048, dtype="bf16"),
        # a single user's token: the time of a launch counts
        dict(name="step-1", kind="step", N=1, D=1000, dtype="f32"),
        # a long document as one sequence (the long workload's length and width)
        dict(name="scan-long", kind="scan", B=1, T=32768, D=2048, dtype="bf16", ragged=False, h0=False),
        # prompts of several users, padded to the longest, continuing kept states
        dict(name="scan-ragged", kind="scan", B=7, T=777, D=1001, dtype="f32", ragged=True, h0=True),
        # a training batch of the language-model workload (B=8, T=4096, 16 heads of 128)
        dict(name="train-lm", kind="train", B=8, T=4096, D=2048, dtype="bf16", ragged=False, h0=False),
        # a small ragged batch in fp32, as a gradient is checked or a small model is trained
        dict(name="train-ragged", kind="train", B=3, T=1000, D=509, dtype="f32", ragged=True, h0=True),
        # the block's norm ahead of 8-bit projections, language-model workload's tokens
        dict(name="norm-lm-8bit", kind="norm", R=32768, D=2048, dtype="bf16", res="bf16", out="row"),
        # the same norm at a decode step, residual stream in fp32
        dict(name="norm-decode", kind="norm", R=256, D=2048, dtype="bf16", res="f32", out="group"),
        # its gradient over the training batch
        dict(name="norm-bwd-lm", kind="norm_bwd", R=32768, D=2048, dtype="bf16", res="bf16"),
        # odd sizes in fp32
        dict(name="norm-bwd-odd", kind="norm_bwd", R=1111, D=777, dtype="f32", res="f32"),
        # the preprocessing's gradient in the training batch of the language-model workload
        dict(name="prep-bwd-lm", kind="prep_bwd", B=8, H=16, T=4096, d=128, W=4, dtype="bf16", hist=False),
        # a short piece of a sequence with its history
        dict(name="prep-bwd-short", kind="prep_bwd", B=2, H=3, T=77, d=64, W=3, dtype="f32", hist=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A model width: a multiple of 64 as models have it, or any number."""
    d = _log_int(rng, lo, hi)
    return max(64, d // 64 * 64) if rng.random() < 0.6 else d


def draw(rng):
    kind = rng.choice(["step", "scan", "train", "norm", "norm_bwd", "prep_bwd"])
    dtype = rng.choice(["bf16", "f32"])
    cap = (1 << 25) if dtype == "f32" else (1 << 26)
    if kind == "step":
        return dict(kind=kind, N=_log_int(rng, 1, 1024), D=_width(rng, 64, 4096), dtype=dtype)
    if kind in ("scan", "train"):
        B, D = _log_int(rng, 1, 16), _width(rng, 64, 4096)
        T = _log_int(rng, 1, max(2, min(32768 if kind == "scan" else 8192, cap // (B * D))))
        return dict(kind=kind, B=B, T=T, D=D, dtype=dtype, ragged=rng.random() < 0.5, h0=rng.random() < 0.5)
    if kind in ("norm", "norm_bwd"):
        D = _width(rng, 64, 8192)
        R = _log_int(rng, 1, min(65536, cap // D))
        res = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
        c = dict(kind=kind, R=R, D=D, dtype=dtype, res=res)
        if kind == "norm":
            c["out"] = rng.choice(["plain", "row", "group"])
        return c
    d, H, B = rng.choice([16, 64, 128]), _log_int(rng, 1, 16), _log_int(rng, 1, 8)
    T = _log_int(rng, 1, min(8192, cap // (B * H * d)))
    return dict(kind=kind, B=B, H=H, T=T, d=d, W=rng.randint(1, 4), dtype=dtype, hist=rng.random() < 0.5)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _decay_parameter(gen, D):
    """lam [D] with exp(-c softplus(lam)) ~ U(0.9, 0.999), the usual initialisation."""
    a0 = torch.rand(D, generator=gen, device="cuda") * 0.099 + 0.9
    return torch.log(torch.expm1(-torch.log(a0) / DECAY))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind, dt = case["kind"], DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)

    f32 = torch.float32
    s = {"case": case}
    if kind == "step":
        N, D = case["N"], case["D"]
        s.update(x=normal(N, D), ga=normal(N, D), gi=normal(N, D), lam=_decay_parameter(gen, D),
                 h=normal(N, D, dtype=f32))
    elif kind in ("scan", "train"):
        B, T, D = case["B"], case["T"], case["D"]
        s.update(x=normal(B, T, D), ga=normal(B, T, D), gi=normal(B, T, D), lam=_decay_parameter(gen, D),
                 h0=normal(B, D, dtype=f32) if case["h0"] else None, lengths=None)
        if case["ragged"]:  # one sequence of each batch is as long as the padding, the others are shorter
            n = np.random.default_rng(seed).integers(0, T + 1, B).astype(np.int32)
            n[0] = T
            s["lengths"] = torch.from_numpy(n).cuda()
        if kind == "train":
            s.update(dy=normal(B, T, D), d_hfinal=normal(B, D, dtype=f32))
    elif kind == "norm":
        R, D = case["R"], case["D"]
        s.update(x=normal(R, D), residual=normal(R, D, dtype=DTYPES[case["res"]], scale=2.0),
                 w=1.0 + normal(D, dtype=f32, scale=0.1))
    elif kind == "norm_bwd":
        R, D = case["R"], case["D"]
        res = DTYPES[case["res"]]
        s.update(s=normal(R, D, dtype=res, scale=2.0), w=1.0 + normal(D, dtype=f32, scale=0.1), dy=normal(R, D),
                 d_residual=normal(R, D, dtype=res))
    else:
        B, H, T, d, W = (case[k] for k in ("B", "H", "T", "d", "W"))
        bound = 1.0 / math.sqrt(W)
        for n in ("q", "k"):
            s[n] = normal(B, H, T, d)
            s["w_" + n] = (torch.rand((H, d, W), generator=gen, device="cuda") * 2 - 1) * bound
            s["d_" + n] = normal(B, H, T, d, dtype=f32)
            s[n + "_hist"] = normal(B, H, W - 1, d) if case["hist"] and W > 1 else None
    return s


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------

def _gates(x, ga, gi, lam):
    """w = -2 log a, the decay a, the input scale m = sqrt(1 - a^2) and the two sigmoids, in fp32."""
    sr, si = torch.sigmoid(ga.float()), torch.sigmoid(gi.float())
    w = (2 * DECAY) * torch.nn.functional.softplus(lam) * sr
    return w, torch.exp(-0.5 * w), torch.sqrt(-torch.expm1(-w)), sr, si


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1 from zero, and the running product of a, by doubling."""
    s = 1
    while s < a.shape[1]:
        u = torch.cat([u[:, :s], torch.addcmul(u[:, s:], a[:, s:], u[:, :-s])], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return u, a


def _valid(s, T):
    """[B, T, 1]: which rows lie within their sequence's length."""
    if s["lengths"] is None:
        return None
    return (torch.arange(T, device="cuda")[None, :] < s["lengths"][:, None])[:, :, None]


def _states(s):
    """a, h_t and h_{t-1} [B, T, D], the final state, and what the gradients need; rows behind a length keep the state."""
    w, a, m, sr, si = _gates(s["x"], s["ga"], s["gi"], s["lam"])
    u = m * si * s["x"].float()
    ok = _valid(s, a.shape[1])
    if ok is not None:
        a, u = torch.where(ok, a, 1.0), torch.where(ok, u, 0.0)
    h, run = _scan(a, u)
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
    if s["h0"] is not None:
        h = torch.addcmul(h, run, first)
    return ok, w, a, m, sr, si, h, torch.cat([first, h[:, :-1]], 1)


def _plain_scan(s):
    ok, _, _, _, _, _, h, _ = _states(s)
    y = h if ok is None else torch.where(ok, h, 0.0)
    return {"y": y.to(s["x"].dtype), "h_final": h[:, -1].contiguous()}


def _plain_train(s):
    dt, x = s["x"].dtype, s["x"].float()
    ok, w, a, m, sr, si, h, before = _states(s)
    y = h if ok is None else torch.where(ok, h, 0.0)
    out = {"y": y.to(dt), "h_final": h[:, -1].contiguous()}
    # g_t = dy_t + a_{t+1} g_{t+1}, the final state's gradient entering behind the last row
    dy = s["dy"].float() if ok is None else torch.where(ok, s["dy"].float(), 0.0)
    a_next = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g, run = _scan(a_next.flip(1), dy.flip(1))
    g = torch.addcmul(g, run, s["d_hfinal"][:, None]).flip(1)
    out["dh0"] = a[:, 0] * g[:, 0]
    gm = g * m
    half = 0.5 * w * g * (torch.where(m > 0, a * a / m, 0.0) * si * x - a * before)  # dL / d log w
    grads = {"dx": gm * si, "dga": half * (1 - sr), "dgi": gm * x * si * (1 - si)}
    if ok is not None:
        grads = {k: torch.where(ok, v, 0.0) for k, v in grads.items()}
        half = torch.where(ok, half, 0.0)
    ratio = torch.sigmoid(s["lam"]) / torch.nn.functional.softplus(s["lam"])
    out["dlam"] = half.sum((0, 1), dtype=torch.float64).float() * ratio
    out.update({k: v.to(dt) for k, v in grads.items()})
    return out


def _plain_step(s):
    _, a, m, _, si = _gates(s["x"], s["ga"], s["gi"], s["lam"])
    h = a * s["h"] + m * si * s["x"].float()
    s["h"].copy_(h)
    return {"y": h.to(s["x"].dtype), "h": s["h"]}


def _plain_norm(s):
    case, x = s["case"], s["x"].float() + s["residual"].float()
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["w"]
    out = {"residual": x.to(s["residual"].dtype)}
    if case["out"] == "plain":
        out["y"] = y.to(s["x"].dtype)
        return out
    R, D = y.shape
    g = D if case["out"] == "row" else GROUP
    n = -(-D // g)
    z = torch.nn.functional.pad(y, (0, n * g - D)).view(R, n, g)
    amax = z.abs().amax(2).clamp_min(AMAX_FLOOR)
    q = (z * (E4M3_MAX / amax)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    out["y"] = q.view(R, n * g)[:, :D].contiguous()
    out["scale"] = amax / E4M3_MAX
    return out


def _plain_norm_bwd(s):
    x, dy = s["s"].float(), s["dy"].float()
    rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    xhat, g = x * rstd, dy * s["w"]
    ds = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True)) + s["d_residual"].float()
    out = {"ds": ds.to(s["s"].dtype), "dw": (dy * xhat).sum(0, dtype=torch.float64).float()}
    if s["s"].dtype != s["dy"].dtype:
        out["dx"] = ds.to(s["dy"].dtype)
    return out


def _plain_prep_bwd(s):
    W, out = s["case"]["W"], {}
    for n in ("q", "k"):
        raw, taps, do, hist = s[n], s["w_" + n], s["d_" + n], s[n + "_hist"]
        B, H, T, d = raw.shape
        first = torch.zeros((B, H, W - 1, d), device="cuda") if hist is None else hist.float()
        seq = torch.cat([first, raw.float()], 2)              # rows -(W-1) .. T-1
        rows = seq.unfold(2, W, 1).flip(-1)                   # [B, H, T, d, W]: tap i weighs token t - i
        y = (rows * taps[None, :, None]).sum(-1)
        norm = torch.sqrt((y * y).sum(-1, keepdim=True))
        unit = y / norm.clamp_min(EPS)
        dot = torch.where(norm > EPS, (unit * do).sum(-1, keepdim=True), 0.0)
        dyc = (do - unit * dot) / norm.clamp_min(EPS)         # gradient at the convolution's output
        out["dw_" + n] = (rows * dyc[..., None]).sum((0, 2), dtype=torch.float64).float()
        tail = torch.nn.functional.pad(dyc, (0, 0, W - 1, W - 1))
        dseq = (tail.unfold(2, W, 1) * taps[None, :, None]).sum(-1)  # rows -(W-1) .. T-1
        out["d%s_raw" % n] = dseq[:, :, W - 1:].to(raw.dtype)
        if hist is not None:
            out["d%s_hist" % n] = dseq[:, :, :W - 1].to(raw.dtype)
    return out


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def _own(s):
    from test_regression_sequence_amd import mesa

    case = s["case"]
    kind = case["kind"]
    if kind == "step":
        r = mesa.lru_step(s["x"], s["ga"], s["gi"], s["lam"], s["h"], c=DECAY)
        return {"y": r["y"], "h": s["h"]}
    if kind == "scan":
        return mesa.lru_fwd(s["x"], s["ga"], s["gi"], s["lam"], c=DECAY, h0=s["h0"], lengths=s["lengths"],
                            return_state=True)
    if kind == "train":
        kw = dict(c=DECAY, h0=s["h0"], lengths=s["lengths"])
        ws = torch.empty(mesa.lru_workspace_bytes(case["B"], case["T"], case["D"], dtype=s["x"].dtype),
                         device="cuda", dtype=torch.uint8)
        args = (s["x"], s["ga"], s["gi"], s["lam"])
        out = mesa.lru_fwd(*args, return_state=True, workspace=ws, **kw)
        out.update(mesa.lru_bwd(*args, s["dy"], d_hfinal=s["d_hfinal"], state_grads=True, workspace=ws,
                                states_in_workspace=True, **kw))
        return out
    if kind == "norm":
        group = {"plain": None, "row": 0, "group": GROUP}[case["out"]]
        return mesa.rmsnorm(s["x"], s["w"], residual=s["residual"], eps=EPS, quant_group=group)
    if kind == "norm_bwd":
        return mesa.rmsnorm_bwd(s["s"], s["w"], s["dy"], d_residual=s["d_residual"], eps=EPS)
    return mesa.qk_preprocess_bwd(s["q"], s["k"], s["w_q"], s["w_k"], s["d_q"], s["d_k"], q_hist=s["q_hist"],
                                  k_hist=s["k_hist"], eps=EPS, history_grads=s["q_hist"] is not None)


_PLAIN = {"step": _plain_step, "scan": _plain_scan, "train": _plain_train, "norm": _plain_norm,
          "norm_bwd": _plain_norm_bwd, "prep_bwd": _plain_prep_bwd}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["kind"]](state)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    """Bytes: every input read once, every output written once.  A training pass
    is two calls with the loss between them in real use, so it counts the
    forward's inputs twice.  The mean length of a ragged sequence is about T/2
    (rows behind a length are not read, and are written as zeros)."""
    kind = case["kind"]
    e = 2 if case["dtype"] == "bf16" else 4
    if kind == "step":
        n = case["N"] * case["D"]
        return {"bytes": n * (4 * e + 8) + 4 * case["D"], "flops": 30 * n}
    if kind in ("scan", "train"):
        B, T, D = case["B"], case["T"], case["D"]
        n = B * T * D
        live = (T + (B - 1) * T / 2) * D if case["ragged"] else n
        states = 4 * B * D * (2 if case["h0"] else 1) + 4 * D
        if kind == "scan":
            return {"bytes": 3 * e * live + e * n + states, "flops": 30 * live}
        return {"bytes": 7 * e * live + 4 * e * n + 2 * states + 4 * B * D + 8 * D, "flops": 90 * live}
    if kind in ("norm", "norm_bwd"):
        n, r = case["R"] * case["D"], 2 if case["res"] == "bf16" else 4
        if kind == "norm_bwd":
            return {"bytes": n * (e + 3 * r + (e if e != r else 0)) + 8 * case["D"], "flops": 14 * n}
        o = {"plain": e, "row": 1, "group": 1}[case["out"]]
        groups = {"plain": 0, "row": 1, "group": -(-case["D"] // GROUP)}[case["out"]]
        return {"bytes": n * (e + 2 * r + o) + 4 * case["D"] + 4 * groups * case["R"], "flops": 8 * n}
    B, H, T, d, W = (case[k] for k in ("B", "H", "T", "d", "W"))
    n = B * H * T * d
    hist = 2 * e * B * H * (W - 1) * d if case["hist"] else 0
    return {"bytes": 2 * (n * (2 * e + 4) + 2 * 4 * H * d * W + hist), "flops": 2 * n * (6 * W + 10)}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def _exact_recurrence(x, ga, gi, lam, h0, lengths, dy=None, d_hfinal=None):
    """Token by token; the gradients through the gates come from torch's automatic differentiation."""
    leaf = [t.double().requires_grad_(dy is not None) for t in (x, ga, gi, lam)]
    x, ga, gi, lam = leaf
    B, T, D = x.shape
    log_a = -DECAY * torch.log1p(torch.exp(lam)) / (1 + torch.exp(-ga))
    a = torch.exp(log_a)
    u = torch.sqrt(-torch.expm1(2 * log_a)) * x / (1 + torch.exp(-gi))
    n = [T] * B if lengths is None else [int(v) for v in lengths.cpu()]
    stop = torch.tensor(n, device="cuda")
    av, uv = a.detach(), u.detach()
    h = torch.zeros((B, D), device="cuda", dtype=torch.float64) if h0 is None else h0.double()
    start, y, prev = h, torch.zeros_like(av), torch.zeros_like(av)
    for t in range(T):
        live = (stop > t)[:, None]
        prev[:, t] = h
        h = torch.where(live, av[:, t] * h + uv[:, t], h)
        y[:, t] = torch.where(live, h, 0.0)
    out = {"y": y, "h_final": h}
    if dy is None:
        return out
    g, after = torch.zeros_like(av), d_hfinal.double()   # after: gradient at the state behind row t
    for t in range(T - 1, -1, -1):
        live = (stop > t)[:, None]
        now = after + dy[:, t].double()
        g[:, t] = torch.where(live, now, 0.0)
        after = torch.where(live, av[:, t] * now, after)
    grads = torch.autograd.grad([a, u], leaf, [g * prev, g])
    out.update(dh0=after, **dict(zip(("dx", "dga", "dgi", "dlam"), grads)))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "step":
        r = _exact_recurrence(s["x"][:, None], s["ga"][:, None], s["gi"][:, None], s["lam"], s["h"], None)
        return {"y": r["y"][:, 0], "h": r["h_final"]}
    if kind == "scan":
        return _exact_recurrence(s["x"], s["ga"], s["gi"], s["lam"], s["h0"], s["lengths"])
    if kind == "train":
        return _exact_recurrence(s["x"], s["ga"], s["gi"], s["lam"], s["h0"], s["lengths"], s["dy"], s["d_hfinal"])
    if kind == "norm":
        v = s["x"].double() + s["residual"].double()
        D = v.shape[1]
        y = s["w"].double() * v / torch.sqrt(v.square().sum(1, keepdim=True) / D + EPS)
        if case["out"] == "plain":
            return {"y": y, "residual": v}
        g = D if case["out"] == "row" else GROUP
        scale = torch.stack([p.abs().amax(1).clamp_min(AMAX_FLOOR) for p in y.split(g, 1)], 1) / E4M3_MAX
        codes = y / scale.repeat_interleave(g, 1)[:, :D]
        return {"y": codes.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double(), "scale": scale, "residual": v}
    if kind == "norm_bwd":
        v, w = s["s"].double().requires_grad_(), s["w"].double().requires_grad_()
        y = w * v / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)
        ds, dw = torch.autograd.grad(y, [v, w], s["dy"].double())
        ds = ds + s["d_residual"].double()
        return {"ds": ds, "dw": dw, "dx": ds if case["res"] != case["dtype"] else None}
    out, W = {}, case["W"]
    for n in ("q", "k"):
        raw, taps = s[n].double().requires_grad_(), s["w_" + n].double().requires_grad_()
        B, H, T, d = raw.shape
        hist = s[n + "_hist"]
        first = (torch.zeros((B, H, W - 1, d), device="cuda", dtype=torch.float64) if hist is None
                 else hist.double()).requires_grad_()
        seq = torch.cat([first, raw], 2)
        y = sum(taps[None, :, None, :, i] * seq[:, :, W - 1 - i:W - 1 - i + T] for i in range(W))
        unit = y / y.square().sum(-1, keepdim=True).sqrt().clamp_min(EPS)
        draw_, dw, dh = torch.autograd.grad(unit, [raw, taps, first], s["d_" + n].double(), allow_unused=True)
        out["d%s_raw" % n], out["dw_" + n] = draw_, dw
        if hist is not None:
            out["d%s_hist" % n] = dh
    return out
