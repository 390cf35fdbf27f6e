"""Host-side validation of the operators around the layer (CPU only).

Every call here fails validation before the first launch or has nothing to do.
"""
import ctypes

import pytest

from test_regression_sequence_amd import mesa

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
P = ctypes.c_void_p


def lru_desc(**kw):
    base = dict(B=2, T=130, D=100, ld=100, c=8.0, dtype=mesa.MESA_BF16)
    base.update(kw)
    return mesa.LruDesc(*[base[f] for f, _ in mesa.LruDesc._fields_])


def lru_ws(d):
    return mesa.lib().mesa_lru_workspace_bytes(ctypes.byref(d))


def call_lru_fwd(d, wbytes=1 << 40, **kw):
    a = dict(x=FAKE, ga=FAKE, gi=FAKE, lam=FAKE, h0=0, lengths=0, y=FAKE, h_final=0, workspace=FAKE)
    a.update(kw)
    return mesa.lib().mesa_lru_fwd(ctypes.byref(d), *[P(v) if v else None for v in a.values()], wbytes, None)


def call_lru_bwd(d, ld_grad=100, flag=0, wbytes=1 << 40, **kw):
    a = dict(x=FAKE, ga=FAKE, gi=FAKE, lam=FAKE, h0=0, lengths=0, dy=FAKE, d_hfinal=0, dx=FAKE, dga=FAKE, dgi=FAKE)
    b = dict(dlam=FAKE, dh0=0)
    ws = kw.pop("workspace", FAKE)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    p = lambda m: [P(v) if v else None for v in m.values()]  # noqa: E731
    return mesa.lib().mesa_lru_bwd(ctypes.byref(d), *p(a), ld_grad, *p(b), flag, P(ws) if ws else None, wbytes, None)


BAD_LRU = [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(D=0, ld=100), 1), (dict(ld=99), 1), (dict(c=0.0), 1), (dict(c=-1.0), 1),
    (dict(c=float("inf")), 1), (dict(c=float("nan")), 1), (dict(dtype=2), 1),
    (dict(ld=(1 << 20) + 1), 2), (dict(D=1), 2), (dict(B=1 << 19, T=64 * 8, D=128, ld=128), 0), (dict(B=1 << 19, T=64 * 8 + 1, D=128, ld=128), 2),
    (dict(B=2 ** 31 - 1, T=2 ** 31 - 1), 2), (dict(B=2 ** 31 - 1, T=0, D=2), 2), (dict(B=(1 << 23) + 1, T=0, D=2), 2),
]


@pytest.mark.parametrize("kw,expect", BAD_LRU)
def test_lru_rejects_bad_descriptors(kw, expect):
    d = lru_desc(**kw)
    if expect == 0:  # the largest: accepted up to the workspace
        assert call_lru_fwd(d, workspace=0) == 4 and call_lru_bwd(d, ld_grad=1 << 20, workspace=0) == 4 and lru_ws(d) > 0
        return
    assert call_lru_fwd(d) == expect
    assert call_lru_bwd(d, ld_grad=1 << 20) == expect
    assert lru_ws(d) == 0


def test_lru_rejects_missing_and_misaligned_pointers_and_small_workspaces():
    d = lru_desc()
    need = lru_ws(d)
    assert need >= 2 * 3 * 100 * 4
    for name in ("x", "ga", "gi", "lam", "y"):
        assert call_lru_fwd(d, **{name: 0}) == 1, name
    for name in ("x", "ga", "gi", "lam", "h0", "lengths", "y", "h_final", "workspace"):
        assert call_lru_fwd(d, **{name: FAKE + 8}) == 3, name
    assert call_lru_fwd(d, workspace=0) == 4
    assert call_lru_fwd(d, wbytes=need - 1) == 4
    for name in ("x", "ga", "gi", "lam", "dy", "dx", "dga", "dgi", "dlam"):
        assert call_lru_bwd(d, **{name: 0}) == 1, name
    for name in ("x", "ga", "gi", "lam", "h0", "lengths", "dy", "d_hfinal", "dx", "dga", "dgi", "dlam", "dh0", "workspace"):
        assert call_lru_bwd(d, **{name: FAKE + 4}) == 3, name
    assert call_lru_bwd(d, ld_grad=99) == 1
    assert call_lru_bwd(d, flag=2) == 1
    assert call_lru_bwd(d, flag=-1) == 1
    assert call_lru_bwd(d, ld_grad=1 << 20, workspace=0) == 4
    assert call_lru_bwd(d, ld_grad=(1 << 20) + 1) == 2
    assert call_lru_bwd(d, wbytes=need - 1) == 4
    assert lru_ws(lru_desc(T=0)) == 0


def test_lru_step_validation():
    def call(N=2, D=100, ld=100, c=8.0, dtype=1, **kw):
        a = dict(x=FAKE, ga=FAKE, gi=FAKE, lam=FAKE, h=FAKE, y=FAKE)
        a.update(kw)
        return mesa.lib().mesa_lru_step(N, D, ld, ctypes.c_float(c), dtype, *[P(v) if v else None for v in a.values()], None)

    assert call(N=-1) == 1
    assert call(D=0) == 1
    assert call(ld=99) == 1
    assert call(D=1) == 2
    assert call(c=0.0) == 1
    assert call(dtype=5) == 1
    assert call(N=0) == 0  # nothing to do, nothing launched
    for name in ("x", "ga", "gi", "lam", "h", "y"):
        assert call(**{name: 0}) == 1
        assert call(**{name: FAKE + 2}) == 3


def call_norm(R=4, D=100, dtype=1, res=1, eps=1e-6, out=0, group=0, **kw):
    a = dict(x=FAKE, residual=FAKE, w=FAKE)
    b = dict(y=FAKE, scale=0, residual_out=0)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    p = lambda m: [P(v) if v else None for v in m.values()]  # noqa: E731
    return mesa.lib().mesa_rmsnorm(R, D, dtype, res, *p(a), ctypes.c_float(eps), out, group, *p(b), None)


def call_norm_bwd(R=4, D=100, dtype=1, res=1, eps=1e-6, wbytes=1 << 40, workspace=FAKE, **kw):
    a = dict(s=FAKE, w=FAKE, dy=FAKE, d_residual=0)
    b = dict(ds=FAKE, dx=0, dw=FAKE)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    p = lambda m: [P(v) if v else None for v in m.values()]  # noqa: E731
    return mesa.lib().mesa_rmsnorm_bwd(R, D, dtype, res, *p(a), ctypes.c_float(eps), *p(b),
                                       P(workspace) if workspace else None, wbytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(R=-1), 1), (dict(D=0), 1), (dict(dtype=2), 1), (dict(res=-1), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1),
    (dict(eps=2.0 ** -127), 1), (dict(eps=float("inf")), 1), (dict(eps=float("nan")), 1), (dict(D=16385), 2),
    (dict(dtype=0, res=1), 2), (dict(R=2 ** 30, D=16384), 2), (dict(R=2 ** 30 + 1, D=1), 2),
])
def test_norm_rejects_bad_sizes_and_types(kw, expect):
    assert call_norm(**kw) == expect
    assert call_norm_bwd(**kw) == expect


def test_norm_rejects_missing_and_misaligned_pointers():
    for name in ("x", "w", "y"):
        assert call_norm(**{name: 0}) == 1, name
    for name in ("x", "residual", "w", "y", "scale", "residual_out"):
        assert call_norm(**{name: FAKE + 4}) == 3, name
    assert call_norm(out=2) == 1
    assert call_norm(out=1) == 1                       # e4m3 needs scales
    assert call_norm(out=1, scale=FAKE, group=-1) == 1
    assert call_norm(out=1, scale=FAKE, group=64) == 2
    assert call_norm(R=0, x=0) == 0                    # nothing to do, nothing launched
    for name in ("s", "w", "dy", "ds", "dw"):
        assert call_norm_bwd(**{name: 0}) == 1, name
    for name in ("s", "w", "dy", "d_residual", "ds", "dx", "dw", "workspace"):
        assert call_norm_bwd(**{name: FAKE + 8}) == 3, name
    need = mesa.lib().mesa_rmsnorm_bwd_workspace_bytes(4, 100)
    assert need > 0
    assert call_norm_bwd(wbytes=need - 1) == 4
    assert call_norm_bwd(workspace=0) == 4
    assert mesa.lib().mesa_rmsnorm_bwd_workspace_bytes(-1, 100) == 0


def test_preprocess_backward_validation():
    L = mesa.lib()
    A, G, O = 0x7F0000000000, 0x7F1000000000, 0x7F2000000000   # distinct 16-byte aligned fake ranges
    M = 0x100000

    def call(B=2, H=2, T=8, d=128, W=4, dtype=1, eps=1e-6, workspace=A + 32 * M, wbytes=1 << 40, **kw):
        ins = dict(q=A, k=A + M, wq=A + 2 * M, wk=A + 3 * M, qh=0, kh=0)
        gin = dict(dq=G, dk=G + M, dqh=0, dkh=0)
        outs = dict(dqr=O, dkr=O + M, dwq=O + 2 * M, dwk=O + 3 * M, dqhist=0, dkhist=0)
        for k, v in kw.items():
            next(m for m in (ins, gin, outs) if k in m)[k] = v
        p = lambda m: [P(v) if v else None for v in m.values()]  # noqa: E731
        return L.mesa_qk_preprocess_bwd(B, H, T, d, W, dtype, *p(ins), ctypes.c_float(eps), *p(gin), *p(outs),
                                        P(workspace) if workspace else None, wbytes, None)

    need = L.mesa_qk_preprocess_bwd_workspace_bytes(2, 2, 8, 128, 4, 1)
    assert need > 0 and L.mesa_qk_preprocess_bwd_workspace_bytes(2, 2, 0, 128, 4, 1) == 0
    assert call(d=96) == 2
    assert call(W=5) == 2
    assert call(B=65536, H=1) == 2
    assert call(T=2 ** 30 + 1) == 2
    assert call(W=0) == 1
    assert call(B=0) == 1
    assert call(T=-1) == 1
    assert call(dtype=3) == 1
    for eps in (0.0, 2.0 ** -64, float("inf"), float("nan")):
        assert call(eps=eps) == 1
    for name in ("q", "k", "wq", "wk", "dq", "dk", "dqr", "dkr", "dwq", "dwk"):
        assert call(**{name: 0}) == 1, name
    for name in ("q", "k", "wq", "wk", "qh", "kh", "dq", "dk", "dqh", "dkh", "dqr", "dkr", "dwq", "dwk", "dqhist", "dkhist"):
        assert call(**{name: O + 8 * M + 4}) == 3, name
    assert call(dqr=A) == 1               # over the raw input
    assert call(dkr=G) == 1               # over the incoming gradient
    assert call(qh=A + 4 * M, dqhist=A + 4 * M) == 1
    assert call(workspace=0) == 4
    assert call(wbytes=need - 1) == 4


def apart(names):
    """Distinct fake ranges, far apart."""
    return {n: 0x7F0000000000 + i * 0x10000000 for i, n in enumerate(names)}


def test_outputs_over_inputs_are_refused():
    """Every output and the workspace against every input, at equal addresses and where one ends in the other."""
    d = lru_desc()
    a = apart(("x", "ga", "gi", "lam", "h0", "lengths", "y", "h_final", "workspace"))
    ins = ("x", "ga", "gi", "lam", "h0", "lengths")
    for o in ("y", "h_final", "workspace"):
        for i in ins:
            if (o, i) != ("h_final", "h0"):
                assert call_lru_fwd(d, **{**a, o: a[i]}) == 1, (o, i)
    assert call_lru_fwd(d, **{**a, "h_final": a["h0"] + 16}) == 1
    assert call_lru_fwd(d, **{**a, "y": a["x"] - 16}) == 1 and call_lru_fwd(d, **{**a, "x": a["y"] - 16}) == 1

    a = apart(ins + ("dy", "d_hfinal", "dx", "dga", "dgi", "dlam", "dh0", "workspace"))
    for o in ("dx", "dga", "dgi", "dlam", "dh0", "workspace"):
        for i in ins + ("dy", "d_hfinal"):
            if (o, i) != ("dh0", "d_hfinal"):
                assert call_lru_bwd(d, **{**a, o: a[i]}) == 1, (o, i)

    a = apart(("x", "ga", "gi", "lam", "h", "y"))
    for o in ("h", "y"):
        for i in ("x", "ga", "gi", "lam"):
            b = {**a, o: a[i]}
            assert mesa.lib().mesa_lru_step(2, 100, 100, ctypes.c_float(8.0), 1, *[P(v) for v in b.values()], None) == 1, (o, i)

    a = apart(("x", "residual", "w", "y", "scale", "residual_out"))
    for kw in (dict(res=1), dict(res=0), dict(res=1, out=1), dict(res=1, out=1, group=128)):
        for o, over in (("y", ("x", "residual", "w", "residual_out")), ("residual_out", ("w",)),
                        ("scale", ("x", "residual", "w", "residual_out"))):
            for i in over:
                if o != "scale" or "out" in kw:
                    assert call_norm(**kw, **{**a, o: a[i]}) == 1, (kw, o, i)
        assert call_norm(**kw, **{**a, "residual_out": a["residual"] + 16}) == 1
    assert call_norm(res=0, **{**a, "residual_out": a["x"]}) == 1  # an fp32 stream over bf16 rows

    a = apart(("s", "w", "dy", "d_residual", "ds", "dx", "dw", "workspace"))
    for o in ("ds", "dx", "dw", "workspace"):
        for i in ("s", "w", "dy", "d_residual"):
            if (o, i) != ("ds", "d_residual"):
                assert call_norm_bwd(**{**a, o: a[i]}) == 1, (o, i)
