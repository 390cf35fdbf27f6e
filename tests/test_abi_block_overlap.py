"""Which buffers of the operators around the layer may share memory (CPU only).

Every call here is refused before the first launch.
"""
import ctypes

import pytest

from test_regression_sequence_amd import mesa

P = ctypes.c_void_p
STEP = 0x10000000
LRU_IN = ("x", "ga", "gi", "lam", "h0", "lengths")


def apart(*names):
    """Distinct fake ranges, far apart, 16-byte aligned, never dereferenced."""
    return {n: 0x7F0000000000 + i * STEP for i, n in enumerate(names)}


def ptrs(a, names):
    return [P(a[n]) if a.get(n) else None for n in names]


def lru_fwd(B=2, T=130, D=100, ld=100, **kw):
    a = {**apart(*LRU_IN, "y", "h_final", "workspace"), **kw}
    d = mesa.LruDesc(B, T, D, ld, 8.0, mesa.MESA_BF16)
    return mesa.lib().mesa_lru_fwd(ctypes.byref(d), *ptrs(a, LRU_IN + ("y", "h_final", "workspace")), 1 << 40, None)


def lru_bwd(B=2, T=130, D=100, ld=100, ld_grad=100, dtype=mesa.MESA_BF16, **kw):
    a = {**apart(*LRU_IN, "dy", "d_hfinal", "dx", "dga", "dgi", "dlam", "dh0", "workspace"), **kw}
    d = mesa.LruDesc(B, T, D, ld, 8.0, dtype)
    return mesa.lib().mesa_lru_bwd(ctypes.byref(d), *ptrs(a, LRU_IN + ("dy", "d_hfinal", "dx", "dga", "dgi")), ld_grad,
                                   *ptrs(a, ("dlam", "dh0")), 0, *ptrs(a, ("workspace",)), 1 << 40, None)


def norm_bwd(R=4, D=100, dtype=1, res=1, **kw):
    a = {**apart("s", "w", "dy", "d_residual", "ds", "dx", "dw", "workspace"), **kw}
    return mesa.lib().mesa_rmsnorm_bwd(R, D, dtype, res, *ptrs(a, ("s", "w", "dy", "d_residual")), ctypes.c_float(1e-6),
                                       *ptrs(a, ("ds", "dx", "dw", "workspace")), 1 << 40, None)


def test_a_permitted_sharing_permits_no_other():
    """h_final over h0, dh0 over d_hfinal, ds over d_residual: everything else over the shared buffer is refused."""
    f = apart(*LRU_IN, "y", "h_final", "workspace")
    for name in ("y", "workspace"):
        assert lru_fwd(h_final=f["h0"], **{name: f["h0"]}) == 1, name
    b = apart(*LRU_IN, "dy", "d_hfinal", "dx", "dga", "dgi", "dlam", "dh0", "workspace")
    for name in ("dx", "dga", "dgi", "dlam", "workspace"):
        assert lru_bwd(dh0=b["d_hfinal"], **{name: b["d_hfinal"]}) == 1, name
    n = apart("s", "w", "dy", "d_residual", "ds", "dx", "dw", "workspace")
    for res in (0, 1):
        for name in ("dx", "dw", "workspace"):
            assert norm_bwd(res=res, ds=n["d_residual"], **{name: n["d_residual"]}) == 1, (res, name)


def distinct(outs):
    """More fake ranges, apart from those of apart()."""
    return {n: 0x7F0000000000 + (50 + i) * STEP for i, n in enumerate(outs)}


def check_pairs(outs, call, **kw):
    f = distinct(outs)
    for i, p in enumerate(outs):
        for q in outs:
            if p != q:
                for over in (0, 16):
                    assert call(**{**kw, **f, q: f[p] + over}) == 1, (kw, p, q, over)


def test_outputs_over_outputs_are_refused():
    for T in (1, 8, 130):
        check_pairs(("y", "h_final", "workspace"), lru_fwd, T=T)
        check_pairs(("dx", "dga", "dgi", "dlam", "dh0", "workspace"), lru_bwd, T=T)
    for res in (0, 1):
        check_pairs(("ds", "dx", "dw", "workspace"), norm_bwd, res=res)

    def step(**kw):
        a = {**apart("x", "ga", "gi", "lam"), **kw}
        return mesa.lib().mesa_lru_step(2, 100, 100, ctypes.c_float(8.0), 1, *ptrs(a, ("x", "ga", "gi", "lam", "h", "y")), None)
    check_pairs(("h", "y"), step)

    def norm(out=0, group=0, **kw):
        a = {**apart("x", "residual", "w"), **kw}
        return mesa.lib().mesa_rmsnorm(4, 100, 1, 1, *ptrs(a, ("x", "residual", "w")), ctypes.c_float(1e-6), out, group,
                                       *ptrs(a, ("y", "scale", "residual_out")), None)
    check_pairs(("y", "residual_out"), norm)
    for group in (0, 128):
        check_pairs(("y", "residual_out"), norm, out=1, group=group, scale=0x7E0000000000)
        f = distinct(("y", "scale", "residual_out"))
        for other in ("y", "residual_out"):
            assert norm(out=1, group=group, **{**f, "scale": f[other]}) == 1
            assert norm(out=1, group=group, **{**f, other: f["scale"]}) == 1

    def prep(**kw):
        a = {**apart("q", "k", "wq", "wk", "qh", "kh", "dq", "dk", "dqh", "dkh"), **kw}
        return mesa.lib().mesa_qk_preprocess_bwd(
            2, 2, 8, 128, 4, 1, *ptrs(a, ("q", "k", "wq", "wk", "qh", "kh")), ctypes.c_float(1e-6),
            *ptrs(a, ("dq", "dk", "dqh", "dkh", "dqr", "dkr", "dwq", "dwk", "dqhist", "dkhist", "workspace")), 1 << 40, None)
    check_pairs(("dqr", "dkr", "dwq", "dwk", "dqhist", "dkhist", "workspace"), prep)


@pytest.mark.parametrize("T", [1, 2, 130])
def test_gradient_slices_that_cut_into_one_another_are_refused(T):
    """dx, dga and dgi as slices of one wider tensor: refused where a row of one reaches into a row of another,
    before or behind it, also between the last row of one and the first of the other."""
    B, D, ld = 2, 104, 400                       # bf16: rows of 208 bytes, 800 apart
    at = 0x7E0000000000
    whole = dict(B=B, T=T, D=D, ld=D, ld_grad=ld)
    ok = dict(dx=at, dga=at + 208, dgi=at + 416)
    for name in ok:
        for other in ok:
            if other != name:
                for by in (16, 192, -16, -192, 800 + 16, 800 - 192, -800 + 16, -800 - 192):
                    if abs(by) < 800 or B * T > 2:
                        assert lru_bwd(**whole, **{**ok, name: ok[other] + by}) == 1, (name, other, by)
    rows = B * T
    last = (rows - 1) * 800
    assert lru_bwd(**whole, **{**ok, "dgi": ok["dx"] + last + 192}) == 1     # only the last row of dx and the first of dgi
    assert lru_bwd(**whole, **{**ok, "dgi": ok["dx"] - last - 192}) == 1
