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
