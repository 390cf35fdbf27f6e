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
    (dict(B=1 << 20, T=1 << 20, ld=1 << 20), 2), (dict(B=1 << 30, T=64, D=1000, ld=1000), 2),
]


@pytest.mark.parametrize("kw,expect", BAD_LRU)
def test_lru_rejects_bad_descriptors(kw, expect):
    d = lru_desc(**kw)
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
    assert call_lru_bwd(d, ld_grad=2 ** 31 - 1, workspace=0) == 4
    assert call_lru_bwd(lru_desc(T=1 << 20), ld_grad=1 << 20) == 2
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
    assert call(c=0.0) == 1
    assert call(dtype=5) == 1
    assert call(N=0) == 0  # nothing to do, nothing launched
    for name in ("x", "ga", "gi", "lam", "h", "y"):
        assert call(**{name: 0}) == 1
        assert call(**{name: FAKE + 2}) == 3
