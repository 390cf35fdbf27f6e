"""Host-side validation of the gated delta rule and of clipping (CPU only).

Every call here fails validation before the first launch.
"""
import ctypes

import pytest

from test_regression_sequence_amd import mesa

P = ctypes.c_void_p
STEP = 0x10000000
IN = ("q", "k", "v", "gamma", "beta", "s0", "lengths")
OUT = ("dq", "dk", "dv", "dgamma", "dbeta", "ds0")


def apart(*names, base=0x7F0000000000):
    """Distinct fake ranges, far apart, 16-byte aligned, never dereferenced."""
    return {n: base + i * STEP for i, n in enumerate(names)}


def heads(H, T, d):
    return mesa.Rows(H * T * d, T * d, d)


def tokens(H, T, d, wide=None):
    row = wide or H * d
    return mesa.Rows(T * row, d, row)


def desc(B=2, H=4, Hk=2, T=130, dk=64, dv=48, dtype=1, **kw):
    rows = dict(q=heads(Hk, T, dk), k=heads(Hk, T, dk), v=heads(H, T, dv), o=heads(H, T, dv), gamma=heads(H, T, 1),
                beta=heads(H, T, 1))
    rows.update(kw)
    return mesa.DeltaDesc(B, H, Hk, T, dk, dv, dtype, *[rows[n] for n in ("q", "k", "v", "o", "gamma", "beta")])


def grad_rows(d, **kw):
    rows = dict(d_o=heads(d.H, d.T, d.dv), dq=heads(d.Hk, d.T, d.dk), dk=heads(d.Hk, d.T, d.dk), dv=heads(d.H, d.T, d.dv),
                dgamma=heads(d.H, d.T, 1), dbeta=heads(d.H, d.T, 1))
    rows.update(kw)
    return mesa.DeltaGradRows(*[rows[n] for n in ("d_o", "dq", "dk", "dv", "dgamma", "dbeta")])


def ptr(v):
    return P(v) if v else None


def need(d, keep):
    return mesa.lib().mesa_delta_workspace_bytes(ctypes.byref(d), keep)


def fwd(d, keep=0, wbytes=1 << 50, **kw):
    a = {**apart(*IN, "o", "s_final", "workspace"), **kw}
    return mesa.lib().mesa_delta_fwd(ctypes.byref(d), *[ptr(a[n]) for n in IN + ("o", "s_final")], keep,
                                     ptr(a["workspace"]), wbytes, None)


def bwd(d, rows=None, flag=0, wbytes=1 << 50, **kw):
    a = {**apart(*IN, "d_o", "d_sfinal", *OUT, "workspace"), **kw}
    rows = grad_rows(d) if rows is None else rows
    return mesa.lib().mesa_delta_bwd(ctypes.byref(d), ctypes.byref(rows), *[ptr(a[n]) for n in IN + ("d_o", "d_sfinal") + OUT],
                                     flag, ptr(a["workspace"]), wbytes, None)


def step(d, **kw):
    a = {**apart("q", "k", "v", "gamma", "beta", "state", "o"), **kw}
    return mesa.lib().mesa_delta_step(ctypes.byref(d), *[ptr(a[n]) for n in ("q", "k", "v", "gamma", "beta", "state", "o")], None)


BAD = [(dict(B=0), 1), (dict(H=0), 1), (dict(Hk=0), 1), (dict(H=3), 1), (dict(T=-1), 1), (dict(dk=0), 1), (dict(dv=0), 1),
       (dict(dtype=2), 1), (dict(q=mesa.Rows(-64, 64, 64)), 1), (dict(gamma=mesa.Rows(0, 0, -1)), 1),
       (dict(beta=mesa.Rows(0, (1 << 40) + 1, 0)), 1), (dict(dk=16), 2), (dict(dk=96), 2), (dict(dk=256), 2), (dict(dv=24), 2),
       (dict(dv=1040), 2), (dict(B=1 << 20, H=4, T=64, dv=64), 0), (dict(B=1 << 20, H=4, T=65, dv=64), 2),
       (dict(B=1 << 20, H=4, T=1, dv=80), 2), (dict(B=2 ** 31 - 1, H=2 ** 31 - 2, T=2 ** 31 - 1, **{n: mesa.Rows(8, 8, 8) for n in ("q", "k", "v", "o", "gamma", "beta")}), 2)]


@pytest.mark.parametrize("kw,expect", BAD)
def test_descriptors(kw, expect):
    d = desc(**kw)
    if expect == 0:  # the largest: accepted up to the workspace
        assert fwd(d, workspace=0) == 4 and bwd(d, workspace=0) == 4 and need(d, 0) > 0
        return
    assert fwd(d) == expect and bwd(d) == expect
    assert need(d, 0) == need(d, 1) == 0
    if "T" not in kw:
        assert step(desc(**{**kw, "T": 1})) == expect


@pytest.mark.parametrize("name", ["d_o", "dq", "dk", "dv", "dgamma", "dbeta"])
def test_gradient_strides(name):
    d = desc()
    assert bwd(d, grad_rows(d, **{name: mesa.Rows(-8, 8, 8)})) == 1
    if name != "d_o":
        assert bwd(d, grad_rows(d, **{name: mesa.Rows(0, 0, 0)})) == 1          # rows over one another
    if name in ("dq", "dk", "dv"):
        assert bwd(d, grad_rows(d, **{name: mesa.Rows(4 * 130 * 64, 130 * 64, 32)})) == 1
    assert bwd(d, grad_rows(d, **{name: mesa.Rows(1 << 28, 64, (1 << 20) + 8)})) == 2
    if name in ("d_o", "dq", "dk", "dv"):
        assert bwd(d, grad_rows(d, **{name: mesa.Rows(1 << 20, 1 << 17, 129 + 3)})) == 3


@pytest.mark.parametrize("name", ["q", "k", "v", "o", "gamma", "beta"])
def test_strides(name):
    """The largest strides pass up to the workspace, larger ones are refused, and those that no index uses do not matter."""
    H, Hk, T = 4, 2, 130
    ok = mesa.Rows(1 << 36, 1 << 30, 1 << 20)
    d = desc(H=H, Hk=Hk, T=T, **{name: ok})
    f = {n: (i + 1) << 44 for i, n in enumerate((*IN, "o", "s_final", "workspace"))}
    assert fwd(d, **{**f, "workspace": 0}) == 4
    assert fwd(desc(**{name: mesa.Rows(1 << 36, 1 << 30, (1 << 20) + 8)}), **f) == 2
    assert fwd(desc(**{name: mesa.Rows((1 << 36) + 8, 1 << 30, 1 << 20)}), **f) == 1
    assert fwd(desc(B=1, T=1, **{name: mesa.Rows(3, 1 << 30, 1 << 30)}), **{**f, "workspace": 0}) == 4


def test_missing_and_misaligned():
    d = desc()
    small, big = need(d, 0), need(d, 1)
    assert 0 < small < big
    assert need(d, 2) == need(d, -1) == 0
    for n in ("q", "k", "v", "gamma", "beta", "o"):
        assert fwd(d, **{n: 0}) == 1, n
    for n in ("q", "k", "v", "gamma", "beta", "d_o", "dq", "dk", "dv", "dgamma", "dbeta"):
        assert bwd(d, **{n: 0}) == 1, n
    for n in ("q", "k", "v", "s0", "lengths", "o", "s_final", "workspace"):
        assert fwd(d, **{n: 0x7F0000000008}) == 3, n
    for n in ("q", "k", "v", "s0", "lengths", "d_o", "d_sfinal", "dq", "dk", "dv", "ds0", "workspace"):
        assert bwd(d, **{n: 0x7F0000000008}) == 3, n
    for n in ("gamma", "beta"):
        assert fwd(d, **{n: 0x7F0000000002}) == 3 and bwd(d, **{n: 0x7F0000000001}) == 3, n
    for n in ("dgamma", "dbeta"):
        assert bwd(d, **{n: 0x7F0000000002}) == 3, n
    for n in ("q", "k", "v", "o"):
        assert fwd(desc(**{n: mesa.Rows(1 << 20, 1 << 17, 131 * 4)})) == 3, n
    assert fwd(d, keep=2) == fwd(d, keep=-1) == bwd(d, flag=2) == bwd(d, flag=-1) == 1
    assert fwd(d, workspace=0) == bwd(d, workspace=0) == 4
    assert fwd(d, wbytes=small - 1) == fwd(d, keep=1, wbytes=big - 1) == bwd(d, wbytes=big - 1) == 4
    assert fwd(desc(o=mesa.Rows(0, 48, 48))) == 1                                 # output rows over one another
    assert fwd(desc(o=mesa.Rows(4 * 130 * 48, 130 * 48, 32))) == 1
    assert mesa.lib().mesa_delta_fwd(None, *[None] * 9, 0, None, 0, None) == 1
    assert mesa.lib().mesa_delta_bwd(ctypes.byref(d), None, *[P(0x10000)] * 15, 0, None, 0, None) == 1


def test_step():
    d = desc(T=1)
    for n in ("q", "k", "v", "gamma", "beta", "state", "o"):
        assert step(d, **{n: 0}) == 1, n
    for n in ("q", "k", "v", "state", "o"):
        assert step(d, **{n: 0x7F0000000008}) == 3, n
    assert step(d, gamma=0x7F0000000002) == 3
    assert step(desc(T=2)) == 1 and step(desc(T=0)) == 1
    f = apart("q", "k", "v", "gamma", "beta", "state", "o")
    for n in ("q", "k", "v", "gamma", "beta"):
        assert step(d, state=f[n]) == 1 and step(d, o=f[n]) == 1, n
    assert step(d, o=f["state"] + 16) == 1


def test_shared_memory():
    d = desc()
    f = apart(*IN, "o", "s_final", "workspace")
    for keep in (0, 1):
        for o in ("o", "s_final", "workspace"):
            for i in IN:
                if (o, i) != ("s_final", "s0"):
                    assert fwd(d, keep=keep, **{o: f[i]}) == 1, (o, i)
            for other in ("o", "s_final", "workspace"):
                if other != o:
                    assert fwd(d, keep=keep, **{o: f[other] + 16}) == 1, (o, other)
    for o in ("o", "workspace"):  # s_final over s0 permits no other
        assert fwd(d, s_final=f["s0"], **{o: f["s0"]}) == 1
    assert fwd(d, s_final=f["s0"] + 16) == 1
    b = apart(*IN, "d_o", "d_sfinal", *OUT, "workspace")
    for o in OUT + ("workspace",):
        for i in IN + ("d_o", "d_sfinal"):
            if (o, i) != ("ds0", "d_sfinal"):
                assert bwd(d, **{o: b[i]}) == 1, (o, i)
        for other in OUT + ("workspace",):
            if other != o:
                assert bwd(d, **{o: b[other] + 16}) == 1, (o, other)
        if o != "ds0":
            assert bwd(d, ds0=b["d_sfinal"], **{o: b["d_sfinal"]}) == 1, o


@pytest.mark.parametrize("T", [1, 2, 130])
def test_gradient_slices_of_one_wider_tensor(T):
    """dq, dk and dv [B, T, heads, d] side by side in one tensor: accepted up to the workspace; one that reaches
    into another's rows is refused."""
    H = Hk = 2
    d = desc(H=H, Hk=Hk, T=T, dk=64, dv=64)
    row = 3 * 2 * 64 + 16
    r = tokens(H, T, 64, wide=row)
    rows = grad_rows(d, dq=r, dk=r, dv=r)
    at = 0x7E0000000000
    ok = dict(dq=at, dk=at + 2 * 128, dv=at + 2 * 256)
    assert bwd(d, rows, workspace=0, **ok) == 4
    for n in ok:
        for other in ok:
            if n != other:
                for by in (16, 240, -16, -240):
                    assert bwd(d, rows, **{**ok, n: ok[other] + by}) == 1, (n, other, by)


def clip(sizes, dtypes=None, max_norm=1.0, eps=1e-6, wbytes=1 << 20, grads=None, outs=None, norm=0x7D0000000000,
         scale=0x7D0000000010, workspace=0x7C0000000000, count=None):
    n = len(sizes)
    dtypes = [0] * n if dtypes is None else dtypes
    grads = [0x7F0000000000 + i * STEP for i in range(n)] if grads is None else grads
    outs = [0x7E0000000000 + i * STEP for i in range(n)] if outs is None else outs
    return mesa.lib().mesa_grad_clip(n if count is None else count, (P * n)(*grads), (P * n)(*outs), (ctypes.c_int64 * n)(*sizes),
                                     (ctypes.c_int * n)(*dtypes), max_norm, eps, ptr(norm), ptr(scale), ptr(workspace), wbytes, None)


def test_clip():
    inf, nan = float("inf"), float("nan")
    G, O = 0x7F0000000000, 0x7E0000000000
    for kw, expect in [
        (dict(count=-1), 1), (dict(dtypes=[0, 2]), 1), (dict(max_norm=-1.0), 1), (dict(max_norm=nan), 1), (dict(eps=0.0), 1),
        (dict(eps=inf), 1), (dict(eps=nan), 1), (dict(grads=[G, 0]), 1), (dict(outs=[0, O]), 1), (dict(norm=0), 1),
        (dict(grads=[G, G + 0x1002]), 3), (dict(outs=[O + 2, O + 0x2000]), 3), (dict(dtypes=[1, 1], outs=[O + 1, O + 0x2000]), 3),
        (dict(norm=0x7D0000000002), 3), (dict(scale=0x7D0000000012), 3), (dict(workspace=0x7C0000000008), 3),
        (dict(workspace=0), 4), (dict(wbytes=mesa.lib().mesa_grad_clip_workspace_bytes() - 1), 4),
        (dict(outs=[G + 4, O]), 1), (dict(outs=[O, O + 396]), 1), (dict(outs=[O, O]), 1), (dict(outs=[G + STEP, O]), 1),
        (dict(grads=[G, G + 200], outs=[G, O]), 1), (dict(grads=[G, G], outs=[G, G]), 1), (dict(norm=O + 4), 1),
        (dict(scale=G + 396), 1), (dict(workspace=O + 16), 1), (dict(norm=0x7C0000000010), 1), (dict(scale=0x7D0000000000), 1),
    ]:
        assert clip([100, 100], **kw) == expect, kw
    assert clip([-1, 4]) == 1
    assert clip([1 << 44, 1]) == 2
    assert clip([1] * 4097) == 2
    assert mesa.lib().mesa_grad_norm(0, None, None, None, None, P(0x10000), 1 << 20, None) == 1
    assert mesa.lib().mesa_grad_clip(2, None, None, None, None, 1.0, 1e-6, P(16), None, P(0x10000), 1 << 20, None) == 1
    # many tensors: the one that lies over another is found wherever it stands in the list
    n = 4096
    grads = [G + i * 4096 for i in range(n)]
    outs = [O + i * 4096 for i in range(n)]
    for i, j in ((0, 4095), (4095, 0), (2000, 2001)):
        assert clip([1024] * n, grads=grads, outs=outs[:i] + [outs[j] + 4] + outs[i + 1:]) == 1
        assert clip([1024] * n, grads=grads, outs=outs[:i] + [grads[j] + 4] + outs[i + 1:]) == 1
