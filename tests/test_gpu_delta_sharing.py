"""Gated delta rule on the GPU: inputs and outputs that lie between one another's rows in padded tensors, whose
rows are not at one stride from the first sequence's first to the last one's last.  Needs an MI355X."""
import pytest
import torch

from test_gpu_delta_calls import BF16, F32, INPUTS, equal, inputs, train
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def parts(layout, B, T, room, heads, d, dtype):
    """One tensor with room for more tokens, and its parts [B, heads, T, d] for each of `heads`."""
    n = sum(heads)
    if layout == "tokens":
        wide = torch.full((B, room, n, d), 7.0, device="cuda", dtype=dtype)
        at = wide[:, 1:1 + T].transpose(1, 2)
    else:
        wide = torch.full((B, n, room, d), 7.0, device="cuda", dtype=dtype)
        at = wide[:, :, 1:1 + T]
    return wide, list(torch.split(at, heads, 1))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2), (3, 1)])
def test_outputs_in_one_padded_tensor(H, Hk, layout, dtype):
    """dq, dk, dv and o side by side in a tensor with room for more tokens, dgamma and dbeta in another; q, k, v and d_o too."""
    B, T, d = 3, 70, 64
    a = inputs(1, B, H, Hk, T, d, d, dtype)
    want = train(a)
    grads, (dq, dk, dv, o) = parts(layout, B, T, 90, [Hk, Hk, H, H], d, dtype)
    gates, (dgamma, dbeta) = parts(layout, B, T, 77, [H, H], 1, F32)
    _, ins = parts(layout, B, T, 72, [Hk, Hk, H, H], d, dtype)
    b = dict(a)
    for n, t in zip(("q", "k", "v", "d_o"), ins):
        b[n] = t.copy_(a[n])
    out = dict(dq=dq, dk=dk, dv=dv, o=o, dgamma=dgamma[..., 0], dbeta=dbeta[..., 0])
    equal(want, train(b, out=out))
    for wide in (grads, gates):
        rest = wide.clone()
        (rest[:, 1:1 + T] if layout == "tokens" else rest[:, :, 1:1 + T]).fill_(7.0)
        assert bool((rest == 7).all())   # nothing beside them was written


def test_parts_of_a_prompt_into_one_tensor():
    """Two parts of a batch of prompts, outputs into their place beside the inputs of the same tensor."""
    B, H, T, d = 2, 2, 150, 32
    a = inputs(2, B, H, H, T, d, d)
    want = mesa.delta_fwd(*(a[n] for n in INPUTS), return_state=True)
    wide = torch.zeros((B, T, 4, H, d), device="cuda", dtype=BF16)
    q, k, v, o = (wide[:, :, i].transpose(1, 2) for i in range(4))
    for n, t in zip(("q", "k", "v"), (q, k, v)):
        t.copy_(a[n])
    state = torch.zeros((B, H, d, d), device="cuda")
    for lo, hi in ((0, 64), (64, 150)):  # (whole chunks, so the same sums)
        cut = [t[:, :, lo:hi] for t in (q, k, v, a["gamma"], a["beta"])]
        mesa.delta_fwd(*cut, s0=state, return_state=True, out={"o": o[:, :, lo:hi], "s_final": state})
    assert torch.equal(o, want["o"]) and torch.equal(state, want["s_final"])


def test_steps_into_slices():
    """One token of a batch whose rows lie in one padded tensor."""
    a = inputs(3, 5, 4, 2, 1, 64, 64)
    x = {n: t[:, :, 0].contiguous() for n, t in a.items() if n in INPUTS}
    s = a["s0"].clone()
    want = mesa.delta_step(*x.values(), s)["o"]
    wide = torch.zeros((5, 14, 64), device="cuda", dtype=BF16)
    q, k, v, o = wide[:, 0:2], wide[:, 2:4], wide[:, 5:9], wide[:, 9:13]
    for n, t in zip(("q", "k", "v"), (q, k, v)):
        t.copy_(x[n])
    s2 = a["s0"].clone()
    mesa.delta_step(q, k, v, x["gamma"], x["beta"], s2, out={"o": o})
    assert torch.equal(o, want) and torch.equal(s, s2)


def test_rows_that_are_shared_are_refused():
    """In the same padded tensors: one that reaches into another's rows, or into the next sequence's."""
    B, H, T, d = 3, 2, 70, 64
    a = inputs(4, B, H, H, T, d, d)
    args = [a[n] for n in INPUTS]
    wide = torch.zeros((B + 1, 90, 4, H * d), device="cuda", dtype=BF16)  # (room for rows that reach too far)

    def rows(token, at):
        return wide.view(-1).as_strided((B, H, T, d), (90 * 4 * H * d, d, 4 * H * d, 1), token * 4 * H * d + at)
    good = dict(dq=rows(3, 0), dk=rows(3, H * d), dv=rows(3, 2 * H * d))
    mesa.delta_bwd(*args, a["d_o"], out=good)
    for n, m in (("dq", "dk"), ("dk", "dv"), ("dv", "dq")):
        lo = {"dq": 0, "dk": H * d, "dv": 2 * H * d}[m]
        for token, at in ((3, lo), (3, lo + 8), (3, lo + H * d - 8), (3, lo - 8 if lo else 8), (12, lo), (72, lo + 56), (0, lo + 8)):
            with pytest.raises(mesa.MesaError):
                mesa.delta_bwd(*args, a["d_o"], out={**good, n: rows(token, at)})
