"""Gated delta rule and clipping where offsets pass 2^31 and 2^32.  Needs an MI355X."""
import math

import pytest
import torch

from test_regression_sequence_amd import mesa
from test_gpu_delta_calls import BF16, INPUTS, equal, inputs, train, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def test_strides_behind_2_to_the_31():
    """Sequences 2^31 + 64 elements apart, inputs and outputs."""
    a = inputs(1, 2, 3, 3, 150, 64, 64)
    want = train(a)
    far = (1 << 31) + 64
    n = a["v"][0].numel()

    def spread(base, slot):
        return base.as_strided(a["v"].shape, (far, 150 * 64, 64, 1), slot * n)
    base, outs = (torch.empty(far + 4 * n, device="cuda", dtype=BF16) for _ in range(2))
    b = dict(a)
    for i, m in enumerate(("q", "k", "v", "d_o")):
        b[m] = spread(base, i)
        b[m].copy_(a[m])
    out = {m: spread(outs, i) for i, m in enumerate(("o", "dq", "dk", "dv"))}
    equal(want, train(b, out=out))


def test_token_strides_at_their_limit():
    a = inputs(2, 1, 2, 2, 130, 32, 32)
    want = train(a)
    far = 1 << 20
    base, outs = (torch.empty(130 * far, device="cuda", dtype=BF16) for _ in range(2))

    def spread(base, slot):
        return base.as_strided(a["v"].shape, (0, 32, far, 1), slot * 64)
    b = dict(a)
    for i, m in enumerate(("q", "k", "v", "d_o")):
        b[m] = spread(base, i)
        b[m].copy_(a[m])
    out = {m: spread(outs, i) for i, m in enumerate(("o", "dq", "dk", "dv"))}
    equal(want, train(b, out=out))


def test_a_workspace_whose_parts_pass_2_to_the_31_elements():
    """131072 chunks' states of 128 x 128: the last sequences against a call of their own (of as many heads as
    let walks go the same way)."""
    B, H, T, d = 32, 32, 8192, 128
    last = inputs(3, B // 2, H, H, T, d, d)
    a = {m: torch.cat([t, t]) for m, t in last.items()}
    want = train(last, workspace(last))
    ws = workspace(a)
    assert ws.numel() > (1 << 33) * 3
    got = train(a, ws)
    equal(want, {m: t[B // 2:] for m, t in got.items()})
    equal(want, {m: t[:B // 2] for m, t in got.items()})


def test_steps_of_states_behind_2_to_the_31():
    N, H, d = 4200, 32, 128
    g = torch.Generator(device="cuda").manual_seed(4)
    a = inputs(5, 8, H, H, 1, d, d)
    state = torch.randn((N, H, d, d), generator=g, device="cuda")
    idx = torch.arange(N, device="cuda") % 8
    x = [a[m][:, :, 0].index_select(0, idx) for m in INPUTS]
    tail = state[-8:].clone()
    want = mesa.delta_step(*(t[-8:].contiguous() for t in x), tail)["o"]
    got = mesa.delta_step(*x, state)["o"]
    assert torch.equal(got[-8:], want) and torch.equal(state[-8:], tail)


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_clipping_a_tensor_of_more_than_2_to_the_32_elements(dtype):
    n = (1 << 32) + 77
    x = torch.zeros(n, device="cuda", dtype=dtype)
    at = torch.tensor([0, (1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, n - 1], device="cuda")
    x[at] = 2.0
    r = mesa.grad_clip([x, torch.ones(1, device="cuda")], 1.0)
    norm = math.sqrt(4 * 6 + 1)
    assert abs(float(r["norm"]) - norm) <= 2.0 ** -23 * norm
    want = torch.tensor(2 / (norm + 1e-6), dtype=torch.float64).to(dtype)
    half = 2.0 ** -8 if dtype is BF16 else 2.0 ** -22
    assert bool(((x[at].double() / want.double() - 1).abs() <= half).all())
    assert int(torch.count_nonzero(x.view(torch.uint8 if dtype is BF16 else torch.int32))) <= 12
