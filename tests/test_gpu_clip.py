"""Global gradient norm and clipping on the GPU against the fp64 definition.  Needs an MI355X.

Squares are exact in 64 bits and n of them add up to n 2^-53: the norm is off by its
rounding to fp32, 2^-24.  The scale adds max_norm's and its own rounding (2^-24 each),
an output one product's and, in bf16, one rounding to it (2^-8).
"""
import math

import numpy as np
import pytest
import torch

from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def gradients(sizes, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(torch.bfloat16 if i % 3 == 1 else torch.float32)
            for i, n in enumerate(sizes)]


def check(grads, max_norm, r, before=None, eps=1e-6):
    before = grads if before is None else before
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in before))
    scale = min(1.0, max_norm / (norm + eps))
    assert abs(float(r["norm"]) - norm) <= 2.0 ** -23 * norm
    assert abs(float(r["scale"]) - scale) <= 3 * 2.0 ** -24 * scale
    for g, o in zip(before, r["grads"]):
        want = g.double() * scale
        half = (2.0 ** -8 if g.dtype is torch.bfloat16 else 0.0) + 5 * 2.0 ** -24
        assert o.dtype is g.dtype and bool(((o.double() - want).abs() <= half * want.abs()).all())


SIZES = [[1], [5], [8], [17, 0, 3], [8191, 8192, 8193], [100] * 7 + [1 << 20, 3], [4096, 77] * 60, [1000003, 65536 * 9 + 1]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("factor", [0.01, 0.999, 100.0])
def test_sizes(sizes, factor):
    grads = gradients(sizes, seed=len(sizes))
    bound = factor * math.sqrt(sum(sizes))
    outs = [torch.full_like(g, 7.0) for g in grads]
    kept = [g.clone() for g in grads]
    r = mesa.grad_clip(grads, bound, out=outs)
    check(grads, bound, r)
    assert all(torch.equal(g, k) for g, k in zip(grads, kept))
    assert abs(float(mesa.grad_norm(grads)["norm"]) - float(r["norm"])) == 0.0
    r = mesa.grad_clip(grads, bound)   # in place
    check(grads, bound, r, before=kept)
    assert all(torch.equal(g, o) for g, o in zip(grads, outs))


def test_tensors_at_any_address():
    flat = gradients([0, 0, 40000])[2]
    half = flat.to(torch.bfloat16)
    grads = [flat[1:1001], half[3:2006], flat[5003:5004], half[20001:33000], flat[10000:33333]]
    outs = [torch.empty(g.numel() + 1, device="cuda", dtype=g.dtype)[1:] for g in grads]
    check(grads, 10.0, mesa.grad_clip(grads, 10.0, out=outs))
    rest = flat.clone()
    mesa.grad_clip([flat[1:1001], flat[5003:5004]], 1.0)
    mask = torch.ones_like(flat, dtype=torch.bool)
    mask[1:1001] = mask[5003:5004] = False
    assert torch.equal(flat[mask], rest[mask])  # nothing beside the slices changes


def test_values_at_the_ends():
    huge = [torch.full((100,), 1e38, device="cuda"), torch.full((3,), -3e38, device="cuda")]
    r = mesa.grad_clip(huge, 1.0, out=[torch.empty_like(g) for g in huge])
    norm = math.sqrt(100 * 1e76 + 3 * 9e76)
    assert math.isinf(float(r["norm"])) or abs(float(r["norm"]) / norm - 1) < 1e-6
    for g, o in zip(huge, r["grads"]):
        assert bool(((o.double() * norm / g.double() - 1).abs() < 1e-6).all())  # the scale itself is 64-bit until rounded
    tiny = [torch.full((100,), 1e-38, device="cuda")]
    r = mesa.grad_clip(tiny, 1.0)
    assert abs(float(r["norm"]) / 1e-37 - 1) < 1e-6 and float(r["scale"]) == 1.0
    zero = [torch.zeros(33, device="cuda")]
    r = mesa.grad_clip(zero, 0.0)
    assert float(r["norm"]) == 0.0 and float(r["scale"]) == 0.0
    x = gradients([1000, 50])
    r = mesa.grad_clip(x, math.inf)
    assert float(r["scale"]) == 1.0
    for bad, norm_ok, scale_ok in ((math.nan, math.isnan, math.isnan), (math.inf, math.isinf, lambda v: v == 0.0)):
        x = gradients([1000, 50])
        x[1][7] = bad
        r = mesa.grad_clip(x, 1.0, out=[torch.empty_like(g) for g in x])
        assert norm_ok(float(r["norm"])) and scale_ok(float(r["scale"]))
        assert math.isnan(float(r["grads"][1][7]))
        assert bool(torch.isnan(r["grads"][0]).all() if math.isnan(bad) else (r["grads"][0] == 0).all())


def test_a_tensor_listed_twice_counts_twice():
    g = gradients([500])[0]
    outs = [torch.empty_like(g), torch.empty_like(g)]
    check([g, g], 1.0, mesa.grad_clip([g, g], 1.0, out=outs))
    with pytest.raises(mesa.MesaError):
        mesa.grad_clip([g, g], 1.0)


def test_refusals():
    g = gradients([64, 64])
    for call in (lambda: mesa.grad_clip([], 1.0), lambda: mesa.grad_clip(g, -1.0), lambda: mesa.grad_clip(g, math.nan),
                 lambda: mesa.grad_clip(g, 1.0, eps=0.0), lambda: mesa.grad_clip(g, 1.0, out=g[:1]),
                 lambda: mesa.grad_clip([g[0].half()], 1.0), lambda: mesa.grad_clip([g[0].cpu()], 1.0),
                 lambda: mesa.grad_clip([g[0][::2]], 1.0), lambda: mesa.grad_clip(g, 1.0, out=[g[1], g[0]]),
                 lambda: mesa.grad_clip([g[0], g[0][:8]], 1.0),
                 lambda: mesa.grad_clip(g, 1.0, workspace=torch.empty(16, device="cuda", dtype=torch.uint8))):
        with pytest.raises(mesa.MesaError):
            call()
