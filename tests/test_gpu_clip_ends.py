"""Clipping where norms, bounds and scales leave fp32's ordinary range.  Needs an MI355X."""
import math

import pytest
import torch

from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def some(dtype, n=1000, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("into", ["place", "outputs"])
def test_no_bound_and_infinite_gradients(into, dtype):
    """max_norm = infinity changes nothing: an infinite gradient gives the norm, a NaN is one everywhere."""
    for bad, scale in ((math.inf, 1.0), (-math.inf, 1.0), (math.nan, math.nan)):
        x = [some(dtype), some(dtype, 50, 2)]
        x[1][7] = bad
        kept = [g.clone() for g in x]
        r = mesa.grad_clip(x, math.inf, out=None if into == "place" else [torch.empty_like(g) for g in x])
        if math.isnan(bad):
            assert math.isnan(float(r["norm"])) and math.isnan(float(r["scale"]))
            assert all(bool(g.isnan().all()) for g in r["grads"])
        else:
            assert float(r["norm"]) == math.inf and float(r["scale"]) == scale
            assert all(torch.equal(g, k) for g, k in zip(r["grads"], kept))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [1e36, 1e38])
@pytest.mark.parametrize("bound", [1.0, 1e-3, 1e-6, 2.0 ** -126])
def test_scales_below_the_normal_numbers(bound, size, dtype):
    """Gradients near fp32's end, whose scale is subnormal or less: outputs are as near as any (the scale's rounding and a
    product's, 2^-24 each, in bf16 one to it, 2^-8), where they are normal numbers themselves."""
    x = [(some(F32) * size).to(dtype), torch.full((3,), -size, device="cuda", dtype=dtype)]
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in x))
    scale = bound / (norm + 1e-6)
    assert scale < 2.0 ** -116
    r = mesa.grad_clip(x, bound, out=[torch.empty_like(g) for g in x])
    half = (2.0 ** -8 if dtype is BF16 else 0.0) + 3 * 2.0 ** -24
    for g, o in zip(x, r["grads"]):
        want = g.double() * scale
        assert bool(((o.double() - want).abs() <= half * want.abs() + 2.0 ** -149 + (2.0 ** -134 if dtype is BF16 else 0.0)).all())
    assert abs(float(r["scale"]) - scale) <= 2.0 ** -23 * scale + 2.0 ** -150
    in_place = [g.clone() for g in x]
    mesa.grad_clip(in_place, bound)
    assert all(torch.equal(g, o) for g, o in zip(in_place, r["grads"]))


def test_bounds_are_taken_as_given():
    """The scale is bound / (norm + eps) in 64 bits, rounded once: a bound or eps of Python is not rounded to fp32 before."""
    x = [torch.tensor([3.0], device="cuda")]
    for i in range(1, 60):
        bound, eps = 0.1 * i / 3, 1e-6 * i
        want = torch.tensor(min(1.0, bound / (3.0 + eps)), dtype=torch.float64).float()
        assert float(mesa.grad_clip(x, bound, eps=eps, out=[torch.empty_like(x[0])])["scale"]) == float(want), (bound, eps)


def test_bounds_above_the_largest_float():
    x = [torch.full((100,), 3e38, device="cuda")]
    kept = x[0].double()
    r = mesa.grad_clip(x, 1e39)
    assert abs(float(r["scale"]) - 1 / 3) <= 2.0 ** -22
    assert bool((x[0].double() / kept * 3 - 1).abs().max() <= 2.0 ** -22)
