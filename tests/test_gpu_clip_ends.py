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
