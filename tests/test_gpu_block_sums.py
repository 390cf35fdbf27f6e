"""Sums over rows, tokens and sequences of the operators around the layer: their error does not grow
with the number of terms.  Equal rows make a sum in fp32 lose in one direction: S + t with S = n t is
rounded the same way for all S between two powers of two, by up to n e t (e = 2^-24), a relative
error of order n e at the end of a chain of n; 64-bit sums of short fp32 ones keep the short ones'.
Needs an MI355X.
"""
import numpy as np
import pytest
import torch

from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def normal(*shape, dtype=torch.float32, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def copies(v, n):
    return v.expand(n, *v.shape[1:]).contiguous()


@pytest.mark.parametrize("R,D,dtype,res", [(1 << 24, 16, "bf16", "bf16"), (1 << 22, 300, "bf16", "f32"),
                                           (1 << 20, 2500, "bf16", "bf16"), (1 << 18, 9000, "bf16", "bf16")])
def test_norm_weight_gradient_over_many_equal_rows(R, D, dtype, res):
    """dw = R dy n.  n = s r is off by (depth / 2 + 4) e with the row sum's depth min(D, 128) + 10; a lane adds at most
    64 rows in fp32, the rest is 64-bit: in all (64 + depth / 2 + 8) e."""
    t = {"bf16": torch.bfloat16, "f32": torch.float32}
    s, dy, w = normal(1, D, dtype=t[res], seed=1), normal(1, D, dtype=t[dtype], seed=2), 1 + 0.1 * normal(D, seed=3)
    dw = mesa.rmsnorm_bwd(copies(s, R), w, copies(dy, R), eps=1e-5)["dw"].double()
    sd = s[0].double()
    want = R * dy[0].double() * sd / torch.sqrt(sd.square().mean() + 1e-5)
    bound = (64 + 0.5 * (min(D, 128) + 10) + 8) * E * want.abs()
    assert ((dw - want).abs() <= bound).all(), float(((dw - want).abs() / want.abs()).max() / E)
