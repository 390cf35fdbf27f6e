"""The norm and the preprocessing's gradient where factors leave the ordinary range, against the
fp64 oracle.  Needs an MI355X.
"""
import numpy as np
import pytest
import torch

from oracle.block_oracle import qk_preprocess_backward, rmsnorm
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


@pytest.mark.parametrize("D", [5, 100, 777, 2048, 5000])
@pytest.mark.parametrize("size,weight", [(1e-17, 1e25), (1e15, 1e-30), (1e-17, 1e-30), (1e15, 1e25)])
def test_norm_of_small_and_large_rows_with_large_and_small_weights(size, weight, D):
    """s / rms(s) is of order 1 whatever the row's size, so y is of the weights' order: finite where w / rms(s) is not,
    with all its bits where that is below the smallest float.  Bounds as in test_gpu_norm.py."""
    g = torch.Generator().manual_seed(D)
    x = torch.randn(4, D, generator=g) * size
    w = (torch.rand(D, generator=g) + 0.5) * weight
    rel = (0.5 * (min(D, 128) + 10) + 8) * E
    for group in (None, 0, 128):
        ref = rmsnorm(x.numpy(), w.numpy(), eps=1e-37, group=group)
        r = mesa.rmsnorm(x.cuda(), w.cuda(), eps=1e-37, quant_group=group)
        y = r["y"].float().cpu().numpy().astype(np.float64)
        if group is None:
            assert (np.abs(y - ref["y"]) <= (rel + E) * np.abs(ref["y"])).all()
        else:
            scale = r["scale"].cpu().numpy().astype(np.float64)
            assert (np.abs(scale - ref["scale"]) <= (rel + 2 * E) * ref["scale"]).all()
            v = ref["y"] / np.repeat(ref["scale"], group or D, axis=1)[:, :D]
            assert (np.abs(y - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) * (1 + 1e-5) + (2 * rel + 8 * E) * np.abs(v)).all()
