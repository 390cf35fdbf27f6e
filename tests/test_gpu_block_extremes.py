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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,T", [(16, 9), (64, 100), (128, 1), (128, 1500)])
def test_nan_in_a_row_reaches_every_gradient_through_its_norm(d, T, dtype):
    """A NaN in a raw row, its history, a tap or an incoming gradient: NaN exactly where the definition has it."""
    B, H, W = 2, 2, 4
    rng = np.random.default_rng(d + T)

    def half(a):
        return torch.from_numpy(a.astype(np.float32)).to(dtype)

    clean = dict(x=half(rng.standard_normal((B, H, T, d))), hist=half(rng.standard_normal((B, H, W - 1, d))),
                 w=torch.from_numpy(rng.standard_normal((H, d, W)).astype(np.float32)),
                 d=torch.from_numpy(rng.standard_normal((B, H, T, d)).astype(np.float32)))
    spots = [("x", (1, 0, t, 3)) for t in {0, T // 2, T - 1}] + [("hist", (1, 0, W - 2, 5)), ("w", (0, 7, 1)), ("d", (1, 0, T // 2, 2))]
    for key, at in spots:
        a = {k: v.clone() for k, v in clean.items()}
        a[key][at] = float("nan")
        t, c = {k: v.cuda() for k, v in a.items()}, {k: v.cuda() for k, v in clean.items()}
        # the NaN in the queries only: the keys are clean
        r = mesa.qk_preprocess_bwd(t["x"], c["x"], t["w"], c["w"], t["d"], c["d"], q_hist=t["hist"], k_hist=c["hist"],
                                   history_grads=True)
        n = {k: v.float().numpy() for k, v in a.items()}
        with np.errstate(invalid="ignore"):
            ref = qk_preprocess_backward(n["x"], n["w"], n["d"], n["hist"])
        for got, want in (("dq_raw", "dx"), ("dw_q", "dw"), ("dq_hist", "dhist")):
            assert np.isnan(ref["dw"]).any()
            assert np.array_equal(np.isnan(r[got].float().cpu().numpy()), np.isnan(ref[want])), (key, at, got)
        for got in ("dk_raw", "dw_k", "dk_hist"):
            assert torch.isfinite(r[got]).all(), (key, at, got)
