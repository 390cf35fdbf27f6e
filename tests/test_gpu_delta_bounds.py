"""Gated delta rule on the GPU: the sweep's configurations with the forward within the bound of its own walk: of one
walk where there are fewer than four chunks.  Needs an MI355X.

The bounds of delta_helpers take every stage's error relative to its result, but q.k is off by 2^-23 of |q||k| = 1,
however small it is itself, and where a head has a few tokens nothing larger may hide that: a head of two tokens whose
o is 0.0085 long was 2.0e-8 off, 2.3e-6 of it.  Token t reads u_j = beta_j w_j times that error from each token j of its
chunk, errors of different tokens in no common direction: 2^-23 sqrt(sum |u_j|^2) is added for o.
"""
import numpy as np
import pytest
import torch

from delta_helpers import draw, e32, to_dev
from oracle.delta_oracle import delta_forward
from test_gpu_delta_sweep import configuration
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "gamma", "beta")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


@pytest.mark.parametrize("seed", range(40, 80))
def test_bounds(seed):
    c, layout, _ = configuration(seed)
    walks = 1 if c["T"] <= 192 else 2
    a = draw(seed=seed, **c)
    t = to_dev(a, c["dtype"], layout)
    args = [t[n] for n in NAMES]
    r = mesa.delta_fwd(*args, s0=t["s0"], lengths=t["lengths"], return_state=True)
    want = delta_forward(*(a[n] for n in NAMES), s0=a["s0"], lengths=a["lengths"])
    e = e32(a, 12 * walks)
    size = lambda x: np.linalg.norm(x.reshape(x.shape[0], x.shape[1], -1), axis=-1)  # noqa: E731  of each head
    u = np.sum((a["beta"][..., None] * want["w"]) ** 2, -1)
    chunks = [np.cumsum(u[:, :, i:i + 64], -1) for i in range(0, u.shape[2], 64)]
    read = size(np.sqrt(np.concatenate(chunks, -1)))
    half = 2.0 ** -8 if c["dtype"] is torch.bfloat16 else 2.0 ** -24
    off = size(r["o"].double().cpu().numpy() - want["o"])
    assert np.all(off <= (e + half) * size(want["o"]) + 2.0 ** -23 * read), off / size(want["o"])
    assert np.all(size(r["s_final"].double().cpu().numpy() - want["s_final"]) <= e * size(want["s_final"]))
