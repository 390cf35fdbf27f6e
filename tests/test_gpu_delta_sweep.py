"""Gated delta rule on the GPU against the fp64 oracle over seeded mixed configurations: types, heads that
share keys, sizes, lengths from none to several segments, layouts, states, gates.  Needs an MI355X."""
import numpy as np
import pytest
import torch

from delta_helpers import check_backward, check_forward, draw, to_dev
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def configuration(seed):
    rng = np.random.default_rng([77, seed])
    Hk = int(rng.integers(1, 4))
    H = Hk * int(rng.integers(1, 4))
    B = int(rng.integers(1, 5))
    T = int(rng.choice([rng.integers(1, 65), rng.integers(65, 400), rng.integers(400, 1500)]))
    c = dict(B=B, H=H, Hk=Hk, T=T, dk=int(rng.choice([32, 64, 128])), dv=16 * int(rng.integers(1, 13)),
             dtype=torch.bfloat16 if rng.integers(2) else torch.float32, gates=str(rng.choice(["usual", "slow", "fast"])),
             s0=bool(rng.integers(2)))
    if rng.integers(2):
        c["lengths"] = rng.integers(-1, T + 3, B)
    return c, str(rng.choice(["heads", "tokens", "slices"])), bool(rng.integers(2))


@pytest.mark.parametrize("seed", range(40))
def test_sweep(seed):
    c, layout, kept = configuration(seed)
    a = draw(seed=seed, **c)
    t = to_dev(a, c["dtype"], layout)
    args = [t[n] for n in ("q", "k", "v", "gamma", "beta")]
    ws = None
    if kept:
        ws = torch.empty(mesa.delta_workspace_bytes(*args, keep_states=True), device="cuda", dtype=torch.uint8).fill_(0xFF)
    r = mesa.delta_fwd(*args, s0=t["s0"], lengths=t["lengths"], return_state=True, keep_states=kept, workspace=ws)
    check_forward(r, a, c["dtype"], walks=2)
    g = mesa.delta_bwd(*args, t["d_o"], s0=t["s0"], lengths=t["lengths"], d_sfinal=t["d_sfinal"], state_grads=True,
                       workspace=ws, states_in_workspace=kept)
    check_backward(g, a, c["dtype"], walks=2)
