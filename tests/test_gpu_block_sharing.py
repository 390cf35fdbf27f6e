"""Buffers of the operators around the layer that share an allocation without sharing memory are
accepted, those that share memory are refused by the binding.  Needs an MI355X.
"""
import pytest
import torch

from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,D", [(1, 1, 8), (2, 1, 24), (1, 2, 64), (3, 70, 72), (2, 300, 64)])
def test_inputs_and_gradients_as_sixths_of_one_tensor(B, T, D, dtype):
    """x, ga, gi and their gradients side by side, with nothing between them, equal dense calls bit for bit."""
    g = torch.Generator(device="cuda").manual_seed(1)
    wide = torch.randn(B, T, 6 * D, generator=g, device="cuda").to(dtype)
    lam, dy = torch.randn(D, generator=g, device="cuda") - 4, torch.randn(B, T, D, generator=g, device="cuda").to(dtype)
    part = [wide[..., i * D:(i + 1) * D] for i in range(6)]
    dense = [p.contiguous() for p in part[:3]]
    want = mesa.lru_bwd(*dense, lam, dy, state_grads=True)
    names = ("dx", "dga", "dgi")
    got = mesa.lru_bwd(*part[:3], lam, dy, state_grads=True, out=dict(zip(names, part[3:])))
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
    for p, q in zip(part, dense):
        assert torch.equal(p, q)


def test_outputs_back_to_back_in_one_buffer():
    """y, the final state and the workspace as neighbours: accepted; moved 16 bytes into one another: refused."""
    B, T, D = 2, 200, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    x, ga, gi = (torch.randn(B, T, D, generator=g, device="cuda") for _ in range(3))
    lam = torch.randn(D, generator=g, device="cuda") - 4
    need, ny, nh = mesa.lru_workspace_bytes(B, T, D, dtype=torch.float32), 4 * B * T * D, 4 * B * D
    buf = torch.empty(need + ny + nh, dtype=torch.uint8, device="cuda")

    def at(start, n):
        return buf[start:start + n]

    def views(y0, h0, w0):
        return dict(out={"y": at(y0, ny).view(torch.float32).view(B, T, D), "h_final": at(h0, nh).view(torch.float32).view(B, D)},
                    workspace=at(w0, need), return_state=True)

    want = mesa.lru_fwd(x, ga, gi, lam, return_state=True)
    for y0, h0, w0 in ((0, ny, ny + nh), (need + nh, need, 0), (nh, 0, nh + ny)):
        r = mesa.lru_fwd(x, ga, gi, lam, **views(y0, h0, w0))
        torch.cuda.synchronize()
        assert torch.equal(r["y"], want["y"]) and torch.equal(r["h_final"], want["h_final"])
    for y0, h0, w0 in ((16, ny, ny + nh), (0, ny - 16, ny + nh), (0, ny, ny + nh - 16), (need + nh - 16, 0, 16 + nh)):
        with pytest.raises(mesa.MesaError):
            mesa.lru_fwd(x, ga, gi, lam, **views(y0, h0, w0))
