"""The gated linear recurrence where values leave the ordinary range: infinities and NaN
in valid rows, parameters and states, against what the definition gives.  Needs an MI355X.
"""
import numpy as np
import pytest
import torch

from oracle.block_oracle import lru_backward, lru_forward, lru_step
from test_regression_sequence_amd import mesa

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mesa.lib()


def draw(B, T, D, dtype=torch.float32, seed=0):
    gen = torch.Generator().manual_seed(seed)
    d = {k: torch.randn(B, T, D, generator=gen).to(dtype) for k in ("x", "ga", "gi", "dy")}
    d["lam"] = torch.rand(D, generator=gen) * 6 - 9
    d["h0"], d["d_hfinal"] = torch.randn(B, D, generator=gen), torch.randn(B, D, generator=gen)
    return d


def run(d, lengths=None, c=8.0):
    t = {k: v.cuda() for k, v in d.items()}
    if lengths is not None:
        lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    args, kw = (t["x"], t["ga"], t["gi"], t["lam"]), dict(c=c, h0=t["h0"], lengths=lengths)
    r = mesa.lru_fwd(*args, return_state=True, **kw)
    r.update(mesa.lru_bwd(*args, t["dy"], d_hfinal=t["d_hfinal"], state_grads=True, **kw))
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in r.items()}


# one tile of 8 tokens, of 32, of 64 (backward), of 128 (forward 64), and several tiles
TILES = [(7, 5), (20, 13), (50, 41), (90, 70), (700, 451)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,n", TILES)
def test_rows_behind_a_length_are_zeros_whatever_the_valid_ones_hold(T, n, dtype):
    """Infinities and NaN in the last valid row, in an earlier one, in the initial state and in the
    final state's gradient: rows behind the length are zeros, other channels and sequences have
    the bits of a call without them."""
    B, D, hit = 3, 70, 37
    lengths = [T, n, n - 1]
    clean = run(draw(B, T, D, dtype), lengths)
    for key, at, bad in [(k, t, v) for k in ("x", "ga", "gi", "dy") for t in (n - 1, 1) for v in (NAN, INF, -INF)] + \
                        [(k, None, v) for k in ("h0", "d_hfinal") for v in (NAN, INF)]:
        d = draw(B, T, D, dtype)
        if at is None:
            d[key][1, hit] = bad
        else:
            d[key][1, at, hit] = bad
        r = run(d, lengths)
        for name in ("y", "dx", "dga", "dgi"):
            for b, m in enumerate(lengths):
                assert (r[name][b, m:] == 0).all(), (key, at, bad, name, b)
        for name in r:
            keep = torch.ones_like(r[name], dtype=torch.bool)
            keep[(hit,) if name == "dlam" else (1, Ellipsis, hit)] = False
            assert torch.equal(r[name][keep], clean[name][keep]), (key, at, bad, name)


@pytest.mark.parametrize("c", [2.5e38, float(np.finfo(np.float32).max)])
def test_largest_decay_scales(c):
    """c up to the largest float: where softplus(lam) is 0 in fp32 the state stays, elsewhere every token starts
    anew, y = sigmoid(gi) x; nothing is NaN."""
    d = draw(2, 200, 5, seed=1)
    d["lam"] = torch.tensor([-INF, -1e30, -200.0, 2.0, INF])
    r = run(d, c=c)
    assert all(torch.isfinite(v).all() for v in r.values())
    assert torch.equal(r["y"][..., :3], d["h0"][:, None, :3].expand(-1, 200, -1))
    assert torch.equal(r["h_final"][:, :3], d["h0"][:, :3])
    assert not any(r[k][..., :3].any() for k in ("dx", "dga", "dgi"))
    want = torch.sigmoid(d["gi"].double()) * d["x"].double()
    assert ((r["y"].double() - want)[..., 3:].abs() <= 16 * E * want[..., 3:].abs()).all()
    h = d["h0"].cuda()
    y = mesa.lru_step(*(d[k][:, 0].contiguous().cuda() for k in ("x", "ga", "gi")), d["lam"].cuda(), h, c=c)["y"].cpu()
    assert torch.equal(y[:, :3], d["h0"][:, :3]) and ((y.double() - want[:, 0])[:, 3:].abs() <= 16 * E * want[:, 0, 3:].abs()).all()


@pytest.mark.parametrize("T", [7, 20, 300])
def test_large_inputs_behind_closed_gates(T):
    """A gate closed in fp32 (a = 1) lets nothing in, whatever x holds: no gradient reaches x, ga, gi or lam through
    it.  One that is barely open (t = -log2(a) of 1e-37 .. 1e-30) has sigmoid(gi) x / m far beyond fp32 but a finite
    v = -log(a) (a^2 / m) sigmoid(gi) x g.

    The bound: -log(a) = ln2 t carries (2 |ga| + 16) e of sigmoid, rate and product, m half as much, the products
    below 16 e together; the state is left out of v (h0 = 0 and inputs of at most m x)."""
    B, D = 2, 8
    d = draw(B, T, D, seed=2)
    d["h0"].zero_()
    big = torch.tensor([1e20, -3e38, 1e30, 3e25])[torch.arange(T) % 4][None, :, None]
    d["x"] = big.expand(B, T, D).clone()
    d["ga"][..., :2] = -200.0
    d["ga"][..., 2:4] = -INF
    r = run(d)
    for k in ("y", "dx", "dga", "dgi"):
        assert not r[k][..., :4].any(), k
    assert not r["dlam"][:4].any() and not r["h_final"][:, :4].any()

    d = draw(B, T, D, seed=3)
    d["h0"].zero_()
    d["d_hfinal"].zero_()
    d["lam"] = torch.full((D,), -6.0)
    d["x"] = torch.full((B, T, D), 4e22)
    d["ga"] = -torch.linspace(66, 80, D).expand(B, T, D).clone()
    r = run(d)
    n = {k: v.numpy() for k, v in d.items()}
    ref = lru_backward(*(n[k] for k in ("x", "ga", "gi", "lam", "dy")), c=8.0, h0=n["h0"], d_hfinal=n["d_hfinal"])
    # the sum of dy up to the token's own carries T e of its magnitudes
    size = lru_backward(*(n[k] for k in ("x", "ga", "gi", "lam")), np.abs(n["dy"]), c=8.0, h0=n["h0"], d_hfinal=n["d_hfinal"])
    assert np.isfinite(ref["dga"]).all() and np.abs(ref["dga"]).max() > 1
    for k in ("dx", "dga", "dgi"):
        tol = (1.5 * (2 * 80 + 16) + 16 + 2 * T) * E * np.abs(size[k]) + 1e-30
        assert (np.abs(r[k].numpy() - ref[k]) <= tol).all(), k


def masks(r, ref, clean, hit):
    """NaN where the definition has it and nowhere else; other channels keep their bits."""
    for name in r:
        assert np.array_equal(np.isnan(r[name].float().numpy()), np.isnan(ref[name])), name
        keep = torch.ones_like(r[name], dtype=torch.bool)
        keep[..., hit] = False
        assert torch.equal(r[name][keep], clean[name][keep]), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,n", TILES)
def test_nan_reaches_what_depends_on_it(T, n, dtype):
    """A NaN in lam, in an element of x, ga, gi or dy, or in a state: forward and backward give NaN exactly where
    the definition does."""
    B, D, hit = 2, 66, 65
    lengths = [n, T]
    clean = run(draw(B, T, D, dtype), lengths)
    for key, at in [("lam", (hit,)), ("h0", (0, hit)), ("d_hfinal", (0, hit))] + \
                   [(k, (0, t, hit)) for k in ("x", "ga", "gi", "dy") for t in (0, n // 2, n - 1)]:
        d = draw(B, T, D, dtype)
        d[key][at] = NAN
        r = run(d, lengths)
        a = {k: v.float().numpy() for k, v in d.items()}
        args, kw = [a[k] for k in ("x", "ga", "gi", "lam")], dict(c=8.0, h0=a["h0"], lengths=lengths)
        with np.errstate(invalid="ignore"):
            ref = lru_forward(*args, **kw)
            ref.update(lru_backward(*args, a["dy"], d_hfinal=a["d_hfinal"], **kw))
        assert any(np.isnan(ref[k]).any() for k in r), key
        masks(r, ref, clean, hit)


@pytest.mark.parametrize("key", ["lam", "x", "ga", "gi", "h0"])
def test_nan_in_a_step(key):
    N, D, hit = 3, 66, 9
    d = draw(N, 1, D, seed=4)
    v = d[key]
    v[(hit,) if key == "lam" else (1, hit) if key == "h0" else (1, 0, hit)] = NAN
    h = d["h0"].cuda()
    y = mesa.lru_step(*(d[k][:, 0].contiguous().cuda() for k in ("x", "ga", "gi")), d["lam"].cuda(), h)["y"].cpu()
    with np.errstate(invalid="ignore"):
        ref = lru_step(*(d[k][:, 0].numpy() for k in ("x", "ga", "gi")), d["lam"].numpy(), d["h0"].numpy())
    assert np.isnan(ref).any()
    assert np.array_equal(np.isnan(y.numpy()), np.isnan(ref)) and np.array_equal(np.isnan(h.cpu().numpy()), np.isnan(ref))
