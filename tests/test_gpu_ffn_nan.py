"""NaNs in the gate of the feed-forward block: what depends on one is a NaN, and nothing else is."""
import math

import pytest

import sparse_top_lookup_gb300 as pk
from operators64 import ACTS

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
ID = {"silu": pk.PKM_ACT_SILU, "gelu": pk.PKM_ACT_GELU, "gelu_tanh": pk.PKM_ACT_GELU_TANH,
      "relu": pk.PKM_ACT_RELU}


def empty(*shape):
    return torch.empty(*shape, dtype=BF16, device="cuda")


def run(x, wg, wu, wd, act, dy=None):
    """y, g, u and with dy the gradients."""
    (B, dim), F = x.shape, wg.shape[0]
    y, g, u = empty(B, dim), empty(B, F), empty(B, F)
    ws = torch.empty(max(pk.pkm_gated_ffn_workspace_bytes(B, dim, F),
                         pk.pkm_gated_ffn_backward_workspace_bytes(B, dim, F)), dtype=torch.uint8,
                     device="cuda")
    pk.check(pk.pkm_gated_ffn(x, wg, wu, wd, B, dim, F, ID[act], ws, y, g, u), "forward")
    if dy is None:
        return y, g, u
    d = [torch.empty_like(t) for t in (x, wg, wu, wd)]
    pk.check(pk.pkm_gated_ffn_backward(x, wg, wu, wd, g, u, dy, B, dim, F, ID[act], ws, *d), "backward")
    return (y, g, u) + tuple(d)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("B", [3, 100, 300])
def test_a_nan_in_one_gate_weight_reaches_what_depends_on_it(act, B):
    dim, F = 64, 136
    gen = torch.Generator(device="cuda").manual_seed(B)
    x, wg, wu, wd, dy = (torch.randn(*s, device="cuda", generator=gen).to(BF16)
                         for s in ((B, dim), (F, dim), (F, dim), (dim, F), (B, dim)))
    want = run(x, wg, wu, wd, act, dy)
    wg[21, 5] = math.nan
    y, g, u, dx, dwg, dwu, dwd = run(x, wg, wu, wd, act, dy)
    rest = torch.arange(F, device="cuda") != 21
    assert bool(g[:, 21].isnan().all()) and torch.equal(g[:, rest], want[1][:, rest])
    assert bool(y.isnan().all()), "y"            # every output has a term of h[:, 21]
    assert bool(dx.isnan().all()), "dx"
    for n, t, w in (("dwg", dwg, want[4]), ("dwu", dwu, want[5]), ("dwd", dwd.T, want[6].T)):
        assert bool(t[21].isnan().all()), n
        assert torch.equal(t[rest], w[rest]), n


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("B", [100, 300])
def test_infinity_less_infinity_in_the_gate_is_a_nan(act, B):
    dim, F = 64, 136
    gen = torch.Generator(device="cuda").manual_seed(B)
    x, wg, wu, wd = (torch.randn(*s, device="cuda", generator=gen).to(BF16)
                     for s in ((B, dim), (F, dim), (F, dim), (dim, F)))
    x[:, 3], x[:, 4], wu[:, 3:5] = 1.0, 1.0, 0.0
    wg[7, 3], wg[7, 4] = math.inf, -math.inf
    y, g, u = run(x, wg, wu, wd, act)
    assert bool(g[:, 7].isnan().all()) and bool(u.isfinite().all()) and bool(y.isnan().all())
