"""The feed-forward block's activations at single values, in both tails.

Weights and inputs are chosen so that every sum has one term that is not zero: g, u, h, dg and du reach
the outputs with no rounding but their own to bf16, at most 2^-8 of the value, and the arithmetic of the
activation in fp32.
"""
import math

import pytest

import sparse_top_lookup_gb300 as pk
import operators64
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


def gates(lo, hi, n):
    return torch.linspace(lo, hi, n, device="cuda").to(BF16).unique()


def act64(g, act):
    """act(g) and act'(g), good relative to themselves in the negative tail too."""
    if act != "gelu_tanh":
        return operators64.act64(g, act)
    c = 2 * math.sqrt(2 / math.pi)
    v = c * (g + 0.044715 * g ** 3)
    s, rest = torch.sigmoid(v), torch.sigmoid(-v)             # (1 + tanh(v / 2)) / 2, and 1 less it
    return g * s, s + g * s * rest * c * (1 + 0.134145 * g * g)


def one_by_one(values):
    """x, Wg, Wu, Wd with g = values (each in a token and a column of its own), u = 1."""
    n = values.numel()
    B, dim, F = n, 16, 8
    x = torch.zeros(B, dim, dtype=BF16, device="cuda")
    x[:, 0], x[:, 1] = values, 1.0
    wg, wu, wd = (torch.zeros(*s, dtype=BF16, device="cuda") for s in ((F, dim), (F, dim), (dim, F)))
    wg[0, 0], wu[0, 1], wd[2, 0] = 1.0, 1.0, 1.0
    return x, wg, wu, wd


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n", [90, 700])
def test_h_is_good_relative_to_itself_in_both_tails(act, n):
    # h = act(g): rounded to bf16 once (y's rounding then changes nothing); fp32's arithmetic: exponents of
    # up to 100 with 2^-24 relative in the argument, and a few ulp
    g = gates(-9.0, 20.0, n)
    y = run(*one_by_one(g), act)[0][:, 2].double()
    want = act64(g.double(), act)[0]
    off = (y - want).abs()
    assert bool((off <= want.abs() * (2.0 ** -8 + 2.0 ** -16)).all()), float((off / want.abs().clamp(
        min=1e-300)).max())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("n", [90, 700])
def test_du_and_dg_are_good_in_both_tails(act, n):
    # dh = 1: du = act(g), relative to itself; dg = act'(g), whose two terms may cancel: relative to
    # the larger, at most |act'| + |g| |act''|-like magnitudes below 2 (|act'| + |act(g)|)
    g = gates(-9.0, 20.0, n)
    x, wg, wu, wd = one_by_one(g)
    dy = torch.zeros_like(x)
    dy[:, 2] = 1.0
    dx = run(x, wg, wu, wd, act, dy)[3].double()
    a, da = act64(g.double(), act)
    assert bool(((dx[:, 1] - a).abs() <= a.abs() * (2.0 ** -8 + 2.0 ** -16)).all()), "du"
    assert bool(((dx[:, 0] - da).abs() <= da.abs() * 2.0 ** -8 + (da.abs() + a.abs()) * 2.0 ** -16).all()), "dg"
