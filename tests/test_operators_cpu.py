"""The feed-forward block and the distillation loss without a GPU: the 64-bit forms that the GPU
tests compare with are pinned by differences and by torch's own gradients, and the C ABI refuses
bad arguments before any CUDA call."""
import ctypes
import math

import pytest

import sparse_top_lookup_gb300 as pk
from operators64 import ACTS, act64, distill64, ffn64, ffn_backward64

torch = pytest.importorskip("torch")
F64 = torch.float64


@pytest.fixture(scope="module")
def L():
    pk.build()
    return pk.lib()


# ------------------------------------------------------------------ the 64-bit forms

@pytest.mark.parametrize("act", ACTS)
def test_activation_slopes_are_differences(act):
    g = torch.linspace(-6, 6, 241, dtype=F64) + 0.0123
    e = 1e-5
    num = (act64(g + e, act)[0] - act64(g - e, act)[0]) / (2 * e)
    # central differences are off by e^2/6 times the third derivative (below 3 for all of
    # these) plus a rounding of 1e-16 * 6 / e
    assert (act64(g, act)[1] - num).abs().max() < 3 * e * e / 6 + 1e-15 * 6 / e


@pytest.mark.parametrize("act", ACTS)
def test_ffn_gradients_are_autograds(act):
    gen = torch.Generator().manual_seed(3)
    x, wg, wu, wd, dy = (torch.randn(*s, dtype=F64, generator=gen)
                         for s in ((5, 6), (7, 6), (7, 6), (6, 7), (5, 6)))
    leaves = [t.requires_grad_() for t in (x, wg, wu, wd)]
    ours = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
            "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh"),
            "relu": torch.relu}[act]
    y = (ours(x @ wg.T) * (x @ wu.T)) @ wd.T
    want = torch.autograd.grad(y, leaves, dy)
    with torch.no_grad():
        g, u, _, y64 = ffn64(*leaves, act)
        got = ffn_backward64(*leaves, g, u, dy, act)
    assert torch.allclose(y64, y, rtol=1e-12, atol=1e-12)
    for n, w in zip(("dx", "dwg", "dwu", "dwd"), want):
        assert torch.allclose(got[n], w, rtol=1e-12, atol=1e-12), n


def test_distill_gradient_is_autograds_and_differences():
    gen = torch.Generator().manual_seed(4)
    B, V, k, T = 4, 11, 3, 1.7
    z = torch.randn(B, V, dtype=F64, generator=gen) * 2
    idx = torch.tensor([[3, 7, 1], [0, 0, 5], [2, -1, -1], [-1, -1, -1]])  # twice, short, none
    t = torch.randn(B, k, dtype=F64, generator=gen)
    dl = torch.tensor([0.3, 1.1, -0.7, 2.0], dtype=F64)
    loss, lse, dz = distill64(z, idx, t, T, dl)
    zz = z.clone().requires_grad_()
    logq = torch.log_softmax(zz / T, 1)
    total = 0
    for b in range(3):
        keep = idx[b] >= 0
        logp = torch.log_softmax(t[b][keep] / T, 0)
        row = T * T * (logp.exp() * (logp - logq[b][idx[b][keep]])).sum()
        assert math.isclose(float(row.detach()), float(loss[b]), rel_tol=1e-12)
        total = total + dl[b] * row
    total.backward()
    assert loss[3] == 0 and torch.allclose(dz, zz.grad, rtol=1e-12, atol=1e-14)
    e = 1e-5
    for b in range(B):
        for v in (0, 3, 10):
            zp, zm = z.clone(), z.clone()
            zp[b, v] += e
            zm[b, v] -= e
            num = dl[b] * (distill64(zp, idx, t, T)[0][b] - distill64(zm, idx, t, T)[0][b]) / (2 * e)
            assert abs(float(num - dz[b, v])) < 1e-8


# ------------------------------------------------------------------ refusals

def ffn(L, x=16, wg=16, wu=16, wd=16, B=4, dim=64, F=64, act=0, ws=16, y=16, g=None, u=None):
    return L.pkm_gated_ffn(x, wg, wu, wd, B, dim, F, act, ws, y, g, u, 16, None)


def ffn_b(L, x=16, wg=16, wu=16, wd=16, g=16, u=16, dy=16, B=4, dim=64, F=64, act=0, ws=16, dx=16,
          dwg=16, dwu=16, dwd=16, gd=pk.PKM_BF16):
    return L.pkm_gated_ffn_backward(x, wg, wu, wd, g, u, dy, B, dim, F, act, ws, dx, dwg, dwu, dwd,
                                    gd, 16, None)


@pytest.mark.parametrize("call", [ffn, ffn_b])
def test_ffn_refusals(L, call):
    for n in ("x", "wg", "wu", "wd", "ws"):
        assert call(L, **{n: None}) == pk.PKM_ERR_INVALID
        assert call(L, **{n: 24}) == pk.PKM_ERR_ALIGN
    assert call(L, B=-1) == pk.PKM_ERR_INVALID
    assert call(L, dim=0) == pk.PKM_ERR_INVALID
    assert call(L, F=-8) == pk.PKM_ERR_INVALID
    assert call(L, dim=60) == pk.PKM_ERR_UNSUPPORTED
    assert call(L, F=63) == pk.PKM_ERR_UNSUPPORTED
    assert call(L, act=4) == pk.PKM_ERR_UNSUPPORTED
    assert call(L, act=-1) == pk.PKM_ERR_UNSUPPORTED
    assert call(L, B=2 ** 31 - 1) == pk.PKM_ERR_RANGE
    assert call(L, B=2 ** 30, F=2 ** 20) == pk.PKM_ERR_RANGE
    assert call(L, dim=2 ** 24, F=2 ** 24) == pk.PKM_ERR_RANGE


def test_ffn_refusals_of_each(L):
    assert ffn(L, y=None) == pk.PKM_ERR_INVALID
    assert ffn(L, g=16) == pk.PKM_ERR_INVALID
    assert ffn(L, u=16) == pk.PKM_ERR_INVALID
    assert ffn(L, g=16, u=20) == pk.PKM_ERR_ALIGN
    assert ffn(L, B=0, x=None, y=None) == pk.PKM_OK
    for n in ("g", "u", "dy"):
        assert ffn_b(L, **{n: None}) == pk.PKM_ERR_INVALID
    assert ffn_b(L, dwg=None) == pk.PKM_ERR_INVALID
    assert ffn_b(L, dwu=None) == pk.PKM_ERR_INVALID
    assert ffn_b(L, dwd=18) == pk.PKM_ERR_ALIGN
    assert ffn_b(L, gd=pk.PKM_FP8_E4M3) == pk.PKM_ERR_UNSUPPORTED
    assert ffn_b(L, B=0, gd=pk.PKM_F32) == pk.PKM_OK


def test_ffn_workspaces(L):
    # at least what is kept between the products: h, and dg, du and h, in bf16
    for B, dim, F in ((1, 8, 8), (37, 512, 1400), (16384, 1024, 4096)):
        assert pk.pkm_gated_ffn_workspace_bytes(B, dim, F) >= 2 * B * F
        assert pk.pkm_gated_ffn_backward_workspace_bytes(B, dim, F) >= 6 * B * F
    assert pk.pkm_gated_ffn_workspace_bytes(-1, 8, 8) == 0
    assert pk.pkm_gated_ffn_backward_workspace_bytes(4, 0, 8) == 0


def dis(L, z=16, dt=pk.PKM_F32, ld=100, B=2, V=100, idx=16, t=16, k=4, T=1.0, loss=16):
    return L.pkm_distill(z, dt, ld, B, V, idx, t, k, T, loss, None, 16, None)


def dis_b(L, z=16, dt=pk.PKM_F32, ld=100, B=2, V=100, idx=16, t=16, k=4, T=1.0, lse=16, dl=16,
          dz=16, ldd=100):
    return L.pkm_distill_backward(z, dt, ld, B, V, idx, t, k, T, lse, dl, dz, ldd, 16, None)


def dis_t(L, z=16, dt=pk.PKM_F32, ld=100, B=2, V=100, idx=16, t=16, k=4, T=1.0, dl=16, loss=16,
          lse=16, dz=16, ldd=100):
    return L.pkm_distill_train(z, dt, ld, B, V, idx, t, k, T, dl, loss, lse, dz, ldd, 16, None)


@pytest.mark.parametrize("call,needs", [(dis, ("z", "idx", "t", "loss")),
                                        (dis_b, ("z", "idx", "t", "lse", "dl", "dz")),
                                        (dis_t, ("z", "idx", "t", "dl", "loss", "lse", "dz"))])
def test_distill_refusals(L, call, needs):
    for n in needs:
        assert call(L, **{n: None}) == pk.PKM_ERR_INVALID
    for bad in (dict(B=-1), dict(V=0), dict(k=0), dict(T=0.0), dict(T=-1.0), dict(T=math.nan),
                dict(T=math.inf)):
        assert call(L, **bad) == pk.PKM_ERR_INVALID
    assert call(L, dt=pk.PKM_FP8_E4M3) == pk.PKM_ERR_UNSUPPORTED
    assert call(L, k=pk.PKM_DISTILL_MAX_K + 1) == pk.PKM_ERR_UNSUPPORTED
    assert call(L, ld=99) == pk.PKM_ERR_RANGE
    assert call(L, z=18) == pk.PKM_ERR_ALIGN
    assert call(L, z=17, dt=pk.PKM_BF16) == pk.PKM_ERR_ALIGN
    assert call(L, B=0, z=None) == pk.PKM_OK
    if "dz" in needs:
        assert call(L, ldd=99) == pk.PKM_ERR_RANGE
        assert call(L, dz=17) == pk.PKM_ERR_ALIGN
        assert call(L, z=32, dz=32, ld=104) == pk.PKM_ERR_RANGE  # in place with two strides


def test_binding_refuses_other_layouts(L):
    x = torch.zeros(8, 16, dtype=torch.bfloat16)
    w = torch.zeros(16, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pk.pkm_gated_ffn(x, w, w.t()[:, ::2], w, 8, 16, 16, 0, x, x, stream=0)
    with pytest.raises(ValueError):
        pk.pkm_gated_ffn_backward(x.t(), w, w, w, x, x, x, 8, 16, 16, 0, x, x, w, w, w, stream=0)
    z, idx, t = torch.zeros(4, 32), torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    v = torch.zeros(4)
    with pytest.raises(ValueError):
        pk.pkm_distill(z[:, ::2], pk.PKM_F32, 32, 4, 16, idx, t, 2, 1.0, v, stream=0)
    with pytest.raises(ValueError):
        pk.pkm_distill(z, pk.PKM_F32, 40, 4, 32, idx, t, 2, 1.0, v, stream=0)
    with pytest.raises(ValueError):
        pk.pkm_distill_train(z, pk.PKM_F32, 32, 4, 32, idx.t(), t, 2, 1.0, v, v, v, z, 32, stream=0)


def test_argument_types(L):
    assert L.pkm_distill.argtypes[8] is ctypes.c_float
    assert (pk.PKM_ACT_SILU, pk.PKM_ACT_GELU, pk.PKM_ACT_GELU_TANH, pk.PKM_ACT_RELU) == (0, 1, 2, 3)
