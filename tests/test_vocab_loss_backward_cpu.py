"""The vocabulary loss's backward pass that takes the forward's loss: the C ABI refuses bad arguments before any
CUDA call."""
import pytest

import sparse_top_lookup_gb300 as pk

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    pk.build()
    return pk.lib()


def call(L, x=16, w=16, t=16, lse=16, loss=16, dl=16, B=4, dim=64, V=100, ws=16, dx=16, dw=16,
         gd=pk.PKM_BF16, st=16):
    return L.pkm_vocab_loss_backward_with_loss(x, w, t, lse, loss, dl, B, dim, V, ws, dx, dw, gd, st, None)


def test_refusals(L):
    for n in ("x", "w", "t", "lse", "loss", "dl", "ws"):
        assert call(L, **{n: None}) == pk.PKM_ERR_INVALID
    for n in ("lse", "loss", "dl", "st"):
        assert call(L, **{n: 18}) == pk.PKM_ERR_ALIGN
    for n in ("x", "w", "ws", "dx", "dw"):
        assert call(L, **{n: 24}) == pk.PKM_ERR_ALIGN
    assert call(L, t=20) == pk.PKM_ERR_ALIGN
    for bad in (dict(B=-1), dict(dim=0), dict(V=0)):
        assert call(L, **bad) == pk.PKM_ERR_INVALID
    assert call(L, dim=60) == pk.PKM_ERR_UNSUPPORTED
    assert call(L, gd=pk.PKM_FP8_E4M3) == pk.PKM_ERR_UNSUPPORTED
    for bad in (dict(B=2 ** 31 - 1), dict(V=2 ** 31 - 1), dict(B=2 ** 30, V=2 ** 24)):
        assert call(L, **bad) == pk.PKM_ERR_RANGE
    assert call(L, B=0, x=None, loss=None, gd=pk.PKM_F32) == pk.PKM_OK
    assert call(L, B=0, x=None, dw=None) == pk.PKM_OK


def test_binding_refuses_other_layouts(L):
    x, f = torch.zeros(8, 16, dtype=torch.bfloat16), torch.zeros(16)
    t = torch.zeros(8, dtype=torch.int64)
    with pytest.raises(ValueError):
        pk.pkm_vocab_loss_backward_with_loss(x, x, t, f, f[::2], f, 8, 16, 8, f, x, x, stream=0)
