"""The sum and norm where the squares of a row leave fp32's range, and rows near it: against the 64-bit form.

Tolerances as in test_gpu_norm.py.
"""
import pytest

import sparse_top_lookup_gb300 as pk
from more_operators64 import norm64
from test_gpu_norm import BF16, F32, F64, U8, backward, check_forward, forward, normal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 2e-38, 1e-30, 1e-20, 1e-5])
@pytest.mark.parametrize("dim", [8, 64, 264, 2048, 8208, 16384])
def test_rows_of_every_size(dim, eps):
    # a row each from 2^-120 to 2^100, most of whose squares are out of range
    at = torch.arange(-120, 101, 4, device="cuda")
    x = normal(len(at), dim, seed=dim) * torch.exp2(at.float())[:, None]
    r = normal(len(at), dim, seed=dim + 1) * torch.exp2(at.float())[:, None]
    x[:, 0] += 3 * torch.exp2(at.float())  # (no row of next to nothing)
    w = 1 + 0.3 * normal(dim, seed=3)
    # (y beyond fp32's range, with eps much below the squares, is none of this: rows are of order one)
    for yt in (F32, BF16) + ((U8,) if dim % 16 == 0 else ()):
        if yt == U8 and eps > 1e-37:
            continue  # (rows below eps: codes of 2^-126 and less)
        check_forward(x, r, w, yt, eps=eps)


def test_one_large_entry_among_tiny_ones():
    x = torch.full((6, 2048), 1e-30, device="cuda")
    x[1, 77], x[2, 2047], x[3, 0], x[4, 9] = 1e-10, 1.0, 1e25, 3e38
    x[5, 5] = 1e-19
    w = 1 + 0.3 * normal(2048, seed=3)
    check_forward(x, None, w, F32, eps=0.0)
    check_forward(x, None, w, F32, eps=1e-5)


def test_rows_in_range_keep_their_bits():
    # beside rows out of it
    x, w = normal(64, 520, seed=1), normal(520, seed=2)
    want = forward(x, None, w, F32, eps=0.0)
    x2 = x.clone()
    x2[::3] *= 1e-25
    got = forward(x2, None, w, F32, eps=0.0)
    rest = torch.arange(64, device="cuda") % 3 != 0
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(got, want))
    assert bool(torch.isfinite(got[1]).all())


@pytest.mark.parametrize("eps", [0.0, 1e-35, 1e-5])
def test_zeros_infinities_and_nan_as_before(eps):
    x, w = normal(5, 264, seed=1), normal(264, seed=2)
    x[0], x[1, 3], x[2, 7] = 0, float("inf"), float("nan")
    x[3] *= 1e-25
    _, y, rstd = forward(x, None, w, F32, eps=eps)
    if eps == 0:
        assert bool(y[0].isnan().all()) and rstd[0].item() == float("inf")
    else:
        assert bool((y[0] == 0).all())
    assert bool(y[1, 3].isnan()) and rstd[1].item() == 0
    assert bool(y[2].isnan().all())
    S, R, Y = norm64(x[3:].to(F64), None, w.to(F64), eps)
    assert bool(((y[3:].to(F64) - Y).abs() <= 300 * 2.0 ** -24 * Y.abs()).all())


@pytest.mark.parametrize("dim", [64, 528, 16384])
def test_in_place_out_of_range(dim):
    x, r, w = 1e-25 * normal(9, dim, seed=1), 1e-25 * normal(9, dim, seed=2), normal(dim, seed=3)
    s, y, rstd = (t.clone() for t in forward(x, r, w, F32, eps=0.0))
    xx, rr = x.clone(), r.clone()
    pk.check(pk.pkm_add_rms_norm(xx, pk.PKM_F32, rr, pk.PKM_F32, w, 0.0, 9, dim, rr, pk.PKM_F32, xx,
                                 pk.PKM_F32), "norm")
    assert torch.equal(rr, s) and torch.equal(xx, y)
    codes = forward(x, r, w, U8, eps=0.0)[1].clone()
    xx = x.clone()
    yy = torch.empty_like(codes)
    pk.check(pk.pkm_add_rms_norm(xx, pk.PKM_F32, r, pk.PKM_F32, w, 0.0, 9, dim, xx, pk.PKM_F32, yy,
                                 pk.PKM_FP8_E4M3), "norm")
    assert torch.equal(xx, s) and torch.equal(yy, codes)


def test_rows_of_denormals_and_wide_weights():
    # rstd is past fp32's range, or only its product with the weight is; y is not
    x = torch.ldexp(normal(3, 264, seed=1), torch.tensor([[-140], [-126], [-118]], device="cuda"))
    w = 1e4 * normal(264, seed=2)
    _, y, rstd = forward(x, None, w, F32, eps=0.0)
    Y = norm64(x.to(F64), None, w.to(F64), 0.0)[2]
    assert bool(((y.to(F64) - Y).abs() <= (264 / 2 + 10) * 2.0 ** -24 * Y.abs()).all())
    assert rstd[0].item() == float("inf") and bool(torch.isfinite(rstd[1:]).all())


@pytest.mark.parametrize("dim", [264, 16384])
def test_the_gradient_of_rows_out_of_range(dim):
    # from the forward's rstd: as a row in range and its multiple, d shrinking as the row grows
    x, dy, w = normal(3, dim, seed=1), normal(3, dim, seed=2), normal(dim, seed=3)
    for e in (-100, -40, 70, 100):
        rows = [x, torch.ldexp(x, torch.tensor(e, device="cuda"))]
        got = []
        for s in rows:
            rstd = forward(s, None, w, F32, eps=0.0)[2].clone()
            got.append(backward(s, w, rstd, dy, None, F32))
        assert torch.equal(torch.ldexp(got[1]["d"], torch.tensor(e, device="cuda")), got[0]["d"]), e
        assert torch.equal(got[1]["dw"], got[0]["dw"]), e
