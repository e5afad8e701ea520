"""Distillation of the longest row that the interface's 32-bit V allows.

Tolerances: a thread's sum joins one partial sum per chunk of 16384 columns in each of 8 slices, all in
fp32: at most V / 131072 + 100 roundings, each 2^-24 of the sum, in lse, loss / T^2 and every q.
"""
import math

import pytest

import sparse_top_lookup_gb300 as pk

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
U = 2.0 ** -24
V, T = 2 ** 31 - 1, 2.0
STEP = 1 << 26


@pytest.fixture(scope="module")
def row():
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    gen = torch.Generator(device="cuda").manual_seed(1)
    z = torch.empty(1, V, dtype=BF16, device="cuda")
    for lo in range(0, V, STEP):
        z[0, lo:lo + STEP].normal_(0.0, 2.0, generator=gen)
    idx = torch.tensor([[0, 5, 1 << 30, V - 1]], device="cuda")
    t = torch.tensor([[1.0, 2.5, 0.5, 2.0]], device="cuda")
    z[0, idx[0]] = torch.tensor([20.0, 38.0, 8.0, 41.0], dtype=BF16, device="cuda")
    total = sum(float(torch.exp(z[0, lo:lo + STEP].double() / T - 20).sum()) for lo in range(0, V, STEP))
    lse = 20 + math.log(total)
    p = torch.softmax(t[0].double() / T, 0)
    logq = z[0, idx[0]].double() / T - lse
    loss = T * T * float((p * (torch.log(p) - logq)).sum())
    yield z, idx, t, p, lse, loss
    torch.cuda.empty_cache()


def test_gradient(row):
    z, idx, t, p, lse, _ = row
    dz = torch.full_like(z, -777.0)
    one = torch.ones(1, device="cuda")
    pk.check(pk.pkm_distill_backward(z, pk.PKM_BF16, V, 1, V, idx, t, 4, T,
                                     torch.tensor([lse], device="cuda"), one, dz, V), "backward")
    q = torch.exp(z[0, idx[0]].double() / T - lse)
    want = T * (q - p)
    assert bool(((dz[0, idx[0]].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4 * q).all())
    dz[0, idx[0]] = 0
    for lo in range(0, V, STEP):
        want = T * torch.exp(z[0, lo:lo + STEP].double() / T - lse)
        at = idx[0][(idx[0] >= lo) & (idx[0] < lo + STEP)] - lo
        want[at] = 0
        off = (dz[0, lo:lo + STEP].double() - want).abs()
        # (U |lse| for lse, U |z / T| for the constant, U |x| twice for the rest; U (64) as elsewhere)
        assert bool((off <= want * (2.0 ** -8 + U * 400)).all()), lo


def test_loss(row):
    z, idx, t, _, lse, loss = row
    got, got_lse = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    pk.check(pk.pkm_distill(z, pk.PKM_BF16, V, 1, V, idx, t, 4, T, got, got_lse), "forward")
    err = U * (V / 131072 + 100)
    assert abs(float(got_lse) - lse) <= err + 2 * U * abs(lse)
    assert abs(float(got) - loss) <= T * T * (err + 64 * U * 40) + 2 * U * abs(loss)
