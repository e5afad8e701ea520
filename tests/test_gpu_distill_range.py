"""Distillation on the GPU where logits are far from zero: finite masks of every size over a few
columns, a stretch, all columns but one and whole rows; rows with a common offset; tiny temperatures.

The 64-bit form takes the row's largest logit away first (a sum of 1e30 and log V has no room in 64
bits either).  Tolerances, per row and column, with U = 2^-24, x = (z - max) log2(e) / T and y the same
of the teacher's list:
  q  an exponential is good to 2 ulp (4 U) and to the rounding of its argument, difference and
     product, each U |x|; the sum of the terms to 40 U (few terms per thread, then a tree), division
     and factors to 10 U:                                              U (64 + 4 |x|)
  p  the same with at most 16 terms per lane:                          U (48 + 4 |y|)
  loss  T^2 sum p (..): p's error times the term's magnitudes M, the terms' own four roundings, the logs'
     error (64 U from their sums), one rounding at the end
  lse   max / T + log(sum): 64 U, one rounding
  dz    q's and p's errors times |dloss| T; one rounding; bf16's exponents may take the scale in, which
     leaves half a step of a number below 1024: 2^-15
  from an fp32 lse: U |lse| for lse and U |z / T| for log2(e) / T more in every exponent.
"""
import math

import pytest

import sparse_top_lookup_gb300 as pk

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F64, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
U = 2.0 ** -24
L2E = 1.4426950408889634
KIND = {F32: pk.PKM_F32, BF16: pk.PKM_BF16}

# rows of a warp each, of one CTA or two, of a cluster
FORMS = [(650, 600), (3, 3000), (3, 40000)]
MASKS = [-1e4, -1e5, -1e6, -1e9, -1e10, -1e20, -1e30, -3e38]
WHERE = ["vector", "stretch", "all but one", "all"]


def rows(B, V, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(B, V, device="cuda", generator=gen) * 2
    t = torch.randn(B, 4, device="cuda", generator=gen) * 3
    idx = torch.arange(4, device="cuda").repeat(B, 1) * 5
    z.scatter_(1, idx, t + torch.randn(B, 4, device="cuda", generator=gen))
    dl = torch.randn(B, device="cuda", generator=gen)
    return z.to(dtype), idx, t, dl


def masked(B, V, dtype, where, value, seed=1):
    z, idx, t, dl = rows(B, V, dtype, seed)
    if where == "vector":
        z[:, V // 2 // 8 * 8:V // 2 // 8 * 8 + 8] = value
    elif where == "stretch":
        z[:, V // 4:V // 2] = value
    elif where == "all but one":
        live = z[:, 5].clone()
        z[:] = value
        z[:, 5] = live
        idx[::2, 0], idx[::2, 2:] = -1, -1        # the live column alone; else masked ones too
    else:
        z[:] = value
    return z, idx, t, dl


class Exact:
    """The definition in 64 bits (every entry with idx >= 0 counts), and what the bounds need."""

    def __init__(self, z, idx, t, T, dl):
        z = z.double()
        self.m = z.amax(1, keepdim=True)
        self.d = (z - self.m) / T
        self.log_sum = torch.logsumexp(self.d, 1)
        self.lse = self.m[:, 0] / T + self.log_sum
        logq = self.d - self.log_sum[:, None]
        there = idx >= 0
        at = idx.clamp(min=0)
        tt = t.double().masked_fill(~there, -math.inf) / T
        y = tt - tt.amax(1, keepdim=True)
        log_mass = torch.logsumexp(y, 1, keepdim=True)
        p = torch.exp(y - log_mass)
        y = y.masked_fill(~there, 0.0)
        lq = logq.gather(1, at)
        self.loss = T * T * torch.where(p > 0, p * (y - log_mass - lq), torch.zeros_like(p)).sum(1)
        self.q = torch.exp(logq)
        self.P = torch.zeros_like(z).scatter_add_(1, at, p)
        self.scale = (dl.double().abs() * T)[:, None]
        self.dz = (dl.double() * T)[:, None] * (self.q - self.P)
        # bounds
        self.rel_q = U * (64 + 4 * L2E * self.d.abs())
        rel_p = U * (48 + 4 * L2E * y.abs())
        self.err_p = torch.zeros_like(z).scatter_add_(1, at, p * rel_p)
        M = y.abs() + self.d.gather(1, at).abs() + self.log_sum.abs()[:, None] + log_mass.abs()
        self.loss_err = (2 * U * self.loss.abs() + T * T * (
            torch.where(p > 0, p * (rel_p + 8 * U) * M, torch.zeros_like(p)).sum(1)
            + 64 * U + 4 * U * self.log_sum.abs()))
        self.lse_err = 2 * U * self.lse.abs() + 64 * U + 2 * U * self.log_sum.abs()

    def dz_err(self, rel_q, dtype):
        half = U if dtype == F32 else 2.0 ** -8
        own = 0.0 if dtype == F32 else 2.0 ** -15
        q = self.q * (rel_q + own)
        return half * self.dz.abs() + 1.01 * self.scale * (q + self.err_p + 2.0 ** -120)


def forward(z, idx, t, T):
    B, V = z.shape
    loss, lse = torch.full((B,), -7.0, device="cuda"), torch.full((B,), -7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.check(pk.pkm_distill(z, KIND[z.dtype], V, B, V, idx, t, idx.shape[1], T, loss, lse, st), "forward")
    assert st.item() == pk.PKM_OK
    return loss, lse


def train(z, idx, t, T, dl):
    B, V = z.shape
    loss, lse, dz = torch.empty(B, device="cuda"), torch.empty(B, device="cuda"), torch.empty_like(z)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.check(pk.pkm_distill_train(z, KIND[z.dtype], V, B, V, idx, t, idx.shape[1], T, dl, loss, lse, dz, V,
                                  st), "train")
    assert st.item() == pk.PKM_OK
    return loss, lse, dz


def within(got, want, err, what):
    got = got.double()
    beyond = want.float().isinf()                 # more than fp32 holds
    assert torch.equal(got[beyond], want.float().double()[beyond]), what
    got, want, err = got[~beyond], want[~beyond], err[~beyond]
    assert bool(torch.isfinite(got).all()), "%s: %d not finite" % (what, int((~torch.isfinite(got)).sum()))
    off = (got - want).abs()
    bad = off > err
    assert not bool(bad.any()), (what, float(off[bad].max()), float(err[bad].min()))


def check_losses(z, idx, t, dl, T):
    e = Exact(z, idx, t, T, dl)
    for what, (loss, lse) in (("forward", forward(z, idx, t, T)), ("train", train(z, idx, t, T, dl)[:2])):
        within(lse, e.lse, e.lse_err, what + " lse")
        within(loss, e.loss, e.loss_err, what + " loss")


@pytest.mark.parametrize("value", MASKS)
@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V", FORMS)
def test_losses_of_rows_with_finite_masks(B, V, dtype, where, value):
    for T in (1.0, 1.7):
        check_losses(*masked(B, V, dtype, where, value), T)


@pytest.mark.parametrize("offset", [1e3, -1e3, 1e5, 1e6, -1e6, 1e10, 1e30])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V", FORMS)
def test_losses_of_rows_with_a_common_offset(B, V, dtype, offset):
    z, idx, t, dl = rows(B, V, F32, 2)
    check_losses((z + offset).to(dtype), idx, t, dl, 0.7)


@pytest.mark.parametrize("dtype,V", [(BF16, 262160), (F32, 131080)])
def test_losses_of_rows_longer_than_a_cluster_holds(dtype, V):
    for value in (-1e9, -1e30):
        check_losses(*masked(2, V, dtype, "stretch", value), 1.0)


@pytest.mark.parametrize("T", [1e-3, 1e-6, 1e-10, 1e-20])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V", FORMS)
def test_losses_of_tiny_temperatures(B, V, dtype, T):
    # p and q are all on their largest entry, or nearly: the loss is T sum p ((t - max t) - (z - max z)),
    # with three roundings a term, and what T^2 leaves of the logs
    z, idx, t, dl = rows(B, V, dtype, 3)
    t = t.round() + torch.arange(4, device="cuda") * 0.25           # no two alike, none near another
    z[:, 7] = 30.0                                                # and the row's largest far ahead
    e = Exact(z, idx, t, T, dl)
    for loss, lse in (forward(z, idx, t, T), train(z, idx, t, T, dl)[:2]):
        within(lse, e.lse, 2 * U * e.lse.abs() + 64 * U, "lse")
        within(loss, e.loss, 64 * U * (e.loss.abs() + T), "loss")


def check_train(z, idx, t, dl, T):
    e = Exact(z, idx, t, T, dl)
    err = e.dz_err(e.rel_q, z.dtype)
    within(train(z, idx, t, T, dl)[2], e.dz, err, "dz")
    B, V = z.shape
    d, loss, lse = z.clone(), torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    pk.check(pk.pkm_distill_train(d, KIND[z.dtype], V, B, V, idx, t, idx.shape[1], T, dl, loss, lse, d, V),
             "train in place")
    within(d, e.dz, err, "dz in place")


@pytest.mark.parametrize("value", MASKS)
@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V", FORMS)
def test_training_gradients_of_rows_with_finite_masks(B, V, dtype, where, value):
    for T in (1.0, 1.7):
        check_train(*masked(B, V, dtype, where, value), T)


@pytest.mark.parametrize("offset", [300.0, 1e3, -1e3, 1e4, 1e5, 1e6, -1e6, 1e10, 1e30])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V", FORMS)
def test_training_gradients_of_rows_with_a_common_offset(B, V, dtype, offset):
    z, idx, t, dl = rows(B, V, F32, 2)
    check_train((z + offset).to(dtype), idx, t, dl, 0.7)


@pytest.mark.parametrize("T", [1e-2, 1e-3, 1e-6, 1e-10, 1e-20])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V", FORMS)
def test_training_gradients_of_tiny_temperatures(B, V, dtype, T):
    z, idx, t, dl = rows(B, V, dtype, 3)
    t = t.round() + torch.arange(4, device="cuda") * 0.25
    z[:, 7] = 30.0
    check_train(z, idx, t, dl, T)


def check_backward(z, idx, t, dl, T):
    """From an lse rounded to fp32: to that rounding; where it says nothing, q within [0, 1]."""
    e = Exact(z, idx, t, T, dl)
    B, V = z.shape
    lse, dz = e.lse.float(), torch.empty_like(z)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.check(pk.pkm_distill_backward(z, KIND[z.dtype], V, B, V, idx, t, idx.shape[1], T, lse, dl, dz, V, st),
             "backward")
    assert st.item() == pk.PKM_OK
    far = 4 * U * e.lse.abs()[:, None]
    err = e.dz_err(torch.expm1(e.rel_q.clamp(max=1.0) + far.clamp(max=1.0)), z.dtype)
    most = e.scale * (1 + e.P) * (1 + 2.0 ** -7)
    known = (far < 0.1).expand_as(dz)
    within(dz[known], e.dz[known], err[known], "dz")
    within(dz, torch.zeros_like(e.dz), most, "dz's range")


@pytest.mark.parametrize("value", MASKS)
@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V", FORMS)
def test_gradients_from_lse_of_rows_with_finite_masks(B, V, dtype, where, value):
    for T in (1.0, 1.7):
        check_backward(*masked(B, V, dtype, where, value), T)


@pytest.mark.parametrize("offset", [300.0, 1e3, -1e3, 1e4, 1e5, 1e6, -1e6, 1e7, 1e8, -1e8, 1e10, 1e30])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V", FORMS)
def test_gradients_from_lse_of_rows_with_a_common_offset(B, V, dtype, offset):
    z, idx, t, dl = rows(B, V, F32, 2)
    check_backward((z + offset).to(dtype), idx, t, dl, 0.7)


@pytest.mark.parametrize("T", [1e-2, 1e-3, 1e-6, 1e-10, 1e-20])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V", FORMS)
def test_gradients_from_lse_of_tiny_temperatures(B, V, dtype, T):
    z, idx, t, dl = rows(B, V, dtype, 3)
    t = t.round() + torch.arange(4, device="cuda") * 0.25
    z[:, 7] = 30.0
    check_backward(z, idx, t, dl, T)
