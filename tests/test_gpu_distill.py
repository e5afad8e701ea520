"""Distillation from a teacher's top logits on the GPU against its 64-bit form.

Tolerances.  exp2f is good to 2 ulp, an argument rounded in fp32 is off by 2^-24 of itself, and
arguments that matter are at most A = (largest - smallest listed logit) / T * log2(e) + 40 away
from the maximum: q and p are good to E = 2^-24 (4 + 2 A).  lse = max / T + log(sum): E for the sum
(its own fp32 sums: 2^-24 * 40, as a thread adds V / 512 terms at most and the rest is a tree), one
fp32 rounding of lse.  The loss adds p-weighted terms that are computed in 64 bits: E times the
terms' magnitudes, and one rounding.  dz: E of each of its two parts and one rounding to its type.
"""
import math

import pytest

import sparse_top_lookup_gb300 as pk
from operators64 import distill64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F64, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
U = 2.0 ** -24
KIND = {F32: pk.PKM_F32, BF16: pk.PKM_BF16}
MARK = -777.0


class Rows:
    """[B, V] with ld elements from row to row, `shift` elements into an aligned buffer, inside
    a buffer whose other values must not change."""

    def __init__(self, B, V, dtype, ld=None, shift=0):
        self.ld = ld or V
        self.buf = torch.full((64 + shift + B * self.ld + 64,), MARK, device="cuda", dtype=dtype)
        self.t = self.buf[64 + shift:64 + shift + B * self.ld].view(B, self.ld)[:, :V]
        self.B, self.V, self.shift = B, V, shift

    def ok(self):
        m = torch.tensor(MARK, dtype=self.buf.dtype).item()
        lo, n = 64 + self.shift, self.B * self.ld
        between = self.buf[lo:lo + n].view(self.B, self.ld)[:, self.V:]
        return all(bool((x == m).all()) for x in (self.buf[:lo], self.buf[lo + n:], between))


def make(B, V, k, dtype, T, seed, ld=None, shift=0, masked=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = Rows(B, V, dtype, ld, shift)
    z.t.copy_(torch.randn(B, V, device="cuda", generator=gen) * 2)
    live = max(1, V - masked)
    idx = torch.randint(0, live, (B, k), device="cuda", generator=gen)
    t = torch.randn(B, k, device="cuda", generator=gen) * 3
    z.t.scatter_(1, idx, (t + torch.randn(B, k, device="cuda", generator=gen)).to(dtype))
    z.t[:, live:] = -math.inf
    length = torch.randint(0, 2 * k + 1, (B, 1), device="cuda", generator=gen)
    if B < 4:
        length.fill_(k)
    idx[torch.arange(k, device="cuda") >= length] = -1
    dl = torch.randn(B, device="cuda", generator=gen)
    dl[::5] = 0
    return z, idx, t, dl


def calls(z, idx, t, dl, T, ld_d=None, shift_d=0, in_place=False):
    """loss, lse of pkm_distill and of pkm_distill_train, dz of backward and of train."""
    B, V, k, dtype = z.B, z.V, idx.shape[1], z.t.dtype
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = {}
    loss, lse = Rows(1, B, F32), Rows(1, B, F32)
    pk.check(pk.pkm_distill(z.t, KIND[dtype], z.ld, B, V, idx, t, k, T, loss.t, lse.t, st), "fwd")
    out["f"] = loss.t[0].clone(), lse.t[0].clone()
    d = Rows(B, V, dtype, ld_d, shift_d)
    pk.check(pk.pkm_distill_backward(z.t, KIND[dtype], z.ld, B, V, idx, t, k, T, lse.t, dl, d.t,
                                     d.ld, st), "bwd")
    out["b"] = d.t.clone()
    loss2, lse2 = Rows(1, B, F32), Rows(1, B, F32)
    if in_place:
        e = Rows(B, V, dtype, z.ld, z.shift)
        e.t.copy_(z.t)
        src = e
    else:
        e, src = Rows(B, V, dtype, ld_d, shift_d), z
    pk.check(pk.pkm_distill_train(src.t, KIND[dtype], src.ld, B, V, idx, t, k, T, dl, loss2.t,
                                  lse2.t, e.t, e.ld, st), "train")
    out["t"] = loss2.t[0], lse2.t[0], e.t
    torch.cuda.synchronize()
    assert all(r.ok() for r in (loss, lse, d, loss2, lse2, e, z))
    out["status"] = st.item()
    return out


def check(z, idx, t, dl, T, out, status=pk.PKM_OK):
    assert out["status"] == status
    Z = z.t.double().cpu()
    loss, lse, dz = distill64(Z, idx.cpu(), t.cpu(), T, dl.double().cpu())
    there = (idx.cpu() >= 0) & (idx.cpu() < z.V) & (t.cpu() > -math.inf)
    spread = 0.0
    if bool(there.any()):
        sel = Z.gather(1, idx.cpu().clamp(0, z.V - 1))[there]
        sel = sel[sel > -math.inf]
        vals = torch.cat((t.cpu().double()[there], sel))
        spread = float(vals.max() - vals.min()) if vals.numel() else 0.0
    A = spread / T * 1.45 + 40
    E = U * (4 + 2 * A + 40)
    top = max(1.0, float(lse[lse > -math.inf].abs().max())) if bool((lse > -math.inf).any()) else 1
    for which in ("f", "t"):
        gl, gs = (x.double().cpu() for x in out[which][:2])
        fin = torch.isfinite(lse)
        assert torch.equal(gs[~fin], lse[~fin])
        assert bool(((gs - lse)[fin].abs() <= 2 * U * lse[fin].abs() + E).all()), which
        fin = torch.isfinite(loss)
        assert torch.equal(gl[~fin], loss[~fin])
        terms = T * T * (spread / T + 2 * top + math.log(idx.shape[1] + 1))
        assert bool(((gl - loss)[fin].abs() <= 2 * U * loss[fin].abs() + 2 * E * terms).all()), which
    half = U if z.t.dtype == F32 else 2.0 ** -8
    for which, got in (("b", out["b"]), ("t", out["t"][2])):
        got = got.double().cpu()
        assert torch.isfinite(got).all(), which
        scale = (dl.double().cpu().abs() * T)[:, None]
        # (the backward pass takes lse in fp32: 2^-24 |lse| more in every exponent)
        bound = half * dz.abs() + (E + 2 * U * top) * (dz.abs() + 2 * scale *
                                                       (dz != 0)) * 1.01
        # where q alone stands, its error is relative
        listed = torch.zeros(z.B, z.V + 1, dtype=torch.bool)
        listed.scatter_(1, torch.where(there, idx.cpu(), torch.full_like(idx.cpu(), z.V)), True)
        rel = (half + 1.01 * (E + 2 * U * top)) * dz.abs() + 1e-44
        bound = torch.where(listed[:, :z.V], bound, rel)
        off = (got - dz).abs()
        assert bool((off <= bound).all()), (which, float((off - bound).max()))
        # what has to be zero is zero
        dead = (dl.cpu() == 0) | ~there.any(1)
        assert bool((got[dead] == 0).all())


SHAPES = [(1, 1, 1), (1, 7, 3), (3, 31, 4), (5, 32, 8), (2, 100, 100), (9, 1000, 17), (4, 4096, 64),
          (3, 8191, 5), (2, 50257, 20), (150, 515, 6), (1, 131072, 64), (2, 100001, 512)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V,k", SHAPES)
def test_matches_64_bits(B, V, k, dtype):
    T = (1.0, 2.0, 0.7)[(B + V) % 3]
    z, idx, t, dl = make(B, V, k, dtype, T, B + V)
    check(z, idx, t, dl, T, calls(z, idx, t, dl, T))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ld,shift,ld_d,shift_d", [(1031, 0, 1031, 0), (1040, 0, 1024, 0),
                                                   (1024, 1, 1025, 3), (1033, 5, 1033, 5),
                                                   (1026, 2, 1024, 8)])
def test_strides_and_alignment(dtype, ld, shift, ld_d, shift_d):
    z, idx, t, dl = make(7, 1021, 9, dtype, 1.5, ld, ld=ld, shift=shift)
    check(z, idx, t, dl, 1.5, calls(z, idx, t, dl, 1.5, ld_d, shift_d))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,ld", [(1000, 1000), (4099, 4103), (40000, 40000)])
def test_in_place(dtype, V, ld):
    z, idx, t, dl = make(6, V, 12, dtype, 2.0, V, ld=ld)
    check(z, idx, t, dl, 2.0, calls(z, idx, t, dl, 2.0, in_place=True))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_rows_than_run_at_once(dtype):
    z, idx, t, dl = make(1700, 333, 5, dtype, 1.0, 6)
    check(z, idx, t, dl, 1.0, calls(z, idx, t, dl, 1.0))


# many rows of every form: a warp each, one CTA each, clusters of two to eight; a row longer than
# a cluster holds
@pytest.mark.parametrize("dtype,B,V,ld", [(BF16, 700, 2001, 2003), (F32, 650, 1000, 1001),
                                          (BF16, 700, 500, 512), (F32, 610, 64, 67),
                                          (BF16, 620, 4000, 4001), (F32, 330, 20000, 20000),
                                          (BF16, 200, 60001, 60001), (F32, 70, 90000, 90001),
                                          (BF16, 4, 262160, 262160), (F32, 3, 131080, 131081),
                                          (F32, 2, 200001, 200001), (BF16, 2, 300003, 300007),
                                          (F32, 5, 390000, 390001), (BF16, 2, 800003, 800003),
                                          (F32, 2, 400001, 400004)])
def test_rows_of_every_form(dtype, B, V, ld):
    z, idx, t, dl = make(B, V, 10, dtype, 2.0, V, ld=ld)
    check(z, idx, t, dl, 2.0, calls(z, idx, t, dl, 2.0))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,V", [(3, 600), (700, 600), (3, 30000)])
def test_rows_whose_every_logit_is_the_lowest_value(dtype, B, V):
    # the softmax of equal logits is uniform; in one call, as lse in fp32 cannot hold log V here
    z, idx, t, _ = make(B, V, 4, dtype, 1.0, 3)
    z.t.fill_(torch.finfo(dtype).min)
    idx[:] = torch.arange(4, device="cuda")
    loss, lse, dz = torch.empty(B, device="cuda"), torch.empty(B, device="cuda"), torch.empty_like(z.t)
    pk.check(pk.pkm_distill_train(z.t, KIND[dtype], V, B, V, idx, t, 4, 1.0,
                                  torch.ones(B, device="cuda"), loss, lse, dz, V), "train")
    p = torch.softmax(t.double(), 1)
    want = torch.full((B, V), 1 / V, dtype=F64, device="cuda")
    want[:, :4] -= p
    half = U if dtype == F32 else 2.0 ** -8
    assert bool(((dz.double() - want).abs() <= (half + 100 * U) * want.abs() + 100 * U / V).all())
    assert torch.isfinite(loss).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_columns_and_lists(dtype):
    z, idx, t, dl = make(12, 700, 6, dtype, 1.0, 31, masked=100)
    dl.fill_(0.5)
    idx[0] = -1                        # no list
    idx[1] = 5                         # one column six times
    idx[2] = torch.arange(6, device="cuda")
    t[2, 1:] = -math.inf               # one entry with any mass
    idx[3], t[3] = 7, -math.inf        # none with any mass
    z.t[4, :600] = -math.inf           # one live logit besides the masked ones
    z.t[4, 11] = 2.0
    idx[4] = 11
    z.t[5] = torch.finfo(dtype).min    # masks of the lowest value, and one live column
    z.t[5, 3] = 1.0
    idx[5] = 3
    z.t[6, :300] = torch.finfo(dtype).min
    idx[6] = torch.arange(400, 406, device="cuda")
    check(z, idx, t, dl, 1.0, calls(z, idx, t, dl, 1.0))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_masked_column_in_the_list_has_infinite_loss(dtype):
    z, idx, t, dl = make(4, 300, 4, dtype, 1.0, 7, masked=50)
    idx[:] = torch.arange(4, device="cuda")
    idx[1, 2] = 280
    idx[2], t[2] = torch.tensor([280, 1, 2, 3], device="cuda"), torch.tensor([-math.inf, 0, 1, 2.])
    z.t[3] = -math.inf                 # nothing is live: lse is -inf
    dl.fill_(1.0)
    out = calls(z, idx, t, dl, 1.0)
    assert out["f"][0][1] == math.inf and torch.isfinite(out["f"][0][2]) and out["f"][0][3] == math.inf
    assert out["f"][1][3] == -math.inf
    check(z, idx, t, dl, 1.0, out)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_an_index_past_the_vocabulary_is_reported_and_absent(dtype):
    z, idx, t, dl = make(3, 200, 4, dtype, 1.0, 8)
    idx[:] = torch.arange(4, device="cuda")
    idx[1, 3] = 200
    idx[2, 0] = 1 << 40
    check(z, idx, t, dl, 1.0, calls(z, idx, t, dl, 1.0), status=pk.PKM_ERR_BAD_INDEX)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [500, 70000])
def test_rows_that_count_for_nothing_may_hold_anything(dtype, V):
    z, idx, t, dl = make(5, V, 4, dtype, 1.0, 9)
    idx[:] = torch.arange(4, device="cuda")
    dl[:] = torch.tensor([1.0, 0.0, 1.0, 1.0, 0.0])
    clean = calls(z, idx, t, dl, 1.0)
    z.t[1, 17] = math.nan
    z.t[4, 3] = math.inf
    out = calls(z, idx, t, dl, 1.0)
    for a, b in ((out["b"], clean["b"]), (out["t"][2], clean["t"][2])):
        assert torch.equal(a, b) and bool((a[1] == 0).all()) and bool((a[4] == 0).all())
    assert bool(out["f"][0][1].isnan()) and torch.equal(out["f"][0][[0, 2, 3]],
                                                        clean["f"][0][[0, 2, 3]])


@pytest.mark.parametrize("T", [0.25, 1.0, 8.0])
def test_gradient_is_the_losses_difference(T):
    # one row shifted by +-e at one column, as rows of one batch; the loss is good to about 1e-5,
    # its third derivative is below 1 / T
    V, k, e = 300, 5, 0.02
    gen = torch.Generator(device="cuda").manual_seed(2)
    base = torch.randn(V, device="cuda", generator=gen) * min(2.0, 2 * T)
    at = [0, 3, 17, 150, 299]
    z = base.repeat(2 * len(at), 1)
    for i, v in enumerate(at):
        z[2 * i, v] += e
        z[2 * i + 1, v] -= e
    idx = torch.tensor([3, 17, 40, 41, 299], device="cuda").repeat(z.shape[0], 1)
    t = (torch.randn(k, device="cuda", generator=gen) * min(2.0, 2 * T)).repeat(z.shape[0], 1)
    loss = torch.empty(z.shape[0], device="cuda")
    pk.check(pk.pkm_distill(z, pk.PKM_F32, V, z.shape[0], V, idx, t, k, T, loss), "forward")
    one, lse, dz = torch.empty(1, device="cuda"), torch.empty(1, device="cuda"), torch.empty(1, V, device="cuda")
    pk.check(pk.pkm_distill_train(base[None], pk.PKM_F32, V, 1, V, idx[:1], t[:1], k, T,
                                  torch.ones(1, device="cuda"), one, lse, dz, V), "train")
    for i, v in enumerate(at):
        step = float(z[2 * i, v].double() - z[2 * i + 1, v].double())
        num = float(loss[2 * i].double() - loss[2 * i + 1].double()) / step
        noise = 2 * (2 * U * abs(float(loss[0])) + 2e-6 * T * T) / step
        assert abs(num - float(dz[0, v])) <= noise + e * e / 6 / T * 2, (v, num, float(dz[0, v]))


def test_on_another_stream_and_in_a_graph():
    z, idx, t, dl = make(9, 5000, 8, BF16, 2.0, 5)
    want = calls(z, idx, t, dl, 2.0)["t"]
    loss, lse, dz = torch.zeros(9, device="cuda"), torch.zeros(9, device="cuda"), torch.zeros_like(z.t)

    def call():
        pk.check(pk.pkm_distill_train(z.t, pk.PKM_BF16, 5000, 9, 5000, idx, t, 8, 2.0, dl, loss,
                                      lse, dz, 5000), "train")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert torch.equal(dz, want[2]) and torch.equal(loss, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for x in (loss, lse, dz):
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dz, want[2]) and torch.equal(loss, want[0]) and torch.equal(lse, want[1])
