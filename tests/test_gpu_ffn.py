"""The gated feed-forward block on the GPU against its 64-bit form.

Tolerances: a value rounded to bf16 is off by at most 2^-8 of itself, and, over many values, by at
most 2^-8 / sqrt(3) in the 2-norm (errors spread evenly over half a step either side, all values
at the bottom of a binade).  Two bounds are derived from that: one for each element, in which
every rounding is at its worst and in the same direction, and one for the 2-norm, in which n
independent roundings add up as sqrt(n) (times 1.05 for the sample; fp32 sums are far below).
"""
import math

import pytest

import sparse_top_lookup_gb300 as pk
from operators64 import ACTS, act64, ffn64, ffn_backward64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, F64 = torch.bfloat16, torch.float64
HALF = 2.0 ** -8
PAD = 64


def act_id(act):
    return {"silu": pk.PKM_ACT_SILU, "gelu": pk.PKM_ACT_GELU, "gelu_tanh": pk.PKM_ACT_GELU_TANH,
            "relu": pk.PKM_ACT_RELU}[act]


class Guarded:
    """A matrix inside a larger buffer whose other values must not change."""

    def __init__(self, *shape, dtype=BF16, fill=None):
        n = math.prod(shape)
        self.all = torch.full((n + 2 * PAD,), -777.0, device="cuda").to(dtype)
        self.t = self.all[PAD:PAD + n].view(shape)
        self.t.fill_(float("nan") if fill is None else fill)

    def ok(self):
        m = self.all[0].item()
        return bool((self.all[:PAD] == m).all()) and bool((self.all[-PAD:] == m).all())


def inputs(B, dim, F, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sd=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * sd).to(BF16)
    return (normal(B, dim, sd=scale), normal(F, dim, sd=dim ** -0.5),
            normal(F, dim, sd=dim ** -0.5), normal(dim, F, sd=F ** -0.5), normal(B, dim))


def forward(x, wg, wu, wd, act, keep=True, stream=None):
    (B, dim), F = x.shape, wg.shape[0]
    y = Guarded(B, dim)
    g, u = (Guarded(B, F), Guarded(B, F)) if keep else (None, None)
    ws = Guarded(pk.pkm_gated_ffn_workspace_bytes(B, dim, F), dtype=torch.uint8, fill=255)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.check(pk.pkm_gated_ffn(x, wg, wu, wd, B, dim, F, act_id(act), ws.t, y.t,
                              g.t if keep else None, u.t if keep else None, status, stream), "ffn")
    torch.cuda.synchronize()
    assert status.item() == pk.PKM_OK
    assert y.ok() and ws.ok() and (not keep or (g.ok() and u.ok()))
    return y.t, (g.t if keep else None), (u.t if keep else None)


def near(got, want, each, roundings, what):
    """Element bound `each` (a tensor), and the 2-norm's for so many independent roundings."""
    got = got.to(F64)
    assert torch.isfinite(got).all(), what
    off = (got - want).abs()
    assert bool((off <= each).all()), "%s: off by %g where %g is allowed" % (
        what, off[off > each].max(), each[off > each].min())
    norm = want.norm()
    if want.numel() >= 4096 and norm > 0:
        rel = float((got - want).norm() / norm)
        assert rel <= 1.05 * math.sqrt(roundings) * HALF / math.sqrt(3), (what, rel)


def check_forward(x, wg, wu, wd, act, keep=True):
    y, g, u = forward(x, wg, wu, wd, act, keep)
    X, G, U, D = (t.to(F64) for t in (x, wg, wu, wd))
    g64, u64, h64, y64 = ffn64(X, G, U, D, act)
    dim, F = G.shape[1], G.shape[0]
    # an fp32 sum of n terms is off by at most n 2^-24 of the sum of their magnitudes
    eg = dim * 2.0 ** -24 * (X.abs() @ G.abs().T)
    eu = dim * 2.0 ** -24 * (X.abs() @ U.abs().T)
    if keep:
        near(g, g64, HALF * g64.abs() + 2 * eg, 1, "g")
        near(u, u64, HALF * u64.abs() + 2 * eu, 1, "u")
    a64, slope = act64(g64, act)
    # (slopes are at most 1.13, and change by at most eg over the error itself; the activations'
    # own fp32 arithmetic is good to 2^-18 of |g|)
    eh = (HALF * h64.abs() + 1.2 * eg * u64.abs() + a64.abs() * eu + eg * eu
          + 2.0 ** -18 * g64.abs() * u64.abs())
    ey = eh @ D.abs().T + F * 2.0 ** -24 * (h64.abs() @ D.abs().T)
    near(y, y64, 1.01 * (HALF * y64.abs() + (1 + HALF) * ey) + 1e-30, 2, "y")


SHAPES = [(1, 8, 8), (1, 64, 256), (2, 72, 136), (7, 200, 520), (31, 64, 64), (64, 256, 512),
          (65, 128, 384), (127, 136, 264), (128, 512, 1400), (129, 264, 520), (255, 64, 128),
          (256, 256, 256), (257, 320, 776), (300, 1024, 2048), (777, 520, 1032), (1030, 72, 2056)]


@pytest.mark.parametrize("B,dim,F", SHAPES)
def test_forward(B, dim, F):
    check_forward(*inputs(B, dim, F, B + dim + F)[:4], act=ACTS[(B + F // 8) % 4])


# few tokens: tiles of every height, shared by one CTA to eight, K tails, more tiles than SMs
@pytest.mark.parametrize("B,dim,F", [(1, 1024, 4096), (16, 1024, 2048), (17, 2048, 520),
                                     (48, 200, 5000), (64, 1032, 4104), (3, 64, 20480),
                                     (2, 4096, 256), (63, 136, 136), (64, 8, 1000)])
def test_few_tokens(B, dim, F):
    check_forward(*inputs(B, dim, F, B + dim + F)[:4], act=ACTS[(dim // 8) % 4])
    check_backward(B, dim, F, ACTS[(F // 8) % 4], seed=F)


# few tiles of long products: tiles cut along K, and joined in a fixed order
@pytest.mark.parametrize("B,dim,F", [(200, 256, 8192), (129, 264, 6000), (513, 136, 5000),
                                     (150, 1024, 4096), (300, 2048, 2048)])
def test_cut_tiles(B, dim, F):
    x, wg, wu, wd, _ = inputs(B, dim, F, B + dim)
    check_forward(x, wg, wu, wd, "silu")
    check_backward(B, dim, F, "gelu_tanh", seed=F)
    check_backward(B, dim, F, "silu", seed=F, grad_dtype=pk.PKM_F32)
    y = forward(x, wg, wu, wd, "silu")[0].clone()
    assert torch.equal(forward(x, wg, wu, wd, "silu")[0], y)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("B", [3, 200])
def test_activations(act, B):
    # gate values out to about +-40: both tails of every activation
    check_forward(*inputs(B, 256, 264, 5, scale=10.0)[:4], act=act, keep=False)


def test_more_tiles_than_clusters():
    check_forward(*inputs(2500, 256, 2304, 9)[:4], act="silu")


def check_backward(B, dim, F, act, seed=1, grad_dtype=None, skip=()):
    grad_dtype = pk.PKM_BF16 if grad_dtype is None else grad_dtype
    f32 = grad_dtype == pk.PKM_F32
    x, wg, wu, wd, dy = inputs(B, dim, F, seed)
    g, u = (x.float() @ wg.float().T).to(BF16), (x.float() @ wu.float().T).to(BF16)
    out = {"dx": Guarded(B, dim)}
    kind = dict(dtype=torch.float32, fill=3.0) if f32 else dict()
    out.update(dwg=Guarded(F, dim, **kind), dwu=Guarded(F, dim, **kind),
               dwd=Guarded(dim, F, **kind))
    ws = Guarded(pk.pkm_gated_ffn_backward_workspace_bytes(B, dim, F), dtype=torch.uint8, fill=255)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    arg = {n: None if n in skip else o.t for n, o in out.items()}
    pk.check(pk.pkm_gated_ffn_backward(x, wg, wu, wd, g, u, dy, B, dim, F, act_id(act), ws.t,
                                       arg["dx"], arg["dwg"], arg["dwu"], arg["dwd"], grad_dtype,
                                       status), "ffn backward")
    torch.cuda.synchronize()
    assert status.item() == pk.PKM_OK and ws.ok() and all(o.ok() for o in out.values())
    X, G, U, D, Y, g64, u64 = (t.to(F64) for t in (x, wg, wu, wd, dy, g, u))
    ref = ffn_backward64(X, G, U, D, g64, u64, Y, act)
    a, da = (t.abs() for t in act64(g64, act))
    edh = dim * 2.0 ** -24 * (Y.abs() @ D.abs())  # the fp32 sum dh
    dh = (Y @ D).abs()
    eps = 2.0 ** -17  # the slopes' own fp32 arithmetic, of at most 1.13 + |g|'s share of it
    edg = HALF * ref["dg"].abs() + (1 + HALF) * u64.abs() * (
        edh * da + dh * eps * (1 + g64.abs()))
    edu = HALF * ref["du"].abs() + (1 + HALF) * (edh * a + dh * eps * g64.abs())
    eh = HALF * ref["h"].abs() + eps * g64.abs() * u64.abs()
    sums = dict(dx=(edg @ G.abs() + edu @ U.abs(), ref["dg"].abs() @ G.abs()
                    + ref["du"].abs() @ U.abs(), 2 * F),
                dwg=(edg.T @ X.abs(), ref["dg"].abs().T @ X.abs(), B),
                dwu=(edu.T @ X.abs(), ref["du"].abs().T @ X.abs(), B),
                dwd=(Y.abs().T @ eh, Y.abs().T @ ref["h"].abs(), B))
    for n, (e, s, terms) in sums.items():
        if n in skip:
            assert bool((out[n].t == 3.0).all() if f32 and n != "dx" else out[n].t.isnan().all())
            continue
        e = e + (terms + 2) * 2.0 ** -24 * s
        if f32 and n != "dx":
            got = out[n].t.to(F64) - 3.0  # added to what was there
            near(got, ref[n], 1.01 * e + 2.0 ** -23 * (3 + ref[n].abs()) + 1e-30, 1, n)
        else:
            near(out[n].t, ref[n], 1.01 * (HALF * ref[n].abs() + (1 + HALF) * e) + 1e-30, 2, n)


@pytest.mark.parametrize("B,dim,F", SHAPES)
def test_backward(B, dim, F):
    check_backward(B, dim, F, ACTS[(B + F // 8 + 1) % 4], seed=B + F)


@pytest.mark.parametrize("act", ACTS)
def test_backward_activations(act):
    check_backward(333, 264, 520, act)


@pytest.mark.parametrize("B,dim,F", [(5, 72, 136), (300, 256, 520), (1500, 512, 1024)])
def test_backward_accumulates_in_fp32(B, dim, F):
    check_backward(B, dim, F, "silu", grad_dtype=pk.PKM_F32)


@pytest.mark.parametrize("skip", [("dx",), ("dwg", "dwu"), ("dwd",), ("dx", "dwd")])
@pytest.mark.parametrize("f32", [False, True])
def test_backward_leaves_out_what_is_not_asked_for(skip, f32):
    check_backward(130, 136, 264, "silu", grad_dtype=pk.PKM_F32 if f32 else None, skip=skip)


def test_gradient_is_the_forward_passes_difference():
    # L = sum(dy * y) along a direction of wd: linear in wd, so a difference over any step is its
    # gradient, up to the roundings of y (2^-8 each, B * dim of them, independent) over the step
    B, dim, F = 256, 128, 256
    x, wg, wu, wd, dy = inputs(B, dim, F, 12)
    _, g, u = forward(x, wg, wu, wd, "silu")
    dwd = torch.empty_like(wd)
    ws = torch.empty(pk.pkm_gated_ffn_backward_workspace_bytes(B, dim, F), dtype=torch.uint8,
                     device="cuda")
    pk.check(pk.pkm_gated_ffn_backward(x, wg, wu, wd, g, u, dy, B, dim, F, 0, ws, None, None, None,
                                       dwd), "backward")
    v = torch.randn(dim, F, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    v = (v * F ** -0.5).to(BF16)
    y1 = forward(x, wg, wu, (wd + v).to(BF16), "silu")[0].to(F64)
    y0 = forward(x, wg, wu, wd, "silu")[0].to(F64)
    step = (wd + v).to(BF16).to(F64) - wd.to(F64)
    num = float((dy.to(F64) * (y1 - y0)).sum())
    got = float((dwd.to(F64) * step).sum())
    # six standard deviations of the roundings of y1 and y0, and of dwd's
    sd = HALF / math.sqrt(3) * math.sqrt(float(((dy.to(F64) * y1) ** 2).sum()
                                               + ((dy.to(F64) * y0) ** 2).sum()
                                               + ((dwd.to(F64) * step) ** 2).sum()))
    assert abs(num - got) <= 6 * sd, (num, got, sd)


def test_empty_batch():
    w = torch.zeros(16, 16, dtype=BF16, device="cuda")
    g = torch.full((16, 16), 5.0, dtype=BF16, device="cuda")
    f = torch.full((16, 16), 5.0, device="cuda")
    none = torch.empty(0, 16, dtype=BF16, device="cuda")
    pk.check(pk.pkm_gated_ffn(none, w, w, w, 0, 16, 16, 0, None, none), "forward")
    pk.check(pk.pkm_gated_ffn_backward(none, w, w, w, none, none, none, 0, 16, 16, 0, None, none, g,
                                       g, None), "backward")
    pk.check(pk.pkm_gated_ffn_backward(none, w, w, w, none, none, none, 0, 16, 16, 0, None, none, f,
                                       f, f, pk.PKM_F32), "backward")
    torch.cuda.synchronize()
    assert bool((g == 0).all()) and bool((f == 5).all())


def test_the_same_bits_every_time():
    a = inputs(300, 264, 520, 3)
    y = forward(*a[:4], "gelu")[0].clone()
    for _ in range(3):
        assert torch.equal(forward(*a[:4], "gelu")[0], y)


@pytest.mark.parametrize("B,dim,F", [(77, 128, 264), (5, 128, 264), (33, 512, 1032)])
def test_on_another_stream_and_in_a_graph(B, dim, F):
    x, wg, wu, wd, _ = inputs(B, dim, F, 4)
    want = forward(x, wg, wu, wd, "silu")[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.zeros(B, dim, dtype=BF16, device="cuda")
    ws = torch.empty(pk.pkm_gated_ffn_workspace_bytes(B, dim, F), dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(s):
        pk.check(pk.pkm_gated_ffn(x, wg, wu, wd, B, dim, F, 0, ws, y), "ffn")
    s.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pk.check(pk.pkm_gated_ffn(x, wg, wu, wd, B, dim, F, 0, ws, y), "ffn")
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_nan_stays_in_its_row():
    x, wg, wu, wd, _ = inputs(140, 64, 128, 8)
    want = forward(x, wg, wu, wd, "silu")[0].clone()
    x[131, 5] = float("nan")
    y = forward(x, wg, wu, wd, "silu")[0]
    assert bool(y[131].isnan().all())
    rest = torch.arange(140, device="cuda") != 131
    assert torch.equal(y[rest], want[rest])
