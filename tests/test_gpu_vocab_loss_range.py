"""The head's product with its cross entropy at the ends of its range: what the calls of pkm_vocab_loss
agree on there.

Tolerances as in test_gpu_vocab_loss.py.
"""
import math

import pytest

import sparse_top_lookup_gb300 as pk
from more_operators64 import Guarded, vocab64
from test_gpu_vocab_loss import (BF16, F64, HALF, check_loss, errors_of_logits, far, forward, gradient,
                                 inputs, loss_bounds, near)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BIG = 1e25  # bf16; its square overflows fp32


def with_infinities(B, dim, V, seed=0):
    """Inputs, and tokens by what their logits hold.  Column 0 of x is BIG in those tokens and 0 in the
    others, column 0 of W is +-BIG in three rows; column 1 of x moves all of a token's logits."""
    x, w, target, dloss = inputs(B, dim, V, seed=seed, absent=0.0)
    up, down, down2 = V // 3, V // 2, V - 1
    w[:, 0], x[:, 0] = 0, 0
    w[:, 1], x[:, 1] = 1, 0
    keep = (target == up) | (target == down) | (target == down2)
    target[keep] = 1
    w[up, 0], w[down, 0], w[down2, 0] = BIG, -BIG, -BIG
    return x, w, target, dloss, up, down


@pytest.mark.parametrize("B,V", [(1, 700), (5, 300), (150, 700), (150, 30000)])
@pytest.mark.parametrize("kind", ["target", "other", "padding"])
def test_a_logit_of_plus_infinity(B, V, kind):
    # inf - inf where it is the target's, the limit where it is another's; in every call
    x, w, target, dloss, up, _ = with_infinities(B, 64, V)
    b = B // 2
    x[b, 0] = BIG
    target[b] = up if kind == "target" else -1 if kind == "padding" else 0
    rest = torch.arange(B, device="cuda") != b
    got = dict(zip(("loss", "lse"), forward(x, w, target)))
    calls = [got, gradient(x, w, target, dloss, True)]
    calls.append(gradient(x, w, target, dloss, False, lse=got["lse"]))
    for c in calls:
        if "loss" in c:
            assert c["lse"][b].item() == math.inf
            want = {"target": math.nan, "other": math.inf, "padding": 0.0}[kind]
            assert c["loss"][b].item() == want or (math.isnan(want) and bool(c["loss"][b].isnan()))
            if B > 1:
                check_loss(x[rest], w, target[rest], (c["loss"][rest], c["lse"][rest]))
        if "dx" in c:
            if kind == "padding":
                assert bool((c["dx"][b] == 0).all()) and bool(torch.isfinite(c["dw"]).all())
            else:
                assert bool(c["dx"][b].isnan().all())
                assert bool(c["dw"][target[b]].isnan().all()) and bool(c["dw"][up].isnan().all())
                others = torch.ones(V, dtype=torch.bool, device="cuda")
                others[[up, int(target[b])]] = False
                assert bool(torch.isfinite(c["dw"][others]).all())
            assert bool(torch.isfinite(c["dx"][rest]).all())


@pytest.mark.parametrize("B,V", [(1, 700), (5, 300), (150, 700), (150, 30000)])
@pytest.mark.parametrize("move", [0.0, -160.0, 300.0])
@pytest.mark.parametrize("kind", ["target", "other", "padding"])
def test_a_logit_of_minus_infinity(B, V, kind, move):
    # a power of 0: only the loss of such a target is infinite
    x, w, target, dloss, up, down = with_infinities(B, 64, V, seed=1)
    w[up, 0] = 0
    b = B // 2
    x[b, 0], x[b, 1] = BIG, move
    target[b] = down if kind == "target" else -1 if kind == "padding" else 0
    X, W = x.to(F64), w.to(F64)
    Z = X @ W.T
    Z[b, [down, V - 1]] = -math.inf
    lse = torch.logsumexp(Z, 1)
    # (the logits' own error, and the sums': as loss_bounds, without the infinite ones)
    finite = torch.ones(V, dtype=torch.bool, device="cuda")
    finite[[down, V - 1]] = False
    same = target.clone()
    same[b] = -1 if kind != "other" else 0
    e_loss, e_lse = loss_bounds(x, w[finite], same.clamp(max=int(finite.sum()) - 1))[2:]
    got = dict(zip(("loss", "lse"), forward(x, w, target)))
    step = gradient(x, w, target, dloss, True)
    back = gradient(x, w, target, dloss, False, lse=lse.float())
    for c in (got, step):
        assert abs(float(c["lse"][b].to(F64) - lse[b])) <= 1.05 * float(e_lse[b])
        if kind == "target":
            assert c["loss"][b].item() == math.inf
        elif kind == "padding":
            assert c["loss"][b].item() == 0
        else:
            assert abs(float(c["loss"][b].to(F64) - (lse[b] - Z[b, 0]))) <= 1.05 * float(e_loss[b])
    # dz in 64 bits; x's column 0 takes part in dW's column 0 alone, W's in dx's
    there = target >= 0
    scale = (dloss.to(F64) * there)[:, None]
    dz = torch.exp(Z - lse[:, None])
    ez = errors_of_logits(x * (torch.arange(64, device="cuda") > 0), w)
    ez += 2.0 ** -20 * (2 + Z.abs().nan_to_num(0, 0, 0) + lse.abs()[:, None])
    eo = 1.05 * scale * dz * ez
    dz[torch.arange(B, device="cuda")[there], target[there]] -= 1
    dz *= scale
    e = HALF * dz.abs() + eo
    for c in (step, back):
        sums = (V + 2) * 2.0 ** -24 * (dz.abs() @ W.abs())
        checks = [("dx", dz @ W, e @ W.abs() + sums)]
        sums = (B + 2) * 2.0 ** -24 * (dz.abs().T @ X.abs())
        checks.append(("dw", dz.T @ X, e.T @ X.abs() + HALF * (dz.abs() + e).T @ X.abs() + sums))
        for name, want, bound in checks:
            each = 1.02 * (HALF * want.abs() + (1 + HALF) * bound) + 1e-38
            near(c[name][:, 1:], want[:, 1:], each[:, 1:], 0, name)


# ------------------------------------------------------------------ weights


def check_kept(x, w, target, dloss):
    """The gradient's calls where a training step keeps powers.  dz is rounded once and the results are; x with
    its factor once more, and in a training step that factor may take a rounding back: it is that of the
    target's power, half a step of bf16 at most, and comes to the row's other elements instead.  Then an element
    of dW is off by four half steps, each of what it sums, and one of dx by two."""
    (B, dim), V = x.shape, w.shape[0]
    assert -(-B // 256) * -(-V // 256) > 76
    X, W = x.to(F64), w.to(F64)
    loss, lse, e_loss, e_lse = loss_bounds(x, w, target)
    _, _, dz = vocab64(X, W, target, dloss.to(F64))
    Z = X @ W.T
    ez = errors_of_logits(x, w) + 2.0 ** -23 * far(Z, target)
    there = (target >= 0) & (target < V)
    at = torch.where(there, target, torch.zeros_like(target))[:, None]
    scale = torch.where(there, dloss.to(F64).abs(), torch.zeros_like(lse))[:, None]
    p = torch.exp(Z - lse[:, None])
    for train in (False, True):
        el = (e_lse if train else torch.zeros_like(lse)) + 2.0 ** -24 * lse.abs()
        eo = 1.05 * scale * p * (ez + el[:, None] + 2.0 ** -20)
        if train:
            eo = eo.scatter(1, at, 1.05 * scale * (e_loss + 2.0 ** -22 * -torch.expm1(-loss))[:, None])
        edz = HALF * dz.abs() + eo
        got = gradient(x, w, target, dloss, train, lse=lse.float())
        if train:
            check_loss(x, w, target, (got["loss"], got["lse"]))
        sums = (V + 2) * 2.0 ** -24 * (dz.abs() @ W.abs())
        want = dz @ W
        near(got["dx"], want, 1.01 * (HALF * want.abs() + (1 + HALF) * (edz @ W.abs() + sums)) + 1e-38, 2,
             "dx", eo @ W.abs() + sums)
        sums = (B + 2) * 2.0 ** -24 * (dz.abs().T @ X.abs())
        want = dz.T @ X
        more = (2 if train else 1) * 1.01 * HALF * ((dz.abs() + edz).T @ X.abs())
        each = HALF * want.abs() + (1 + HALF) * (edz.T @ X.abs() + sums + more)
        near(got["dw"], want, 1.01 * each + 1e-38, 4 if train else 3, "dw", eo.T @ X.abs() + sums)


def far_rows(B, dim, V, seed):
    """Tokens whose target lies 40 to 65 below their best logit."""
    x, w, target, _ = inputs(B, dim, V, seed=seed, absent=0.0, sd=7.0, lift=0.0)
    z = x.to(F64) @ w.to(F64).T
    gap = z.amax(1, keepdim=True) - z
    gen = torch.Generator(device="cuda").manual_seed(seed)
    aim = 40 + 25 * torch.rand(B, 1, device="cuda", generator=gen, dtype=F64)
    target = (gap - aim).abs().argmin(1)
    at = gap.gather(1, target[:, None])
    assert float(at.min()) > 35 and float(at.max()) < 67
    return x, w, target


@pytest.mark.parametrize("dim", [64, 200])
@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-8, 1e-10, 1e-12, 1e-16])
def test_tokens_far_from_their_targets_with_small_weights(size, dim):
    # a step that keeps powers: rows' factors down to 2^-94 of dloss
    B = 100
    x, w, target = far_rows(B, dim, 30000, seed=3)
    dloss = size * (0.5 + torch.rand(B, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)))
    check_kept(x, w, target, dloss)


@pytest.mark.parametrize("first", [0.0, 1e-30, 1e30, math.nan])
def test_tokens_of_very_different_weight_in_a_step_that_keeps_powers(first):
    x, w, target, dloss = inputs(100, 64, 30000, seed=8, absent=0.0)
    target[:40] = -1
    dloss[:40] = first  # (padding: whatever it holds)
    check_kept(x, w, target, dloss)
    if first == 0.0:
        dloss[50], dloss[60:] = 1e-6, 1e-12
        check_kept(x, w, target, dloss)
        dloss[:] *= 1e-16
        check_kept(x, w, target, dloss)


def test_one_light_token_far_from_its_target():
    # its target's row and its best logit's get next to nothing from the others
    x, w, target = far_rows(100, 64, 30000, seed=5)
    dloss = torch.full((100,), 1.0, device="cuda")
    dloss[1:] = 1e-10
    check_kept(x, w, target, dloss)
    check_kept(x, w, target, dloss.flip(0).contiguous())


@pytest.mark.parametrize("B,dim,V", [(2000, 256, 10000), (500, 512, 30000)])
def test_a_steps_dw_in_the_2_norm(B, dim, V):
    # tokens learnt to some part: the target's element is most of dz, and its rounding is not in dW.  What is:
    # x's with the factor and the result's, which are formed here, and both of the other elements' share
    x, w, target, _ = inputs(B, dim, V, seed=1, absent=0.0, lift=math.log(V))
    dloss = torch.full((B,), 1 / B, device="cuda")
    X, W = x.to(F64), w.to(F64)
    loss, lse, dz = vocab64(X, W, target, dloss.to(F64))
    want = dz.T @ X
    factor = (torch.exp((X * W[target]).sum(1) - lse) / B)[:, None]
    xs = (X * factor).to(BF16).to(F64) / factor
    fewest = (dz.T @ xs).to(BF16).to(F64) - want
    size = X.square().sum(1)
    own = dz.gather(1, target[:, None])[:, 0].square()
    share = float(((dz.square().sum(1) - own) * size).sum() / (dz.square().sum(1) * size).sum())
    dw = gradient(x, w, target, dloss, True)["dw"].to(F64)
    off, norm = float((dw - want).norm() / want.norm()), float(fewest.norm() / want.norm())
    assert off <= 1.03 * math.sqrt(norm ** 2 + 2 * share * HALF ** 2 / 3), (off, norm, share)



# ------------------------------------------------------------------ learnt tokens


def learnt(dim, V, far, move, seed):
    """One token, some `far` ahead in its target's logit, which is a sum of terms of either sign; all
    logits are moved by `move`."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(V, dim, device="cuda", generator=gen) * 0.05).to(BF16)
    target = torch.tensor([V // 2], device="cuda")
    w[target] = torch.randn(1, dim, device="cuda", generator=gen).to(BF16)
    x = torch.randn(1, dim, device="cuda", generator=gen)
    t = w[target].float()
    x += t * (far - (x * t).sum()) / t.square().sum()
    x[:, 0], w[:, 0] = move, 1
    return x.to(BF16), w, target, torch.ones(1, device="cuda")


def with_loss(x, w, target, lse, loss, dloss, grad_dtype=pk.PKM_BF16, status=None, stream=None):
    (B, dim), V = x.shape, w.shape[0]
    f32 = grad_dtype == pk.PKM_F32
    dx = Guarded(B, dim, dtype=BF16)
    dw = Guarded(V, dim, dtype=torch.float32, fill=3.0) if f32 else Guarded(V, dim, dtype=BF16)
    ws = Guarded(pk.pkm_vocab_loss_backward_workspace_bytes(B, dim, V, grad_dtype), dtype=torch.uint8,
                 fill=255)
    pk.check(pk.pkm_vocab_loss_backward_with_loss(x, w, target, lse, loss, dloss, B, dim, V, ws.t, dx.t,
                                                  dw.t, grad_dtype, status, stream), "backward")
    torch.cuda.synchronize()
    assert dx.ok() and dw.ok() and ws.ok()
    return {"dx": dx.t, "dw": dw.t}


@pytest.mark.parametrize("dim", [64, 512, 2048])
@pytest.mark.parametrize("V", [500, 40000])
@pytest.mark.parametrize("move", [0, -100])
def test_a_learnt_tokens_gradient(V, dim, move):
    # from lse: off by the lse's rounding and the logit's fp32 sum; with the loss: by three roundings of
    # its own size
    for i, far in enumerate(range(10, 60, 3)):
        x, w, target, dloss = learnt(dim, V, far, move, seed=i)
        X, W = x.to(F64), w.to(F64)
        loss64, lse64, dz = vocab64(X, W, target, dloss.to(F64))
        want = dz[0, target[0]] * X[0]
        sizes = (X[0].abs() * W[target[0]].abs()).sum()
        got = gradient(x, w, target, dloss, False, lse=lse64.float())["dw"][target[0]].to(F64)
        # a lane's sum of dim / 32 products and five additions; lse and its difference are rounded
        e = (dim / 32 + 6) * 2.0 ** -24 * sizes + 2 * 2.0 ** -24 * lse64.abs()
        each = 1.01 * (3 * HALF * want.abs() + e * X[0].abs()) + 1e-38
        off = (got - want).abs()
        assert bool((off <= each).all()), (far, float((off - each).max()))
        # the forward's own loss, good to its bound
        loss, lse = forward(x, w, target)
        got = with_loss(x, w, target, lse, loss, dloss)["dw"][target[0]].to(F64)
        e = loss_bounds(x, w, target)[2] / loss64 + 2.0 ** -20
        assert bool(((got - want).abs() <= 1.01 * (3 * HALF + e) * want.abs() + 1e-38).all()), far


@pytest.mark.parametrize("V", [500, 40000])
@pytest.mark.parametrize("off", [-0.03, 0.03, -3.0])
def test_the_backward_pass_from_an_lse_of_other_logits(off, V):
    # exp(z - lse) - [target] of the lse it is given, which may be above 0 at a target
    B, dim = 150, 128
    x, w, target, dloss = inputs(B, dim, V, seed=6, lift=14.0)
    X, W = x.to(F64), w.to(F64)
    Z = X @ W.T
    lse = (torch.logsumexp(Z, 1) + off).float()
    got = gradient(x, w, target, dloss, False, lse=lse)
    there = target >= 0
    scale = (dloss.to(F64) * there)[:, None]
    p = torch.exp(Z - lse.to(F64)[:, None])
    dz = p.scatter_add(1, target.clamp(min=0)[:, None], -torch.ones(B, 1, dtype=F64, device="cuda")) * scale
    if off < 0:
        at = dz.gather(1, target.clamp(min=0)[:, None])[there]
        assert bool((at > 0).any())
    eo = 1.05 * scale * p * (errors_of_logits(x, w) + 2.0 ** -20 * (1 + lse.to(F64).abs()[:, None] + Z.abs()))
    e = HALF * dz.abs() + eo
    sums = (V + 2) * 2.0 ** -24 * (dz.abs() @ W.abs())
    want = dz @ W
    near(got["dx"], want, 1.01 * (HALF * want.abs() + (1 + HALF) * (e @ W.abs() + sums)) + 1e-38, 2, "dx",
         eo @ W.abs() + sums)
    sums = (B + 2) * 2.0 ** -24 * (dz.abs().T @ X.abs())
    want = dz.T @ X
    bound = e.T @ X.abs() + sums + 1.01 * HALF * ((dz.abs() + e).T @ X.abs())
    near(got["dw"], want, 1.01 * (HALF * want.abs() + (1 + HALF) * bound) + 1e-38, 3, "dw",
         eo.T @ X.abs() + sums)


@pytest.mark.parametrize("B,dim,V", [(1, 64, 40000), (130, 136, 4099), (257, 264, 513), (1001, 520, 3001),
                                     (33000, 16, 300), (20, 264, 50257)])
def test_the_forward_and_the_backward_pass_with_its_loss(B, dim, V):
    # are the step that forms all products
    x, w, target, dloss = inputs(B, dim, V, seed=V)
    loss, lse = forward(x, w, target)
    X, W = x.to(F64), w.to(F64)
    _, _, dz = vocab64(X, W, target, dloss.to(F64))
    e_loss, e_lse = loss_bounds(x, w, target)[2:]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = with_loss(x, w, target, lse, loss, dloss, status=status)
    assert status.item() == pk.PKM_OK
    eo = 1.05 * (dz.abs() * (errors_of_logits(x, w) + e_lse[:, None] + 2.0 ** -20 * (1 + lse.to(F64).abs()[:, None])))
    there = target >= 0
    at = target.clamp(min=0)[:, None]
    mine = 1.05 * (dloss.to(F64) * there * (e_loss + 2.0 ** -22))[:, None]
    eo = eo.scatter(1, at, mine)
    e = HALF * dz.abs() + eo
    sums = (V + 2) * 2.0 ** -24 * (dz.abs() @ W.abs())
    want = dz @ W
    near(got["dx"], want, 1.01 * (HALF * want.abs() + (1 + HALF) * (e @ W.abs() + sums)) + 1e-38, 2, "dx",
         eo @ W.abs() + sums)
    sums = (B + 2) * 2.0 ** -24 * (dz.abs().T @ X.abs())
    want = dz.T @ X
    bound = e.T @ X.abs() + sums + 1.01 * HALF * ((dz.abs() + e).T @ X.abs())
    near(got["dw"], want, 1.01 * (HALF * want.abs() + (1 + HALF) * bound) + 1e-38, 3, "dw",
         eo.T @ X.abs() + sums)
    added = with_loss(x, w, target, lse, loss, dloss, pk.PKM_F32)
    assert torch.equal(added["dx"], got["dx"])
    near(added["dw"].to(F64) - 3.0, want, 1.01 * bound + 2.0 ** -23 * (3 + want.abs()), 0, "dw")
    if -(-B // 256) * -(-V // 256) <= 76:  # (one round of tiles: the training step does the same)
        step = gradient(x, w, target, dloss, True)
        assert torch.equal(step["loss"], loss) and torch.equal(step["lse"], lse)
        assert torch.equal(step["dx"], got["dx"]) and torch.equal(step["dw"], got["dw"])


def test_the_backward_pass_with_its_loss_on_another_stream_and_in_a_graph():
    x, w, target, dloss = inputs(300, 136, 5001, seed=2)
    B, dim, V = 300, 136, 5001
    target[7] = V  # (counts for nothing, and is reported)
    loss, lse = forward(x, w, target, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = with_loss(x, w, target, lse, loss, dloss, status=status)
    assert status.item() == pk.PKM_ERR_BAD_INDEX and bool((want["dx"][7] == 0).all())
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = with_loss(x, w, target, lse, loss, dloss)
    assert all(torch.equal(got[n], want[n]) for n in want)
    out = {n: torch.empty_like(t) for n, t in want.items()}
    ws = torch.full((pk.pkm_vocab_loss_backward_workspace_bytes(B, dim, V),), 255, dtype=torch.uint8,
                    device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pk.check(pk.pkm_vocab_loss_backward_with_loss(x, w, target, lse, loss, dloss, B, dim, V, ws,
                                                      out["dx"], out["dw"]), "backward")
    for _ in range(2):
        for t in out.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in want)
