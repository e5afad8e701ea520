"""The operators around a memory layer, as they are measured.

Two operators, each with its gradient:

gated feed-forward block (the dense block that a product-key memory layer stands beside or in
place of), x [B, dim] -> y [B, dim]:
    g = x Wg^T,  u = x Wu^T,  h = act(g) * u,  y = h Wd^T
  "forward"   y alone (serving: one token up to a long prompt)
  "backward"  from dy and the kept g, u: dx, dWg, dWu, dWd
  "train"     the forward pass that keeps g and u, then the backward pass

distillation from a teacher's top logits (idx, teacher [B, k]: a row's k best in the layout that a
lookup returns, -1 where the list is shorter), student logits z [B, V], temperature T:
    p = softmax(teacher / T) over the row's list, q = softmax(z / T) over all V,
    loss[b] = T^2 * sum_j p_j (log p_j - log q[idx_j])
    dz = dloss[b] * T * (sum_j p_j * q - p scattered to idx)
  "forward"   loss and the log-sum-exp of z / T (evaluation)
  "backward"  dz from the kept log-sum-exp
  "train"     loss, log-sum-exp and dz in one call

With `own` false, run() computes them from elementary torch operations in 32 bits, rounded once
at the end; with `own` true it makes the calls of sparse_top_lookup_gb300 that a user makes.
"""
import math

import torch

own = False

ACTS = ("silu", "gelu", "gelu_tanh", "relu")
BF16 = torch.bfloat16


def listed():
    ffn, dis = "ffn", "distill"
    return [
        # one token of one sequence: latency, the weights are read once
        dict(name="ffn one token", op=ffn, mode="forward", B=1, dim=1024, F=4096, act="silu"),
        # a serving batch of single tokens, an odd number of them, wide block
        dict(name="ffn 37 tokens", op=ffn, mode="forward", B=37, dim=2048, F=8192, act="gelu"),
        # one ragged prompt; F a multiple of 8 only
        dict(name="ffn prompt 777", op=ffn, mode="forward", B=777, dim=1024, F=2728, act="silu"),
        # a batch of prompts, the page workload's width
        dict(name="ffn prompt 16384", op=ffn, mode="forward", B=16384, dim=1024, F=4096,
             act="gelu_tanh"),
        # the backward pass of a small odd batch, as in fine-tuning
        dict(name="ffn backward 1001", op=ffn, mode="backward", B=1001, dim=520, F=1400,
             act="relu"),
        # a training step at the mid workload's batch, page width
        dict(name="ffn train 4096", op=ffn, mode="train", B=4096, dim=1024, F=4096, act="silu"),
        # the largest training step: the large workload's width
        dict(name="ffn train 16384", op=ffn, mode="train", B=16384, dim=2048, F=8192, act="silu"),
        # scoring one held-out row: latency
        dict(name="distill one row", op=dis, mode="forward", B=1, V=32000, k=16, dtype="f32",
             T=1.0, pad=0, masked=0),
        # evaluation of a batch, rows padded to another stride, odd vocabulary
        dict(name="distill eval 2000", op=dis, mode="forward", B=2000, V=50257, k=32,
             dtype="bf16", T=2.0, pad=47, masked=0),
        # the gradient alone, from an autograd graph's upstream gradient
        dict(name="distill backward 1500", op=dis, mode="backward", B=1500, V=50257, k=20,
             dtype="f32", T=1.5, pad=0, masked=0),
        # fine-tuning on a small vocabulary
        dict(name="distill train 4096", op=dis, mode="train", B=4096, V=32000, k=32,
             dtype="bf16", T=1.0, pad=0, masked=0),
        # a training step on a large vocabulary whose last columns are padding, masked with -inf
        dict(name="distill train 8192", op=dis, mode="train", B=8192, V=131072, k=64,
             dtype="bf16", T=2.0, pad=0, masked=72),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.55:
        return dict(op="ffn", mode=rng.choice(("forward", "forward", "backward", "train")),
                    B=_log_uniform(rng, 1, 16384), dim=8 * _log_uniform(rng, 16, 256),
                    F=8 * _log_uniform(rng, 32, 1024), act=rng.choice(ACTS))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    V = _log_uniform(rng, 100, 131072)
    B = _log_uniform(rng, 1, min(16384, (8192 if dtype == "bf16" else 4096) * 131072 // V))
    return dict(op="distill", mode=rng.choice(("forward", "backward", "train", "train")), B=B,
                V=V, k=rng.randint(4, 64), dtype=dtype, T=rng.choice((1.0, 1.5, 2.0, 4.0)),
                pad=rng.choice((0, 0, rng.randint(1, 64))),
                masked=rng.choice((0, rng.randint(1, V // 10))))


def _normal(gen, *shape, sd=1.0, dtype=BF16):
    t = torch.empty(shape, device="cuda", dtype=dtype)
    return t.normal_(0.0, sd, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    B = case["B"]
    if case["op"] == "ffn":
        dim, F = case["dim"], case["F"]
        s["x"] = _normal(gen, B, dim)
        s["wg"] = _normal(gen, F, dim, sd=dim ** -0.5)
        s["wu"] = _normal(gen, F, dim, sd=dim ** -0.5)
        s["wd"] = _normal(gen, dim, F, sd=F ** -0.5)
        if case["mode"] != "forward":
            s["dy"] = _normal(gen, B, dim)
        if case["mode"] == "backward":  # what the forward pass kept
            s["g"] = s["x"] @ s["wg"].T
            s["u"] = s["x"] @ s["wu"].T
        return s
    V, k = case["V"], case["k"]
    dtype = BF16 if case["dtype"] == "bf16" else torch.float32
    live = V - case["masked"]
    z = torch.empty(B, V + case["pad"], device="cuda", dtype=dtype)
    z.normal_(0.0, 2.0, generator=gen)
    z = z[:, :V]
    # the teacher's list: best first; where it is shorter than k, and in about one row of 16
    # (padding tokens, which count for nothing) everywhere, -1
    # (distinct columns: one in each of k stretches of the vocabulary, in a random order)
    idx = torch.rand(B, k, device="cuda", generator=gen).argsort(dim=1) * (live // k)
    idx += torch.randint(0, live // k, (B, k), device="cuda", generator=gen)
    # the best of the list weighs about as much as the rest of the vocabulary does together
    centre = math.log(V) + 2 - 3 * math.sqrt(2 * math.log(k))
    teacher = torch.empty(B, k, device="cuda").normal_(centre, 3.0, generator=gen)
    teacher = teacher.sort(dim=1, descending=True).values
    # a student that has learnt some of it
    lift = teacher + torch.empty(B, k, device="cuda").normal_(0.0, 1.5, generator=gen)
    z.scatter_(1, idx, lift.to(dtype))
    if case["masked"]:
        z[:, live:] = -math.inf
    length = torch.randint((k + 1) // 2, 2 * k + 1, (B, 1), device="cuda", generator=gen)
    keep = torch.rand(B, 1, device="cuda", generator=gen) >= 1 / 16
    if B == 1:
        keep.fill_(True)
    idx.masked_fill_((torch.arange(k, device="cuda") >= length) | ~keep, -1)
    s.update(z=z, idx=idx, teacher=teacher)
    s["dloss"] = keep[:, 0].float() / keep.sum().clamp(min=1)
    if case["mode"] == "backward":  # what the forward pass kept
        s["lse"] = torch.logsumexp(z.float() / case["T"], dim=1)
    return s


# ---------------------------------------------------------------- plain form, 32 bits


def _act32(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        e = 1 / (1 + torch.exp(-g))
        return g * e, e * (1 + g * (1 - e))
    if act == "relu":
        return g.clamp(min=0), (g > 0).to(g.dtype)
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * 0.5 ** 0.5))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (0.5 / math.pi) ** 0.5
    c = (2 / math.pi) ** 0.5
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return (0.5 * g * (1 + t),
            0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g))


def _plain_ffn(s):
    x, wg, wu, wd = (s[n].float() for n in ("x", "wg", "wu", "wd"))
    out = {}
    if s["mode"] == "backward":
        g, u = s["g"].float(), s["u"].float()
    else:
        g, u = x @ wg.T, x @ wu.T
    a, da = _act32(g, s["act"])
    h = a * u
    if s["mode"] != "backward":
        out["y"] = (h @ wd.T).to(BF16)
    if s["mode"] == "forward":
        return out
    if s["mode"] == "train":
        out["g"], out["u"] = g.to(BF16), u.to(BF16)
    dy = s["dy"].float()
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    out["dx"] = (dg @ wg + du @ wu).to(BF16)
    out["dwg"], out["dwu"] = (dg.T @ x).to(BF16), (du.T @ x).to(BF16)
    out["dwd"] = (dy.T @ h).to(BF16)
    return out


def _plain_distill(s):
    T, idx = s["T"], s["idx"]
    z = s["z"].float() / T
    at = idx.clamp(min=0)
    if s["mode"] == "backward":
        lse = s["lse"][:, None]
    else:
        top = z.amax(dim=1, keepdim=True)
        total = torch.exp(z - top).sum(dim=1, keepdim=True)
        lse = top + torch.log(total)
    # a row's few listed entries in 64 bits: the loss is a small difference of its terms
    there = idx >= 0
    some = there.any(dim=1, keepdim=True)
    t = s["teacher"].double() / T
    t = t - t.masked_fill(~there, -math.inf).amax(dim=1, keepdim=True)
    e = torch.where(there, torch.exp(t), torch.zeros_like(t))
    mass = torch.where(some, e.sum(dim=1, keepdim=True), torch.ones_like(t[:, :1]))
    p = e / mass
    out = {}
    if s["mode"] != "backward":
        logq = s["z"].gather(1, at).double() / T - (top.double() + torch.log(total.double()))
        term = torch.where(p > 0, p * (t - torch.log(mass) - logq), torch.zeros_like(p))
        out["loss"] = (T * T * term.sum(dim=1)).float()
        out["lse"] = lse[:, 0]
    if s["mode"] != "forward":
        d = torch.exp(z - lse)
        d *= p.sum(dim=1, keepdim=True).float()
        d.scatter_add_(1, at, -p.float())
        d *= s["dloss"][:, None] * T
        out["dz"] = d.to(s["z"].dtype)
    return out


# ------------------------------------------------------------ the framework's operators


def _own_ffn(s):
    import sparse_top_lookup_gb300 as pk
    B, dim, F, mode = s["B"], s["dim"], s["F"], s["mode"]
    act = {"silu": pk.PKM_ACT_SILU, "gelu": pk.PKM_ACT_GELU, "gelu_tanh": pk.PKM_ACT_GELU_TANH,
           "relu": pk.PKM_ACT_RELU}[s["act"]]
    x, wg, wu, wd = s["x"], s["wg"], s["wu"], s["wd"]
    out, g, u = {}, s.get("g"), s.get("u")
    if mode != "backward":
        if mode == "train":
            g, u = (torch.empty(B, F, dtype=BF16, device="cuda") for _ in range(2))
            out["g"], out["u"] = g, u
        out["y"] = torch.empty(B, dim, dtype=BF16, device="cuda")
        ws = torch.empty(pk.pkm_gated_ffn_workspace_bytes(B, dim, F), dtype=torch.uint8,
                         device="cuda")
        pk.check(pk.pkm_gated_ffn(x, wg, wu, wd, B, dim, F, act, ws, out["y"], g, u),
                 "pkm_gated_ffn")
    if mode != "forward":
        out["dx"] = torch.empty_like(x)
        out["dwg"], out["dwu"], out["dwd"] = (torch.empty_like(w) for w in (wg, wu, wd))
        ws = torch.empty(pk.pkm_gated_ffn_backward_workspace_bytes(B, dim, F),
                         dtype=torch.uint8, device="cuda")
        pk.check(pk.pkm_gated_ffn_backward(x, wg, wu, wd, g, u, s["dy"], B, dim, F, act, ws,
                                           out["dx"], out["dwg"], out["dwu"], out["dwd"]),
                 "pkm_gated_ffn_backward")
    return out


def _own_distill(s):
    import sparse_top_lookup_gb300 as pk
    B, V, k, T, z, mode = s["B"], s["V"], s["k"], s["T"], s["z"], s["mode"]
    dtype = pk.PKM_BF16 if s["dtype"] == "bf16" else pk.PKM_F32
    ld = z.stride(0)
    loss, lse = (torch.empty(B, device="cuda") for _ in range(2))
    if mode == "forward":
        pk.check(pk.pkm_distill(z, dtype, ld, B, V, s["idx"], s["teacher"], k, T, loss, lse),
                 "pkm_distill")
        return {"loss": loss, "lse": lse}
    dz = torch.empty(B, V, dtype=z.dtype, device="cuda")
    if mode == "backward":
        pk.check(pk.pkm_distill_backward(z, dtype, ld, B, V, s["idx"], s["teacher"], k, T,
                                         s["lse"], s["dloss"], dz, V), "pkm_distill_backward")
        return {"dz": dz}
    pk.check(pk.pkm_distill_train(z, dtype, ld, B, V, s["idx"], s["teacher"], k, T, s["dloss"],
                                  loss, lse, dz, V), "pkm_distill_train")
    return {"loss": loss, "lse": lse, "dz": dz}


def run(state):
    if state["op"] == "ffn":
        return _own_ffn(state) if own else _plain_ffn(state)
    return _own_distill(state) if own else _plain_distill(state)


def work(case):
    B, mode = case["B"], case["mode"]
    if case["op"] == "ffn":
        dim, F = case["dim"], case["F"]
        weights, acts, kept = 2 * 3 * dim * F, 2 * B * dim, 2 * 2 * B * F
        forward = dict(bytes=weights + 2 * acts, flops=6 * B * dim * F)
        # x, dy, dx; the weights and their gradients; g and u
        backward = dict(bytes=2 * weights + 3 * acts + kept, flops=12 * B * dim * F)
        if mode == "forward":
            return forward
        if mode == "backward":
            return backward
        # x and the weights once for both, g and u written and kept
        return dict(bytes=2 * weights + 4 * acts + kept, flops=18 * B * dim * F)
    V, k = case["V"], case["k"]
    e = 2 if case["dtype"] == "bf16" else 4
    lists, rows = 12 * B * k, 8 * B
    reads = e * B * V
    if mode == "forward":
        return dict(bytes=reads + lists + rows, flops=4 * B * V)
    return dict(bytes=2 * reads + lists + rows + 4 * B, flops=(6 if mode == "train" else 4) * B * V)


# ------------------------------------------------------------- the definition, 64 bits


def _exact_ffn(case, s):
    mode, act, dim, F, B = (case[n] for n in ("mode", "act", "dim", "F", "B"))
    wg, wu, wd = (s[n].double() for n in ("wg", "wu", "wd"))
    names = {"forward": ("y",), "backward": ("dx",), "train": ("y", "g", "u", "dx")}[mode]
    parts = {n: [] for n in names}
    grads = [torch.zeros(shape, dtype=torch.float64, device="cuda")
             for shape in ((F, dim), (F, dim), (dim, F))]
    for lo in range(0, B, 2048):
        x = s["x"][lo:lo + 2048].double()
        if mode == "backward":
            g, u = s["g"][lo:lo + 2048].double(), s["u"][lo:lo + 2048].double()
        else:
            g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        if act == "silu":
            gate = torch.sigmoid(g)
            a, slope = gate * g, gate + gate * (1 - gate) * g
        elif act == "relu":
            a, slope = torch.relu(g), torch.heaviside(g, torch.zeros_like(g))
        elif act == "gelu":
            cdf = torch.special.ndtr(g)
            a, slope = cdf * g, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        else:
            # 0.5 (1 + tanh v) = sigmoid(2 v)
            w = 2 * math.sqrt(2 / math.pi)
            gate = torch.sigmoid(w * (g + 0.044715 * g ** 3))
            a = gate * g
            slope = gate + gate * (1 - gate) * g * w * (1 + 0.134145 * g ** 2)
        h = u * a
        if mode != "backward":
            parts["y"].append(torch.mm(h, wd.t()).float())
        if mode == "train":
            parts["g"].append(g.float())
            parts["u"].append(u.float())
        if mode != "forward":
            dy = s["dy"][lo:lo + 2048].double()
            dh = torch.mm(dy, wd)
            du, dg = dh * a, dh * u * slope
            parts["dx"].append(torch.addmm(torch.mm(du, wu), dg, wg).float())
            grads[0].addmm_(dg.t(), x)
            grads[1].addmm_(du.t(), x)
            grads[2].addmm_(dy.t(), h)
    out = {n: torch.cat(v) for n, v in parts.items()}
    if mode != "forward":
        out.update(zip(("dwg", "dwu", "dwd"), grads))
    return out


def _exact_distill(case, s):
    T, B, V, mode = case["T"], case["B"], case["V"], case["mode"]
    out = {n: [] for n in {"forward": ("loss", "lse"), "backward": ("dz",),
                           "train": ("loss", "lse", "dz")}[mode]}
    step = max(1, (1 << 27) // V)
    for lo in range(0, B, step):
        z = s["z"][lo:lo + step].double() / T
        idx, n = s["idx"][lo:lo + step], z.shape[0]
        t = s["teacher"][lo:lo + step].double() / T
        t = torch.where(idx < 0, torch.full_like(t, -math.inf), t)
        none = (idx < 0).all(dim=1)
        t[none] = 0.0
        logp = torch.log_softmax(t, dim=1)
        p = torch.softmax(t, dim=1)
        p[none] = 0.0
        # one more column takes what the absent entries would add
        col = torch.where(idx < 0, torch.full_like(idx, V), idx)
        lse = (s["lse"][lo:lo + step].double() if mode == "backward"
               else torch.logsumexp(z, dim=1))
        logq = z - lse[:, None]
        if mode != "backward":
            at = torch.cat((logq, torch.zeros(n, 1, dtype=z.dtype, device="cuda")), 1)
            at = at.gather(1, col)
            out["loss"].append(T * T * (torch.xlogy(p, p).sum(1) - (p * at).sum(1)))
            out["lse"].append(lse)
            del at, logp
        if mode != "forward":
            target = torch.zeros(n, V + 1, dtype=z.dtype, device="cuda")
            target.scatter_add_(1, col, p)
            rest = target[:, :V]
            grad = (torch.exp(logq) * p.sum(1, keepdim=True) - rest) * T
            out["dz"].append((grad * s["dloss"][lo:lo + step].double()[:, None]).float())
            del target, rest, grad
    return {n: torch.cat(v) for n, v in out.items()}


def exact(case, seed):
    if case["op"] == "ffn" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    return _exact_ffn(case, s) if case["op"] == "ffn" else _exact_distill(case, s)
