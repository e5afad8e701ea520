"""Plain 64-bit forms of the gated feed-forward block and of distillation from a teacher's top
logits, with their gradients, written out from the formulas (torch, float64, any device)."""
import math

import torch

ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def act64(g, act):
    """act(g) and act'(g)."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 0.134145 * g * g)
    return torch.clamp(g, min=0), (g > 0).to(g.dtype)


def ffn64(x, wg, wu, wd, act):
    """g, u, h, y."""
    g, u = x @ wg.T, x @ wu.T
    h = act64(g, act)[0] * u
    return g, u, h, h @ wd.T


def ffn_backward64(x, wg, wu, wd, g, u, dy, act):
    """dict of dg, du, h, dx, dwg, dwu, dwd."""
    a, da = act64(g, act)
    dh = dy @ wd
    dg, du, h = dh * u * da, dh * a, a * u
    return dict(dg=dg, du=du, h=h, dx=dg @ wg + du @ wu, dwg=dg.T @ x, dwu=du.T @ x, dwd=dy.T @ h)


def distill64(z, idx, teacher, T, dloss=None):
    """loss, lse and (with dloss) dz, row by row from the definition."""
    B, V = z.shape
    loss, lse = torch.zeros(B, dtype=z.dtype), torch.zeros(B, dtype=z.dtype)
    dz = torch.zeros(B, V, dtype=z.dtype)
    for b in range(B):
        zb = z[b].cpu() / T
        lse[b] = torch.logsumexp(zb, 0)
        there = [j for j in range(idx.shape[1]) if 0 <= int(idx[b, j]) < V
                 and float(teacher[b, j]) != -math.inf]
        if not there:
            continue
        at = idx[b].cpu()[there]
        t = teacher[b].cpu().to(z.dtype)[there] / T
        logp = torch.log_softmax(t, 0)
        p = torch.exp(logp)
        logq = torch.where(zb == -math.inf, zb, zb - lse[b])
        term = torch.where(p > 0, p * (logp - logq[at]), torch.zeros_like(p))
        loss[b] = T * T * term.sum()
        if dloss is not None and float(dloss[b]) != 0:
            row = torch.exp(logq)
            row.index_add_(0, at, -p)
            dz[b] = float(dloss[b]) * T * row
    return loss, lse, dz
