"""A transformer block's feed-forward half with a memory layer beside it, trained from a
teacher's top logits.

    f = gated feed-forward block(x)                    pkm_gated_ffn
    m = memory layer(x): query network, lookup, read   pkm_query_net, pkm_forward
    logits = (x + f + m) head^T                        (torch)
    loss = distillation from the teacher's k best      pkm_distill_train

and back: dlogits replace the logits, the block's gradients come from pkm_gated_ffn_backward
(the weights' added to in fp32) and the memory's from pkm_backward.  The parameters are stepped by
plain SGD.  Run as `python examples/distill_block.py` on a GPU; it prints the mean loss per step.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_top_lookup_gb300 as pk  # noqa: E402

BF16 = torch.bfloat16


def train(steps=20, B=512, dim=256, F=704, V=4000, n_keys=32, heads=2, k=8, teacher_k=16, T=2.0,
          rate=1.0, seed=0):
    """Trains for `steps` steps on one batch; the list of mean losses."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sd=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device="cuda", generator=gen) * sd).to(dtype)

    x, head = normal(B, dim, dtype=BF16), normal(V, dim, sd=dim ** -0.5, dtype=BF16)
    # the teacher: another block's logits on the same tokens, kept as its best teacher_k
    other = torch.tanh(x.float() @ normal(dim, dim, sd=dim ** -0.5)) * 2
    teacher, idx = ((x.float() + other) @ head.float().T * 2).topk(teacher_k, dim=1)
    # parameters, in fp32
    wg, wu, wd = normal(F, dim, sd=dim ** -0.5), normal(F, dim, sd=dim ** -0.5), normal(dim, F, sd=F ** -0.5)
    wq = normal(heads * dim, dim, sd=dim ** -0.5, dtype=BF16)
    scale, shift = torch.ones(heads * dim, device="cuda"), torch.zeros(heads * dim, device="cuda")
    subkeys = normal(heads, 2, n_keys, dim // 2, sd=(2 / dim) ** 0.5)
    values = normal(n_keys ** 2, dim, sd=dim ** -0.5)
    params = [wg, wu, wd, subkeys, values]
    grads = [torch.zeros_like(p) for p in params]
    # a training program's buffers
    h = pk.pkm_create(pk.make_config(dim, dim, B, heads, n_keys, k, with_backward=1))
    f, g, u = (torch.empty(B, n, dtype=BF16, device="cuda") for n in (dim, F, F))
    q = torch.empty(B, heads, dim, dtype=BF16, device="cuda")
    sel = torch.empty(B, heads, k, dtype=torch.int64, device="cuda")
    w = torch.empty(B, heads, k, device="cuda")
    m = torch.empty(B, dim, device="cuda")
    loss, lse = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    dloss = torch.full((B,), 1.0 / B, device="cuda")
    dx, dq = torch.empty_like(x), torch.empty(B, heads, dim, device="cuda")
    ws = torch.empty(max(pk.pkm_gated_ffn_workspace_bytes(B, dim, F),
                         pk.pkm_gated_ffn_backward_workspace_bytes(B, dim, F)),
                     dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    losses = []
    try:
        for _ in range(steps):
            bg, bu, bd, bC, bV = (p.to(BF16) for p in params)
            # forward
            pk.check(pk.pkm_gated_ffn(x, bg, bu, bd, B, dim, F, pk.PKM_ACT_SILU, ws, f, g, u,
                                      status), "pkm_gated_ffn")
            pk.check(pk.pkm_query_net(x, wq, B, dim, heads * dim, scale, shift, q, status),
                     "pkm_query_net")
            pk.check(pk.pkm_forward(h, q, bC, bV, B, heads, n_keys, k, m, sel, w), "pkm_forward")
            logits = (x.float() + f.float() + m).to(BF16) @ head.T
            # the loss, its gradient in the logits' place
            pk.check(pk.pkm_distill_train(logits, pk.PKM_BF16, V, B, V, idx, teacher, teacher_k,
                                          T, dloss, loss, lse, logits, V, status),
                     "pkm_distill_train")
            losses.append(loss.mean())
            # backward
            dout = logits @ head
            for t in grads:
                t.zero_()
            pk.check(pk.pkm_gated_ffn_backward(x, bg, bu, bd, g, u, dout, B, dim, F,
                                               pk.PKM_ACT_SILU, ws, dx, *grads[:3], pk.PKM_F32,
                                               status), "pkm_gated_ffn_backward")
            pk.check(pk.pkm_backward(h, q, bC, bV, B, heads, n_keys, k, sel, w, dout.float(), dq,
                                     grads[3], grads[4]), "pkm_backward")
            for p, t in zip(params, grads):
                p.sub_(t, alpha=rate)
        losses = torch.stack(losses).tolist()
        for st in (status.item(), pk.pkm_get_status(h)):
            pk.check(st, "device status")
    finally:
        pk.pkm_destroy(h)
    return losses


if __name__ == "__main__":
    for i, v in enumerate(train()):
        print("step %2d  loss %.4f" % (i, v))
