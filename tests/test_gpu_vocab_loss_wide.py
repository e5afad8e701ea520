"""The vocabulary loss's gradient of x over a weight of more than 2^31 elements, all of whose rows it sums.

Tolerances as in test_gpu_vocab_loss.py; a sum over the vocabulary is formed in at most 64 stretches.
"""
import pytest

from test_gpu_vocab_loss import BF16, F64, HALF, SUM, gradient, inputs, near

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [1, 5, 200])
def test_dx_past_32_bits(B):
    V, dim, block = 2100000, 1032, 100000  # 2.2e9 weights
    x, _, _, dloss = inputs(B, dim, 10, seed=B, absent=0.0)
    w = torch.empty(V, dim, dtype=BF16, device="cuda")
    w.normal_(0.0, dim ** -0.5, generator=torch.Generator(device="cuda").manual_seed(1))
    # targets on both sides of 2^31 elements, and in the last row
    target = torch.linspace(0, V - 1, B, device="cuda").long() if B > 1 else torch.tensor([V - 1], device="cuda")
    got = gradient(x, w, target, dloss, True, skip=("dw",))["dx"]
    X = x.to(F64)
    lse = torch.full((B,), -float("inf"), dtype=F64, device="cuda")
    for i in range(0, V, block):
        lse = torch.logaddexp(lse, torch.logsumexp(X @ w[i:i + block].to(F64).T, 1))
    want, sizes = torch.zeros(B, dim, dtype=F64, device="cuda"), torch.zeros(B, dim, dtype=F64, device="cuda")
    for i in range(0, V, block):
        W = w[i:i + block].to(F64)
        dz = torch.exp(X @ W.T - lse[:, None])
        here = (target >= i) & (target < i + block)
        dz[torch.arange(B, device="cuda")[here], target[here] - i] -= 1
        dz *= dloss.to(F64)[:, None]
        want += dz @ W
        sizes += dz.abs() @ W.abs()
    # a logit's error, and what the log-sum-exp's adds to a power
    e = 2 * (dim + 2) * 2.0 ** -24 * float((X.abs() @ w[-1000:].to(F64).abs().T).max()) + 2 * SUM
    e += 2.0 ** -20 * (1 + float(lse.max()))
    other = (e + 2 * (V / 64 + 66) * 2.0 ** -24) * sizes
    near(got, want, 1.01 * (HALF * want.abs() + (1 + HALF) * (HALF * sizes + other)) + 1e-38, 2, "dx", other)
