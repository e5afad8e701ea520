"""Distillation on the GPU: long lists and columns that occur several times in them, in the forms
for short rows, one CTA's rows and rows of a cluster, with more rows than run at one time.

Tolerances are test_gpu_distill's.
"""
import pytest
import torch

import test_gpu_distill as d

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype,B,V,k", [
    (BF16, 650, 300, 100), (F32, 620, 1000, 128), (BF16, 640, 37, 64), (F32, 5, 300, 300),
    (BF16, 3, 3, 512), (F32, 330, 5000, 301), (BF16, 170, 60001, 512), (F32, 90, 40000, 130),
    (BF16, 90, 131072, 65), (F32, 85, 130001, 40)])
def test_columns_that_occur_several_times(dtype, B, V, k, in_place):
    z, idx, t, dl = d.make(B, V, k, dtype, 2.0, V + k)
    g = torch.Generator().manual_seed(V)
    few = torch.randint(0, V, (B, 5), generator=g).cuda()
    idx[1::3, 1::2] = idx[1::3, 0:k - k % 2:2]                 # pairs of neighbours
    idx[2::3] = few[2::3][:, torch.arange(k) % 5]              # five columns
    idx[3::6, k // 2:] = idx[3::6, :k - k // 2].flip(1)        # pairs far apart
    idx[4::6, ::3] = -1
    d.check(z, idx, t, dl, 2.0, d.calls(z, idx, t, dl, 2.0, in_place=in_place))


@pytest.mark.parametrize("dtype,V", [(F32, 600), (BF16, 30000), (F32, 130000)])
def test_the_same_bits_each_time(dtype, V):
    z, idx, t, dl = d.make(400, V, 70, dtype, 1.0, V)
    idx[:, 1::2] = idx[:, ::2]
    first = d.calls(z, idx, t, dl, 1.0)
    for _ in range(3):
        out = d.calls(z, idx, t, dl, 1.0)
        assert torch.equal(out["b"], first["b"])
        assert all(torch.equal(a, b) for w in "ft" for a, b in zip(out[w], first[w]))
