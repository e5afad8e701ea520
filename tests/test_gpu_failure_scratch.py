"""A selection that gives up leaves its lists as its scratch's memory was.

The merge that follows reads them.  Its results are not meaningful then, but it has to stay
within its shared memory whatever they hold: NaNs leave places of the best-k unfilled, whose
codes are what shared memory held.  The scratch here is memory that was filled with NaNs (as
fp32 and as 16-bit codes) before the handle was made.
"""
import pytest

import oracle
import synth
from helpers import compare_lookup, to_device

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
pk = pytest.importorskip("sparse_top_lookup_gb300")


@pytest.mark.parametrize("k", [16, 32])
@pytest.mark.parametrize("form", [1, 2])
@pytest.mark.parametrize("bits", [0x7FC07FC0, 0x0007FFFF, -1])
def test_a_lookup_that_gave_up_stays_in_bounds(form, k, bits):
    B, H, d_q, n, d_v = 256, 1, 128, 256, 64
    fill = [torch.full((1 << 20,), bits, dtype=torch.int32, device="cuda") for _ in range(4)]
    fill += [torch.full((m,), bits, dtype=torch.int32, device="cuda")
             for m in (512, 4096, 8192, 16384, 65536) for _ in range(4)]
    torch.cuda.synchronize()
    del fill
    torch.cuda.empty_cache()
    s = synth.seed_of(dict(cfg_id=161))
    q = synth.normal(s, 1, B * H * d_q, 1.0, dtype="bf16")
    C = synth.normal(s, 2, H * 2 * n * (d_q // 2), 2.0 / d_q, dtype="bf16")
    h = pk.pkm_create(pk.make_config(d_q, d_v, B, H, n, k, q_dtype=pk.PKM_BF16))
    try:
        tq, tC = to_device(q, "bf16"), to_device(C, "bf16")
        idx = torch.empty(B, H, k, dtype=torch.int64, device="cuda")
        w = torch.empty(B, H, k, device="cuda")
        pk.check(pk.pkm_set_option(h, pk.PKM_OPT_SELECT_FORM, form), "set_option")
        pk.check(pk.pkm_set_option(h, pk.PKM_OPT_TEST_STALL, 1), "set_option")
        pk.check(pk.pkm_lookup(h, tq, tC, B, H, n, k, idx, w), "pkm_lookup")
        assert pk.pkm_get_status(h) == pk.PKM_ERR_TIMEOUT
        pk.check(pk.pkm_set_option(h, pk.PKM_OPT_TEST_STALL, 0), "set_option")
        pk.check(pk.pkm_lookup(h, tq, tC, B, H, n, k, idx, w), "pkm_lookup")
        assert pk.pkm_get_status(h) == pk.PKM_OK
        ref = oracle.lookup(q, C, B, H, d_q, n, k)
        res = compare_lookup(idx.cpu().numpy(), w.cpu().numpy(), ref, q, C, "bf16", H, d_q, n)
        assert res["failures"] == 0 and res["w_ok"], res
    finally:
        pk.pkm_destroy(h)
    torch.cuda.synchronize()
