"""Calls of different sizes on several host threads at once, each with its own context, stream and buffers: what
one call is granted of a kernel's shared memory is not taken back by a smaller one."""
import sys
import threading

import pytest

import sparse_top_lookup_gb300 as pk

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def together(sizes, make, calls=20000, threads=4):
    """make(size) -> handle, call, result: `calls` calls on each of `threads` threads a size; all are taken, and
    the last results are a single thread's."""
    want, got = {}, []
    for size in sizes:
        h, call, result = make(size)
        try:
            pk.check(call(None), "call")
            torch.cuda.synchronize()
            want[size] = result.clone()
        finally:
            pk.pkm_destroy(h)

    def many(size):
        h, call, result = make(size)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.default_stream())
        refused = 0
        for i in range(calls):
            refused += call(stream.cuda_stream) != pk.PKM_OK
            if i % 500 == 499:
                stream.synchronize()
        stream.synchronize()
        got.append((size, refused, result))
        pk.pkm_destroy(h)
    switch = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    workers = [threading.Thread(target=many, args=(s,)) for s in sizes for _ in range(threads)]
    for t in workers:
        t.start()
    for t in workers:
        t.join()
    sys.setswitchinterval(switch)
    torch.cuda.synchronize()
    assert len(got) == threads * len(sizes) and all(g[1] == 0 for g in got), [g[:2] for g in got]
    assert all(torch.equal(result, want[size]) for size, _, result in got)


def test_reads_of_many_rows():
    # a bag's rows are staged in shared memory: 64 and 96 KB
    n, d_v, k = 16, 8, 8
    gen = torch.Generator(device="cuda").manual_seed(1)
    V = torch.randn(n * n, d_v, device="cuda", generator=gen).bfloat16()
    ins = {H: (torch.randint(0, n * n, (1, H, k), device="cuda", generator=gen),
               torch.rand(1, H, k, device="cuda", generator=gen)) for H in (1000, 1500)}

    def make(H):
        h = pk.pkm_create(pk.make_config(32, d_v, 1, H, n, k, q_dtype=pk.PKM_BF16))
        out = torch.empty(1, d_v, device="cuda")
        return h, lambda s: pk.pkm_gather(h, V, 1, H, n, k, *ins[H], out, s), out
    together((1000, 1500), make)


def test_lookups_on_the_cuda_cores():
    # a query, both halves' scores and the candidates: 51 and 67 KB
    H, k = 1, 4
    gen = torch.Generator(device="cuda").manual_seed(2)
    ins = {n: (torch.randn(2, H, d_q, device="cuda", generator=gen),
               torch.randn(H, 2, n, d_q // 2, device="cuda", generator=gen))
           for n, d_q in ((2560, 8192), (4096, 8192))}

    def make(n):
        h = pk.pkm_create(pk.make_config(8192, 8, 2, H, n, k, q_dtype=pk.PKM_F32))
        idx, w = torch.empty(2, H, k, dtype=torch.int64, device="cuda"), torch.empty(2, H, k, device="cuda")
        return h, lambda s: pk.pkm_lookup(h, *ins[n], 2, H, n, k, idx, w, s), idx
    together((2560, 4096), make, calls=200, threads=2)
