"""The norm's backward pass of wide rows from host threads at once, each with its own width, stream and
workspace: a block's shared memory differs by width, and no call takes from another what it was granted."""
import threading

import pytest

import sparse_top_lookup_gb300 as pk
from test_gpu_norm import F32, backward, normal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_two_widths_from_several_threads():
    B, dims, calls = 2, (12288, 16384), 4000
    s, dy = ({d: normal(B, d, seed=i) for d in dims} for i in (1, 2))
    w, rstd = {d: normal(d, seed=3) for d in dims}, torch.ones(B, device="cuda")
    want = {d: backward(s[d], w[d], rstd, dy[d], None, F32)["dw"].clone() for d in dims}
    got = []

    def many(d):
        stream = torch.cuda.Stream()
        ws = torch.empty(pk.pkm_add_rms_norm_backward_workspace_bytes(B, d), dtype=torch.uint8, device="cuda")
        dw = torch.empty(d, device="cuda")
        stream.wait_stream(torch.cuda.default_stream())
        refused = 0
        for i in range(calls):
            refused += pk.PKM_OK != pk.pkm_add_rms_norm_backward(
                s[d], pk.PKM_F32, w[d], rstd, dy[d], pk.PKM_F32, None, B, d, ws, None, pk.PKM_F32, None,
                pk.PKM_F32, dw, stream.cuda_stream)
            if i % 100 == 99:
                stream.synchronize()
        got.append((d, refused, dw))
    torch.cuda.synchronize()
    threads = [threading.Thread(target=many, args=(d,)) for d in dims for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(got) == 6 and all(refused == 0 for _, refused, _ in got), [g[:2] for g in got]
    assert all(torch.equal(dw, want[d]) for d, _, dw in got)


def test_a_graph_of_wide_rows_after_narrower_calls():
    B, d = 3, 16384
    s, dy, w = normal(B, d, seed=1), normal(B, d, seed=2), normal(d, seed=3)
    rstd = torch.ones(B, device="cuda")
    want = backward(s, w, rstd, dy, None, F32)["dw"].clone()
    ws = torch.empty(pk.pkm_add_rms_norm_backward_workspace_bytes(B, d), dtype=torch.uint8, device="cuda")
    dw = torch.empty(d, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pk.check(pk.pkm_add_rms_norm_backward(s, pk.PKM_F32, w, rstd, dy, pk.PKM_F32, None, B, d, ws, None,
                                              pk.PKM_F32, None, pk.PKM_F32, dw), "norm backward")
    for narrow in (12288, 10248):
        t = normal(B, narrow, seed=4)
        backward(t, w[:narrow].contiguous(), rstd, t, None, F32)
        dw.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw, want)
