"""The feed-forward block's tiles that are cut along K and joined through the workspace: captured and
replayed, call after call on one workspace, and on two streams.

A part's flag is good for one launch: it holds that launch's number, which a replay repeats, and is
cleared when it has been seen.  Were it left, a replay would add the last replay's parts.  Results are
compared with those of the same calls on a quiet GPU, bit by bit.
"""
import pytest

import sparse_top_lookup_gb300 as pk
from test_gpu_ordering import Step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# cut in the down projection and dx; in the gate and the backward gate
SHAPES = [(200, 256, 8192), (513, 136, 5000), (300, 4096, 1000)]
FLAGS = 80 * 2 * 8 * 8  # bytes at a workspace's end: clusters, CTAs, epilogue warps, 64 bits


def align256(n):
    return (n + 255) // 256 * 256


class Ffn(Step):
    def __init__(self, B, dim, F):
        super().__init__(B, dim, F, 64)
        self.ws.zero_()

    def forward(self):
        pk.check(pk.pkm_gated_ffn(self.x, *self.w, self.B, self.dim, self.F, 0, self.ws, self.y, self.g,
                                  self.u), "forward")

    def backward(self):
        pk.check(pk.pkm_gated_ffn_backward(self.x, *self.w, self.g, self.u, self.dy, self.B, self.dim,
                                           self.F, 0, self.ws, self.dx, *self.dw), "backward")

    def calls(self):
        self.forward()
        self.backward()

    def results(self):
        return [self.y, self.g, self.u, self.dx] + self.dw


@pytest.mark.parametrize("shape", SHAPES)
def test_these_shapes_are_cut_and_their_flags_cleared(shape):
    s = Ffn(*shape)
    for a, b in zip(s.targets(), s.source(1)):
        a.copy_(b)
    B, dim, F = shape
    for call, kept, n in ((s.forward, align256(2 * B * F), pk.pkm_gated_ffn_workspace_bytes(B, dim, F)),
                          (s.backward, 3 * align256(2 * B * F),
                           pk.pkm_gated_ffn_backward_workspace_bytes(B, dim, F))):
        assert n - kept > FLAGS
        s.ws.zero_()
        call()
        torch.cuda.synchronize()
        assert bool((s.ws[kept:n - FLAGS] != 0).any()), "no parts were written"
        assert not bool((s.ws[n - FLAGS:n] != 0).any()), "a flag was left"


@pytest.mark.parametrize("shape", SHAPES)
def test_replays_with_other_inputs(shape):
    s = Ffn(*shape)
    sources = [s.source(30 * i) for i in range(3)]
    want = [s.quiet(src) for src in sources]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.calls()
    for i in (0, 1, 2, 2, 1, 0, 1):
        for a, b in zip(s.targets(), sources[i]):
            a.copy_(b)
        for r in s.results():
            r.fill_(-1.0)
        graph.replay()
        got = [r.clone() for r in s.results()]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i


@pytest.mark.parametrize("shape", SHAPES)
def test_calls_and_replays_by_turns_on_one_workspace(shape):
    s = Ffn(*shape)
    sources = [s.source(30 * i + 7) for i in range(2)]
    want = [s.quiet(src) for src in sources]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.calls()
    got = []
    for i in (0, 1, 1, 0, 0, 1):
        for a, b in zip(s.targets(), sources[i]):
            a.copy_(b)
        s.calls()
        got.append([r.clone() for r in s.results()])
        for r in s.results():
            r.fill_(-1.0)
        graph.replay()
        got.append([r.clone() for r in s.results()])
    torch.cuda.synchronize()
    for n, i in enumerate((0, 0, 1, 1, 1, 1, 0, 0, 0, 0, 1, 1)):
        assert all(torch.equal(a, b) for a, b in zip(got[n], want[i])), n


def test_on_two_streams():
    steps = [Ffn(*SHAPES[0]) for _ in range(2)]
    src = [s.source(50 + i) for i, s in enumerate(steps)]
    want = [s.quiet(c) for s, c in zip(steps, src)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(6):
        for s, c, st in zip(steps, src, streams):
            with torch.cuda.stream(st):
                for a, b in zip(s.targets(), c):
                    a.copy_(b)
                s.calls()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), w))
