"""The feed-forward block and the distillation between other work of their stream: what they read
was written just before, what they write was read just before and is read just after, outside and
inside of CUDA graphs, behind kernels, copies, memsets and joined streams.

Results are compared with those of the same call on a quiet GPU, bit by bit.
"""
import pytest

import sparse_top_lookup_gb300 as pk

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale)


class Step:
    """A forward and a backward pass and a training step of the loss on buffers that stay."""

    def __init__(self, B, dim, F, V, k=8):
        self.B, self.dim, self.F, self.V, self.k = B, dim, F, V, k
        self.x, self.dy = torch.empty(B, dim, dtype=BF16, device="cuda"), rand(B, dim).to(BF16)
        self.w = [torch.empty(*s, dtype=BF16, device="cuda") for s in ((F, dim), (F, dim), (dim, F))]
        self.y, self.dx = torch.empty_like(self.x), torch.empty_like(self.x)
        self.dw = [torch.empty_like(w) for w in self.w]
        self.g, self.u = (torch.empty(B, F, dtype=BF16, device="cuda") for _ in range(2))
        n = max(pk.pkm_gated_ffn_workspace_bytes(B, dim, F),
                pk.pkm_gated_ffn_backward_workspace_bytes(B, dim, F))
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.z = torch.empty(B, V, dtype=BF16, device="cuda")
        self.idx = torch.randint(0, V, (B, k), device="cuda")
        self.t, self.dl = rand(B, k, seed=3), torch.full((B,), 1.0, device="cuda")
        self.loss, self.lse = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")

    def source(self, seed):
        B, dim, F, V = self.B, self.dim, self.F, self.V
        return ([rand(B, dim, seed=seed).to(BF16)] +
                [rand(*s, seed=seed + i + 1, scale=0.1).to(BF16)
                 for i, s in enumerate(((F, dim), (F, dim), (dim, F)))] +
                [rand(B, V, seed=seed + 7).to(BF16)])

    def targets(self):
        return [self.x] + self.w + [self.z]

    def calls(self):
        B, dim, F, V, k = self.B, self.dim, self.F, self.V, self.k
        pk.check(pk.pkm_gated_ffn(self.x, *self.w, B, dim, F, 0, self.ws, self.y, self.g, self.u), "f")
        pk.check(pk.pkm_gated_ffn_backward(self.x, *self.w, self.g, self.u, self.dy, B, dim, F, 0,
                                           self.ws, self.dx, *self.dw), "b")
        pk.check(pk.pkm_distill_train(self.z, pk.PKM_BF16, V, B, V, self.idx, self.t, k, 1.0, self.dl,
                                      self.loss, self.lse, self.z, V), "d")

    def results(self):
        return [self.y, self.dx] + self.dw + [self.loss, self.lse, self.z]

    def quiet(self, source):
        for a, b in zip(self.targets(), source):
            a.copy_(b)
        torch.cuda.synchronize()
        self.calls()
        torch.cuda.synchronize()
        return [r.clone() for r in self.results()]


SHAPES = [(1, 256, 1024, 3000), (37, 512, 2048, 20000), (300, 256, 1000, 1000), (700, 512, 1024, 200)]


@pytest.mark.parametrize("shape", SHAPES)
def test_inputs_written_just_before_and_results_read_just_after(shape):
    s = Step(*shape)
    sources = [s.source(10 * i) for i in range(3)]
    want = [s.quiet(src) for src in sources]
    busy = rand(4096, 4096)
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for src in sources:
            busy = busy @ busy.t() * 1e-4         # keeps the GPU behind the host
            for a, b in zip(s.targets(), src):
                a.copy_(b)                        # the old ones may still be being read
            s.calls()
            got.append([r.clone() for r in s.results()])
            for r in s.results()[:-1]:
                r.fill_(-1.0)
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 3])), i


@pytest.mark.parametrize("before", ["nothing", "kernel", "memset", "memcpy", "join"])
@pytest.mark.parametrize("shape", SHAPES)
def test_in_a_graph_behind(shape, before):
    s = Step(*shape)
    src = s.source(5)
    want = s.quiet(src)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if before == "kernel":
            for a, b in zip(s.targets(), src):
                torch.add(b, 0, out=a)
        elif before == "memset":
            s.y.zero_(), s.ws.zero_()
        elif before == "memcpy":
            for a, b in zip(s.targets(), src):
                a.copy_(b)
        elif before == "join":
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                for a, b in zip(s.targets()[::2], src[::2]):
                    torch.add(b, 0, out=a)
            for a, b in zip(s.targets()[1::2], src[1::2]):
                torch.add(b, 0, out=a)
            main.wait_stream(side)
        s.calls()
    for _ in range(3):
        for a, b in zip(s.targets(), src):
            a.copy_(b) if before in ("nothing", "memset") else a.zero_()
        for r in s.results()[:-1]:
            r.fill_(-1.0)
        graph.replay()
        got = [r.clone() for r in s.results()]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("B", [3, 300])
def test_calls_on_two_streams(B):
    steps = [Step(B, 256, 1024, 5000) for _ in range(2)]
    src = [s.source(20 + i) for i, s in enumerate(steps)]
    want = [s.quiet(c) for s, c in zip(steps, src)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, c, st in zip(steps, src, streams):
            with torch.cuda.stream(st):
                for a, b in zip(s.targets(), c):
                    a.copy_(b)
                s.calls()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, b) for a, b in zip(s.results(), w))
