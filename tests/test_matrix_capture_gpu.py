"""What the feed-forward block and the orthogonalised update promise as calls: captured
into a graph they give the same bits on new inputs, two graphs may share a
workspace, they keep to the stream they are given, two streams with a workspace
each do not disturb one another, and what is not theirs stays as it was."""
import pytest
import torch

import rms_backward_gb300 as m

from matrix_cases import DEV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Step:
    """A block forward and backward and the update of its three matrices, as a training step has them."""

    def __init__(self, T, D, F, workspace=None):
        self.T, self.D, self.F = T, D, F
        b16 = lambda *s: torch.zeros(*s, dtype=BF, device=DEV)  # noqa: E731
        self.x, self.dy = b16(T, D), b16(T, D)
        self.w = [b16(F, D), b16(F, D), b16(D, F)]
        self.y, self.gate, self.up, self.dx = b16(T, D), b16(T, F), b16(T, F), b16(T, D)
        self.grads = [torch.zeros(w.shape, device=DEV) for w in self.w]
        self.out = [torch.zeros_like(w) for w in self.w]
        self.ws = torch.zeros(self.size(), dtype=torch.uint8, device=DEV) if workspace is None else workspace

    def size(self):
        T, D, F = self.T, self.D, self.F
        return max(m.mhc_ffn_forward_workspace_bytes(T, D, F), m.mhc_ffn_backward_workspace_bytes(T, D, F),
                   m.mhc_orthogonalize_workspace_bytes(F, D), m.mhc_orthogonalize_workspace_bytes(D, F))

    def new_inputs(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        for t in (self.x, self.dy, *self.w):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV) * t.shape[-1] ** -0.5)

    def run(self, **stream):
        m.mhc_ffn_forward(self.x, *self.w, self.y, self.ws, self.gate, self.up, **stream)
        m.mhc_ffn_backward(self.x, *self.w, self.gate, self.up, self.dy, self.dx, *self.grads, self.ws, **stream)
        for g, o in zip(self.grads, self.out):
            m.mhc_orthogonalize(g, o, self.ws, **stream)

    def results(self):
        written = [self.y, self.gate, self.up, self.dx, *self.grads, *self.out]
        copies = [t.clone() for t in written]
        for t in written:
            t.fill_(float("nan"))
        return copies


# few tokens and a short side, single blocks, odd sizes, pairs of blocks
SHAPES = [(2, 32, 200), (40, 136, 264), (33, 75, 141), (1100, 1600, 1608)]


@pytest.mark.parametrize("T,D,F", SHAPES)
def test_captured_step(T, D, F):
    step = Step(T, D, F)
    want = []
    for seed in (1, 2, 3):
        step.new_inputs(seed)
        step.run()
        want.append(step.results())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for seed, expected in zip((2, 1, 3), (want[1], want[0], want[2])):
        step.new_inputs(seed)
        graph.replay()
        for got, e in zip(step.results(), expected):
            assert torch.equal(got, e) and bool(torch.isfinite(e).all())
    assert not torch.equal(want[0][0], want[1][0])
    assert m.mhc_operators_device_status() == 0


def test_two_graphs_share_a_workspace():
    a, b = Step(40, 136, 264), Step(33, 75, 141)
    ws = torch.zeros(max(a.size(), b.size()), dtype=torch.uint8, device=DEV)
    a.ws = b.ws = ws
    want, graphs = [], []
    for s in (a, b):
        s.new_inputs(7)
        s.run()
        want.append(s.results())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 1)):
        for i in order:
            graphs[i].replay()
    for s, w in zip((a, b), want):
        assert all(torch.equal(p, q) for p, q in zip(s.results(), w))


@pytest.mark.parametrize("T,D,F", SHAPES)
@pytest.mark.parametrize("named", [False, True])
def test_step_on_a_side_stream(T, D, F, named):
    """The inputs arrive late on a side stream; the calls run there."""
    step, side = Step(T, D, F), torch.cuda.Stream()
    step.new_inputs(1)
    step.run()
    want = step.results()
    step.new_inputs(2)
    step.results()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(4_000_000)
        step.new_inputs(1)
        if not named:
            step.run()
    if named:
        step.run(stream=side)
    with torch.cuda.stream(side):
        got = step.results()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_two_streams_at_once():
    steps = [Step(1100, 1600, 1608), Step(40, 136, 264), Step(2, 32, 200)]
    want = []
    for i, s in enumerate(steps):
        s.new_inputs(i)
        s.run()
        want.append(s.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for s, t in zip(steps, streams):
            s.run(stream=t)
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(p, q) for p, q in zip(s.results(), w))
    assert m.mhc_operators_device_status() == 0


def test_calls_back_to_back_reuse_buffers():
    """Each call starts before the one ahead has ended; none reads or overwrites what that still needs:
    the output of one block is the input of the next, through one workspace and one pair of buffers."""
    T, D, F = 300, 264, 520
    s = Step(T, D, F)
    s.new_inputs(3)
    for w in s.w:
        w.mul_(4)
    # root mean squares: x 0.06, then 0.12, 0.6 and 12 (each call about squares them); a fourth call's
    # would be some 10^3, a tenth's overflow
    bufs = [s.x.clone(), torch.empty_like(s.x)]

    def chain(wait):
        bufs[0].copy_(s.x)
        for i in range(3):
            m.mhc_ffn_forward(bufs[i % 2], *s.w, bufs[1 - i % 2], s.ws)
            if wait:
                torch.cuda.synchronize()
        return bufs[1].clone()

    want = chain(True)
    assert bool(torch.isfinite(want).all()) and want.abs().max() > 1
    for _ in range(20):
        assert torch.equal(chain(False), want)
    assert m.mhc_operators_device_status() == 0


def test_inputs_are_left_alone():
    s = Step(33, 75, 141)
    s.new_inputs(4)
    kept = [t.clone() for t in (s.x, s.dy, *s.w)]
    s.run()
    g = [t.clone() for t in s.grads]
    m.mhc_orthogonalize(s.grads[0], s.out[0], s.ws)
    assert all(torch.equal(p, q) for p, q in zip(kept, (s.x, s.dy, *s.w)))
    assert all(torch.equal(p, q) for p, q in zip(g, s.grads))
