"""What every call of the operators promises, over a chain of all of them:
captured into a CUDA graph it gives the same bits on new inputs, and on a side
stream it waits for what that stream holds.  The chain has every multi-launch
call: an embedding gradient with two merges and a join, and norm gradients of
each path with their parameter sums."""
import pytest
import torch

import rms_backward_gb300 as m

import operators_cases as C
from operators_cases import DEV, empty, gen, normal, rng_state

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
P = 0.2


class Chain:
    """Token ids -> streams -> a sublayer -> streams, a plain norm and dropout,
    and everything back to the table."""

    def __init__(self, T, D, V):
        self.T, self.D, self.V = T, D, V
        g = gen(T + D)
        self.ids = torch.zeros(T, dtype=torch.int64, device=DEV)
        self.table, self.h = normal(g, V, D).to(DEV), C.gates(g, T).to(DEV)
        self.gamma, self.beta = normal(g, D).to(DEV), normal(g, D).to(DEV)
        self.grad_out = torch.zeros(T, 4 * D, dtype=BF, device=DEV)
        self.rng = rng_state()
        b16, f32 = (lambda *s: empty(*s, dtype=BF)), (lambda *s: empty(*s))
        self.x, self.y, self.n, self.d, self.out = b16(T, 4 * D), b16(T, D), b16(T, D), b16(T, D), b16(T, 4 * D)
        self.stats = [f32(T) for _ in range(4)]
        self.gy, self.gd, self.gn, self.gh, self.gx = b16(T, D), b16(T, D), b16(T, D), torch.zeros(T, 24, device=DEV), b16(T, 4 * D)
        self.params = [torch.zeros(D, device=DEV) for _ in range(4)]
        self.gt, self.gt_added = f32(V, D), torch.zeros(V, D, device=DEV)
        size = max(m.mhc_embed_workspace_bytes(T, V, D), m.mhc_collapse_norm_workspace_bytes(T, D))
        self.ws = torch.zeros(size, dtype=torch.uint8, device=DEV)

    def new_inputs(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        ids = torch.randint(-1, self.V, (self.T,), generator=g, device=DEV)
        self.ids.copy_(torch.where(torch.rand(self.T, generator=g, device=DEV) < 0.4, 3, ids))
        self.grad_out.copy_(torch.randn(self.T, 4 * self.D, generator=g, device=DEV))
        self.rng[1] = seed
        self.gt_added.fill_(1.0)

    def run(self, **stream):
        s = self.stats
        m.mhc_embed_forward(self.ids, self.table, self.x, **stream)
        m.mhc_collapse_norm_forward(self.x, self.h, self.gamma, self.beta, self.y, s[0], s[1], **stream)
        m.mhc_layernorm_forward(self.y, self.gamma, self.beta, self.n, s[2], s[3], **stream)
        m.mhc_dropout(self.n, self.d, self.rng, p=P, sequence=1, **stream)
        m.mhc_update_forward(self.x, self.d, self.h, self.out, self.rng, p=P, **stream)
        m.mhc_update_backward(self.x, self.d, self.h, self.grad_out, self.gy, self.gh, self.rng, p=P, **stream)
        m.mhc_dropout(self.gy, self.gd, self.rng, p=P, sequence=1, **stream)
        m.mhc_layernorm_backward(self.y, self.gd, self.gamma, s[2], s[3], self.gn, *self.params[:2], self.ws, **stream)
        m.mhc_collapse_norm_backward(self.x, self.h, self.gn, self.gamma, s[0], s[1], self.gx, self.gh, *self.params[2:],
                                     self.ws, grad_x_out=self.grad_out, **stream)
        m.mhc_embed_backward(self.ids, self.gx, self.gt, self.ws, **stream)
        m.mhc_embed_backward(self.ids, self.gx, self.gt_added, self.ws, accumulate=True, **stream)

    def results(self):
        """Copies of all that was written, which is then spoiled."""
        written = [self.x, self.y, self.n, self.d, self.out, *self.stats, self.gy, self.gd, self.gn, self.gh, self.gx,
                   *self.params, self.gt, self.gt_added]
        copies = [t.clone() for t in written]
        for t in written:
            t.fill_(float("nan"))
        return copies


# one row per block's groups, rows at any address, and rows that are read again
SHAPES = [(17000, 40, 300), (600, 1285, 50), (40, 10248, 20)]


@pytest.mark.parametrize("T,D,V", SHAPES)
def test_captured_chain(T, D, V):
    chain = Chain(T, D, V)
    want = []
    for seed in (1, 2, 3):
        chain.new_inputs(seed)
        chain.run()
        want.append(chain.results())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain.run()
    for seed, expected in zip((2, 1, 3), (want[1], want[0], want[2])):
        chain.new_inputs(seed)
        graph.replay()
        for got, e in zip(chain.results(), expected):
            assert torch.equal(got, e) and bool(torch.isfinite(e).all())
    assert not torch.equal(want[0][-1], want[1][-1])


@pytest.mark.parametrize("T,D,V", SHAPES)
@pytest.mark.parametrize("named", [False, True])
def test_chain_on_a_side_stream(T, D, V, named):
    """The inputs arrive late on a side stream; the calls run there, given that
    stream or under it as the current one."""
    chain, side = Chain(T, D, V), torch.cuda.Stream()
    chain.new_inputs(1)
    chain.run()
    want = chain.results()
    chain.new_inputs(2)
    chain.results()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(4_000_000)
        chain.new_inputs(1)
        if not named:
            chain.run()
    if named:
        chain.run(stream=side)
    with torch.cuda.stream(side):
        got = chain.results()
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
