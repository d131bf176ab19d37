"""The whole-number check of embedding gradients (operators_exact.py) on the
CPU, with planted mistakes: what a wrong merge or join of a long run would do."""
import torch

import operators_exact as X

T, V, D, N = 40000, 64, 8, 4
CHUNK = 32   # ordered tokens a block sums


def test_planted_mistakes_are_rejected():
    ids, grad_x, _, want = X.case(T, V, D, N, seed=1, frequent=0.8)
    run = (ids == V // 2).nonzero().flatten()
    assert len(run) > 512 * CHUNK
    assert X.equal(want.float(), want)

    def without(tokens):
        keep = torch.ones(T, dtype=torch.bool)
        keep[tokens] = False
        return X.sums(ids[keep], grad_x[keep], V, D).float()

    doubled = X.sums(torch.cat([ids, ids[run[:CHUNK]]]), torch.cat([grad_x, grad_x[run[:CHUNK]]]), V, D).float()
    zero = want.float()
    zero[V // 2] = 0
    one = want.float()
    one[3, 5] += 1
    for wrong in (without(run[:CHUNK]), without(run[-1:]), without(run[512 * CHUNK:]), doubled, zero, one, want.float() * 1.5,
                  torch.full((V, D), float("nan")), want[:-1].float()):
        assert not X.equal(wrong, want)


def test_order_does_not_matter():
    """Whatever the order, the FP32 sums are the whole numbers."""
    ids, grad_x, table, want = X.case(3000, 7, 3, 2, seed=2, frequent=0.5, pad=0.1, start=True)
    order = torch.randperm(3000, generator=torch.Generator().manual_seed(3))
    ok = ids[order] >= 0
    got = table.clone()
    for k in range(2):
        got.index_add_(0, ids[order][ok], grad_x[order][ok][:, 3 * k:3 * k + 3].float())
    assert X.equal(got, want)
