"""Embedding gradients that leave no room for an error (not a test module): the
gradients are small whole numbers and so few that every partial sum, in any
order, is a whole number below 2^24, exact in FP32.  The result has to be
equal to the sums in whole numbers; a lost or doubled token shows.

(A bound by the length of the row's chain says little about a row that is the
sum of a hundred thousand terms.)"""
import torch


def case(T, V, D, n, seed, frequent=0.0, pad=0.0, start=False):
    """ids [T], grad_x [T, n D], the table's start or None, and the wanted
    gradient, on the CPU.  A share `frequent` of the tokens are id V // 2."""
    assert 3 * T * n + 100 < 2**24
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, V, (T,), generator=g)
    if frequent:
        ids[torch.rand(T, generator=g) < frequent] = V // 2
    if pad:
        ids[torch.rand(T, generator=g) < pad] = -1
    grad_x = torch.randint(1, 4, (T, n * D), generator=g).to(torch.bfloat16)   # positive: nothing cancels
    table = torch.randint(-100, 101, (V, D), generator=g).float() if start else None
    return ids, grad_x, table, sums(ids, grad_x, V, D, table)


def sums(ids, grad_x, V, D, table=None):
    want = torch.zeros(V, D, dtype=torch.int64) if table is None else table.long()
    ok = (ids >= 0) & (ids < V)
    return want.index_add_(0, ids[ok], grad_x.view(len(ids), -1, D)[ok].long().sum(1))


def equal(got, want):
    return got.shape == want.shape and torch.equal(got.double().cpu(), want.double())
