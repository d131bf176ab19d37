"""examples/train_streams.py with the library's feed-forward block and orthogonalised
updates: one step's gradients against autograd of the same model in FP64, and a
run of a few steps."""
import os
import sys

import pytest
import torch

import rms_backward_gb300 as mhc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import train_streams as E  # noqa: E402

pytestmark = pytest.mark.gpu


def _reference(model, ids, targets):
    """Gradients of the model in FP64 with the model's dropout masks and BF16 matrices."""
    p = {k: v.double().requires_grad_() for k, v in model.params.items()}
    T, D = model.T, model.D
    x = p["table"][ids].repeat(1, 4)
    norm = lambda u, a, b: torch.nn.functional.layer_norm(u, (D,), a, b, 1e-5)  # noqa: E731
    for i in range(model.L):
        r = (x.square().mean(1) + 1e-6).sqrt()
        l = (x @ p[f"w{i}"].t()) / r[:, None] * torch.repeat_interleave(
            p[f"alpha{i}"], torch.tensor([4, 4, 16], device=x.device)) + p[f"bias{i}"]
        m = l[:, 8:].reshape(T, 4, 4).exp()
        for _ in range(20):
            m = m / m.sum(2, keepdim=True)
            m = m / m.sum(1, keepdim=True)
        xs = x.view(T, 4, D)
        n = norm((torch.sigmoid(l[:, :4])[:, :, None] * xs).sum(1), p[f"gamma{i}"], p[f"beta{i}"])
        y = (torch.nn.functional.silu(n @ p[f"gate{i}"].t()) * (n @ p[f"up{i}"].t())) @ p[f"down{i}"].t()
        mask = torch.empty(T, D, device=x.device)
        mhc.mhc_dropout(torch.ones(T, D, device=x.device), mask, model.rng, p=model.p, sequence=i)
        x = (torch.bmm(m, xs) + 2 * torch.sigmoid(l[:, 4:8])[:, :, None] * (y * mask.double())[:, None]).reshape(T, 4 * D)
    out = norm(x.view(T, 4, D).mean(1), p["norm"], p["norm_bias"])
    torch.nn.functional.cross_entropy(out @ p["head"].t(), targets).backward()
    return {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("tokens,hidden", [(96, 64), (130, 42)])
def test_gradients_match_autograd(tokens, hidden):
    """Between the loss and a parameter lie some dozen roundings to BF16 of activations and, in the
    block, three of matrices and five of what its products read; twenty independent ones of a relative
    size of 2^-8 / sqrt(3) on average come to 1 % of a gradient's norm: twice that."""
    model = E.Model(tokens, hidden, 128, layers=2, p=0.1, seed=3, block="gated")
    ids, targets = E.batch(tokens, 128, torch.Generator(device="cuda:0").manual_seed(5))
    model.loss_and_gradients(ids, targets)
    grads = _reference(model, ids, targets)
    assert {f"{k}{i}" for k in ("gate", "up", "down") for i in (0, 1)} <= set(grads)
    for k, g in grads.items():
        err = (model.grads[k].double() - g).norm() / g.norm()
        assert err < 0.02, (k, err.item())


def test_training_runs():
    """Every step's loss is a number and every matrix moves by the update's size."""
    losses = E.train(steps=4, tokens=256, hidden=128, vocab=128, say=lambda *_: None, block="gated")
    assert len(losses) == 4 and all(v == v and v < 100 for v in losses)
    model = E.Model(256, 128, 128, block="gated")
    matrices = E.Orthogonalised(model, lr=1e-2)
    model.loss_and_gradients(*E.batch(256, 128, torch.Generator(device="cuda:0").manual_seed(1)))
    before = {k: model.params[k].clone() for k in matrices.names}
    matrices.step()
    for k, w in before.items():
        m, n = w.shape
        # singular values in [0.68, 1.21] of min(m, n) directions that the gradient has; none adds more
        rms = (model.params[k] - w).norm().item() / (m * n) ** 0.5
        assert 0 < rms <= 1.22 * 1e-2 * 0.2
