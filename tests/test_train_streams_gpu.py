"""examples/train_streams.py: the operators, the projection stage and the gates
together.  One step's gradients against autograd of the same model in FP64, and
a short training run."""
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
    """Loss and gradients of the model in FP64 with the model's dropout masks."""
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
        y = torch.nn.functional.silu(n @ p[f"up{i}"]) @ p[f"down{i}"]
        mask = torch.empty(T, D, device=x.device)
        mhc.mhc_dropout(torch.ones(T, D, device=x.device), mask, model.rng, p=model.p, sequence=i)
        x = (torch.bmm(m, xs) + 2 * torch.sigmoid(l[:, 4:8])[:, :, None] * (y * mask.double())[:, None]).reshape(T, 4 * D)
    out = norm(x.view(T, 4, D).mean(1), p["norm"], p["norm_bias"])
    loss = torch.nn.functional.cross_entropy(out @ p["head"].t(), targets)
    loss.backward()
    return loss.item(), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("tokens,hidden", [(96, 64), (130, 42)])
def test_gradients_match_autograd(tokens, hidden):
    """Activations are rounded to BF16 (2^-9 relative, on average less) some
    dozen times between the loss and a parameter; independent roundings of
    relative size 2^-9 add up to under 2 % of a gradient's norm."""
    model = E.Model(tokens, hidden, 128, layers=2, p=0.1, seed=3)
    ids, targets = E.batch(tokens, 128, torch.Generator(device="cuda:0").manual_seed(5))
    loss = model.loss_and_gradients(ids, targets).item()
    want, grads = _reference(model, ids, targets)
    assert abs(loss - want) < 0.02 * want
    for k, g in grads.items():
        err = (model.grads[k].double() - g).norm() / g.norm()
        assert err < 0.02, (k, err.item())
    unused = torch.ones(128, dtype=torch.bool, device=ids.device)
    unused[ids] = False
    assert not model.grads["table"][unused].any()


def test_training_lowers_the_loss():
    losses = E.train(steps=30, tokens=512, hidden=128, vocab=128, say=lambda *_: None)
    assert losses[-1] < 0.5 * losses[0], losses
