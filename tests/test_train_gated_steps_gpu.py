"""examples/train_streams.py with orthogonalised updates: every step moves every matrix against its
momentum by the formula's update."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle.mhcm_oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import train_streams as E  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden", [128, 42])
def test_steps_follow_the_formula(hidden):
    """Three steps with new gradients each.  The update's operands are FP16 (2^-9 of its 2-norm), it is stored in
    BF16 (2^-8 of an element), and the weight that it is taken from is FP32, so the difference of two weights
    holds 2^-24 of the weight for either."""
    model = E.Model(256, hidden, 128, seed=1, block="gated")
    lr = 1e-2
    matrices = E.Orthogonalised(model, lr)
    assert set(matrices.names) == {f"{k}{i}" for k in ("gate", "up", "down") for i in range(model.L)}
    g = torch.Generator(device="cuda:0").manual_seed(1)
    momentum = {k: np.zeros(tuple(model.params[k].shape)) for k in matrices.names}
    for _ in range(3):
        model.loss_and_gradients(*E.batch(256, 128, g))
        before = {k: model.params[k].clone() for k in matrices.names}
        for k in matrices.names:
            momentum[k] = matrices.momentum * momentum[k] + model.grads[k].double().cpu().numpy()
        matrices.step()
        for k, w in before.items():
            step = (model.params[k].double() - w.double()).cpu().numpy()
            want = -lr * 0.2 * max(w.shape) ** 0.5 * O.orthogonalize(momentum[k])
            norm = np.linalg.norm
            assert norm(want) > 0 and (step * momentum[k]).sum() < 0
            assert norm(step - want) <= (2.0 ** -8 + 2.0 ** -9) * norm(want) + 2.0 ** -23 * norm(w.double().cpu().numpy()), k
