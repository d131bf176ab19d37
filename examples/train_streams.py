"""Trains a small model of mHC sublayers with the library's calls: token ids to
streams, sublayers between collapse and update, the gates, every gradient.

    python examples/train_streams.py [--steps 40] [--tokens 2048] [--hidden 256] [--block gated]

Each sublayer is forward_gates (projection, RMS, gates) -> collapse and norm ->
a block -> stream update with dropout.  The block is two matrices in torch
("plain"), or the library's gated feed-forward block ("gated"), whose matrices
are then trained by orthogonalised updates, the other parameters by Adam.  The backward
runs the same calls in reverse: update, the block, collapse and norm (with the
residual path's gradient), gates, projection with that gradient as its addend;
the embedding table's gradient comes last.  The task is synthetic: predict the
next token of sequences that step through the vocabulary by a fixed stride.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import rms_backward_gb300 as mhc  # noqa: E402

BF = torch.bfloat16


class Model:
    """Parameters (FP32), buffers and one training step.  Gradients land in
    ``grads`` under the parameters' names."""

    def __init__(self, tokens: int, hidden: int, vocab: int, layers: int = 2, p: float = 0.1, seed: int = 0,
                 device: str = "cuda:0", block: str = "plain"):
        self.T, self.D, self.V, self.L, self.p, self.block = tokens, hidden, vocab, layers, p, block
        g = torch.Generator(device=device).manual_seed(seed)
        new = lambda *s, std=1.0: torch.randn(*s, generator=g, device=device) * std  # noqa: E731
        K, D = 4 * hidden, hidden
        self.params = {"table": new(vocab, D), "head": new(vocab, D, std=D ** -0.5), "norm": torch.ones(D, device=device),
                       "norm_bias": torch.zeros(D, device=device)}
        for i in range(layers):
            bias = torch.zeros(24, device=device)
            bias[:4] = -1.0                                        # sigmoid(-1) of each stream enters the sublayer
            bias[8:] = 2.0 * torch.eye(4, device=device).reshape(-1)   # streams mostly keep to themselves
            self.params.update({
                f"w{i}": new(24, K, std=K ** -0.5), f"alpha{i}": torch.full((3,), 0.5, device=device), f"bias{i}": bias,
                f"gamma{i}": torch.ones(D, device=device), f"beta{i}": torch.zeros(D, device=device)})
            if block == "gated":
                self.params.update({f"gate{i}": new(2 * D, D, std=D ** -0.5), f"up{i}": new(2 * D, D, std=D ** -0.5),
                                    f"down{i}": new(D, 2 * D, std=(2 * D) ** -0.5)})
            else:
                self.params.update({f"up{i}": new(D, 2 * D, std=D ** -0.5), f"down{i}": new(2 * D, D, std=(2 * D) ** -0.5)})
        self.grads = {k: torch.zeros_like(v) for k, v in self.params.items()}
        self.rng = torch.tensor([1234 + seed, 0], dtype=torch.int64, device=device)   # key, step
        self.plan = mhc.Plan(self.T, K, torch.device(device).index or 0, addend=True)
        f32 = lambda *s: torch.empty(*s, device=device)  # noqa: E731
        b16 = lambda *s: torch.empty(*s, dtype=BF, device=device)  # noqa: E731
        T = self.T
        self.layers = [dict(x=b16(T, K), proj=f32(T, 32), r=f32(T), h=f32(T, 24), n=b16(T, D), mean=f32(T), rstd=f32(T),
                            y=b16(T, D)) for _ in range(layers)]
        if block == "gated":   # the matrices in BF16 and the projections that the backward needs
            for i, a in enumerate(self.layers):
                a.update(weights=[self.params[f"{k}{i}"].to(BF) for k in ("gate", "up", "down")], gate=b16(T, 2 * D), up=b16(T, 2 * D))
        self.x, self.out, self.mean, self.rstd = b16(T, K), b16(T, D), f32(T), f32(T)
        self.mean_gates = torch.zeros(T, 24, device=device)
        self.mean_gates[:, :4] = 0.25                              # the readout: the streams' mean
        self.grad_x, self.grad_part, self.grad_in = b16(T, K), b16(T, K), b16(T, K)
        self.grad_y, self.grad_n, self.grad_h = b16(T, D), b16(T, D), f32(T, 24)
        self.grad_proj, self.grad_r, self.grad_l = f32(T, 32), f32(T), f32(T, 24)
        size = max(self.plan.workspace_bytes, self.plan.forward_workspace_bytes,
                   mhc.mhc_embed_workspace_bytes(T, vocab, D), mhc.mhc_collapse_norm_workspace_bytes(T, D))
        if block == "gated":
            size = max(size, mhc.mhc_ffn_forward_workspace_bytes(T, D, 2 * D), mhc.mhc_ffn_backward_workspace_bytes(T, D, 2 * D),
                       mhc.mhc_orthogonalize_workspace_bytes(2 * D, D), mhc.mhc_orthogonalize_workspace_bytes(D, 2 * D))
        self.workspace = torch.empty(size, dtype=torch.uint8, device=device)

    def forward(self, ids):
        p, ws = self.params, self.workspace
        first = self.layers[0]["x"] if self.L else self.x
        mhc.mhc_embed_forward(ids, p["table"], first)
        for i, a in enumerate(self.layers):
            self.plan.forward_gates(a["x"], p[f"w{i}"], p[f"alpha{i}"], p[f"bias{i}"], a["proj"], a["r"], a["h"], ws)
            mhc.mhc_collapse_norm_forward(a["x"], a["h"], p[f"gamma{i}"], p[f"beta{i}"], a["n"], a["mean"], a["rstd"])
            if self.block == "gated":
                for w, k in zip(a["weights"], ("gate", "up", "down")):
                    w.copy_(p[f"{k}{i}"])
                mhc.mhc_ffn_forward(a["n"], *a["weights"], a["y"], ws, a["gate"], a["up"])
            else:
                a["u"] = a["n"].float() @ p[f"up{i}"]
                a["y"].copy_(torch.nn.functional.silu(a["u"]) @ p[f"down{i}"])
            out = self.layers[i + 1]["x"] if i + 1 < self.L else self.x
            mhc.mhc_update_forward(a["x"], a["y"], a["h"], out, self.rng, p=self.p, sequence=i)
        mhc.mhc_collapse_norm_forward(self.x, self.mean_gates, p["norm"], p["norm_bias"], self.out, self.mean, self.rstd)
        return self.out.float() @ p["head"].t()

    def backward(self, ids, grad_logits):
        p, g, ws = self.params, self.grads, self.workspace
        g["head"].copy_(grad_logits.t() @ self.out.float())
        self.grad_y.copy_(grad_logits @ p["head"])
        mhc.mhc_collapse_norm_backward(self.x, self.mean_gates, self.grad_y, p["norm"], self.mean, self.rstd, self.grad_x,
                                       self.grad_h, g["norm"], g["norm_bias"], ws)
        for i in reversed(range(self.L)):
            a = self.layers[i]
            mhc.mhc_update_backward(a["x"], a["y"], a["h"], self.grad_x, self.grad_y, self.grad_h, self.rng, p=self.p,
                                    sequence=i)
            if self.block == "gated":
                mhc.mhc_ffn_backward(a["n"], *a["weights"], a["gate"], a["up"], self.grad_y, self.grad_n, g[f"gate{i}"],
                                     g[f"up{i}"], g[f"down{i}"], ws)
            else:
                dy, s = self.grad_y.float(), torch.sigmoid(a["u"])
                g[f"down{i}"].copy_((a["u"] * s).t() @ dy)
                du = (dy @ p[f"down{i}"].t()) * s * (1 + a["u"] * (1 - s))
                g[f"up{i}"].copy_(a["n"].float().t() @ du)
                self.grad_n.copy_(du @ p[f"up{i}"].t())
            mhc.mhc_collapse_norm_backward(a["x"], a["h"], self.grad_n, p[f"gamma{i}"], a["mean"], a["rstd"], self.grad_part,
                                           self.grad_h, g[f"gamma{i}"], g[f"beta{i}"], ws, grad_x_out=self.grad_x)
            mhc.mhc_gate_backward(a["proj"], a["r"], p[f"alpha{i}"], p[f"bias{i}"], self.grad_h, self.grad_proj,
                                  self.grad_r, self.grad_l)
            scaled = self.grad_l * a["proj"][:, :24] / a["r"][:, None]   # the gates' parameters are the caller's
            g[f"alpha{i}"].copy_(torch.stack([scaled[:, :4].sum(), scaled[:, 4:8].sum(), scaled[:, 8:].sum()]))
            g[f"bias{i}"].copy_(self.grad_l.sum(0))
            self.plan.execute(a["x"], p[f"w{i}"], self.grad_proj, self.grad_r, a["r"], self.grad_in, g[f"w{i}"], ws,
                              addend=self.grad_part)
            self.grad_x, self.grad_in = self.grad_in, self.grad_x
        mhc.mhc_embed_backward(ids, self.grad_x, g["table"], ws)

    def loss_and_gradients(self, ids, targets):
        logits = self.forward(ids)
        loss = torch.nn.functional.cross_entropy(logits, targets)
        grad = torch.softmax(logits, 1)
        grad[torch.arange(self.T, device=grad.device), targets] -= 1.0
        self.backward(ids, grad / self.T)
        return loss


class Orthogonalised:
    """Momentum, then the orthogonalised update, of a model's block matrices."""

    def __init__(self, model: Model, lr: float, momentum: float = 0.95):
        self.model, self.lr, self.momentum = model, lr, momentum
        self.names = [f"{k}{i}" for i in range(model.L) for k in ("gate", "up", "down")] if model.block == "gated" else []
        self.state = {k: torch.zeros_like(model.params[k]) for k in self.names}
        self.out = {k: torch.empty_like(model.params[k], dtype=BF) for k in self.names}

    def step(self):
        for k in self.names:
            m, out, w = self.state[k], self.out[k], self.model.params[k]
            m.mul_(self.momentum).add_(self.model.grads[k])
            # scaled so that an element's root mean square is 0.2, about an Adam step's
            mhc.mhc_orthogonalize(m, out, self.model.workspace, scale=0.2 * max(w.shape) ** 0.5)
            w.sub_(out.float(), alpha=self.lr)


def batch(tokens: int, vocab: int, generator, device: str = "cuda:0"):
    """Ids and next ids of sequences of 32 that step by 7."""
    start = torch.randint(0, vocab, (-(-tokens // 32), 1), generator=generator, device=device)
    ids = ((start + 7 * torch.arange(33, device=device)) % vocab)
    return ids[:, :-1].reshape(-1)[:tokens].contiguous(), ids[:, 1:].reshape(-1)[:tokens].contiguous()


def train(steps: int = 40, tokens: int = 2048, hidden: int = 256, vocab: int = 512, layers: int = 2, p: float = 0.1,
          lr: float = 3e-3, seed: int = 0, say=print, block: str = "plain"):
    model = Model(tokens, hidden, vocab, layers, p, seed, block=block)
    g = torch.Generator(device="cuda:0").manual_seed(seed + 1)
    matrices = Orthogonalised(model, lr)
    names = [k for k in model.params if k not in matrices.names]
    optimizer = torch.optim.Adam([torch.nn.Parameter(model.params[k]) for k in names], lr=lr)
    for k, q in zip(names, optimizer.param_groups[0]["params"]):
        model.params[k], q.grad = q.data, model.grads[k]
    losses = []
    for step in range(steps):
        ids, targets = batch(tokens, vocab, g)
        loss = model.loss_and_gradients(ids, targets)
        optimizer.step()
        matrices.step()
        model.rng[1] += layers            # new masks: one sequence number per layer was used
        losses.append(loss)
        if step % 10 == 0 or step + 1 == steps:
            say(f"step {step:4d}  loss {loss.item():.4f}")
    if model.plan.device_status() != 0 or mhc.mhc_operators_device_status() != 0:
        raise RuntimeError("a wait inside a kernel timed out")
    return [v.item() for v in losses]


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--steps", type=int, default=40)
    a.add_argument("--tokens", type=int, default=2048)
    a.add_argument("--hidden", type=int, default=256)
    a.add_argument("--vocab", type=int, default=512)
    a.add_argument("--layers", type=int, default=2)
    a.add_argument("--block", choices=("plain", "gated"), default="plain")
    args = a.parse_args()
    train(args.steps, args.tokens, args.hidden, args.vocab, args.layers, block=args.block)
