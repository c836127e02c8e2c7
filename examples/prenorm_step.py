"""Training steps of a small language model with layer norms, a residual branch and a tied embedding.

    x = E[ids]    h = x + norm(x) W^T    logits = norm(h) E^T    loss = -mean log p(next token)

Every part of the step that is not a matrix product or an addition is a call of the library:

* token_logprobs and token_logprobs_backward: the loss and its gradient;
* layer_norm and layer_norm_backward: the norms, whose weights' gradients go into main_grads;
* accumulate_embedding_wgrad: the gradient of the input rows, into E's main_grad;
* adamw_step: E (states in 8 bits, and the bf16 copy that the next forward pass reads) and the norms'
  weights and biases (states in 32 bits), the gradients scaled to a norm of at most 1;
* orthogonalize_update: W's update from its momentum.

    python examples/prenorm_step.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import embedding_weight_grad_gb300 as ewg  # noqa: E402


class PrenormModel:
    def __init__(self, vocab: int, hidden: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        # fp32 masters, their main_grads, and what the forward pass reads of E
        self.E = torch.randn(vocab, hidden, generator=g, device=device) * hidden ** -0.5
        self.W = hidden ** -0.5 * torch.randn(hidden, hidden, generator=g, device=device)
        self.norms = [torch.full((hidden,), v, device=device) for v in (1.0, 0.0, 1.0, 0.0)]   # weight, bias of two
        self.E16 = self.E.bfloat16()
        self.E_grad, self.W_grad = torch.zeros_like(self.E), torch.zeros_like(self.W)
        self.norm_grads = [torch.zeros_like(v) for v in self.norms]
        self.W_momentum = torch.zeros_like(self.W)
        self.table = ewg.adamw_plan([self.E], [self.E_grad], state_bits=8, copies=[self.E16], weight_decay=0.01)
        self.vectors = ewg.adamw_plan(self.norms, self.norm_grads, weight_decay=0.0)
        self.steps = 0

    def forward_backward(self, ids: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        """Adds the batch's gradients to the main_grads; returns the mean loss (targets < 0: none at
        that position)."""
        E, W = self.E16, self.W.bfloat16()
        w1, b1, w2, b2 = self.norms
        x = E[ids]
        first = ewg.layer_norm(x, w1, b1)
        h = x + first.out @ W.T
        second = ewg.layer_norm(h, w2, b2)
        logits = second.out @ E.T
        r = ewg.token_logprobs(logits, targets)
        counted = (targets >= 0).sum()
        grad = torch.full_like(r.logprobs, -1.0) / counted
        dlogits = ewg.token_logprobs_backward(logits, targets, r.row_max, r.log_sum, grad, out=logits)
        self.E_grad += dlogits.T @ second.out          # the embedding as the output layer
        dy = dlogits @ E
        dh = ewg.layer_norm_backward(dy, h, second.mean, second.rstd, w2, weight_main_grad=self.norm_grads[2],
                                     bias_main_grad=self.norm_grads[3], out=dy)
        self.W_grad += dh.T @ first.out
        da = dh @ W
        dx = ewg.layer_norm_backward(da, x, first.mean, first.rstd, w1, weight_main_grad=self.norm_grads[0],
                                     bias_main_grad=self.norm_grads[1], out=da)
        ewg.accumulate_embedding_wgrad(ids, dx + dh, self.E_grad)     # ... and as the input's table
        return -r.logprobs.sum() / counted

    def update(self, lr: float, lr_matrix: float, momentum: float = 0.9) -> None:
        self.steps += 1
        # a clipping factor that stays on the device
        size = torch.stack([g.square().sum() for g in (self.E_grad, *self.norm_grads)]).sum().sqrt()
        scale = (1.0 / size).clamp_max(1.0)
        ewg.adamw_step(self.table, self.steps, lr=lr, grad_scale=scale)
        ewg.adamw_step(self.vectors, self.steps, lr=lr, grad_scale=scale)
        self.W_momentum.mul_(momentum).add_(self.W_grad)
        self.W.add_(ewg.orthogonalize_update(self.W_momentum), alpha=-lr_matrix)
        for g in (self.E_grad, self.W_grad, *self.norm_grads):
            g.zero_()


def batch(vocab: int, tokens: int, seed: int, device="cuda"):
    """Tokens whose successor is (5 id + 1) mod vocab; one in sixteen without a target."""
    g = torch.Generator(device=device).manual_seed(seed)
    ids = torch.randint(vocab, (tokens,), generator=g, device=device)
    targets = (ids * 5 + 1) % vocab
    return ids, torch.where(torch.rand(tokens, generator=g, device=device) < 1 / 16, -100, targets)


def train(steps: int = 30, vocab: int = 1000, hidden: int = 256, tokens: int = 4096):
    model = PrenormModel(vocab, hidden)
    losses = []
    for step in range(steps):
        losses.append(model.forward_backward(*batch(vocab, tokens, step)))
        model.update(lr=3e-3, lr_matrix=0.02)
    return model, [float(x) for x in losses]


if __name__ == "__main__":
    model, losses = train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
    for i in range(0, len(losses), 5):
        print(f"step {i:3d}  loss {losses[i]:.4f}")
