"""Training steps of a small language model whose output layer is its token embedding.

    x = E[ids]    h = x W^T    logits = h E^T    loss = -mean log p(next token)

The library's calls carry the two ends of the vocabulary and the update:

* token_logprobs gives the loss and, in place of the logits, token_logprobs_backward its gradient;
* accumulate_embedding_wgrad adds the gradient of the input rows to E's fp32 main_grad, into
  which the output layer's gradient went before;
* orthogonalize_update turns W's momentum into its update; E takes a plain step.

    python examples/tied_embedding_step.py [steps]

The matrix products between them are torch's.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import embedding_weight_grad_gb300 as ewg  # noqa: E402


class TiedModel:
    def __init__(self, vocab: int, hidden: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.E = torch.randn(vocab, hidden, generator=g, device=device) * hidden ** -0.5   # fp32 masters
        self.W = torch.eye(hidden, device=device) + 0.1 * hidden ** -0.5 * torch.randn(
            hidden, hidden, generator=g, device=device)
        self.E_grad = torch.zeros_like(self.E)         # fp32 main_grads
        self.W_grad = torch.zeros_like(self.W)
        self.W_momentum = torch.zeros_like(self.W)

    def forward_backward(self, ids: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        """Adds the batch's gradients to the main_grads; returns the mean loss (targets < 0:
        no loss at that position)."""
        E, W = self.E.bfloat16(), self.W.bfloat16()
        x = E[ids]
        h = x @ W.T
        logits = h @ E.T
        r = ewg.token_logprobs(logits, targets)
        counted = (targets >= 0).sum()
        grad = torch.full_like(r.logprobs, -1.0) / counted
        dlogits = ewg.token_logprobs_backward(logits, targets, r.row_max, r.log_sum, grad, out=logits)
        dh = dlogits @ E
        dx = dh @ W
        self.E_grad += dlogits.T @ h                   # the embedding as the output layer ...
        ewg.accumulate_embedding_wgrad(ids, dx, self.E_grad)      # ... and as the input's table
        self.W_grad += dh.T @ x
        return -r.logprobs.sum() / counted

    def update(self, lr_matrix: float, lr_embedding: float, momentum: float = 0.9) -> None:
        self.W_momentum.mul_(momentum).add_(self.W_grad)
        self.W.add_(ewg.orthogonalize_update(self.W_momentum), alpha=-lr_matrix)
        self.E.add_(self.E_grad, alpha=-lr_embedding)
        self.E_grad.zero_()
        self.W_grad.zero_()

    def likely_next(self, id_: int, top: int = 5):
        """The most likely tokens after a token, with their log probabilities."""
        row = self.E[id_].bfloat16() @ self.W.bfloat16().T @ self.E.bfloat16().T
        r = ewg.token_logprobs(row, torch.zeros((), dtype=torch.int64, device=row.device), top=top)
        return list(zip(r.top_ids.tolist(), r.top_logprobs.tolist()))


def batch(vocab: int, tokens: int, seed: int, device="cuda"):
    """Tokens whose successor is (5 id + 1) mod vocab; one in sixteen without a target."""
    g = torch.Generator(device=device).manual_seed(seed)
    ids = torch.randint(vocab, (tokens,), generator=g, device=device)
    targets = (ids * 5 + 1) % vocab
    return ids, torch.where(torch.rand(tokens, generator=g, device=device) < 1 / 16, -100, targets)


def train(steps: int = 30, vocab: int = 1000, hidden: int = 256, tokens: int = 4096):
    model = TiedModel(vocab, hidden)
    losses = []
    for step in range(steps):
        losses.append(model.forward_backward(*batch(vocab, tokens, step)))
        model.update(lr_matrix=0.02, lr_embedding=60.0)
    return model, [float(x) for x in losses]


if __name__ == "__main__":
    model, losses = train(int(sys.argv[1]) if len(sys.argv) > 1 else 30)
    for i in range(0, len(losses), 5):
        print(f"step {i:3d}  loss {losses[i]:.4f}")
    print("after token 7 (36 follows it):", [(i, round(p, 2)) for i, p in model.likely_next(7)])
