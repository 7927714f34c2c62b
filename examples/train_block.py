"""A gated feed-forward block and an output head, trained with the library end to end.

One step is what one owner's micro-batch looks like:
  1. the block's forward pass, its gate and up projections kept in 8 bits;
  2. the head's cross entropy with the gradients of the hidden states and of the head,
     some tokens masked (padding);
  3. the block's backward pass from the 8-bit projections;
  4. one Muon step on gate, up and down, one AdamW step on the head.
The task is to name the successor of a token under a fixed permutation of the
vocabulary; token embeddings are fixed random vectors.

    python examples/train_block.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def train(steps=40, tokens=768, hidden=256, ffn=640, vocab=2000, seed=0, device="cuda",
          verbose=False):
    """Mean loss over the unmasked tokens of each step."""
    from newton_schulz_owner_gb300 import dmuon

    bf16 = torch.bfloat16
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(shape, std):
        return torch.randn(shape, generator=gen, device=device).mul_(std).to(bf16)

    embedding = normal((vocab, hidden), 1.0)
    successor = torch.randperm(vocab, generator=gen, device=device)
    weights = [normal((ffn, hidden), hidden ** -0.5), normal((ffn, hidden), hidden ** -0.5),
               normal((hidden, ffn), ffn ** -0.5)]                    # gate, up, down
    head = normal((vocab, hidden), hidden ** -0.5)

    block = dmuon.GatedFFN(tokens, hidden, ffn, save=dmuon.SAVE_ACT8, device=device)
    loss_fn = dmuon.LinearXent(tokens, hidden, vocab, device=device)
    owner = dmuon.MuonOwner([tuple(w.shape) for w in weights], device=device)
    momenta = [torch.zeros(w.shape, device=device) for w in weights]
    m, v = torch.zeros(head.shape, device=device), torch.zeros(head.shape, device=device)
    adam_ws = torch.zeros(dmuon.adamw_workspace_bytes(1), dtype=torch.uint8, device=device)

    saved = block.empty_saved(tokens)
    y, dx, dh = (torch.empty((tokens, hidden), dtype=bf16, device=device) for _ in range(3))
    grads = [torch.empty_like(w) for w in weights]
    dhead = torch.empty_like(head)
    loss, lse = torch.empty(tokens, device=device), torch.empty(tokens, device=device)

    means = []
    for step in range(1, steps + 1):
        ids = torch.randint(vocab, (tokens,), generator=gen, device=device)
        target = successor[ids]
        target[torch.rand(tokens, generator=gen, device=device) < 0.1] = -100   # padding
        live = (target >= 0).float()
        grad_loss = live / live.sum()

        x = embedding[ids]
        block.forward(x, *weights, y, saved)
        h = x + y
        loss_fn.loss_and_grads(h, head, target, grad_loss, loss, lse, dh, dhead)
        block.backward(dh, x, *weights, saved, dx, *grads)
        owner.step(grads, momenta, weights, lr=0.02)
        dmuon.adamw([head], [dhead], [m], [v], step, adam_ws, lr=3e-3, weight_decay=0.0)
        means.append((loss.sum() / live.sum()).detach())
        if verbose and (step % 10 == 0 or step == 1):
            print(f"step {step:4d}  loss {means[-1].item():.4f}")
    for op in (block, loss_fn, owner):
        if op.status() != dmuon.OK:
            raise dmuon.DMuonError(op.status(), "train_block")
    return [float(t) for t in means]


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 100, verbose=True)
