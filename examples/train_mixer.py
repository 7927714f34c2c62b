"""A whole layer -- norms and rotation, linear attention, a gated feed-forward block -- and an
output head, trained with the library on packed documents, then run token by token.

One step is what one owner's micro-batch looks like:
  1. one projection to queries, keys and values; the norms and the rotation of queries and keys;
     linear attention within each document; the output projection;
  2. the feed-forward block and the head's cross entropy with its gradients;
  3. backward through all of them, the gradients of queries, keys and values written side by side
     where the projection's gradient reads them;
  4. one Muon step on the projections, gate, up and down, one AdamW step on the head and the gains.
The task is to name the token that came two places earlier in the document, which takes a mixer
that knows positions.  Token embeddings are fixed random vectors.

    python examples/train_mixer.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Layer:
    def __init__(self, tokens, documents, hidden=256, heads=4, dim=64, ffn=512, vocab=512, seed=0,
                 device="cuda"):
        from newton_schulz_owner_gb300 import dmuon

        self.dm, self.tokens, self.heads, self.dim, self.vocab = dmuon, tokens, heads, dim, vocab
        self.gen = torch.Generator(device=device).manual_seed(seed)
        width = heads * dim
        self.embedding = self.normal((vocab, hidden), 1.0)
        self.w_qkv = self.normal((3 * width, hidden), hidden ** -0.5)
        self.w_o = self.normal((hidden, width), 0.1 * width ** -0.5)   # sums over many tokens are large
        self.ffn = [self.normal((ffn, hidden), hidden ** -0.5), self.normal((ffn, hidden), hidden ** -0.5),
                    self.normal((hidden, ffn), ffn ** -0.5)]
        self.head = self.normal((vocab, hidden), hidden ** -0.5)
        self.gains = [torch.ones(dim, dtype=torch.bfloat16, device=device) for _ in range(2)]
        # heads that remember from a few tokens to a few hundred; slow to fast rotations
        self.log_decay = -torch.exp2(-8 * torch.arange(1, heads + 1, device=device).float() / heads)
        self.inv_freq = (10000.0 ** (-torch.arange(dim // 2, device=device).double() * 2 / dim)).float()

        self.rope = dmuon.QKNormRope(tokens, heads, heads, dim, device=device)
        self.mix = dmuon.LinearAttention(tokens, heads, dim, max_sequences=documents, device=device)
        self.block = dmuon.GatedFFN(tokens, hidden, ffn, device=device)
        self.loss_fn = dmuon.LinearXent(tokens, hidden, vocab, device=device)

    def normal(self, shape, std):
        return torch.randn(shape, generator=self.gen, device=self.gen.device).mul_(std).to(torch.bfloat16)

    def parts(self, qkv):
        """Queries, keys and values of a packed projection."""
        t, w = qkv.shape[0], self.heads * self.dim
        return [qkv[:, i * w:(i + 1) * w].view(t, self.heads, self.dim) for i in range(3)]

    def forward(self, ids, position, offsets):
        """What the head reads, and what backward needs."""
        x = self.embedding[ids]
        qkv = x @ self.w_qkv.t()
        q, k, v = self.parts(qkv)
        qr, kr, o = (torch.zeros(q.shape, dtype=q.dtype, device=q.device) for _ in range(3))
        self.rope.forward(q, k, *self.gains, self.inv_freq, position, qr, kr)
        self.mix.forward(qr, kr, v, self.log_decay, o, offsets=offsets)
        h = x + o.flatten(1) @ self.w_o.t()
        y, saved = torch.empty_like(h), self.block.empty_saved(h.shape[0])
        self.block.forward(h, *self.ffn, y, saved)
        return h + y, (x, qkv, qr, kr, o, h, saved)

    def gradients(self, ids, position, offsets, target, grad_loss):
        """Per-token loss; gradients of qkv, the output projection, gate, up, down, head and gains."""
        out, (x, qkv, qr, kr, o, h, saved) = self.forward(ids, position, offsets)
        q, k, v = self.parts(qkv)
        loss, lse = torch.empty_like(grad_loss), torch.empty_like(grad_loss)
        dout, dh, dhead = torch.empty_like(out), torch.empty_like(h), torch.empty_like(self.head)
        dffn = [torch.empty_like(w) for w in self.ffn]
        self.loss_fn.loss_and_grads(out, self.head, target, grad_loss, loss, lse, dout, dhead)
        self.block.backward(dout, h, *self.ffn, saved, dh, *dffn)
        dh = dh + dout
        do = (dh @ self.w_o).view(o.shape)
        dqkv = torch.zeros_like(qkv)
        dq, dk, dv = self.parts(dqkv)
        dqr, dkr = torch.zeros_like(qr), torch.zeros_like(kr)
        self.mix.backward(do, qr, kr, v, self.log_decay, dqr, dkr, dv, offsets=offsets)
        dgains = [torch.empty_like(g) for g in self.gains]
        self.rope.backward(dqr, dkr, q, k, *self.gains, self.inv_freq, position, dq, dk, *dgains)
        return loss, [dqkv.t() @ x, dh.t() @ o.flatten(1), *dffn], [dhead, *dgains]

    def step(self, ids, position, state):
        """The head's logits of one token for each of a few streams, whose states go on."""
        x = self.embedding[ids]
        qkv = x @ self.w_qkv.t()
        q, k, v = self.parts(qkv)
        qr, kr, o = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        self.rope.forward(q, k, *self.gains, self.inv_freq, position, qr, kr)
        self.mix.step(qr, kr, v, self.log_decay, state, o)
        h = x + o.flatten(1) @ self.w_o.t()
        y, saved = torch.empty_like(h), self.block.empty_saved(h.shape[0])
        self.block.forward(h, *self.ffn, y, saved)
        return (h + y) @ self.head.t()

    def check(self):
        for op in (self.rope, self.mix, self.block, self.loss_fn):
            if op.status() != self.dm.OK:
                raise self.dm.DMuonError(op.status(), type(op).__name__)


def documents(gen, tokens, count, vocab):
    """Packed random documents: ids, positions, offsets and targets (two places back; none for a
    document's first two tokens)."""
    device = gen.device
    cuts = torch.randint(1, tokens, (count - 1,), generator=gen, device=device).sort().values
    ends = torch.cat([torch.zeros(1, dtype=torch.long, device=device), cuts,
                      torch.full((1,), tokens, device=device)])
    at = torch.arange(tokens, device=device)
    position = at - ends[torch.bucketize(at, ends[1:-1], right=True)]
    ids = torch.randint(vocab, (tokens,), generator=gen, device=device)
    target = torch.where(position >= 2, ids.roll(2), -100)
    return ids, position.int(), ends.int(), target


def train(steps=40, tokens=2048, count=6, seed=0, device="cuda", verbose=False):
    """Mean loss over the tokens with a target, of each step; and the trained layer."""
    layer = Layer(tokens, count, seed=seed, device=device)
    dm = layer.dm
    matrices = [layer.w_qkv, layer.w_o, *layer.ffn]
    others = [layer.head, *layer.gains]
    owner = dm.MuonOwner([tuple(w.shape) for w in matrices], device=device)
    momenta = [torch.zeros(w.shape, device=device) for w in matrices]
    m, v = ([torch.zeros(w.shape, device=device) for w in others] for _ in range(2))
    adam_ws = torch.zeros(dm.adamw_workspace_bytes(len(others)), dtype=torch.uint8, device=device)
    means = []
    for step in range(1, steps + 1):
        ids, position, offsets, target = documents(layer.gen, tokens, count, layer.vocab)
        live = (target >= 0).float()
        loss, grads, rest = layer.gradients(ids, position, offsets, target, live / live.sum())
        owner.step(grads, momenta, matrices, lr=0.02)
        dm.adamw(others, rest, m, v, step, adam_ws, lr=3e-3, weight_decay=0.0)
        means.append((loss.sum() / live.sum()).detach())
        if verbose and (step % 10 == 0 or step == 1):
            print(f"step {step:4d}  loss {means[-1].item():.4f}")
    layer.check()
    return [float(x) for x in means], layer


if __name__ == "__main__":
    losses, layer = train(int(sys.argv[1]) if len(sys.argv) > 1 else 150, verbose=True)
    # four streams, token by token: how often the token two places back is named
    ids = torch.randint(layer.vocab, (40, 4), generator=layer.gen, device="cuda")
    state = torch.zeros((4, layer.heads, layer.dim, layer.dim), device="cuda")
    right = 0
    for t in range(40):
        position = torch.full((4,), t, dtype=torch.int32, device="cuda")
        best = layer.step(ids[t], position, state).float().argmax(dim=1)
        right += int((best == ids[t - 2]).sum()) if t >= 2 else 0
    print(f"named {right} of {38 * 4}")
