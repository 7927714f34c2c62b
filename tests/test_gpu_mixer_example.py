"""The example of a whole layer runs, repeats bit for bit, has the gradients of its loss, and its
single-token steps agree with its packed forward pass."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from newton_schulz_owner_gb300 import build_lib
    if not os.path.exists(build_lib.LIB):
        build_lib.build()
    spec = importlib.util.spec_from_file_location(
        "train_mixer", os.path.join(ROOT, "examples", "train_mixer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_it_runs_and_repeats_bit_for_bit(example):
    a, la = example.train(steps=4, seed=3)
    b, lb = example.train(steps=4, seed=3)
    assert a == b and all(math.isfinite(x) for x in a)
    assert torch.equal(la.w_qkv, lb.w_qkv) and torch.equal(la.gains[0], lb.gains[0])


def test_its_gradients_are_those_of_its_loss(example):
    """Against autograd of the same layer in fp64.  Each gradient is a chain of about ten bf16
    roundings of u = 2^-8, independent: relative Frobenius error at most 10 u."""
    t, n = 300, 4
    layer = example.Layer(t, n, seed=5)
    ids, position, offsets, target = example.documents(layer.gen, t, n, layer.vocab)
    live = target >= 0
    gl = live.float() / live.sum()
    _, grads, rest = layer.gradients(ids, position, offsets, target, gl)
    names = ["w_qkv", "w_o", "gate", "up", "down", "head", "gain_q", "gain_k"]
    leaf = [w.double().requires_grad_() for w in
            [layer.w_qkv, layer.w_o, *layer.ffn, layer.head, *layer.gains]]
    x, h, d = layer.embedding[ids].double(), layer.heads, layer.dim
    q, k, v = ((x @ leaf[0].t())[:, i * h * d:(i + 1) * h * d].view(t, h, d) for i in range(3))
    angle = torch.outer(position.double(), layer.inv_freq.double())[:, None]

    def turned(z, w):
        z = z / torch.sqrt(z.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = z[..., :d // 2], z[..., d // 2:]
        return torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1)

    q, k = turned(q, leaf[6]), turned(k, leaf[7])
    at = torch.arange(t, device="cuda")
    doc = torch.bucketize(at, offsets[1:-1].long(), right=True)
    gap = at[:, None] - at
    see = (gap >= 0) & (doc[:, None] == doc)
    decay = torch.where(see, torch.exp(layer.log_decay.double()[:, None, None] * gap.clamp_min(0)), 0.0)
    o = torch.einsum("hij,jhd->ihd", torch.einsum("ihd,jhd->hij", q, k) * decay * d ** -0.5, v)
    y = x + o.flatten(1) @ leaf[1].t()
    y = y + (torch.nn.functional.silu(y @ leaf[2].t()) * (y @ leaf[3].t())) @ leaf[4].t()
    logp = torch.log_softmax(y @ leaf[5].t(), -1)
    loss = -(logp[live, target[live]]).sum() / live.sum()
    for name, got, want in zip(names, grads + rest, torch.autograd.grad(loss, leaf)):
        err = float((got.double() - want).norm() / want.norm())
        assert err <= 10 * U, (name, err)
    layer.check()


def test_steps_agree_with_the_packed_pass(example):
    """Three streams of 20 tokens, as packed documents and token by token: logits within the bf16
    roundings of either way, about six each."""
    n, t = 3, 20
    layer = example.Layer(n * t, n, seed=7)
    ids = torch.randint(layer.vocab, (n, t), generator=layer.gen, device="cuda")
    position = torch.arange(t, device="cuda").int().repeat(n)
    offsets = torch.arange(n + 1, device="cuda").int() * t
    want = (layer.forward(ids.flatten(), position, offsets)[0] @ layer.head.t()).view(n, t, -1).float()
    state = torch.zeros((n, layer.heads, layer.dim, layer.dim), device="cuda")
    for i in range(t):
        got = layer.step(ids[:, i], torch.full((n,), i, dtype=torch.int32, device="cuda"), state).float()
        assert float((got - want[:, i]).norm() / want[:, i].norm()) <= 6 * U
    layer.check()
