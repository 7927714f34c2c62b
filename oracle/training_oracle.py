"""Plain fp64 numpy forms of the training-side operators: activations in 8 bits,
the gated feed-forward block and its gradients, softmax cross entropy of
``hidden W^T`` and its gradients.

TEST INFRASTRUCTURE ONLY, like :mod:`oracle.muon_oracle`: shares no code with the
CUDA library.  The gradients are pinned against central differences of the
forward forms, the 8-bit rounding against its definition in exact fractions
(``tests/test_training_oracle.py``).
"""
from __future__ import annotations

import math
from typing import Dict, Tuple

import numpy as np

ACT8_BLOCK = 32


def act8_codes(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(codes, scales) of a 2-D array: blocks of 32 columns, scale the smallest bf16
    number >= max|x| / 127 and >= 2^-126 (0 for zeros, NaN with codes 0 for a
    non-finite block), code = x / scale to the nearest integer, ties to even."""
    rows, cols = x.shape
    nb = -(-cols // ACT8_BLOCK)
    codes = np.zeros((rows, cols))
    scales = np.zeros((rows, nb))
    for r in range(rows):
        for b in range(nb):
            v = x[r, b * ACT8_BLOCK:(b + 1) * ACT8_BLOCK].astype(np.float64)
            if not np.all(np.isfinite(v)):
                scales[r, b] = np.nan
                continue
            top = float(np.max(np.abs(v)))
            if top == 0.0:
                continue
            mant, expo = math.frexp(max(top / 127.0, 2.0 ** -126))
            s = math.ldexp(math.ceil(mant * 256.0) / 256.0, expo)
            scales[r, b] = s
            codes[r, b * ACT8_BLOCK:(b + 1) * ACT8_BLOCK] = np.rint(v / s)
    return codes, scales


def act8_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return codes * np.repeat(scales, ACT8_BLOCK, axis=1)[:, :codes.shape[1]]


def act(kind: str, g: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """act(g) and act'(g) for "silu", "gelu" or "gelu_tanh"."""
    if kind == "silu":
        s = 0.5 * (1.0 + np.tanh(0.5 * g))
        return g * s, s + g * s * (1.0 - s)
    if kind == "gelu":
        phi = 0.5 * (1.0 + np.vectorize(math.erf)(g / math.sqrt(2.0)))
        return g * phi, phi + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (g + 0.044715 * g ** 3))
        return (0.5 * g * (1.0 + t),
                0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g))
    raise ValueError(kind)


def ffn_forward(x, w_gate, w_up, w_down, kind: str = "silu") -> Dict[str, np.ndarray]:
    gate, up = x @ w_gate.T, x @ w_up.T
    h = act(kind, gate)[0] * up
    return {"gate": gate, "up": up, "h": h, "y": h @ w_down.T}


def ffn_backward(dy, x, w_gate, w_up, w_down, gate, up, kind: str = "silu") -> Dict[str, np.ndarray]:
    a, da = act(kind, gate)
    dh = dy @ w_down
    dgate, dup = dh * up * da, dh * a
    return {"dx": dgate @ w_gate + dup @ w_up, "dw_gate": dgate.T @ x, "dw_up": dup.T @ x,
            "dw_down": dy.T @ (a * up)}


def xent(hidden, weight, target, grad_loss=None) -> Dict[str, np.ndarray]:
    """Per-token loss and log-sum-exp; with grad_loss the gradients of
    sum(grad_loss * loss).  A target outside [0, vocab) masks its token."""
    t, v = hidden.shape[0], weight.shape[0]
    live = np.nonzero((target >= 0) & (target < v))[0]
    h, tg = hidden[live], target[live]
    z = h @ weight.T
    top = z.max(axis=1, keepdims=True) if v else np.zeros((len(live), 1))
    e = np.exp(z - top)
    total = e.sum(axis=1, keepdims=True)
    lse = (np.log(total) + top)[:, 0]
    out = {"loss": np.zeros(t), "lse": np.zeros(t)}
    out["loss"][live] = lse - z[np.arange(len(live)), tg]
    out["lse"][live] = lse
    if grad_loss is not None:
        g = e / total
        g[np.arange(len(live)), tg] -= 1.0
        g *= grad_loss[live][:, None]
        out["dhidden"] = np.zeros_like(hidden)
        out["dhidden"][live] = g @ weight
        out["dweight"] = g.T @ h
    return out
