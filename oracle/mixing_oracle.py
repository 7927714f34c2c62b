"""Plain fp64 numpy forms of the operators that mix tokens: the norm and rotation of query and
key heads, linear attention with a decay for each head, and their gradients.

TEST INFRASTRUCTURE ONLY, like :mod:`oracle.muon_oracle`: shares no code with the CUDA library.
Token by token, as the definitions read; the gradients are pinned against central differences
(``tests/test_mixing_oracle.py``).
"""
from __future__ import annotations

from typing import Dict, Optional

import numpy as np


def _pairs(rotary: int, interleaved: bool):
    i = np.arange(rotary // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)


def _rotate(x, inv_freq, position, interleaved, sign):
    """x (tokens, heads, dim) with the first 2 * len(inv_freq) elements of each head turned."""
    y = x.copy()
    a, b = _pairs(2 * len(inv_freq), interleaved)
    t = sign * np.outer(position.astype(np.float64), inv_freq)[:, None, :]
    y[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
    y[..., b] = x[..., a] * np.sin(t) + x[..., b] * np.cos(t)
    return y


def norm_rope(x, w, inv_freq, position, eps, interleaved=False):
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return _rotate(n * w, inv_freq, position, interleaved, 1.0)


def norm_rope_backward(dy, x, w, inv_freq, position, eps, interleaved=False):
    g = _rotate(dy, inv_freq, position, interleaved, -1.0)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    n = x * r
    gw = g * w
    dx = r * (gw - n * np.mean(gw * n, axis=-1, keepdims=True))
    return dx, np.sum(g * n, axis=(0, 1))


def _bounds(offsets, tokens):
    return [(0, tokens)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def linattn(q, k, v, log_decay, scale, offsets=None, state=None) -> Dict[str, np.ndarray]:
    """out (tokens, heads, value_dim) and the state after each sequence; tokens of no sequence
    come out zero."""
    spans = _bounds(offsets, q.shape[0])
    h, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    out = np.zeros((q.shape[0], h, dv))
    final = np.zeros((len(spans), h, dk, dv)) if state is None else state.astype(np.float64)
    a = np.exp(log_decay)[:, None, None]
    for s, (b, e) in enumerate(spans):
        for t in range(b, e):
            final[s] = a * final[s] + k[t][:, :, None] * v[t][:, None, :]
            out[t] = scale * np.einsum("hi,hij->hj", q[t], final[s])
    return {"out": out, "state": final}


def linattn_backward(dout, q, k, v, log_decay, scale, offsets=None, state=None,
                     dfinal: Optional[np.ndarray] = None) -> Dict[str, np.ndarray]:
    spans = _bounds(offsets, q.shape[0])
    h, dk, dv = q.shape[1], q.shape[2], v.shape[2]
    dq, dkk, dvv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dstate = np.zeros((len(spans), h, dk, dv)) if dfinal is None else dfinal.astype(np.float64)
    a = np.exp(log_decay)[:, None, None]
    for s, (b, e) in enumerate(spans):
        st = np.zeros((h, dk, dv)) if state is None else state[s].astype(np.float64)
        for t in range(b, e):
            st = a * st + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * np.einsum("hij,hj->hi", st, dout[t])
        d = dstate[s]
        for t in range(e - 1, b - 1, -1):
            d = d + scale * q[t][:, :, None] * dout[t][:, None, :]
            dkk[t] = np.einsum("hij,hj->hi", d, v[t])
            dvv[t] = np.einsum("hij,hi->hj", d, k[t])
            d = a * d
        dstate[s] = d
    return {"dq": dq, "dk": dkk, "dv": dvv, "dstate": dstate}
