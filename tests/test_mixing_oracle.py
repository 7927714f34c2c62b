"""Pins of the fp64 forms of the operators that mix tokens: gradients against central
differences, rotations and norms against their invariants, the recurrence against the sum it
stands for."""
import numpy as np
import pytest

import oracle

STEP = 1e-5
# central differences: truncation ~ STEP^2 |f'''| and rounding ~ 2^-53 |f| / STEP, both below
# 1e-8 for the functions here
TOL = 1e-6


def differences(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + STEP
        up = f()
        x[i] = keep - STEP
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * STEP)
    return g


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [0, 4, 8])
def test_norm_rope_gradients_match_differences(rotary, interleaved):
    r = np.random.default_rng(1)
    x, dy, w = r.standard_normal((3, 2, 8)), r.standard_normal((3, 2, 8)), r.standard_normal(8)
    f, pos = 1.0 / 7.0 ** np.arange(rotary // 2), np.array([0, 5, -9])
    loss = lambda: float(np.sum(dy * oracle.norm_rope(x, w, f, pos, 1e-3, interleaved)))
    dx, dw = oracle.norm_rope_backward(dy, x, w, f, pos, 1e-3, interleaved)
    assert np.max(np.abs(dx - differences(loss, x))) < TOL
    assert np.max(np.abs(dw - differences(loss, w))) < TOL


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance_only(interleaved):
    r = np.random.default_rng(2)
    a, b = r.standard_normal((1, 1, 16)), r.standard_normal((1, 1, 16))
    w, f = np.ones(16), 1.0 / 10.0 ** np.arange(8)
    at = lambda x, p: oracle.norm_rope(x, w, f, np.array([p]), 0.0, interleaved)[0, 0]
    assert abs(np.sum(at(a, 12345) ** 2) - 16) < 1e-9
    assert abs(at(a, 3) @ at(b, 10) - at(a, 1003) @ at(b, 1010)) < 1e-9
    assert abs(at(a, 3) @ at(b, 10) - at(a, 3) @ at(b, 11)) > 1e-3


def case(r, t=7, h=2, dk=3, dv=4):
    return (r.standard_normal((t, h, dk)), r.standard_normal((t, h, dk)),
            r.standard_normal((t, h, dv)), -np.array([0.3, 0.0])[:h])


def test_linattn_is_the_decayed_sum_of_earlier_tokens():
    q, k, v, g = case(np.random.default_rng(3))
    got = oracle.linattn(q, k, v, g, 0.5)["out"]
    for t in range(7):
        for h in range(2):
            want = sum(0.5 * np.exp(g[h] * (t - s)) * (q[t, h] @ k[s, h]) * v[s, h]
                       for s in range(t + 1))
            assert np.allclose(got[t, h], want, atol=1e-12)


def test_linattn_sequences_are_apart_and_continue_from_states():
    q, k, v, g = case(np.random.default_rng(4))
    off = [1, 4, 4, 6]
    st = np.random.default_rng(5).standard_normal((3, 2, 3, 4))
    whole = oracle.linattn(q, k, v, g, 0.7, off, st)
    assert not whole["out"][0].any() and not whole["out"][6].any()
    assert np.array_equal(whole["state"][1], st[1])                       # an empty sequence
    one = oracle.linattn(q[1:3], k[1:3], v[1:3], g, 0.7, None, st[:1])
    two = oracle.linattn(q[3:4], k[3:4], v[3:4], g, 0.7, None, one["state"])
    assert np.allclose(np.concatenate([one["out"], two["out"]]), whole["out"][1:4], atol=1e-12)
    assert np.allclose(two["state"][0], whole["state"][0], atol=1e-12)


def test_linattn_gradients_match_differences():
    r = np.random.default_rng(6)
    q, k, v, g = case(r)
    off, st = [0, 3, 3, 6], r.standard_normal((3, 2, 3, 4))
    dout, dfin = r.standard_normal((7, 2, 4)), r.standard_normal((3, 2, 3, 4))

    def loss():
        y = oracle.linattn(q, k, v, g, 0.6, off, st)
        return float(np.sum(dout * y["out"]) + np.sum(dfin * y["state"]))

    got = oracle.linattn_backward(dout, q, k, v, g, 0.6, off, st, dfin)
    for name, x in [("dq", q), ("dk", k), ("dv", v), ("dstate", st)]:
        assert np.max(np.abs(got[name] - differences(loss, x))) < TOL, name


def test_a_planted_mistake_is_seen():
    """Without the decay, or with the state read before its own token, the pins above fail."""
    q, k, v, g = case(np.random.default_rng(7))
    right = oracle.linattn(q, k, v, g, 1.0)["out"]
    assert np.max(np.abs(oracle.linattn(q, k, v, 0 * g, 1.0)["out"] - right)) > 1e-2
    late = oracle.linattn(q[1:], k[:-1], v[:-1], g, 1.0)["out"]
    assert np.max(np.abs(late - right[1:])) > 1e-2
