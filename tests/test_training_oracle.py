"""Pins of the fp64 forms of the training-side operators: gradients against central
differences, the 8-bit rounding against its definition in exact fractions, masks
against removal of the masked tokens."""
from fractions import Fraction

import numpy as np
import pytest

import oracle

STEP = 1e-5
# central differences: truncation ~ STEP^2 |f'''| and rounding ~ 2^-53 |f| / STEP, both
# below 1e-9 for the O(1) functions here; 1e-7 leaves two digits
TOL = 1e-7


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


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_ffn_gradients_match_differences(kind):
    r = np.random.default_rng(1)
    t, d, f = 3, 4, 5
    x, wg, wu, wd = (r.standard_normal(s) for s in [(t, d), (f, d), (f, d), (d, f)])
    dy = r.standard_normal((t, d))
    fwd = oracle.ffn_forward(x, wg, wu, wd, kind)
    got = oracle.ffn_backward(dy, x, wg, wu, wd, fwd["gate"], fwd["up"], kind)
    loss = lambda: float(np.sum(dy * oracle.ffn_forward(x, wg, wu, wd, kind)["y"]))
    for name, v in [("dx", x), ("dw_gate", wg), ("dw_up", wu), ("dw_down", wd)]:
        assert np.max(np.abs(got[name] - differences(loss, v))) < TOL, name


def test_xent_gradients_match_differences_with_masked_tokens():
    r = np.random.default_rng(2)
    h, w = r.standard_normal((5, 3)), r.standard_normal((7, 3))
    target = np.array([2, -100, 6, 7, 0])          # -100 and 7 (= vocab) mask
    gl = r.standard_normal(5)
    got = oracle.xent(h, w, target, gl)
    loss = lambda: float(np.sum(gl * oracle.xent(h, w, target)["loss"]))
    assert np.max(np.abs(got["dhidden"] - differences(loss, h))) < TOL
    assert np.max(np.abs(got["dweight"] - differences(loss, w))) < TOL
    live = [0, 2, 4]
    alone = oracle.xent(h[live], w, target[live], gl[live])
    assert np.array_equal(got["dweight"], alone["dweight"])
    for k in (1, 3):
        assert got["loss"][k] == 0 and got["lse"][k] == 0 and not got["dhidden"][k].any()


def test_xent_of_equal_logits_is_log_vocab():
    out = oracle.xent(np.zeros((2, 4)), np.ones((9, 4)), np.array([0, 8]))
    assert np.allclose(out["loss"], np.log(9), rtol=0, atol=1e-15)


def bf16_fraction_up(v: Fraction) -> Fraction:
    """Smallest number with 8 significant bits that is >= v > 0."""
    e = 0
    while v >= Fraction(2) ** (e + 1):
        e += 1
    while v < Fraction(2) ** e:
        e -= 1
    unit = Fraction(2) ** (e - 7)
    return -((-v) // unit) * unit


def test_act8_codes_follow_the_definition_in_exact_fractions():
    r = np.random.default_rng(3)
    for trial in range(200):
        # bf16 values: 8 significant bits
        v = oracle.round_bf16(r.standard_normal((1, 32)) * 2.0 ** r.integers(-20, 20))
        if trial % 5 == 0:
            v[0, 1:9] = v[0, 0] * np.array([127, 63.5, 31.5, 0.5, 1.5, 2.5, -0.5, -1.5]) / 128
            v = oracle.round_bf16(v)
        codes, scales = oracle.act8_codes(v)
        top = max(abs(Fraction(float(x))) for x in v[0])
        s = bf16_fraction_up(top / 127)
        assert Fraction(float(scales[0, 0])) == s
        for x, c in zip(v[0], codes[0]):
            q = Fraction(float(x)) / s
            assert abs(q - int(c)) <= Fraction(1, 2)
            if abs(q - int(c)) == Fraction(1, 2):
                assert int(c) % 2 == 0
            else:  # the margin that lets fp32 decide like exact arithmetic
                k = q - Fraction(1, 2)
                near = abs(k - round(k))
                assert near >= Fraction(1, 510) or abs(q) < Fraction(1, 2)


def test_act8_edges():
    v = np.zeros((1, 70))
    v[0, 33] = 2.0 ** -130      # below the smallest scale: rounds to a code of it
    v[0, 64:70] = [1.0, -1.0, 0.5, np.inf, 0.0, 3.0]
    codes, scales = oracle.act8_codes(v)
    assert scales[0, 0] == 0 and not codes[0, :32].any()
    assert scales[0, 1] == 2.0 ** -126 and not codes[0, 32:64].any()
    assert np.isnan(scales[0, 2]) and not codes[0, 64:].any()
    back = oracle.act8_values(codes, scales)
    assert back.shape == v.shape and np.isnan(back[0, 64:]).all() and not back[0, :64].any()
