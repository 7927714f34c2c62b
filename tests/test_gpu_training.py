"""GPU parity of the training-side operators (activations in 8 bits, the gated
feed-forward block with its gradients, softmax cross entropy with its gradients)
against their fp64 forms, at the sizes, strides and masks where they can go wrong.

Tolerances.  u = 2^-8 is bf16's unit roundoff.  An output is rounded once and is a
sum of products in which one factor was rounded once before (h, dgate, dup, the
gradient of the logits), so element by element
  |error| <= u |value| + 1.01 u sum |a||b|
with the sum over the products of that element (1.01: second order and fp32
accumulation).  Roundings of independent inputs are independent, so the relative
Frobenius error is about sqrt(2) u / sqrt(3) and at most 2 u.
Losses are fp32: a logit's error is at most 2^-22 sum_k |h_k W_k| (products exact in
fp32, at most a few roundings per partial sum), exp and log add 2^-20 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import os
    from newton_schulz_owner_gb300 import build_lib
    if not os.path.exists(build_lib.LIB):
        build_lib.build()
    from newton_schulz_owner_gb300 import dmuon
    return dmuon


def np64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def near(got, ref, what, mass):
    """`mass`: per element the sum of |a||b| over the products it sums, where one
    factor is rounded to bf16; 0.01 of it for a value that no operand rounding reaches."""
    got = np64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, what
    if ref.size == 0:
        return
    norm = np.linalg.norm(ref)
    err = got - ref
    assert np.all(np.isfinite(got)), what
    assert np.linalg.norm(err) <= 2 * U * norm, (what, np.linalg.norm(err) / norm)
    assert np.all(np.abs(err) <= U * np.abs(ref) + 1.01 * U * mass), what


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def __call__(self, shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=self.g, device="cuda").mul_(std).to(dtype)


SENTINEL = 7.0


class Rows:
    """A (rows, cols) view inside a larger buffer of sentinels, `pad` columns apart
    and `off` elements in."""

    def __init__(self, rows, cols, pad=0, off=0, fill=None):
        self.buf = torch.full((off + rows * (cols + pad) + 8,), SENTINEL, dtype=torch.bfloat16,
                              device="cuda")
        self.off, self.rows, self.cols, self.ld = off, rows, cols, cols + pad
        self.t = self.buf[off:off + rows * self.ld].view(rows, self.ld)[:, :cols]
        if fill is not None:
            self.t.copy_(fill)

    def intact(self):
        mask = torch.ones_like(self.buf, dtype=torch.bool)
        mask[self.off:self.off + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = False
        return bool((self.buf[mask] == SENTINEL).all())


# ------------------------------------------------------------------ 8-bit activations
def act8_check(dm, x, values_dt):
    rows, cols = x.shape
    codes, scales = dm.act8_empty(rows, cols)
    dm.act8_save(x, codes, scales)
    out = Rows(rows, cols, pad=3, off=1).t if values_dt == torch.bfloat16 else \
        torch.empty((rows, cols), device="cuda")
    dm.act8_load(codes, scales, out)
    return codes, scales, out


@pytest.mark.parametrize("shape", [(1, 1), (1, 4096), (3, 31), (3, 32), (5, 33), (2, 2047), (2, 2049),
                                   (7, 4104), (300, 100)])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 8), (5, 1)])
def test_act8_bf16_is_exact(dm, shape, pad, off):
    """bf16 inputs: codes, scales and restored values equal the definition's."""
    x = Rows(*shape, pad, off, Draw(3)(shape, 2.0) * torch.exp2(Draw(4)(shape, 3.0).float()).bfloat16())
    want_c, want_s = oracle.act8_codes(np64(x.t))
    for dt in (torch.bfloat16, torch.float32):
        codes, scales, out = act8_check(dm, x.t, dt)
        assert np.array_equal(np64(codes), want_c) and np.array_equal(np64(scales), want_s)
        want = torch.from_numpy(oracle.act8_values(want_c, want_s)).to(dt)
        assert torch.equal(out.cpu(), want)
    assert x.intact()


def test_act8_ties_go_to_even(dm):
    """Blocks whose largest value makes the scale 2^k: every half-integer quotient."""
    k = torch.arange(-127, 127, device="cuda").float() + 0.5
    x = torch.zeros((8, 64), device="cuda")
    x[:, :62] = k[:248].reshape(4, 62).repeat(2, 1)
    x[:, 31] = 127.0
    x[:, 63] = -127.0
    x[4:] *= 2.0 ** -20
    x = x.to(torch.bfloat16)
    want_c, want_s = oracle.act8_codes(np64(x))
    codes, scales, _ = act8_check(dm, x, torch.bfloat16)
    assert np.array_equal(np64(codes), want_c) and np.array_equal(np64(scales), want_s)


def test_act8_fp32_inputs(dm):
    """fp32 quotients round once before the nearest integer is taken, so a code may
    differ from exact arithmetic only where the quotient is a tie to within 2^-16."""
    x = Draw(5)((64, 1000), 1.0, torch.float32)
    want_c, want_s = oracle.act8_codes(np64(x))
    codes, scales, out = act8_check(dm, x, torch.float32)
    assert np.array_equal(np64(scales), want_s)
    q = np64(x) / np.repeat(want_s, 32, axis=1)[:, :1000]
    tie = np.abs(np.abs(q - np.floor(q)) - 0.5) < 2.0 ** -16
    assert np.all((np64(codes) == want_c) | tie)
    assert np.array_equal(np64(out), oracle.act8_values(np64(codes), want_s).astype(np.float32))


def test_act8_zero_tiny_and_non_finite_blocks(dm):
    x = torch.zeros((2, 160), device="cuda")
    x[:, 32] = 2.0 ** -130
    x[:, 64:96] = 3.0e38
    x[0, 100], x[1, 100] = float("inf"), float("nan")
    x[:, 101] = 1.0
    x[:, 128:] = 2.0 ** -120
    for dt in (torch.bfloat16, torch.float32):
        codes, scales, out = act8_check(dm, x.to(dt), torch.float32)
        want_c, want_s = oracle.act8_codes(np64(x.to(dt)))
        assert np.array_equal(np64(codes), want_c)
        assert np.array_equal(np64(scales), want_s, equal_nan=True)
        assert torch.isnan(out[:, 96:128]).all() and not torch.isnan(out[:, :96]).any()
        assert (out[:, :64] == 0).all() and torch.isfinite(out[:, 128:]).all()


# ------------------------------------------------------------------ feed-forward block
def ffn_case(seed, t, d, f):
    g = Draw(seed)
    return dict(x=g((t, d)), wg=g((f, d), 1.5 / np.sqrt(d)), wu=g((f, d), 1.5 / np.sqrt(d)),
                wd=g((d, f), 1 / np.sqrt(f)), dy=g((t, d), 1e-2))


def kept_values(op, dm, saved, t):
    if op.save == dm.SAVE_BF16:
        return [np64(s) for s in saved]
    return [oracle.act8_values(np64(saved[i]), np64(saved[i + 1])) for i in (0, 2)]


def check_kept(dm, op, saved, fwd, c, f):
    if op.save == dm.SAVE_BF16:
        for s, name, w in zip(saved, ("gate", "up"), ("wg", "wu")):
            near(s, fwd[name], name, 0.01 * (np.abs(np64(c["x"])) @ np.abs(np64(c[w])).T))
    elif op.save == dm.SAVE_ACT8:
        for i, name in ((0, "gate"), (2, "up")):
            c, s = np64(saved[i]), np64(saved[i + 1])
            _, want_s = oracle.act8_codes(fwd[name])
            # the scale rounds up to 8 bits: an fp32-sized difference moves it by one step at most
            assert np.all(np.abs(s - want_s) <= 2.0 ** -7 * want_s), name
            # half a step of rounding, and fp32 differences far below a step
            wide = np.repeat(s, 32, axis=1)[:, :f]
            assert np.all(np.abs(c * wide - fwd[name]) <= 0.51 * wide), name


FFN_SHAPES = [(1, 8, 8), (1, 64, 128), (3, 1032, 40), (8, 200, 1000), (5, 36, 64), (2, 100, 33), (17, 256, 129), (64, 129, 257), (65, 512, 384),
              (255, 72, 100), (256, 128, 128), (257, 520, 136), (513, 264, 640), (300, 1000, 2050),
              (33, 4096, 330), (97, 2048, 900), (250, 2900, 520), (700, 640, 1100)]


@pytest.mark.parametrize("t,d,f", FFN_SHAPES)
@pytest.mark.parametrize("save", [0, 1, 2])
def test_ffn_forward(dm, t, d, f, save):
    kind = ["silu", "gelu", "gelu_tanh"][(t + save) % 3]
    c = ffn_case(11, t, d, f)
    op = dm.GatedFFN(t, d, f, activation=ACTS[kind], save=save)
    fwd = oracle.ffn_forward(np64(c["x"]), np64(c["wg"]), np64(c["wu"]), np64(c["wd"]), kind)
    # rows in place, 16-byte aligned rows inside a wider tensor, and unaligned ones
    for pad, off in ((0, 0), (8, 8), (3, 1)):
        x, y = Rows(t, d, pad, off, c["x"]), Rows(t, d, pad, off)
        saved = op.empty_saved(t)
        op.forward(x.t, c["wg"], c["wu"], c["wd"], y.t, saved)
        assert op.status() == dm.OK
        near(y.t, fwd["y"], "y", np.abs(fwd["h"]) @ np.abs(np64(c["wd"])).T)
        check_kept(dm, op, saved, fwd, c, f)
        assert x.intact() and y.intact() and torch.equal(x.t, c["x"])


@pytest.mark.parametrize("t,d,f", FFN_SHAPES)
@pytest.mark.parametrize("save", [1, 2])
def test_ffn_backward(dm, t, d, f, save):
    kind = ["silu", "gelu", "gelu_tanh"][(t + f) % 3]
    c = ffn_case(12, t, d, f)
    op = dm.GatedFFN(t + 3, d, f, activation=ACTS[kind], save=save)
    saved = op.empty_saved(t)
    y = torch.empty_like(c["x"])
    op.forward(c["x"], c["wg"], c["wu"], c["wd"], y, saved)
    gate, up = kept_values(op, dm, saved, t)
    ref = oracle.ffn_backward(np64(c["dy"]), np64(c["x"]), np64(c["wg"]), np64(c["wu"]),
                              np64(c["wd"]), gate, up, kind)
    a, da = oracle.act(kind, gate)
    dh = np64(c["dy"]) @ np64(c["wd"])
    dg, du, ax = np.abs(dh * up * da), np.abs(dh * a), np.abs(np64(c["x"]))
    mass = {"dx": dg @ np.abs(np64(c["wg"])) + du @ np.abs(np64(c["wu"])), "dw_gate": dg.T @ ax,
            "dw_up": du.T @ ax, "dw_down": np.abs(np64(c["dy"])).T @ np.abs(a * up)}
    for pad, off in ((0, 0), (8, 8), (3, 1)):
        x, dy, dx = Rows(t, d, pad, off, c["x"]), Rows(t, d, pad, off, c["dy"]), Rows(t, d, pad, off)
        dw = [torch.full_like(c[k], SENTINEL) for k in ("wg", "wu", "wd")]
        op.backward(dy.t, x.t, c["wg"], c["wu"], c["wd"], saved, dx.t, *dw)
        assert op.status() == dm.OK
        near(dx.t, ref["dx"], "dx", mass["dx"])
        for got, name in zip(dw, ("dw_gate", "dw_up", "dw_down")):
            near(got, ref[name], name, mass[name])
        assert x.intact() and dy.intact() and dx.intact()


def test_ffn_gradient_matches_differences_of_the_forward_pass(dm):
    """Directional derivative of sum(dy * y) along a random direction of each input,
    from the library's own forward pass at two points.  The step is 1/8 of the input's
    size; y is rounded to bf16, so the difference carries noise of about
    u |y| sqrt(T D) against a signal of |gradient . direction|."""
    t, d, f = 128, 256, 512
    c = ffn_case(13, t, d, f)
    op = dm.GatedFFN(t, d, f)
    saved, y = op.empty_saved(t), torch.empty_like(c["x"])
    op.forward(c["x"], c["wg"], c["wu"], c["wd"], y, saved)
    dx = torch.empty_like(y)
    dw = [torch.empty_like(c[k]) for k in ("wg", "wu", "wd")]
    op.backward(c["dy"], c["x"], c["wg"], c["wu"], c["wd"], saved, dx, *dw)
    for name, grad in zip(("x", "wg", "wu", "wd"), (dx, *dw)):
        # along the gradient, scaled to 1/16 of the input: both ends representable closely
        g = grad.float()
        step = g * (c[name].float().norm() / g.norm() / 16)
        ends = []
        for sign in (1, -1):
            moved = {**c, name: (c[name].float() + sign * step).to(torch.bfloat16)}
            op.forward(moved["x"], moved["wg"], moved["wu"], moved["wd"], y, saved)
            ends.append((float((c["dy"].double() * y.double()).sum()), moved[name].double()))
        got = ends[0][0] - ends[1][0]
        want = float((grad.double() * (ends[0][1] - ends[1][1])).sum())
        # third-order terms: (1/16)^2 relative to the slope, with room for their constant
        noise = U * float(c["dy"].double().norm()) * float(y.double().norm()) / np.sqrt(t * d) * 4
        assert abs(got - want) <= 0.05 * abs(want) + noise, name


def test_ffn_nan_stays_in_its_token(dm):
    t, d, f = 70, 64, 96
    c = ffn_case(14, t, d, f)
    c["x"][5, 3] = float("nan")
    op = dm.GatedFFN(t, d, f, save=dm.SAVE_NONE)
    y = torch.empty_like(c["x"])
    op.forward(c["x"], c["wg"], c["wu"], c["wd"], y)
    bad = torch.isnan(y).any(dim=1)
    assert bad[5] and int(bad.sum()) == 1 and torch.isnan(y[5]).all()


def test_ffn_gradient_at_saturated_gates(dm):
    """Kept gates of any finite size: act' is 0 or 1 there, whatever its terms overflow to."""
    t, d, f = 40, 64, 96
    c = ffn_case(16, t, d, f)
    gate, up = Draw(17)((t, f)), Draw(18)((t, f))
    big = torch.tensor([40.0, 1e4, 1e13, 1e20, 3e38], device="cuda").to(torch.bfloat16)
    gate[::2, :5], gate[1::2, 5:10] = -big, -big       # act = act' = 0
    up[:, 10:15], gate[:, 10:15] = 0, big              # act' = 1, h = 0
    c["dy"][:] = c["dy"].abs()
    c["wd"][:, 10:15] = 0                               # and dup = dh act = 0
    for kind, n in ACTS.items():
        op = dm.GatedFFN(t, d, f, activation=n)
        ref = oracle.ffn_backward(np64(c["dy"]), np64(c["x"]), np64(c["wg"]), np64(c["wu"]),
                                  np64(c["wd"]), np64(gate), np64(up), kind)
        dx = torch.empty_like(c["x"])
        dw = [torch.empty_like(c[k]) for k in ("wg", "wu", "wd")]
        op.backward(c["dy"], c["x"], c["wg"], c["wu"], c["wd"], (gate, up), dx, *dw)
        assert op.status() == dm.OK
        a, da = oracle.act(kind, np64(gate))
        dh, ax = np64(c["dy"]) @ np64(c["wd"]), np.abs(np64(c["x"]))
        dg, du = np.abs(dh * np64(up) * da), np.abs(dh * a)
        near(dx, ref["dx"], kind, dg @ np.abs(np64(c["wg"])) + du @ np.abs(np64(c["wu"])))
        near(dw[0], ref["dw_gate"], kind, dg.T @ ax)
        near(dw[1], ref["dw_up"], kind, du.T @ ax)
        near(dw[2], ref["dw_down"], kind, np.abs(np64(c["dy"])).T @ np.abs(a * np64(up)))


def test_ffn_no_tokens(dm):
    op = dm.GatedFFN(4, 64, 96)
    c = ffn_case(15, 4, 64, 96)
    none = c["x"][:0]
    op.forward(none, c["wg"], c["wu"], c["wd"], none.clone(), op.empty_saved(0))
    dw = [torch.full_like(c[k], SENTINEL) for k in ("wg", "wu", "wd")]
    op.backward(none, none, c["wg"], c["wu"], c["wd"], op.empty_saved(0), none.clone(), *dw)
    assert op.status() == dm.OK and all(not w.any() for w in dw)


# ------------------------------------------------------------------ cross entropy
def xent_case(seed, t, d, v, scale=1.0):
    g = Draw(seed)
    w = g((v, d), 1.0 / np.sqrt(d))
    r = np.random.default_rng(seed)
    target = torch.from_numpy(r.integers(0, v, t)).cuda()
    h = g((t, d), scale)
    gl = torch.rand(t, generator=g.g, device="cuda") + 0.5
    return h, w, target, gl


def grad_mass(h, w, target, gl):
    """Sums of |G||W| and |G||h|, with what the exponentials' 16 bits add to G's
    rounding: 2^-11 relative and 2^-25 grad_loss absolute."""
    z = h @ w.T
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    live = (target >= 0) & (target < w.shape[0])
    p[np.arange(len(h))[live], target[live]] -= 1
    g = np.where(live, np.abs(gl), 0)[:, None] * (1.25 * np.abs(p) + 2.0 ** -16)
    return g @ np.abs(w), g.T @ np.abs(h)


def loss_bound(h, w, lse):
    prod = np.abs(h) @ np.abs(w).T
    return 2.0 ** -22 * prod.max(axis=1) * 2 + 2.0 ** -20 * (1 + np.abs(lse))


XENT_SHAPES = [(1, 8, 8), (1, 64, 1), (2, 100, 127), (17, 256, 128), (64, 129, 129), (65, 72, 1000),
               (255, 64, 256), (256, 520, 257), (257, 128, 3001), (40, 512, 20011),
               (33, 1500, 9000), (520, 1100, 4000)]


@pytest.mark.parametrize("t,d,v", XENT_SHAPES)
@pytest.mark.parametrize("grads", [False, True])
def test_xent(dm, t, d, v, grads):
    h, w, target, gl = xent_case(21, t, d, v, 2.0)
    if t > 2:
        target[1], target[2] = -100, v     # both outside [0, vocab)
    ref = oracle.xent(np64(h), np64(w), target.cpu().numpy(), np64(gl) if grads else None)
    bound = loss_bound(np64(h), np64(w), ref["lse"])
    mass = grad_mass(np64(h), np64(w), target.cpu().numpy(), np64(gl))
    op = dm.LinearXent(t + 5, d, v, grads=grads)
    for pad, off in ((0, 0), (8, 8), (3, 1)):
        hr, dh = Rows(t, d, pad, off, h), Rows(t, d, pad, off)
        loss, lse = (torch.full((t,), SENTINEL, device="cuda") for _ in range(2))
        if grads:
            dw = torch.full_like(w, SENTINEL)
            op.loss_and_grads(hr.t, w, target, gl, loss, lse, dh.t, dw)
        else:
            op.loss(hr.t, w, target, loss, lse)
        assert op.status() == dm.OK
        assert np.all(np.abs(np64(loss) - ref["loss"]) <= bound)
        assert np.all(np.abs(np64(lse) - ref["lse"]) <= bound)
        if grads and v > 1:                 # one entry: the gradient is exactly zero
            near(dh.t, ref["dhidden"], "dhidden", mass[0])
            near(dw, ref["dweight"], "dweight", mass[1])
        elif grads:
            assert not dh.t.any() and not dw.any()
        assert hr.intact() and dh.intact()


@pytest.mark.parametrize("t,d,v", [(64, 2048, 300), (160, 3592, 520), (300, 2056, 700),
                                   (350, 2600, 1000), (1000, 3400, 300)])
@pytest.mark.parametrize("grads", [False, True])
def test_xent_long_rows(dm, t, d, v, grads):
    """Rows long enough for the orientation with the vocabulary along the tile's rows, with
    one token tile and several, of 64 to 256 tokens."""
    test_xent(dm, t, d, v, grads)


def test_xent_masked_rows_leave_no_trace(dm):
    """NaN and infinities in masked rows: every other result as if they were not there."""
    t, d, v = 300, 128, 1500
    h, w, target, gl = xent_case(22, t, d, v)
    target[::3] = -1
    target[1::7] = v + 5
    live = (target >= 0) & (target < v)
    op = dm.LinearXent(t, d, v)
    outs = []
    for fill in (0.0, float("nan"), float("inf"), -3e38):
        hh = h.clone()
        hh[~live] = fill
        gg = gl.clone()
        gg[~live] = fill
        loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        op.loss_and_grads(hh, w, target, gg, loss, lse, dh, dw)
        assert op.status() == dm.OK
        assert not loss[~live].any() and not lse[~live].any() and not dh[~live].any()
        only = [torch.empty(t, device="cuda") for _ in range(2)]
        op.loss(hh, w, target, *only)
        assert torch.equal(only[0], loss) and torch.equal(only[1], lse)
        outs.append((loss, lse, dh, dw))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    target.fill_(-1)                        # no live token at all
    op.loss_and_grads(h, w, target, gl, loss, lse, dh, dw)
    assert not loss.any() and not lse.any() and not dh.any() and not dw.any()


def test_xent_wide_and_confident_logits(dm):
    """Logits hundreds apart: some tokens certain of their target, some of another."""
    t, d, v = 96, 64, 700
    h, w, target, gl = xent_case(23, t, d, v)
    hot = torch.where(torch.arange(t, device="cuda") % 2 == 0, target, (target + 1) % v)
    h = (h.float() * 0.1 + w[hot].float() * 300).to(torch.bfloat16)
    ref = oracle.xent(np64(h), np64(w), target.cpu().numpy(), np64(gl))
    op = dm.LinearXent(t, d, v)
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    op.loss_and_grads(h, w, target, gl, loss, lse, dh, dw)
    bound = loss_bound(np64(h), np64(w), ref["lse"])
    assert ref["loss"].max() > 100 and ref["loss"].min() < 1e-3
    assert np.all(np.abs(np64(loss) - ref["loss"]) <= bound)
    mass = grad_mass(np64(h), np64(w), target.cpu().numpy(), np64(gl))
    near(dh, ref["dhidden"], "dhidden", mass[0])
    near(dw, ref["dweight"], "dweight", mass[1])


def test_xent_nan_and_infinite_logits_stay_in_their_token(dm):
    t, d, v = 70, 64, 300
    h, w, target, gl = xent_case(24, t, d, v)
    h[3, 0] = float("nan")
    h[9, 0] = float("inf")
    op = dm.LinearXent(t, d, v, grads=False)
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    op.loss(h, w, target, loss, lse)
    bad = ~torch.isfinite(loss)
    assert bad[3] and bad[9] and int(bad.sum()) == 2


def test_xent_infinite_weight_of_one_token(dm):
    """An overflowed grad_loss reaches its own row of dhidden and every row of dweight
    that its token weighs in, no other row of dhidden."""
    t, d, v = 70, 64, 300
    h, w, target, gl = xent_case(27, t, d, v)
    op = dm.LinearXent(t, d, v)
    outs = []
    for bad in (0.0, float("inf"), float("nan")):
        gl[5] = bad
        loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        op.loss_and_grads(h, w, target, gl, loss, lse, dh, dw)
        assert op.status() == dm.OK
        outs.append((loss, lse, dh, dw))
    others = torch.arange(t, device="cuda") != 5
    assert not outs[0][2][5].any() and torch.isfinite(outs[0][3]).all()
    for loss, lse, dh, dw in outs[1:]:
        assert torch.equal(loss, outs[0][0]) and torch.equal(lse, outs[0][1])
        assert torch.equal(dh[others], outs[0][2][others])
        assert not torch.isfinite(dh[5]).any() and not torch.isfinite(dw).any()


def test_xent_in_several_pieces(dm):
    """A vocabulary so large that 300 tokens take two pieces (256 tokens at a time)."""
    t, d, v = 300, 8, 1 << 22
    h, w, target, gl = xent_case(25, t, d, v, 2.0)
    target[7] = -100
    op = dm.LinearXent(t, d, v)
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    op.loss_and_grads(h, w, target, gl, loss, lse, dh, dw)
    assert op.status() == dm.OK
    # the fp64 form on the GPU: 300 x 4M logits are too many for numpy here
    z = h.double() @ w.double().T
    norm = torch.logsumexp(z, 1)
    live = target >= 0
    at = target.clamp_min(0)
    want = torch.where(live, norm - z.gather(1, at[:, None])[:, 0], torch.zeros_like(norm))
    assert float((loss.double() - want).abs().max()) <= 2.0 ** -16
    z.sub_(norm[:, None]).exp_()
    z[torch.arange(t, device="cuda"), at] -= 1
    z *= torch.where(live, gl.double(), torch.zeros_like(norm))[:, None]
    g = 1.25 * z.abs() + 2.0 ** -16 * torch.where(live, gl.double(), torch.zeros_like(norm))[:, None]
    near(dh, np64(z @ w.double()), "dhidden", np64(g @ w.double().abs()))
    near(dw, np64(z.T @ h.double()), "dweight", np64(g.T @ h.double().abs()))


def test_xent_no_tokens(dm):
    h, w, target, gl = xent_case(26, 4, 64, 96)
    op = dm.LinearXent(4, 64, 96)
    e = torch.empty(0, device="cuda")
    op.loss(h[:0], w, target[:0], e, e.clone())
    dw = torch.full_like(w, SENTINEL)
    op.loss_and_grads(h[:0], w, target[:0], e, e.clone(), e.clone(), h[:0].clone(), dw)
    assert op.status() == dm.OK and not dw.any()


# ------------------------------------------------------------------ offsets past 32 bits
def test_act8_offsets_past_32_bits(dm):
    rows, cols = 70000, 65536                 # 4.6e9 elements
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-3:] = Draw(31)((3, cols))
    codes, scales = dm.act8_empty(rows, cols)
    dm.act8_save(x, codes, scales)
    small = dm.act8_empty(3, cols)
    dm.act8_save(x[-3:], *small)
    assert torch.equal(codes[-3:], small[0]) and torch.equal(scales[-3:], small[1])
    assert not codes[:-3].any() and not scales[:-3].any()
    want = torch.empty_like(x[-3:])
    dm.act8_load(*small, want)
    x.fill_(SENTINEL)
    dm.act8_load(codes, scales, x)
    assert torch.equal(x[-3:], want) and not x[:-3].any()
    del codes, scales
    # three rows of odd length, 2^32 elements and more between the first and the last
    wide = x.view(-1).as_strided((3, 2049), (2200000001, 1))
    wide.copy_(Draw(32)((3, 2049)))
    codes, scales = dm.act8_empty(3, 2049)
    dm.act8_save(wide, codes, scales)
    want_c, want_s = oracle.act8_codes(np64(wide))
    assert np.array_equal(np64(codes), want_c) and np.array_equal(np64(scales), want_s)
    wide.fill_(SENTINEL)
    dm.act8_load(codes, scales, wide)
    back = oracle.act8_values(want_c, want_s)
    assert np.all(np.abs(np64(wide) - back) <= U * np.abs(back))


@pytest.mark.parametrize("save", [1, 2])
@pytest.mark.parametrize("f", [18944, 18949])
def test_ffn_offsets_past_32_bits(dm, save, f):
    """More than 2^31 kept elements, 2^32 bytes of each: only the last tokens weigh."""
    t, d, n = 120000, 64, 300
    c = ffn_case(33, n, d, f)
    op = dm.GatedFFN(t, d, f, save=save)
    x, dy = (torch.zeros((t, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-n:], dy[-n:] = c["x"], c["dy"]
    y, saved = torch.empty_like(x), op.empty_saved(t)
    op.forward(x, c["wg"], c["wu"], c["wd"], y, saved)
    assert op.status() == dm.OK and not y[:-n].any()
    fwd = oracle.ffn_forward(np64(c["x"]), np64(c["wg"]), np64(c["wu"]), np64(c["wd"]))
    near(y[-n:], fwd["y"], "y", np.abs(fwd["h"]) @ np.abs(np64(c["wd"])).T)
    last = tuple(s[-n:] for s in saved)
    check_kept(dm, op, last, fwd, c, f)
    gate, up = kept_values(op, dm, last, n)
    ref = oracle.ffn_backward(np64(c["dy"]), np64(c["x"]), np64(c["wg"]), np64(c["wu"]),
                              np64(c["wd"]), gate, up)
    dw = [torch.empty_like(c[k]) for k in ("wg", "wu", "wd")]
    op.backward(dy, x, c["wg"], c["wu"], c["wd"], saved, y, *dw)
    assert op.status() == dm.OK and not y[:-n].any()
    a, da = oracle.act("silu", gate)
    dh, ax = np64(c["dy"]) @ np64(c["wd"]), np.abs(np64(c["x"]))
    dg, du = np.abs(dh * up * da), np.abs(dh * a)
    near(y[-n:], ref["dx"], "dx", dg @ np.abs(np64(c["wg"])) + du @ np.abs(np64(c["wu"])))
    near(dw[0], ref["dw_gate"], "dw_gate", dg.T @ ax)
    near(dw[1], ref["dw_up"], "dw_up", du.T @ ax)
    near(dw[2], ref["dw_down"], "dw_down", np.abs(np64(c["dy"])).T @ np.abs(a * up))


@pytest.mark.parametrize("t", [40, 300])
@pytest.mark.parametrize("d", [1032, 1033])
def test_xent_offsets_past_32_bits(dm, t, d):
    """A head of 4.3e9 elements, zero but for its last rows, which hold the targets;
    300 tokens take two pieces."""
    v, n = 1 << 22, 500
    h, tail, target, gl = xent_case(34, t, d, n, 2.0)
    tail = (tail.float() * 4).to(torch.bfloat16)
    w = torch.zeros((v, d), dtype=torch.bfloat16, device="cuda")
    w[-n:] = tail
    op = dm.LinearXent(t, d, v)
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    op.loss_and_grads(h, w, target + (v - n), gl, loss, lse, dh, dw)
    assert op.status() == dm.OK
    hd, wd, gd = np64(h), np64(tail), np64(gl)
    z = hd @ wd.T
    norm = np.log(np.exp(z).sum(1) + (v - n))
    at = np.arange(t), target.cpu().numpy()
    bound = loss_bound(hd, wd, norm)
    assert np.all(np.abs(np64(lse) - norm) <= bound)
    assert np.all(np.abs(np64(loss) - (norm - z[at])) <= bound)
    p = np.exp(z - norm[:, None])
    p[at] -= 1
    g = gd[:, None] * p
    # what the roundings leave is in grad_mass: 1.25 |G| and 2^-16 grad_loss of each entry
    room = gd[:, None] * (1.25 * np.abs(p) + 2.0 ** -16)
    near(dh, g @ wd, "dhidden", room @ np.abs(wd))
    near(dw[-n:], g.T @ hd, "dweight", room.T @ np.abs(hd))
    rest = (gd * np.exp(-norm)) @ hd           # the same for every zero row
    first = np64(dw[0])
    assert np.all(np.abs(first - rest) <= 1.01 * U * np.abs(rest)
                  + U * ((gd * np.exp(-norm) * 1.25 + gd * 2.0 ** -25) @ np.abs(hd)))
    # all the same, but for those whose exponentials are taken relative to a tail row
    same = (v - n) // 256 * 256
    for lo in range(0, same, 1 << 19):
        assert (dw[lo:min(lo + (1 << 19), same)] == dw[0]).all()


# ------------------------------------------------------------------ streams, graphs, repeats
def test_results_repeat_bit_for_bit_on_another_stream_and_in_a_graph(dm):
    t, d, f, v = 333, 256, 520, 2000
    c = ffn_case(31, t, d, f)
    h, w, target, gl = xent_case(32, t, d, v)
    ffn, head = dm.GatedFFN(t, d, f, save=dm.SAVE_ACT8), dm.LinearXent(t, d, v)

    def outputs():
        return dict(y=torch.zeros_like(c["x"]), saved=ffn.empty_saved(t), dx=torch.zeros_like(c["x"]),
                    dw=[torch.zeros_like(c[k]) for k in ("wg", "wu", "wd")],
                    loss=torch.zeros(t, device="cuda"), lse=torch.zeros(t, device="cuda"),
                    dh=torch.zeros_like(h), dhead=torch.zeros_like(w))

    def step(o):
        ffn.forward(c["x"], c["wg"], c["wu"], c["wd"], o["y"], o["saved"])
        ffn.backward(c["dy"], c["x"], c["wg"], c["wu"], c["wd"], o["saved"], o["dx"], *o["dw"])
        head.loss_and_grads(h, w, target, gl, o["loss"], o["lse"], o["dh"], o["dhead"])

    def flat(o):
        return [o["y"], *o["saved"], o["dx"], *o["dw"], o["loss"], o["lse"], o["dh"], o["dhead"]]

    first = outputs()
    step(first)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = outputs()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(again)
    side.synchronize()
    graphed = outputs()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(graphed)
    g.replay()
    torch.cuda.synchronize()
    for o in (again, graphed):
        for a, b in zip(flat(o), flat(first)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert ffn.status() == dm.OK and head.status() == dm.OK
