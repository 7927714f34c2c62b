"""GPU tests of the training-side operators where a wrong result hides behind a large norm:
losses near zero against their own size, entries far below their neighbours, logits at
minus infinity, gates where the normal CDF is small, sums over millions of elements.
Their fp64 forms are in oracle/training_oracle.py; u = 2^-8 is bf16's unit roundoff."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


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


def normal(seed, shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dtype)


def run_xent(dm, h, w, target, gl=None):
    t = h.shape[0]
    op = dm.LinearXent(t, h.shape[1], w.shape[0], grads=gl is not None)
    out = dict(loss=torch.full((t,), 7.0, device="cuda"), lse=torch.full((t,), 7.0, device="cuda"))
    if gl is None:
        op.loss(h, w, target, out["loss"], out["lse"])
    else:
        out.update(dhidden=torch.full_like(h, 7.0), dweight=torch.full_like(w, 7.0))
        op.loss_and_grads(h, w, target, gl, out["loss"], out["lse"], out["dhidden"], out["dweight"])
    assert op.status() == dm.OK
    return out


def xent64(h, w, target):
    """loss, lse and softmax minus one-hot without cancellation, in 64 bits."""
    z = h @ w.T
    at = np.arange(len(h)), target
    zt = z[at].copy()
    z[at] = -np.inf
    top = z.max(1)
    others = np.log(np.exp(z - top[:, None]).sum(1)) + top
    loss = np.logaddexp(0, others - zt)
    loss = np.where(others < zt, np.log1p(np.exp(np.minimum(others - zt, 0))), loss)
    g = np.exp(z - (zt + loss)[:, None])
    g[at] = np.expm1(-loss)
    return loss, zt + loss, g


# ------------------------------------------------------------------ logits at minus infinity
@pytest.mark.parametrize("t,d", [(5, 64), (300, 64), (300, 2048)])
@pytest.mark.parametrize("v,gone", [(700, (128, 384)), (700, (32, 64)), (515, (512, 515)), (130, (0, 128))])
def test_xent_entries_at_minus_infinity_weigh_nothing(dm, t, d, v, gone):
    """Whole groups of neighbouring entries (the last, shorter one too) whose logits fall
    below fp32's range: every result as if their rows were not there, in both orientations."""
    h, w = normal(41, (t, d)), normal(42, (v, d), d ** -0.5)
    h[:, 0] = 8.0
    w[gone[0]:gone[1]] = 0
    w[gone[0]:gone[1], 0] = -3e38                  # 8 * -3e38: the product is below fp32's range
    rest = [i for i in range(v) if not gone[0] <= i < gone[1]]
    r = np.random.default_rng(43)
    at = r.integers(0, len(rest), t)
    target = torch.tensor(np.asarray(rest)[at], device="cuda")
    gl = torch.full((t,), 1.0 / t, device="cuda")
    ref = oracle.xent(np64(h), np64(w)[rest], at, np64(gl))
    # the bounds of test_gpu_training.py: fp32 losses, gradients with one operand rounded
    hd, wd = np64(h), np64(w)[rest]
    bound = 2.0 ** -21 * (np.abs(hd) @ np.abs(wd).T).max(1) + 2.0 ** -20 * (1 + np.abs(ref["lse"]))
    for grads in (None, gl):
        out = run_xent(dm, h, w, target, grads)
        assert np.all(np.abs(np64(out["loss"]) - ref["loss"]) <= bound)
        assert np.all(np.abs(np64(out["lse"]) - ref["lse"]) <= bound)
    assert not out["dweight"][gone[0]:gone[1]].any()
    for got, want in ((out["dhidden"], ref["dhidden"]), (out["dweight"][rest], ref["dweight"])):
        assert np.linalg.norm(np64(got) - want) <= 2 * U * np.linalg.norm(want)


# ------------------------------------------------------------------ entries far below their group
@pytest.mark.parametrize("t", [40, 300])
@pytest.mark.parametrize("v", [31, 120, 300])
def test_xent_gradient_of_entries_far_below_their_neighbours(dm, t, v):
    """Neighbouring entries whose logits spread over 20: each row of dweight against its own
    size (the exponentials keep 11 bits down to e^-20 of their group's largest)."""
    d = 64
    w = torch.zeros((v, d), dtype=torch.bfloat16, device="cuda")
    w[:, 0] = -(torch.arange(v, device="cuda") * 7 % 31).to(torch.bfloat16) * (19.5 / 30)
    w[:, 1] = normal(61, (v,), 0.01)
    h = normal(62, (t, d))
    h[:, 0] = 1.0
    target = torch.full((t,), 5, dtype=torch.int64, device="cuda")
    hd, wd, tg = np64(h), np64(w), target.cpu().numpy()
    g = xent64(hd, wd, tg)[2]
    out = run_xent(dm, h, w, target, torch.ones(t, device="cuda"))
    err = np.abs(np64(out["dweight"]) - g.T @ hd)
    assert np.all(err <= U * np.abs(g.T @ hd) + 1.25 * U * (np.abs(g).T @ np.abs(hd)))


# ------------------------------------------------------------------ sure tokens
def sure_case(seed, t, d, v, lo=1e-5, hi=1e-1):
    """Tokens whose loss runs from `hi` down to `lo`: the hidden state is pulled towards the
    target's row until that logit is as far above all others together."""
    h, w = normal(seed, (t, d)).double(), normal(seed + 1, (v, d), d ** -0.5)
    wd = w.double()
    r = np.random.default_rng(seed)
    target = torch.from_numpy(r.integers(0, v, t)).cuda()
    rows = wd[target]
    rows = rows / rows.square().sum(1, keepdim=True)
    want = torch.logspace(np.log10(hi), np.log10(lo), t, device="cuda", dtype=torch.float64)
    if t == 1:
        want = torch.tensor([1e-3], device="cuda", dtype=torch.float64)
    at = torch.arange(t, device="cuda")
    for _ in range(20):                            # others move a little with the pull
        z = h @ wd.T
        zt = z[at, target].clone()
        z[at, target] = -float("inf")
        h = h + rows * (torch.logsumexp(z, 1) - zt - torch.log(torch.expm1(want)))[:, None]
    return h.to(torch.bfloat16), w, target


SURE = [(1, 64, 300), (1, 4096, 5000), (3, 1024, 40), (40, 4096, 300), (64, 512, 129), (300, 64, 5000),
        (300, 2048, 700), (300, 4096, 260), (600, 1000, 2000)]


@pytest.mark.parametrize("t,d,v", SURE)
@pytest.mark.parametrize("seed", [51, 52])
def test_xent_of_sure_tokens_relative_to_the_loss(dm, t, d, v, seed):
    """loss = log(1 + sum of exp(z_v - z_target)), so its relative error is that of the
    exponentials: 2e-6 for their arithmetic and the difference's rounding, and 2^-22 of their
    terms' sizes for the other entries' logits.  Nothing is granted for the target's own
    logit, a sum of one sign of 5 to 25, nor for the sum that 1 is added to."""
    h, w, target = sure_case(seed, t, d, v)
    hd, wd, tg = np64(h), np64(w), target.cpu().numpy()
    loss, lse, g = xent64(hd, wd, tg)
    assert loss.max() < 0.2 and loss.min() > 5e-6
    others = np.abs(hd) @ np.abs(wd).T
    others[np.arange(t), tg] = 0
    rel = 2e-6 + 2.0 ** -22 * others.max(1)
    gl = torch.full((t,), 1.0 / t, device="cuda")
    for grads in (None, gl):
        out = run_xent(dm, h, w, target, grads)
        err = np.abs(np64(out["loss"]) - loss)
        assert np.all(err <= rel * loss), (err / loss).max()
        assert np.all(np.abs(np64(out["lse"]) - lse) <= 3e-7 * np.abs(lse))
    # gradients, element by element: G's entries and the outputs are rounded once each
    g /= t
    for got, want, mass in ((out["dhidden"], g @ wd, np.abs(g) @ np.abs(wd)),
                            (out["dweight"], g.T @ hd, np.abs(g).T @ np.abs(hd))):
        assert np.all(np.abs(np64(got) - want) <= U * np.abs(want) + 1.25 * U * mass)


def test_xent_gradient_rows_of_sure_tokens_balance(dm):
    """Two entries, 10 to 20 apart: G is (-p, p) with p = exp(-gap) whatever the gap."""
    t, d = 40, 64
    w = torch.zeros((2, d), dtype=torch.bfloat16, device="cuda")
    w[0, 0] = 1.0
    w[1, 1] = 1.0
    h = torch.zeros((t, d), dtype=torch.bfloat16, device="cuda")
    gap = torch.linspace(10, 20, t, device="cuda").to(torch.bfloat16)
    h[:, 0] = gap
    target = torch.zeros(t, dtype=torch.int64, device="cuda")
    out = run_xent(dm, h, w, target, torch.ones(t, device="cuda"))
    p = 1 / (1 + np.exp(np64(gap)))
    assert np.all(np.abs(np64(out["loss"]) + np.log1p(-p)) <= 1e-6 * p)
    for col, sign in ((0, -1), (1, 1)):
        assert np.all(np.abs(np64(out["dhidden"])[:, col] - sign * p) <= 2 * U * p)


# ------------------------------------------------------------------ small values of the normal CDF
GATES = [-0.5, -1.0, -2.0, -3.0, -4.0, -4.75, -5.0, -5.5, -5.75, -6.0, -7.0, -8.0, -9.0, -10.0, 0.25, 3.0, 6.0]


def gelu64(g):
    """x Phi(x) and its derivative without cancellation (Phi through erfc)."""
    import math
    phi = np.array([0.5 * math.erfc(-x / math.sqrt(2)) for x in g])
    return g * phi, phi + g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


@pytest.mark.parametrize("t", [1, 9, 40, 300])
def test_gelu_of_negative_gates_relative_to_its_size(dm, t):
    """Every product of the block is with one row of an identity, so y is act(gate) rounded
    twice (h, y), dw_gate's first column act'(gate) and dw_up's act(gate) likewise."""
    gates = torch.tensor(GATES, device="cuda").to(torch.bfloat16)
    n = len(GATES)
    d = f = 64
    eye = torch.eye(d, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((t, d), dtype=torch.bfloat16, device="cuda")
    x[0, :n], x[0, 63] = gates, 1.0
    w_up = torch.zeros((f, d), dtype=torch.bfloat16, device="cuda")
    w_up[:, 63] = 1.0                                              # up = 1
    op = dm.GatedFFN(t, d, f, activation=dm.ACT_GELU)
    saved, y = op.empty_saved(t), torch.empty_like(x)
    op.forward(x, eye, w_up, eye, y, saved)
    a, da = gelu64(np64(gates))
    assert np.all(np.abs(np64(y[0, :n]) - a) <= 1.01 * U * np.abs(a))
    # the gradients of one live token, whose x and dy are the first unit vector
    x.zero_()
    x[0, 0] = 1.0
    dy = x.clone()
    w_down = torch.zeros((d, f), dtype=torch.bfloat16, device="cuda")
    w_down[0] = 1.0                                                # dh = 1
    gate, up = torch.zeros((t, f), dtype=torch.bfloat16, device="cuda"), torch.ones(
        (t, f), dtype=torch.bfloat16, device="cuda")
    gate[0, :n] = gates
    dx, dw = torch.empty_like(x), [torch.empty_like(eye) for _ in range(3)]
    op.backward(dy, x, eye, w_up, w_down, (gate, up), dx, *dw)
    assert op.status() == dm.OK
    # act' crosses zero near -0.75: there two terms of half its size each cancel
    assert np.all(np.abs(np64(dw[0][:n, 0]) - da) <= 1.01 * U * np.abs(da) + 1e-6 * np.exp(-0.5 * np64(gates) ** 2))
    assert np.all(np.abs(np64(dw[1][:n, 0]) - a) <= 1.01 * U * np.abs(a))
    assert np.all(np.abs(np64(dw[2][0, :n]) - a) <= 1.01 * U * np.abs(a))


# ------------------------------------------------------------------ sums over millions of elements
# The accumulator truncates, a bias that no averaging removes.  Allowed of it: 2^-11 of the
# terms' sizes, here at most twice the result's.  The operands' roundings average out over
# millions; the output's is at most u / sqrt(3) as a relative norm.  0.58 u + 0.25 u < u.
LONG = U


def far(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("t", [20, 256, 300])
@pytest.mark.parametrize("d", [64, 72, 33])
def test_xent_hidden_gradient_over_millions_of_entries(dm, t, d):
    """A vocabulary at the limit, weights of one sign: dhidden is a sum of four million terms
    (300 tokens: in two pieces)."""
    v = 1 << 22
    h, w = normal(71, (t, d), 0.1), normal(72, (v, d)).abs_()
    target = torch.arange(t, device="cuda") * 13001
    gl = torch.ones(t, device="cuda")
    out = run_xent(dm, h, w, target, gl)
    want = torch.empty((t, d), dtype=torch.float64, device="cuda")
    for lo in range(0, t, 64):
        z = h[lo:lo + 64].double() @ w.double().T
        z = torch.softmax(z, 1)
        z[torch.arange(len(z), device="cuda"), target[lo:lo + 64]] -= 1
        want[lo:lo + 64] = z @ w.double()
        del z
    assert far(out["dhidden"], want) <= LONG


@pytest.mark.parametrize("d,f", [(64, 64), (40, 33)])
def test_ffn_weight_gradients_over_millions_of_tokens(dm, d, f):
    """All tokens at the limit of four million, every term of the sums positive."""
    t = 1 << 22
    x, dy = normal(73, (t, d)).abs_(), normal(74, (t, d)).abs_()
    wg, wu, wd = (normal(75 + i, s, 0.1).abs_() for i, s in enumerate([(f, d), (f, d), (d, f)]))
    gate, up = normal(78, (t, f)).abs_(), normal(79, (t, f)).abs_()
    op = dm.GatedFFN(t, d, f)
    dx, dw = torch.empty_like(x), [torch.empty_like(w) for w in (wg, wu, wd)]
    op.backward(dy, x, wg, wu, wd, (gate, up), dx, *dw)
    assert op.status() == dm.OK
    want = [torch.zeros(w.shape, dtype=torch.float64, device="cuda") for w in (wg, wu, wd)]
    for lo in range(0, t, 1 << 18):
        s = slice(lo, lo + (1 << 18))
        g, u, y, xs = gate[s].double(), up[s].double(), dy[s].double(), x[s].double()
        sg = torch.sigmoid(g)
        dh = y @ wd.double()
        want[0] += (dh * u * (sg + g * sg * (1 - sg))).T @ xs
        want[1] += (dh * g * sg).T @ xs
        want[2] += y.T @ (g * sg * u)
    for got, ref in zip(dw, want):
        assert far(got, ref) <= LONG


def test_xent_weight_gradient_over_millions_of_tokens(dm):
    """A small vocabulary and four million tokens, hidden states of one sign; the rows that are
    no token's target are sums of one sign."""
    t, d, v = 1 << 22, 64, 40
    h, w = normal(81, (t, d)).abs_(), normal(82, (v, d), 0.05)
    target = torch.zeros(t, dtype=torch.int64, device="cuda")
    out = run_xent(dm, h, w, target, torch.full((t,), 2.0 ** -22, device="cuda"))
    want = torch.zeros((v, d), dtype=torch.float64, device="cuda")
    for lo in range(0, t, 1 << 18):
        hs = h[lo:lo + (1 << 18)].double()
        p = torch.softmax(hs @ w.double().T, 1)
        p[:, 0] -= 1
        want += p.T @ hs * 2.0 ** -22
    assert far(out["dweight"], want) <= LONG
    assert far(out["dweight"][1:], want[1:]) <= LONG


def kinds(shape, seed):
    """A positive matrix whose rows repeat four random ones, and these in 64 bits."""
    four = normal(seed, (4, shape[1])).abs_()
    return four.expand(shape[0] // 4, 4, shape[1]).reshape(shape), four.double()


def bias(got, want):
    """Mean relative error: roundings to bf16, 2^-8 / sqrt(3) each, average out over the
    thousands of elements of a row; what truncation takes does not."""
    return abs(float(((got.double() - want) / want).mean()))


# 2^-11 for the truncation (above), and four times what the roundings leave
BIAS = 2.0 ** -11 + 1e-4


def test_xent_hidden_gradient_of_full_tiles_is_not_biased(dm):
    """A million entries, hidden states and tiles so many that each sums all of them: with
    hidden states of zero every entry weighs 2^-20, exactly."""
    t, d, v = 1024, 5120, 1 << 20
    w, four = kinds((v, d), 83)
    w[0] = 0
    target = torch.zeros(t, dtype=torch.int64, device="cuda")
    out = run_xent(dm, torch.zeros((t, d), dtype=torch.bfloat16, device="cuda"), w, target,
                   torch.ones(t, device="cuda"))
    assert bias(out["dhidden"], (four.sum(0) * (v // 4) - four[0]) / v) <= BIAS


def test_xent_weight_gradient_of_full_tiles_is_not_biased(dm):
    t, d, v = 1 << 20, 5120, 1024
    h, four = kinds((t, d), 84)
    target = torch.zeros(t, dtype=torch.int64, device="cuda")
    out = run_xent(dm, h, torch.zeros((v, d), dtype=torch.bfloat16, device="cuda"), target,
                   torch.full((t,), 2.0 ** -20, device="cuda"))
    assert bias(out["dweight"][1:], four.mean(0) / v) <= BIAS


def test_ffn_weight_gradients_of_full_tiles_are_not_biased(dm):
    t, d, f = 1 << 20, 1024, 1792
    (x, x4), (dy, dy4), (gate, g4), (up, u4) = (kinds((t, n), 85 + i) for i, n in enumerate((d, d, f, f)))
    wg, wu, wd = (normal(89 + i, s, 0.1).abs_() for i, s in enumerate([(f, d), (f, d), (d, f)]))
    op = dm.GatedFFN(t, d, f)
    dx, dw = torch.empty_like(x), [torch.empty_like(w) for w in (wg, wu, wd)]
    op.backward(dy, x, wg, wu, wd, (gate, up), dx, *dw)
    assert op.status() == dm.OK
    sg, dh = torch.sigmoid(g4), dy4 @ wd.double()
    a = g4 * sg
    for got, left, right in zip(dw, (dh * u4 * (sg + a * (1 - sg)), dh * a, dy4), (x4, x4, a * u4)):
        assert bias(got, left.T @ right * (t // 4)) <= BIAS


# ------------------------------------------------------------------ results in place
@pytest.mark.parametrize("t,d,f", [(1, 64, 96), (3, 65, 96), (40, 64, 96), (300, 136, 264), (600, 64, 96)])
def test_forward_and_hidden_gradient_in_place(dm, t, d, f):
    """y may be x, dhidden may be hidden: the same bits as into tensors of their own."""
    x = normal(98, (t, d))
    ws = [normal(99 + i, s, s[1] ** -0.5) for i, s in enumerate([(f, d), (f, d), (d, f)])]
    op = dm.GatedFFN(t, d, f, save=dm.SAVE_NONE)
    y, place = torch.empty_like(x), x.clone()
    op.forward(x, *ws, y)
    op.forward(place, *ws, place)
    assert torch.equal(y, place)
    head, target, gl = normal(103, (500, d)), torch.arange(t, device="cuda") % 500, torch.ones(t, device="cuda")
    want = run_xent(dm, x, head, target, gl)
    place = x.clone()
    op = dm.LinearXent(t, d, 500)
    loss, lse, dw = torch.empty(t, device="cuda"), torch.empty(t, device="cuda"), torch.empty_like(head)
    op.loss_and_grads(place, head, target, gl, loss, lse, place, dw)
    assert op.status() == dm.OK
    assert torch.equal(place, want["dhidden"]) and torch.equal(dw, want["dweight"])


# ------------------------------------------------------------------ the orientations' ranges
@pytest.mark.parametrize("t", [1030, 1100, 1290, 1344, 1345, 1540, 1568, 1569])
def test_ffn_with_five_to_seven_token_tiles(dm, t):
    """Products with the weight's rows as the tile's rows run up to 1568 tokens; sizes on both
    sides of where the orientation changes, forward and backward."""
    d, f = 200, 392
    x, dy = normal(91, (t, d)), normal(92, (t, d), 1e-2)
    wg, wu, wd = (normal(93 + i, s, s[1] ** -0.5) for i, s in enumerate([(f, d), (f, d), (d, f)]))
    for save in (dm.SAVE_BF16, dm.SAVE_ACT8):
        op = dm.GatedFFN(t, d, f, save=save)
        saved, y = op.empty_saved(t), torch.full_like(x, 7.0)
        op.forward(x, wg, wu, wd, y, saved)
        dx, dw = torch.full_like(x, 7.0), [torch.full_like(w, 7.0) for w in (wg, wu, wd)]
        op.backward(dy, x, wg, wu, wd, saved, dx, *dw)
        assert op.status() == dm.OK
        fwd = oracle.ffn_forward(np64(x), np64(wg), np64(wu), np64(wd))
        if save == dm.SAVE_BF16:
            gate, up = np64(saved[0]), np64(saved[1])
        else:
            gate, up = (oracle.act8_values(np64(saved[i]), np64(saved[i + 1])) for i in (0, 2))
        ref = oracle.ffn_backward(np64(dy), np64(x), np64(wg), np64(wu), np64(wd), gate, up)
        a, da = oracle.act("silu", gate)
        dh, ax = np64(dy) @ np64(wd), np.abs(np64(x))
        dg, du = np.abs(dh * up * da), np.abs(dh * a)
        for got, want, mass in (
                (y, fwd["y"], np.abs(fwd["h"]) @ np.abs(np64(wd)).T),
                (dx, ref["dx"], dg @ np.abs(np64(wg)) + du @ np.abs(np64(wu))),
                (dw[0], ref["dw_gate"], dg.T @ ax), (dw[1], ref["dw_up"], du.T @ ax),
                (dw[2], ref["dw_down"], np.abs(np64(dy)).T @ np.abs(a * up))):
            err = np.abs(np64(got) - want)
            assert np.all(err <= U * np.abs(want) + 1.01 * U * mass)


@pytest.mark.parametrize("t", [1030, 1100, 1290, 1568, 1569])
def test_xent_gradients_with_five_to_seven_token_tiles(dm, t):
    d, v = 136, 900
    h, w = normal(95, (t, d), 2.0), normal(96, (v, d), d ** -0.5)
    target = torch.from_numpy(np.random.default_rng(97).integers(0, v, t)).cuda()
    hd, wd, tg = np64(h), np64(w), target.cpu().numpy()
    loss, lse, g = xent64(hd, wd, tg)
    out = run_xent(dm, h, w, target, torch.ones(t, device="cuda"))
    bound = 2.0 ** -21 * (np.abs(hd) @ np.abs(wd).T).max(1) + 2.0 ** -20 * (1 + np.abs(lse))
    assert np.all(np.abs(np64(out["loss"]) - loss) <= bound)
    assert np.all(np.abs(np64(out["lse"]) - lse) <= bound)
    for got, want, mass in ((out["dhidden"], g @ wd, np.abs(g) @ np.abs(wd)),
                            (out["dweight"], g.T @ hd, np.abs(g).T @ np.abs(hd))):
        assert np.all(np.abs(np64(got) - want) <= U * np.abs(want) + 1.26 * U * mass)
