"""GPU parity of the operators that mix tokens (norms and rotation of query and key heads, linear
attention with a decay for each head, their gradients, the step of single tokens) against their
fp64 forms, at the sizes, strides, sequences and decays where they can go wrong.

Tolerances.  u = 2^-8 is bf16's half step relative to the value.
Norm and rotation: computed in fp32 and rounded once.  rsqrt, sine and cosine are within 2^-21,
a handful of fp32 operations adds 2^-22 each: |error| <= u |value| + 2^-19 (|a| + |b|), a and b
the pair before the turn.  The gains' gradients add at most 2^14 terms one after another in any
lane: u |value| + 2^-10 sum |terms| at worst, 2^-14 of it for the sizes here (fewer than 1024 one
after another).
Linear attention: the weighted scores, the entering state and the decayed keys are rounded to bf16
once, the output once.  Element by element
  |error| <= u |value| + 2.1 u mass,   mass = scale sum_s a^(t-s) (|q_t| . |k_s|) |v_s| + |q| |S|
(the state's share has two roundings, the scores' one; 0.1: second order and accumulation); of
independent roundings the relative Frobenius error is about sqrt(4) u 0.43, at most 2 u.
States: keys keep 16 bits, half a step of each of two roundings, 2^-16 of every term; products of a
block are truncated to 2^-20 of their sum, blocks add in fp32: 1.25 * 2^-16 mass.
Single tokens: fp32 throughout, d products one after another: state 2^-22, output u |value| +
2^-17 mass."""
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
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def __call__(self, shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(shape, generator=self.g, device="cuda").mul_(std).to(dtype)


SENTINEL = 7.0


class Place:
    """A (tokens, heads, dim) tensor inside a buffer of sentinels.  "rows": token after token,
    packed beside `others` more dims; "heads": head after head; "mixed": the heads' slices of
    several tensors interleaved.  `off` elements in."""

    def __init__(self, tokens, heads, dim, layout="rows", off=0, pad=0, fill=None):
        if layout == "rows":
            ts, hs = heads * dim + pad, dim
        elif layout == "heads":
            ts, hs = dim + pad, tokens * (dim + pad) + pad
        else:
            ts, hs = heads * (3 * dim + pad) + pad, 3 * dim + pad
        size = off + (max(tokens, 1) - 1) * ts + (heads - 1) * hs + dim + 8
        self.buf = torch.full((size,), SENTINEL, dtype=torch.bfloat16, device="cuda")
        self.at = ((tokens, heads, dim), (ts, hs, 1), off)
        self.t = self.buf.as_strided(*self.at)
        if fill is not None:
            self.t.copy_(fill)

    def intact(self):
        seen = self.buf.clone()
        seen.as_strided(*self.at).fill_(SENTINEL)
        return bool((seen == SENTINEL).all())


LAYOUTS = [("rows", 0, 0), ("rows", 8, 64), ("heads", 16, 8), ("mixed", 8, 0)]


def no_worse(got, ref, bound, what):
    got = np64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, what
    assert np.all(np.isfinite(got)), what
    over = np.abs(got - ref) - bound
    assert np.all(over <= 0), (what, float(over.max()), np.unravel_index(over.argmax(), over.shape))


# ------------------------------------------------------------------ norms and rotation
def rope_reference(dim, rotary, base=10000.0):
    i = torch.arange(rotary // 2, device="cuda", dtype=torch.float64)
    return (base ** (-2 * i / max(1, rotary))).float()


def rope_bound(x, w, eps, y):
    """u |y| + 2^-19 of the pair's magnitudes (at most sqrt(2) the largest of a head)."""
    n = np.abs(x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * w)
    return U * np.abs(y) + 2.0 ** -18 * n.max(axis=-1, keepdims=True)


ROPE = [(1, 32, 8, 128, 128), (3, 1, 1, 8, 8), (5, 3, 2, 64, 32), (70, 12, 2, 128, 64),
        (33, 5, 5, 96, 96), (9, 7, 3, 256, 256), (300, 28, 4, 80, 0), (2, 4, 0, 128, 128),
        (2100, 3, 1, 40, 24), (17, 40, 40, 16, 8)]


@pytest.mark.parametrize("tokens,hq,hk,dim,rotary", ROPE)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("layout,off,pad", LAYOUTS + [("rows", 3, 5), ("heads", 4, 4)])
def test_norm_rope_both_ways(dm, tokens, hq, hk, dim, rotary, interleaved, layout, off, pad):
    """Forward and gradients, aligned or not, gains or none."""
    d, eps = Draw(tokens + dim), 1e-5
    f = rope_reference(dim, rotary)
    pos = torch.randint(-50, 200000, (tokens,), generator=d.g, device="cuda", dtype=torch.int32)
    op = dm.QKNormRope(tokens + 2, hq, hk, dim, rotary, eps=eps, interleaved=interleaved)
    place = lambda h, std=None: None if h == 0 else Place(
        tokens, h, dim, layout, off, pad, None if std is None else d((tokens, h, dim), std))
    tens = lambda p: None if p is None else p.t
    x = [place(hq, 1.7), place(hk, 0.01)]
    w = [d((dim,), 0.5), None if tokens == 5 else d((dim,), 2.0)]
    out = [place(hq), place(hk)]
    op.forward(*map(tens, x), *w, f, pos, *map(tens, out))
    g = [place(hq, 1.0), place(hk, 1e-3)]
    dx = [place(hq), place(hk)]
    dw = [torch.full((dim,), SENTINEL, dtype=torch.bfloat16, device="cuda") for _ in w]
    if w[1] is None or hk == 0:
        dw[1] = None
    op.backward(*map(tens, g), *map(tens, x), *w, f, pos, *map(tens, dx), *dw)
    for i in range(2):
        if x[i] is None:
            continue
        xn, wn = np64(x[i].t), np64(w[i]) if w[i] is not None else np.ones(dim)
        y = oracle.norm_rope(xn, wn, np64(f), np64(pos), eps, interleaved)
        no_worse(out[i].t, y, rope_bound(xn, wn, eps, y), f"out {i}")
        gn = np64(g[i].t)
        want, want_w = oracle.norm_rope_backward(gn, xn, wn, np64(f), np64(pos), eps, interleaved)
        r = 1 / np.sqrt(np.mean(xn * xn, axis=-1, keepdims=True) + eps)
        n, top = np.abs(xn * r), np.abs(gn).max(axis=-1, keepdims=True) * np.sqrt(2)
        most = np.abs(wn).max()
        no_worse(dx[i].t, want, U * np.abs(want) + 2.0 ** -18 * r * top * most * (
            1 + n * n.max(axis=-1, keepdims=True)), f"dx {i}")
        if dw[i] is not None:
            terms = np.sum(top * n, axis=(0, 1))
            no_worse(dw[i], want_w, U * np.abs(want_w) + 2.0 ** -14 * terms, f"dw {i}")
        assert all(p.intact() for p in (x[i], out[i], g[i], dx[i]))


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_far_positions(dm, interleaved):
    """The angle loses nothing up to the ends of int32, with frequencies above one turn too."""
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 1 << 24, -1, 0], dtype=torch.int32,
                       device="cuda")
    f = torch.tensor([1.0, 0.3337, 6.5, 100.25, 1e-7, 2.0 ** -20, 0.0, 0.77], device="cuda")
    op = dm.QKNormRope(6, 3, 1, 16, interleaved=interleaved, eps=0.0)
    q, k = Draw(1)((6, 3, 16)), Draw(2)((6, 1, 16))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    op.forward(q, k, None, None, f, pos, qo, ko)
    one = np.ones(16)
    for x, y in ((q, qo), (k, ko)):
        want = oracle.norm_rope(np64(x), one, np64(f), np64(pos), 0.0, interleaved)
        # position * frequency is exact in the reference to 2^-53 * 2^31 * 100 = 2^-15
        slack = 2.0 ** -15 * np.abs(np64(x)).max()
        no_worse(y, want, rope_bound(np64(x), one, 0.0, want) + slack * 4, "far")


def test_norm_rope_in_place_and_packed(dm):
    """q and k as slices of one projection, normalised where they lie; v is not touched."""
    t, hq, hk, d = 77, 8, 2, 64
    qkv = Draw(3)((t, (hq + 2 * hk) * d))
    keep = qkv.clone()
    q, k = qkv[:, :hq * d].view(t, hq, d), qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
    w, f = Draw(4)((d,)), rope_reference(d, d)
    pos = torch.arange(t, device="cuda", dtype=torch.int32)
    op = dm.QKNormRope(t, hq, hk, d)
    want = [torch.empty((t, h, d), dtype=torch.bfloat16, device="cuda") for h in (hq, hk)]
    op.forward(q, k, w, w, f, pos, *want)
    op.forward(q, k, w, w, f, pos, q, k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, (hq + hk) * d:], keep[:, (hq + hk) * d:])
    # gradients over the outputs' gradients
    g = [Draw(5)(x.shape) for x in want]
    x = [keep[:, :hq * d].view(t, hq, d), keep[:, hq * d:(hq + hk) * d].view(t, hk, d)]
    dx, dw = [torch.empty_like(v) for v in want], [torch.empty_like(w) for _ in want]
    op.backward(*g, *x, w, w, f, pos, *dx, *dw)
    dw2 = [torch.empty_like(w) for _ in want]
    op.backward(*g, *x, w, w, f, pos, *g, *dw2)
    assert all(torch.equal(a, b) for a, b in zip(g + dw2, dx + dw))


def test_norm_rope_bad_values_stay_in_their_head(dm):
    q, k = Draw(6)((4, 3, 64)), Draw(7)((4, 2, 64))
    f, pos = rope_reference(64, 64), torch.arange(4, device="cuda", dtype=torch.int32)
    op = dm.QKNormRope(4, 3, 2, 64)
    run = lambda: [x for x in (torch.empty_like(q), torch.empty_like(k))]
    a, b = run(), run()
    op.forward(q, k, None, None, f, pos, *a)
    q[1, 2, 5] = float("nan")
    k[3, 0, 63] = float("inf")
    op.forward(q, k, None, None, f, pos, *b)
    assert bool(b[0][1, 2].isnan().all()) and bool(b[1][3, 0, 63].isnan())
    a[0][1, 2] = 0
    b[0][1, 2] = 0
    a[1][3, 0] = 0
    b[1][3, 0] = 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_norm_rope_zero_tokens_and_zero_rows(dm):
    op = dm.QKNormRope(8, 2, 2, 64)
    f = rope_reference(64, 64)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    op.forward(e, e, None, None, f, none, e, e)
    dw = [torch.full((64,), SENTINEL, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    op.backward(e, e, e, e, None, None, f, none, e, e, *dw)
    assert not dw[0].any() and not dw[1].any()
    z = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(3, device="cuda", dtype=torch.int32)
    y = [torch.empty_like(z), torch.empty_like(z)]
    op.forward(z, z, None, None, f, pos, *y)
    assert not y[0].any() and not y[1].any()


# ------------------------------------------------------------------ linear attention
def mix_case(seed, tokens, heads, dk, dv, sequences, states, layout=("rows", 0, 0)):
    d = Draw(seed)
    lay, off, pad = layout
    c = {}
    for n, w in (("q", dk), ("k", dk), ("v", dv), ("dout", dv)):
        c[n] = Place(tokens, heads, w, lay, off, pad, d((tokens, heads, w)))
    for n, w in (("out", dv), ("dq", dk), ("dk", dk), ("dv", dv)):
        c["to_" + n] = Place(tokens, heads, w, lay, off, pad)
    g = -torch.exp2(-8 * torch.rand(heads, generator=d.g, device="cuda"))
    if heads > 2:
        g[1] = 0.0
        g[2] = -float("inf")
    if heads > 3:
        g[3] = -20.0
    c["g"] = g
    n = len(sequences) - 1 if sequences is not None else 1
    c["offsets"] = None if sequences is None else torch.tensor(sequences, dtype=torch.int32,
                                                                device="cuda")
    shape = (n, heads, dk, dv)
    c["state"] = d(shape, 3.0, torch.float32) if states else None
    c["dfinal"] = d(shape, 1.0, torch.float32) if states else None
    c["final"], c["dstate"] = (torch.full(shape, SENTINEL, device="cuda") if states else None
                               for _ in range(2))
    return c


def near_mix(got, ref, mass, what, live=None):
    got = np64(got)
    if live is not None:
        got, ref, mass = got[live], ref[live], mass[live]
    if ref.size == 0:
        return
    no_worse(got, ref, U * np.abs(ref) + 2.1 * U * mass, what)
    lim = 2 * U if ref.size >= 1000 else 3 * U
    assert np.linalg.norm(got - ref) <= lim * np.linalg.norm(ref), \
        (what, np.linalg.norm(got - ref) / np.linalg.norm(ref))


def mix_check(dm, c, scale, what):
    tokens, heads, dk = c["q"].t.shape
    dv = c["v"].t.shape[2]
    n = 1 if c["offsets"] is None else len(c["offsets"]) - 1
    op = dm.LinearAttention(tokens, heads, dk, dv, max_sequences=n, scale=scale)
    q, k, v, dout = (c[x].t for x in ("q", "k", "v", "dout"))
    op.forward(q, k, v, c["g"], c["to_out"].t, offsets=c["offsets"], state=c["state"],
               final_state=c["final"])
    op.backward(dout, q, k, v, c["g"], c["to_dq"].t, c["to_dk"].t, c["to_dv"].t,
                offsets=c["offsets"], state=c["state"], dfinal_state=c["dfinal"],
                dstate=c["dstate"])
    assert op.status() == dm.OK
    off = None if c["offsets"] is None else c["offsets"].tolist()
    live = np.zeros(tokens, bool)
    for b, e in ([(0, tokens)] if off is None else zip(off, off[1:])):
        live[b:e] = True
    a = [np64(x) for x in (q, k, v, dout)]
    g, st, df = np64(c["g"]), np64(c["state"]), np64(c["dfinal"])
    mag = [np.abs(x) for x in a]
    ab = lambda x: None if x is None else np.abs(x)
    ref = oracle.linattn(a[0], a[1], a[2], g, scale, off, st)
    mass = oracle.linattn(mag[0], mag[1], mag[2], g, abs(scale), off, ab(st))
    near_mix(c["to_out"].t, ref["out"], mass["out"], what + " out", live)
    back = oracle.linattn_backward(a[3], a[0], a[1], a[2], g, scale, off, st, df)
    bmass = oracle.linattn_backward(mag[3], mag[0], mag[1], mag[2], g, abs(scale), off, ab(st), ab(df))
    for x in ("dq", "dk", "dv"):
        near_mix(c["to_" + x].t, back[x], bmass[x], what + " " + x, live)
    if st is not None:
        tiny = 2.0 ** -100
        no_worse(c["final"], ref["state"], 1.25 * 2.0 ** -16 * mass["state"] + tiny, what + " final")
        no_worse(c["dstate"], back["dstate"], 1.25 * 2.0 ** -16 * bmass["dstate"] + tiny,
                 what + " dstate")
    for x in ("to_out", "to_dq", "to_dk", "to_dv"):
        assert c[x].intact(), (what, x)
        if not live.all():
            assert bool((c[x].t[torch.from_numpy(~live).cuda()] == SENTINEL).all()), (what, x)
    return op


DIMS = [(128, 128), (64, 64), (64, 128), (128, 64), (8, 8), (40, 96), (120, 24), (72, 128)]


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("tokens", [1, 2, 127, 128, 129, 300])
def test_linattn_one_sequence(dm, dk, dv, tokens):
    c = mix_case(tokens + dk, tokens, 5, dk, dv, None, tokens != 2)
    mix_check(dm, c, dk ** -0.5, f"{dk} {dv} {tokens}")


RAGGED = [[0, 0, 1, 129, 129, 385, 400], [5, 6, 7, 135, 300], [0, 128, 256, 384], [3, 3], [17, 400, 400]]


@pytest.mark.parametrize("offsets", RAGGED)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (64, 128), (24, 112)])
@pytest.mark.parametrize("states", [False, True])
def test_linattn_packed_sequences(dm, offsets, dk, dv, states):
    """Empty sequences, single tokens, ends inside a block; rows of no sequence hold NaN, and
    stay as they were in the outputs."""
    c = mix_case(7, 400, 4, dk, dv, offsets, states)
    dead = torch.ones(400, dtype=torch.bool, device="cuda")
    dead[offsets[0]:offsets[-1]] = False
    for x in ("q", "k", "v", "dout"):
        c[x].t[dead] = float("nan")
    for x in ("q", "k", "v", "dout"):      # the reference never looks at them
        c[x].t[dead] = float("nan")
    clean = {x: c[x].t.clone() for x in ("q", "k", "v", "dout")}
    mix_check(dm, c, -0.4, f"{offsets}")
    assert all(torch.equal(torch.nan_to_num(clean[x]), torch.nan_to_num(c[x].t)) for x in clean)


@pytest.mark.parametrize("layout", LAYOUTS[1:])
def test_linattn_strides(dm, layout):
    mix_check(dm, mix_case(8, 333, 3, 64, 128, [0, 100, 333], True, layout), 0.2, str(layout))


@pytest.mark.parametrize("tokens,heads", [(1500, 1), (1024, 3), (2600, 4)])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
def test_linattn_long_sequences_of_few_heads(dm, tokens, heads, dk, dv):
    """Sequences that several CTAs share."""
    mix_check(dm, mix_case(9, tokens, heads, dk, dv, None, True), 0.1, f"{tokens} {heads}")


def test_linattn_many_sequences(dm):
    rng = np.random.default_rng(3)
    ends = np.concatenate([[0], np.cumsum(rng.integers(0, 9, 200))]).tolist()
    mix_check(dm, mix_case(10, ends[-1], 3, 64, 64, ends, True), 1.0, "many")


def test_linattn_states_in_place(dm):
    c = mix_case(11, 1300, 2, 128, 128, None, True)
    op = dm.LinearAttention(1300, 2, 128)
    args = [c[x].t for x in ("q", "k", "v")] + [c["g"]]
    op.forward(*args, c["to_out"].t, state=c["state"], final_state=c["final"])
    s, out = c["state"].clone(), torch.empty_like(c["v"].t)
    op.forward(*args, out, state=s, final_state=s)
    assert torch.equal(s, c["final"]) and torch.equal(out, c["to_out"].t)
    grads = [c[x].t for x in ("to_dq", "to_dk", "to_dv")]
    op.backward(c["dout"].t, *args, *grads, state=c["state"], dfinal_state=c["dfinal"],
                dstate=c["dstate"])
    d, again = c["dfinal"].clone(), [torch.empty_like(x) for x in grads]
    op.backward(c["dout"].t, *args, *again, state=c["state"], dfinal_state=d, dstate=d)
    assert torch.equal(d, c["dstate"]) and all(torch.equal(a, b) for a, b in zip(again, grads))


def test_linattn_bad_values_stay_in_their_sequence_and_head(dm):
    off = [0, 50, 300, 420]
    a, b = (mix_case(12, 420, 3, 128, 128, off, True) for _ in range(2))
    for x in (a, b):
        x["g"].fill_(-0.05)
    for x, at in (("q", (60, 1, 3)), ("k", (61, 1, 0)), ("v", (200, 1, 127)), ("dout", (250, 1, 9))):
        b[x].t[at] = float("nan")
    op = dm.LinearAttention(420, 3, 128, max_sequences=3)
    for x in (a, b):
        args = [x[n].t for n in ("q", "k", "v")] + [x["g"]]
        op.forward(*args, x["to_out"].t, offsets=x["offsets"], state=x["state"], final_state=x["final"])
        op.backward(x["dout"].t, *args, *(x[n].t for n in ("to_dq", "to_dk", "to_dv")),
                    offsets=x["offsets"], state=x["state"], dfinal_state=x["dfinal"],
                    dstate=x["dstate"])
    for n in ("to_out", "to_dq", "to_dk", "to_dv"):
        bad = b[n].t.isnan()
        assert bool(bad[50:300, 1].any()), n
        bad[50:300, 1] = False
        assert not bool(bad.any()), n
        for s in (slice(0, 50), slice(300, 420)):
            assert torch.equal(a[n].t[s], b[n].t[s]), n
        assert torch.equal(a[n].t[:, 0], b[n].t[:, 0]) and torch.equal(a[n].t[:, 2], b[n].t[:, 2]), n
    # causal: the first of them is at token 60, in its own row only
    assert torch.equal(a["to_out"].t[50:60], b["to_out"].t[50:60])
    for n in ("final", "dstate"):
        assert torch.equal(a[n][0], b[n][0]) and torch.equal(a[n][2], b[n][2])
        assert bool(b[n][1, 1].isnan().any()) and torch.equal(a[n][1, 0], b[n][1, 0])


def test_linattn_offsets_out_of_range_are_cut(dm):
    c = mix_case(13, 200, 2, 64, 64, [-5, 90, 500], False)
    want = mix_case(13, 200, 2, 64, 64, [0, 90, 200], False)
    op = dm.LinearAttention(200, 2, 64, max_sequences=2)
    for x in (c, want):
        op.forward(x["q"].t, x["k"].t, x["v"].t, x["g"], x["to_out"].t, offsets=x["offsets"])
    assert torch.equal(c["to_out"].t, want["to_out"].t)
    down = torch.tensor([150, 20, 60], dtype=torch.int32, device="cuda")   # the first is empty
    op.forward(c["q"].t, c["k"].t, c["v"].t, c["g"], c["to_out"].t, offsets=down)
    torch.cuda.synchronize()
    assert op.status() == dm.OK


def test_linattn_no_tokens(dm):
    op = dm.LinearAttention(10, 2, 64, 32, max_sequences=2)
    e, ev = (torch.empty((0, 2, w), dtype=torch.bfloat16, device="cuda") for w in (64, 32))
    st = Draw(14)((2, 2, 64, 32), 1.0, torch.float32)
    out, g = torch.empty_like(st), torch.zeros(2, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    op.forward(e, e, ev, g, ev, offsets=off)
    op.forward(e, e, ev, g, ev, offsets=off, state=st, final_state=out)
    assert torch.equal(out, st)
    op.forward(e, e, ev, g, ev, offsets=off, final_state=out)
    assert not out.any()
    op.backward(ev, e, e, ev, g, e, e, ev, offsets=off, dfinal_state=st, dstate=out)
    assert torch.allclose(out, st, rtol=2 ** -22, atol=0)


# ------------------------------------------------------------------ single tokens
@pytest.mark.parametrize("rows,heads,dk,dv", [(1, 32, 128, 128), (3, 5, 64, 64), (17, 2, 8, 8),
                                              (5, 3, 40, 96), (130, 1, 120, 24), (2, 4, 72, 128)])
@pytest.mark.parametrize("layout", [("rows", 0, 0), ("heads", 1, 3)])
def test_step_matches_the_recurrence(dm, rows, heads, dk, dv, layout):
    c = mix_case(rows + dk, rows, heads, dk, dv, None, False, layout)
    st = Draw(15)((rows + 1, heads, dk, dv), 2.0, torch.float32)
    op = dm.LinearAttention(rows, heads, dk, dv, scale=0.3)
    q, k, v = (c[x].t for x in ("q", "k", "v"))
    new = torch.full_like(st, SENTINEL)
    op.step(q, k, v, c["g"], st, c["to_out"].t, new_state=new)
    each = list(range(rows + 1))
    ref = oracle.linattn(np64(q), np64(k), np64(v), np64(c["g"]), 0.3, each, np64(st)[:rows])
    mass = oracle.linattn(*(np.abs(np64(x)) for x in (q, k, v)), np64(c["g"]), 0.3, each,
                          np.abs(np64(st))[:rows])
    no_worse(new[:rows], ref["state"], 2.0 ** -22 * mass["state"] + 2.0 ** -100, "state")
    no_worse(c["to_out"].t, ref["out"], U * np.abs(ref["out"]) + 2.0 ** -17 * mass["out"], "out")
    assert bool((new[rows] == SENTINEL).all()) and c["to_out"].intact()
    keep, out = st.clone(), torch.empty_like(v)
    op.step(q, k, v, c["g"], st, out)                                   # in place
    assert torch.equal(st[:rows], new[:rows]) and torch.equal(out, c["to_out"].t)
    assert torch.equal(st[rows], keep[rows])


@pytest.mark.parametrize("in_place", [False, True])
def test_step_slots(dm, in_place):
    """Rows name their slots; padding rows are skipped, shared slots taken in order."""
    rows, heads, dk, dv, slots = 300, 3, 64, 40, 9
    c = mix_case(16, rows, heads, dk, dv, None, False)
    st = Draw(17)((slots, heads, dk, dv), 1.0, torch.float32)
    rng = np.random.default_rng(18)
    names = rng.integers(-2, slots + 2, rows)
    names[names == 4] = 3
    op = dm.LinearAttention(rows, heads, dk, dv)
    q, k, v = (c[x].t for x in ("q", "k", "v"))
    new = st.clone() if in_place else torch.full_like(st, SENTINEL)
    op.step(q, k, v, c["g"], new if in_place else st, c["to_out"].t,
            new_state=None if in_place else new,
            slots=torch.tensor(names, dtype=torch.int32, device="cuda"))
    out = c["to_out"].t
    for s in range(slots):
        at = np.nonzero(names == s)[0]
        if len(at) == 0:
            assert s == 4 and torch.equal(new[s], st[s] if in_place else torch.full_like(st[s], SENTINEL))
            continue
        want_new, w = st[s:s + 1].clone(), []
        for r in at:                               # one row after another
            o = torch.empty_like(v[r:r + 1])
            op.step(q[r:r + 1], k[r:r + 1], v[r:r + 1], c["g"], want_new, o)
            w.append(o)
        assert torch.equal(new[s], want_new[0])
        assert torch.equal(out[torch.from_numpy(at).cuda()], torch.cat(w))
    pad = (names < 0) | (names >= slots)
    assert bool((out[torch.from_numpy(pad).cuda()] == SENTINEL).all())


def test_prompt_then_steps_equal_the_whole(dm):
    """A state from forward carries on token by token."""
    heads, d, n, more = 4, 128, 260, 5
    c = mix_case(19, n + more, heads, d, d, None, False)
    c["g"].fill_(-0.02)
    op = dm.LinearAttention(n + more, heads, d)
    q, k, v = (c[x].t for x in ("q", "k", "v"))
    st = torch.empty((1, heads, d, d), device="cuda")
    op.forward(q[:n], k[:n], v[:n], c["g"], c["to_out"].t[:n], final_state=st)
    for t in range(n, n + more):
        op.step(q[t:t + 1], k[t:t + 1], v[t:t + 1], c["g"], st, c["to_out"].t[t:t + 1])
    ref = oracle.linattn(np64(q), np64(k), np64(v), np64(c["g"]), d ** -0.5)
    mass = oracle.linattn(*(np.abs(np64(x)) for x in (q, k, v)), np64(c["g"]), d ** -0.5)
    near_mix(c["to_out"].t, ref["out"], mass["out"], "prompt and steps")
    no_worse(st, ref["state"], 1.5 * 2.0 ** -16 * mass["state"], "state")


# ------------------------------------------------------------------ repeats, streams, graphs
def test_results_repeat_bit_for_bit(dm):
    c = mix_case(20, 3000, 6, 128, 128, [0, 900, 1000, 3000], True)
    op = dm.LinearAttention(3000, 6, 128, max_sequences=3)
    rope = dm.QKNormRope(3000, 6, 6, 128)
    f, pos = rope_reference(128, 128), torch.arange(3000, device="cuda", dtype=torch.int32)
    w = Draw(21)((128,))
    seen = []
    for _ in range(3):
        args = [c[x].t for x in ("q", "k", "v")] + [c["g"]]
        out, fin, dst = torch.empty_like(c["v"].t), torch.empty_like(c["state"]), \
            torch.empty_like(c["state"])
        gr = [torch.empty_like(c["q"].t) for _ in range(3)]
        op.forward(*args, out, offsets=c["offsets"], state=c["state"], final_state=fin)
        op.backward(c["dout"].t, *args, *gr, offsets=c["offsets"], state=c["state"],
                    dfinal_state=c["dfinal"], dstate=dst)
        dx, dw = [torch.empty_like(gr[0]) for _ in range(2)], [torch.empty_like(w) for _ in range(2)]
        rope.backward(gr[0], gr[1], c["q"].t, c["k"].t, w, w, f, pos, *dx, *dw)
        seen.append([out, fin, dst] + gr + dx + dw)
    for other in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], other))


def mixer(dm, t, hidden, heads, d):
    """A layer as a model runs it: one projection, norms and rotation where q and k lie, mixing,
    the feed-forward block, the head's loss, and everything's gradients."""
    r = Draw(22)
    f = 192
    s = {"x": r((t, hidden)), "w_qkv": r((3 * heads * d, hidden), hidden ** -0.5),
         "w_o": r((hidden, heads * d), (heads * d) ** -0.5), "w_q": 1 + r((d,), 0.1),
         "w_k": 1 + r((d,), 0.1), "ffn": [r((f, hidden), hidden ** -0.5), r((f, hidden), hidden ** -0.5),
                                          r((hidden, f), f ** -0.5)], "head": r((500, hidden), 0.1)}
    s["g"] = -torch.exp2(-torch.arange(1, heads + 1, device="cuda").float())
    s["off"] = torch.tensor([0, t // 3, t // 3, t - 4], dtype=torch.int32, device="cuda")
    s["pos"] = torch.arange(t, device="cuda", dtype=torch.int32)
    s["f"] = rope_reference(d, d)
    s["target"] = torch.randint(500, (t,), generator=r.g, device="cuda")
    s["target"][t - 4:] = -100                                 # the padding is not learnt from
    s["rope"] = dm.QKNormRope(t, heads, heads, d)
    s["mix"] = dm.LinearAttention(t, heads, d, max_sequences=3)
    s["block"] = dm.GatedFFN(t, hidden, f, save=dm.SAVE_BF16)
    s["loss"] = dm.LinearXent(t, hidden, 500)
    e = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    s["o"], s["do"] = e(t, heads, d), e(t, heads, d)
    s["qk"], s["dqkv"], s["dqk"] = e(2, t, heads, d), e(t, 3 * heads * d), e(2, t, heads, d)
    s["y"], s["dh"], s["dx"] = e(t, hidden), e(t, hidden), e(t, hidden)
    s["saved"] = s["block"].empty_saved(t)
    s["dw"] = [torch.empty_like(w) for w in s["ffn"]]
    s["dhead"], s["dw_q"], s["dw_k"] = e(500, hidden), e(d), e(d)
    s["l"], s["lse"] = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    s["gl"] = torch.full((t,), 1.0 / t, device="cuda")

    def run():
        qkv = s["x"] @ s["w_qkv"].t()
        q, k, v = (qkv[:, i * heads * d:(i + 1) * heads * d].view(t, heads, d) for i in range(3))
        s["rope"].forward(q, k, s["w_q"], s["w_k"], s["f"], s["pos"], s["qk"][0], s["qk"][1])
        s["mix"].forward(s["qk"][0], s["qk"][1], v, s["g"], s["o"], offsets=s["off"])
        h = s["x"] + s["o"].view(t, -1) @ s["w_o"].t()
        s["block"].forward(h, *s["ffn"], s["y"], s["saved"])
        s["loss"].loss_and_grads(h + s["y"], s["head"], s["target"], s["gl"], s["l"], s["lse"],
                                 s["dh"], s["dhead"])
        s["block"].backward(s["dh"], h, *s["ffn"], s["saved"], s["dx"], *s["dw"])
        dhid = s["dh"] + s["dx"]
        s["do"].copy_((dhid @ s["w_o"]).view(t, heads, d))
        dv = s["dqkv"][:, 2 * heads * d:].view(t, heads, d)
        s["mix"].backward(s["do"], s["qk"][0], s["qk"][1], v, s["g"], s["dqk"][0], s["dqk"][1], dv,
                          offsets=s["off"])
        dq, dk = (s["dqkv"][:, i * heads * d:(i + 1) * heads * d].view(t, heads, d) for i in (0, 1))
        s["rope"].backward(s["dqk"][0], s["dqk"][1], q, k, s["w_q"], s["w_k"], s["f"], s["pos"], dq,
                           dk, s["dw_q"], s["dw_k"])
        s["dw_qkv"] = s["dqkv"].t() @ s["x"]
        return [s["l"], s["dw_qkv"], s["dw_q"], s["dw_k"], s["dhead"], *s["dw"], s["dqkv"]]
    return s, run


def test_a_layer_and_its_gradients(dm):
    """The operators together against the same layer in fp64 through autograd: gradients of the
    projection, of the gains and of the feed-forward weights.  Each is a chain of about ten bf16
    roundings (u each, independent): relative Frobenius error at most 10 u."""
    t, hidden, heads, d = 391, 128, 3, 64
    s, run = mixer(dm, t, hidden, heads, d)
    got = [x.clone() for x in run()]
    leaf = {n: s[n].double().requires_grad_() for n in ("w_qkv", "w_q", "w_k", "head")}
    ffn = [w.double().requires_grad_() for w in s["ffn"]]
    x, w_o = s["x"].double(), s["w_o"].double()
    qkv = x @ leaf["w_qkv"].t()
    q, k, v = (qkv[:, i * heads * d:(i + 1) * heads * d].view(t, heads, d) for i in range(3))
    ang = torch.outer(s["pos"].double(), s["f"].double())[:, None]

    def nr(z, w):
        z = z / torch.sqrt(z.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = z[..., :d // 2], z[..., d // 2:]
        return torch.cat((a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()), -1)

    q, k = nr(q, leaf["w_q"]), nr(k, leaf["w_k"])
    i = torch.arange(t, device="cuda")
    seq = torch.bucketize(i, s["off"][1:].long(), right=True)
    gap = i[:, None] - i
    see = (gap >= 0) & (seq[:, None] == seq) & (i < t - 4)[:, None]
    wgt = torch.where(see, torch.exp(s["g"].double()[:, None, None] * gap.clamp_min(0)), 0.0)
    p = torch.einsum("ihd,jhd->hij", q, k) * wgt * d ** -0.5
    o = torch.einsum("hij,jhd->ihd", p, v).reshape(t, -1)
    h = x + o @ w_o.t()
    gate, up = h @ ffn[0].t(), h @ ffn[1].t()
    h = h + (torch.nn.functional.silu(gate) * up) @ ffn[2].t()
    lsm = torch.log_softmax(h @ leaf["head"].t(), -1)
    live = torch.arange(t - 4, device="cuda")
    loss = -(lsm[live, s["target"][live]]).sum() / t
    want = torch.autograd.grad(loss, [leaf["w_qkv"], leaf["w_q"], leaf["w_k"], leaf["head"], *ffn])
    for name, a, b in zip(["dw_qkv", "dw_q", "dw_k", "dhead", "gate", "up", "down"], got[1:], want):
        err = float((a.double() - b).norm() / b.norm())
        assert err <= 10 * U, (name, err)
    for op in ("rope", "mix", "block", "loss"):
        assert s[op].status() == dm.OK


def test_a_layer_captured_into_a_graph_replays(dm):
    s, run = mixer(dm, 300, 64, 2, 32)
    want = [x.clone() for x in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = run()
    for _ in range(2):
        for x in outs:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # other inputs in the same memory
    s["x"].mul_(-0.5)
    fresh = [x.clone() for x in run()]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, fresh))


def test_two_streams_with_their_own_handles(dm):
    cases = [mix_case(23 + i, 1800, 4, 128, 64, [0, 700, 1800], True) for i in range(2)]
    ops = [dm.LinearAttention(1800, 4, 128, 64, max_sequences=2) for _ in cases]

    def go(c, op, stream=None):
        args = [c[x].t for x in ("q", "k", "v")] + [c["g"]]
        op.forward(*args, c["to_out"].t, offsets=c["offsets"], state=c["state"],
                   final_state=c["final"], stream=stream)
        op.backward(c["dout"].t, *args, *(c[n].t for n in ("to_dq", "to_dk", "to_dv")),
                    offsets=c["offsets"], state=c["state"], dfinal_state=c["dfinal"],
                    dstate=c["dstate"], stream=stream)
        return [c[n].t for n in ("to_out", "to_dq", "to_dk", "to_dv")] + [c["final"], c["dstate"]]

    want = [[x.clone() for x in go(c, op)] for c, op in zip(cases, ops)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for c, op, st in zip(cases, ops, streams):
        go(c, op, st.cuda_stream)
    torch.cuda.synchronize()
    for c, w, op in zip(cases, want, ops):
        have = [c[n].t for n in ("to_out", "to_dq", "to_dk", "to_dv")] + [c["final"], c["dstate"]]
        assert all(torch.equal(a, b) for a, b in zip(have, w)) and op.status() == dm.OK


# ------------------------------------------------------------------ many sequences, far addresses
@pytest.mark.parametrize("heads,sequences,tokens", [(2, 100, 6000), (1, 33, 9000), (12, 70, 3000),
                                                    (3, 800, 2500)])
def test_linattn_many_sequences_of_few_heads(dm, heads, sequences, tokens):
    """More sequences than a warp has lanes, shared among clusters and CTAs wherever they end, the
    states over themselves; every output against the fp64 recurrence."""
    rng = np.random.default_rng(tokens)
    cuts = np.sort(rng.integers(0, tokens, sequences - 1))
    cuts[: sequences // 4] = cuts[sequences // 4]                # a run of empty ones
    off = [0] + np.sort(cuts).tolist() + [tokens]
    c = mix_case(31, tokens, heads, 64, 128, off, True)
    mix_check(dm, c, 0.3, f"{heads} {sequences}")
    op = dm.LinearAttention(tokens, heads, 64, 128, max_sequences=sequences, scale=0.3)
    args = [c[x].t for x in ("q", "k", "v")] + [c["g"]]
    s, out = c["state"].clone(), torch.empty_like(c["v"].t)
    op.forward(*args, out, offsets=c["offsets"], state=s, final_state=s)
    assert torch.equal(s, c["final"]) and torch.equal(out, c["to_out"].t)


def test_rows_past_2_to_the_32_elements(dm):
    """Tokens so far apart that offsets pass 32 bits give the bits of the same tokens side by side."""
    tokens, heads, d, apart = 300, 2, 64, 1 << 24
    far = [torch.empty(tokens * apart, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    f, pos = rope_reference(d, d), torch.arange(tokens, device="cuda", dtype=torch.int32)

    def at(buf, i):       # five tensors to a buffer
        return buf.as_strided((tokens, heads, d), (apart, d, 1), i * heads * d)

    def run(place):
        draw = Draw(32)
        q, k, v, dout = (place(0, i).copy_(draw((tokens, heads, d))) for i in range(4))
        qo, ko = place(1, 0), place(1, 1)
        dm.QKNormRope(tokens, heads, heads, d).forward(q, k, None, None, f, pos, qo, ko)
        op, g = dm.LinearAttention(tokens, heads, d), torch.full((heads,), -0.01, device="cuda")
        out = place(1, 2)
        op.forward(qo, ko, v, g, out)
        grads = [place(1, 3), place(1, 4), place(0, 4)]
        op.backward(dout, qo, ko, v, g, *grads)
        dx, dw = [place(1, 0), place(1, 1)], [torch.empty(d, dtype=torch.bfloat16, device="cuda")] * 2
        rows = [x.clone() for x in (qo, ko, out, *grads)]
        dm.QKNormRope(tokens, heads, heads, d).backward(grads[0], grads[1], q, k, None, None, f, pos, *dx,
                                                        None, None)
        return rows + [x.clone() for x in dx]

    near = {}
    want = run(lambda b, i: near.setdefault((b, i), torch.empty((tokens, heads, d), dtype=torch.bfloat16,
                                                                device="cuda")))
    assert (tokens - 1) * apart > 1 << 32
    assert all(torch.equal(a, b) for a, b in zip(run(lambda b, i: at(far[b], i)), want))


def test_step_states_past_2_to_the_32_elements(dm):
    heads, d, slots, rows = 2, 128, 140000, 5
    pool = torch.empty((slots, heads, d, d), device="cuda")
    assert pool.numel() > 1 << 32
    names = torch.tensor([slots - 1, 3, 131080, 70000, slots - 2], dtype=torch.int32, device="cuda")
    small = Draw(33)((rows, heads, d, d), 1.0, torch.float32)
    for i, n in enumerate(names.tolist()):
        pool[n] = small[i]
    draw = Draw(34)
    q, k, v = (draw((rows, heads, d)) for _ in range(3))
    g = torch.full((heads,), -0.1, device="cuda")
    op, want, out = dm.LinearAttention(rows, heads, d), torch.empty_like(v), torch.empty_like(v)
    op.step(q, k, v, g, small, want)
    op.step(q, k, v, g, pool, out, slots=names)
    assert torch.equal(out, want)
    assert all(torch.equal(pool[n], small[i]) for i, n in enumerate(names.tolist()))


# ------------------------------------------------------------------ sequences dealt whole
@pytest.mark.parametrize("heads,cuts,dk,dv", [(160, [0, 700, 700, 701, 1100, 1500], 8, 24),
                                              (57, [3, 303, 304, 304, 433, 590], 128, 128),
                                              (155, [3, 303, 304, 433], 64, 128),
                                              (52, [0, 900, 901, 1400, 2000], 24, 40),
                                              (160, [5, 5, 5, 5], 64, 64),
                                              (160, [0, 0, 600, 600], 128, 64),
                                              (101, list(range(0, 600, 37)), 64, 64)])
def test_linattn_sequences_of_many_heads(dm, heads, cuts, dk, dv):
    """More heads, or heads and gradients, than SMs: a CTA takes sequences of several of them, one
    after another.  From states, but to none."""
    tokens = max(600, cuts[-1])
    c = mix_case(41, tokens, heads, dk, dv, cuts, False)
    op = mix_check(dm, c, 0.3, f"{heads}")
    first = [c[x].t.clone() for x in ("to_out", "to_dq", "to_dk", "to_dv")]
    q, k, v, dout = (c[x].t for x in ("q", "k", "v", "dout"))
    op.forward(q, k, v, c["g"], c["to_out"].t, offsets=c["offsets"])
    op.backward(dout, q, k, v, c["g"], c["to_dq"].t, c["to_dk"].t, c["to_dv"].t, offsets=c["offsets"])
    assert all(torch.equal(a, c[x].t) for a, x in zip(first, ("to_out", "to_dq", "to_dk", "to_dv")))

    n = len(cuts) - 1
    state, dfinal = (torch.randn(n, heads, dk, dv, device="cuda") for _ in range(2))
    op.forward(q, k, v, c["g"], c["to_out"].t, offsets=c["offsets"], state=state)
    op.backward(dout, q, k, v, c["g"], c["to_dq"].t, c["to_dk"].t, c["to_dv"].t, offsets=c["offsets"],
                state=state, dfinal_state=dfinal)
    assert op.status() == dm.OK
    a, g = [np64(x) for x in (q, k, v, dout)], np64(c["g"])
    st, df = np64(state), np64(dfinal)
    mag = [np.abs(x) for x in a]
    live = np.zeros(tokens, bool)
    live[cuts[0]:cuts[-1]] = True
    near_mix(c["to_out"].t, oracle.linattn(a[0], a[1], a[2], g, 0.3, cuts, st)["out"],
             oracle.linattn(mag[0], mag[1], mag[2], g, 0.3, cuts, np.abs(st))["out"], "out", live)
    back = oracle.linattn_backward(a[3], a[0], a[1], a[2], g, 0.3, cuts, st, df)
    mass = oracle.linattn_backward(mag[3], mag[0], mag[1], mag[2], g, 0.3, cuts, np.abs(st), np.abs(df))
    for x in ("dq", "dk", "dv"):
        near_mix(c["to_" + x].t, back[x], mass[x], x, live)


# ------------------------------------------------------------------ ends inside blocks
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
def test_linattn_queries_after_the_ends_of_sequences(dm, dk, dv):
    """A CTA walks 40 sequences that end inside blocks, some of one row only: the queries that are
    loaded over such an end's output are whole.  Bit for bit what each sequence gives alone, which is
    too short for any place in shared memory to be used twice."""
    heads, lengths = 160, [1, 129, 33, 200, 95, 130, 0, 255, 64, 3] * 4
    cuts = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    c = mix_case(43, cuts[-1], heads, dk, dv, cuts, False)
    op = dm.LinearAttention(cuts[-1], heads, dk, dv, max_sequences=len(lengths), scale=0.2)
    names = ("q", "k", "v", "dout")
    outs = ("to_out", "to_dq", "to_dk", "to_dv")

    def run(offsets, at):
        q, k, v, dout = (c[x].t[at] for x in names)
        out, dq, dkk, dvv = (torch.zeros_like(x) for x in (v, q, k, v))
        op.forward(q, k, v, c["g"], out, offsets=offsets)
        op.backward(dout, q, k, v, c["g"], dq, dkk, dvv, offsets=offsets)
        return out, dq, dkk, dvv

    whole = run(c["offsets"], slice(None))
    assert op.status() == dm.OK
    for b, e in sorted(set(zip(cuts, cuts[1:]))):
        if b == e:
            continue
        for n, x, y in zip(outs, whole, run(None, slice(b, e))):
            assert torch.equal(x[b:e], y), (n, b, e)


# ------------------------------------------------------------------ the binding
def test_attributes_changed_after_a_call_hold(dm):
    """What a handle says of itself is what its next call does."""
    draw = Draw(48)
    q, k, v = (draw((9, 2, 64)) for _ in range(3))
    f, pos = rope_reference(64, 64), torch.arange(9, device="cuda", dtype=torch.int32)
    rope = dm.QKNormRope(9, 2, 2, 64)
    rope.forward(q, k, None, None, f, pos, torch.empty_like(q), torch.empty_like(k))
    for name, value in (("eps", 0.5), ("interleaved", True), ("rotary_dim", 32)):
        setattr(rope, name, value)
        fresh = dm.QKNormRope(9, 2, 2, 64, rope.rotary_dim, rope.eps, rope.interleaved)
        got, want = ([torch.empty_like(q), torch.empty_like(k)] for _ in range(2))
        freq = f[:rope.rotary_dim // 2].contiguous()
        rope.forward(q, k, None, None, freq, pos, *got)
        fresh.forward(q, k, None, None, freq, pos, *want)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    g = torch.full((2,), -0.1, device="cuda")
    mix, got, want = dm.LinearAttention(9, 2, 64), torch.empty_like(v), torch.empty_like(v)
    mix.forward(q, k, v, g, want)
    mix.scale *= 2
    mix.forward(q, k, v, g, got)
    assert torch.equal(got, want * 2)
    one = mix.heads = rope.q_heads = 1
    out = torch.empty_like(v[:, :one])
    mix.forward(q[:, :one], k[:, :one], v[:, :one], g[:one], out)
    assert torch.equal(out, got[:, :one])
    with pytest.raises(ValueError):
        mix.forward(q, k, v, g, got)
    with pytest.raises(ValueError):
        rope.forward(q, k, None, None, freq, pos, q, k)


# ------------------------------------------------------------------ gradients of states
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (72, 40)])
def test_linattn_gradients_of_states_keep_their_size(dm, dk, dv):
    """The final states' gradient is large and the scale small: nothing on the way leaves fp32."""
    tokens, heads, off, scale = 300, 3, [0, 0, 140, 300, 300], 2.0 ** -60
    c = mix_case(46, tokens, heads, dk, dv, off, True)
    c["dfinal"] *= 2.0 ** 70
    op = dm.LinearAttention(tokens, heads, dk, dv, max_sequences=4, scale=scale)
    q, k, v, dout = (c[x].t for x in ("q", "k", "v", "dout"))
    dq, dkk, dvv = (c[x].t for x in ("to_dq", "to_dk", "to_dv"))
    args = [np64(x) for x in (dout, q, k, v, c["g"])] + [scale, off, np64(c["state"]), np64(c["dfinal"])]
    ref = oracle.linattn_backward(*args)
    mass = oracle.linattn_backward(*(np.abs(x) for x in args[:4]), *args[4:7], *(np.abs(x) for x in args[7:]))
    for want_dstate in (True, False):
        op.backward(dout, q, k, v, c["g"], dq, dkk, dvv, offsets=c["offsets"], state=c["state"],
                    dfinal_state=c["dfinal"], dstate=c["dstate"] if want_dstate else None)
        for n, got in (("dq", dq), ("dk", dkk), ("dv", dvv)):
            near_mix(got, ref[n], mass[n], n)
    no_worse(c["dstate"], ref["dstate"], 1.25 * 2.0 ** -16 * mass["dstate"] + 2.0 ** -30, "dstate")


@pytest.mark.parametrize("scale", [0.3, -7.0, 2.0 ** -64])
def test_linattn_states_pass_empty_sequences_bit_for_bit(dm, scale):
    heads, d, off = 3, 64, [0, 0, 140, 140]
    c = mix_case(47, 140, heads, d, d, off, True)
    c["dfinal"][0] *= 1e30
    c["dfinal"][2] *= 1e-37
    op = dm.LinearAttention(140, heads, d, max_sequences=3, scale=scale)
    q, k, v, dout = (c[x].t for x in ("q", "k", "v", "dout"))
    op.forward(q, k, v, c["g"], c["to_out"].t, offsets=c["offsets"], state=c["state"], final_state=c["final"])
    op.backward(dout, q, k, v, c["g"], *(c[x].t for x in ("to_dq", "to_dk", "to_dv")), offsets=c["offsets"],
                state=c["state"], dfinal_state=c["dfinal"], dstate=c["dstate"])
    for i in (0, 2):
        assert torch.equal(c["final"][i], c["state"][i]) and torch.equal(c["dstate"][i], c["dfinal"][i])


# ------------------------------------------------------------------ slow heads
def test_states_of_slow_heads_do_not_drift(dm):
    """2^20 tokens in one chain of blocks (a CTA to a head), terms of one sign: what a decay loses when
    it is rounded to fp32 must not add up over the blocks that a slow head remembers.  A term is within
    1.25 * 2^-16; two roundings of 2^-24 a block fall to either side (terms are random): six deviations
    of their sum, at most sqrt(2 blocks / 3) * 2^-24, two blocks' worth of a state that grew to its size
    over all of them counting for no more than their average of a third."""
    tokens, heads, d = 1 << 20, 152, 8
    g = torch.tensor([-1e-6, -2e-7, -5e-8, -5e-7, -2e-3, 0.0, -7e-9, -3.3e-5], device="cuda")
    draw = Draw(44)
    k, v = (draw((tokens, heads, d)).abs_() for _ in range(2))
    final = torch.empty((1, heads, d, d), device="cuda")
    op, out = dm.LinearAttention(tokens, heads, d), torch.empty_like(v)
    op.forward(k, k, v, g.repeat(heads // 8), out, final_state=final)
    assert op.status() == dm.OK
    far = torch.arange(tokens - 1, -1, -1, device="cuda", dtype=torch.float64)
    tolerance = 1.25 * 2.0 ** -16 + 6 * 2.0 ** -24 * (2 * tokens / 128 / 9) ** 0.5
    for h in range(8):
        want = (k[:, h].double() * torch.exp(g[h].double() * far)[:, None]).T @ v[:, h].double()
        err = float((final[0, h].double() / want - 1).abs().max())
        assert err <= tolerance, (float(g[h]), err)
    # against time, k for queries: the first state's gradient, every term decayed once more
    op.backward(v, k, k, v, g.repeat(heads // 8), *(torch.empty_like(v) for _ in range(3)), dstate=final)
    assert op.status() == dm.OK
    for h in range(8):
        weight = d ** -0.5 * torch.exp(g[h].double() * (far.flip(0) + 1))
        want = (k[:, h].double() * weight[:, None]).T @ v[:, h].double()
        err = float((final[0, h].double() / want - 1).abs().max())
        assert err <= tolerance, ("dstate", float(g[h]), err)


def test_steps_of_slow_heads_do_not_drift(dm):
    """8000 single tokens of one sign: what exp(log_decay) loses when it is rounded to fp32 must not add
    up.  Three roundings of 2^-24 a step fall to either side (terms are random): six deviations of
    their sum, each counting as the state's size then did, a third of its last on average."""
    heads, d, n = 8, 64, 8000
    g = torch.tensor([-1e-6, -2e-7, -4.5e-8, -1e-7, -2e-4, 0.0, -7e-9, -3.3e-5], device="cuda")
    draw = Draw(45)
    k, v = (draw((n, heads, d)).abs_() for _ in range(2))
    s, op = torch.zeros((1, heads, d, d), device="cuda"), dm.LinearAttention(1, heads, d)
    out = torch.empty_like(v[:1])
    for t in range(n):
        op.step(k[t:t + 1], k[t:t + 1], v[t:t + 1], g, s, out)
    w = torch.exp(g.double() * torch.arange(n - 1, -1, -1, device="cuda").double()[:, None])
    want = torch.einsum("th,thi,thj->hij", w, k.double(), v.double())
    err = (s[0].double() / want - 1).abs().amax(dim=(1, 2))
    assert float(err.max()) <= 6 * 2.0 ** -24 * (3 * n / 9) ** 0.5, err.tolist()


def test_steps_keep_infinities(dm):
    """An infinity in a state stays one in slow and in fast heads, and a zero a zero."""
    heads, d = 4, 32
    g = torch.tensor([-1e-6, 0.0, -3.0, -0.3], device="cuda")
    z = torch.zeros((1, heads, d), dtype=torch.bfloat16, device="cuda")
    s = torch.zeros((1, heads, d, d), device="cuda")
    s[0, :, 3, 5], s[0, :, 7, 9] = float("inf"), -float("inf")
    want = s.clone()
    dm.LinearAttention(1, heads, d).step(z, z, z, g, s, torch.empty_like(z))
    assert torch.equal(s, want)


def test_required_tensors_may_not_be_none(dm):
    draw = Draw(49)
    q, k, v = (draw((4, 2, 64)) for _ in range(3))
    f, pos = rope_reference(64, 64), torch.arange(4, device="cuda", dtype=torch.int32)
    rope, mix, g = dm.QKNormRope(4, 2, 2, 64), dm.LinearAttention(4, 2, 64), torch.zeros(2, device="cuda")
    state = torch.zeros((4, 2, 64, 64), device="cuda")
    e = [torch.empty_like(q) for _ in range(3)]

    def each(call, args, optional=()):
        for i in range(len(args)):
            if i not in optional:
                with pytest.raises(TypeError):
                    call(*args[:i], None, *args[i + 1:])
        call(*args)

    each(rope.forward, [q, k, None, None, f, pos, e[0], e[1]], (2, 3))
    each(rope.backward, [q, k, q, k, None, None, f, pos, e[0], e[1]], (4, 5))
    each(mix.forward, [q, k, v, g, e[0]])
    each(mix.backward, [v, q, k, v, g, *e])
    each(mix.step, [q, k, v, g, state, e[0]])


def test_gains_gradients_at_far_addresses(dm):
    """Tokens so far apart that offsets pass 32 bits give the gains' gradients of the same tokens
    side by side."""
    tokens, heads, d, apart = 300, 2, 64, 1 << 24
    far = torch.empty(tokens * apart, dtype=torch.bfloat16, device="cuda")
    f, pos = rope_reference(d, d), torch.arange(tokens, device="cuda", dtype=torch.int32)
    w, seen = [Draw(50 + i)((d,)) for i in range(2)], []
    for i in range(2):
        draw = Draw(52)
        rows = [draw((tokens, heads, d)) for _ in range(4)]
        to = [torch.empty_like(rows[0]) for _ in range(2)]
        if i == 1:
            place = [far.as_strided((tokens, heads, d), (apart, d, 1), j * heads * d) for j in range(6)]
            rows, to = [p.copy_(r) for p, r in zip(place, rows)], place[4:]
        dw = [torch.full((d,), SENTINEL, dtype=torch.bfloat16, device="cuda") for _ in w]
        dm.QKNormRope(tokens, heads, heads, d).backward(*rows, *w, f, pos, *to, *dw)
        seen.append([x.clone() for x in to] + dw)
    assert all(torch.equal(a, b) for a, b in zip(*seen))
