"""Host-side tests of the C ABI of the operators that mix tokens: workspace sizes, and bad
arguments refused before anything touches a GPU (addresses here are never read)."""
import ctypes
import itertools

import pytest
import torch


@pytest.fixture(scope="module")
def dm():
    import os
    from newton_schulz_owner_gb300 import build_lib
    if not os.path.exists(build_lib.LIB):
        build_lib.build()
    from newton_schulz_owner_gb300 import dmuon
    return dmuon


P, W = 1 << 30, 1 << 40          # tensors lie GAP bytes apart
GAP = 1 << 28


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


def place(i, ts=256, hs=64, off=0):
    return Heads(P + i * GAP + off, ts, hs)


def ref(h):
    return None if h is None else ctypes.byref(h)


# Past the argument checks a call asks for the device: without one that is no argument error.
ARGUMENT = {-1, -2, -3}


def qk(dm, shape=(4, 4, 4, 64, 64, 0, 1e-6), q=0, k=1, f=W, pos=W, out=(2, 3), w=(W, W)):
    h = [place(x) if isinstance(x, int) else x for x in (q, k, *out)]
    return dm.lib().dmuon_qk_norm_rope(ctypes.byref(dm.QkShape(*shape)), ref(h[0]), ref(h[1]), *w, f,
                                       pos, ref(h[2]), ref(h[3]), None)


def qk_back(dm, shape=(4, 4, 4, 64, 64, 0, 1e-6), t=(0, 1, 2, 3, 4, 5), f=W, pos=W, w=(W, W),
            dw=(W, W), ws=W, nb=0):
    h = [place(x) if isinstance(x, int) else x for x in t]
    s = dm.QkShape(*shape)
    need = dm.lib().dmuon_qk_norm_rope_workspace_bytes(ctypes.byref(s))
    return dm.lib().dmuon_qk_norm_rope_backward(ctypes.byref(s), *(ref(x) for x in h[:4]), *w, f, pos,
                                                ref(h[4]), ref(h[5]), *dw, ws, need + nb, None)


def test_qk_refuses_bad_arguments(dm):
    bad, al = dm.ERR_INVALID_ARG, dm.ERR_ALIGNMENT
    assert dm.lib().dmuon_qk_norm_rope(None, *[None] * 9) == bad
    for s in [(-1, 4, 4, 64, 64, 0, 0), (4, 0, 4, 64, 64, 0, 0), (4, 4, -1, 64, 64, 0, 0),
              (4, 4, 4, 60, 32, 0, 0), (4, 4, 4, 264, 64, 0, 0), (4, 4, 4, 0, 0, 0, 0),
              (4, 4, 4, 64, 72, 0, 0), (4, 4, 4, 64, 20, 0, 0), (4, 4, 4, 64, -8, 0, 0),
              (4, 4, 4, 64, 64, 0, -1.0), (4, 4, 4, 64, 64, 0, float("nan")),
              (4, 4, 4, 64, 64, 0, float("inf")), ((1 << 22) + 1, 4, 4, 64, 64, 0, 0)]:
        assert qk(dm, shape=s) == bad, s
        assert dm.lib().dmuon_qk_norm_rope_workspace_bytes(ctypes.byref(dm.QkShape(*s))) == 0, s
        assert qk_back(dm, shape=s) == bad, s
    assert qk(dm) not in ARGUMENT
    assert qk(dm, q=None) == bad and qk(dm, k=None) == bad and qk(dm, out=(2, None)) == bad
    assert qk(dm, shape=(4, 4, 0, 64, 64, 0, 0), k=None, out=(2, None)) not in ARGUMENT
    assert qk(dm, f=None) == bad and qk(dm, pos=None) == bad
    assert qk(dm, shape=(4, 4, 4, 64, 0, 0, 0), f=None, pos=None) not in ARGUMENT
    assert qk(dm, q=place(0, 255)) == bad and qk(dm, q=place(0, 256, 63)) == bad
    assert qk(dm, q=place(0, 64, 128)) == bad                       # tokens inside the heads' span
    assert qk(dm, q=place(0, 64, 256)) not in ARGUMENT              # head after head
    assert qk(dm, q=place(0, 0, 64)) == bad and qk(dm, q=place(0, 256, 0)) == bad
    assert qk(dm, q=place(0, off=1)) == al and qk(dm, out=(place(2, off=1), 3)) == al
    assert qk(dm, q=place(0, off=2)) not in ARGUMENT                # slow, but taken
    assert qk(dm, w=(W + 1, W)) == al and qk(dm, f=W + 2) == al and qk(dm, pos=W + 1) == al
    assert qk(dm, shape=(0, 4, 4, 64, 64, 0, 0), q=None, k=None, out=(None, None), pos=None) == dm.OK
    # outputs: their own input, or apart
    assert qk(dm, out=(0, 1)) not in ARGUMENT
    assert qk(dm, out=(1, 0)) == bad and qk(dm, out=(2, 2)) == bad and qk(dm, out=(0, 0)) == bad
    assert qk(dm, out=(place(0, off=64), 3)) == bad


def test_qk_backward_refuses_bad_arguments(dm):
    bad, al = dm.ERR_INVALID_ARG, dm.ERR_ALIGNMENT
    assert qk_back(dm) not in ARGUMENT and qk_back(dm, dw=(None, None)) not in ARGUMENT
    for i in range(6):
        t = [0, 1, 2, 3, 4, 5]
        t[i] = None
        assert qk_back(dm, t=t) == bad, i
        t[i] = place(i, off=1)
        assert qk_back(dm, t=t) == al, i
    assert qk_back(dm, ws=None) == bad and qk_back(dm, ws=W + 16) == al
    assert qk_back(dm, nb=-1) == dm.ERR_WORKSPACE and qk_back(dm, dw=(W + 1, W)) == al
    assert qk_back(dm, t=(0, 1, 2, 3, 0, 1)) not in ARGUMENT        # over the gradients they come from
    assert qk_back(dm, t=(0, 1, 2, 3, 2, 5)) == bad                 # q is read again for nothing else,
    assert qk_back(dm, t=(0, 1, 2, 3, 1, 0)) == bad                 # but one rule is easier to keep
    assert qk_back(dm, t=(0, 1, 2, 3, 4, 4)) == bad


def lin(dm, shape=(4, 1, 4, 64, 64, 0.5), t=(0, 1, 2, 3), g=W, off=None, st=None, fin=None, ws=W, nb=0):
    h = [place(x) if isinstance(x, int) else x for x in t]
    s = dm.LinattnShape(*shape)
    need = dm.lib().dmuon_linattn_workspace_bytes(ctypes.byref(s), 0)
    return dm.lib().dmuon_linattn_forward(ctypes.byref(s), *(ref(x) for x in h[:3]), g, off, st, fin,
                                          ref(h[3]), ws, need + nb, None)


def lin_back(dm, shape=(4, 1, 4, 64, 64, 0.5), t=(0, 1, 2, 3, 4, 5, 6), g=W, off=None, st=None, dfin=None,
             dst=None, ws=W, nb=0):
    h = [place(x) if isinstance(x, int) else x for x in t]
    s = dm.LinattnShape(*shape)
    need = dm.lib().dmuon_linattn_workspace_bytes(ctypes.byref(s), 1)
    return dm.lib().dmuon_linattn_backward(ctypes.byref(s), *(ref(x) for x in h[:4]), g, off, st, dfin,
                                           *(ref(x) for x in h[4:]), dst, ws, need + nb, None)


BAD_SHAPES = [(-1, 1, 4, 64, 64, 0.5), (4, 0, 4, 64, 64, 0.5), (4, 1, 0, 64, 64, 0.5),
              (4, 1, 4, 60, 64, 0.5), (4, 1, 4, 64, 4, 0.5), (4, 1, 4, 136, 64, 0.5),
              (4, 1, 4, 64, 136, 0.5), (4, 1, 4, 0, 64, 0.5), (4, 1, 4, 64, 64, 0.0),
              (4, 1, 4, 64, 64, float("nan")), (4, 1, 4, 64, 64, float("inf")),
              ((1 << 22) + 1, 1, 4, 64, 64, 0.5), (4, (1 << 16) + 1, 4, 64, 64, 0.5),
              (4, 1, (1 << 16) + 1, 64, 64, 0.5), (4, 1 << 16, 1 << 16, 64, 64, 0.5)]


def test_linattn_refuses_bad_arguments(dm):
    bad, al = dm.ERR_INVALID_ARG, dm.ERR_ALIGNMENT
    for s in BAD_SHAPES:
        assert dm.lib().dmuon_linattn_workspace_bytes(ctypes.byref(dm.LinattnShape(*s)), 1) == 0, s
        assert lin(dm, shape=s) == bad and lin_back(dm, shape=s) == bad, s
    assert dm.lib().dmuon_linattn_workspace_bytes(None, 0) == 0
    assert lin(dm) not in ARGUMENT and lin_back(dm) not in ARGUMENT
    for call, n in ((lin, 4), (lin_back, 7)):
        for i in range(n):
            t = list(range(n))
            t[i] = None
            assert call(dm, t=t) == bad, i
            for off in (2, 8):
                t[i] = place(i, off=off)
                assert call(dm, t=t) == al, i
            t[i] = place(i, 260)
            assert call(dm, t=t) == al, i
            t[i] = place(i, 0)
            assert call(dm, t=t) == bad, i                          # broadcast along tokens
            t[i] = place(i, 256, 0)
            assert call(dm, t=t) == bad, i                          # and along heads
        assert call(dm, g=None) == bad and call(dm, ws=None) == bad and call(dm, g=W + 2) == al
        assert call(dm, ws=W + 128) == al and call(dm, nb=-1) == dm.ERR_WORKSPACE
        assert call(dm, shape=(4, 2, 4, 64, 64, 0.5)) == bad        # sequences without offsets
        assert call(dm, shape=(4, 2, 4, 64, 64, 0.5), off=W) not in ARGUMENT
        assert call(dm, off=W + 2) == al and call(dm, st=W + 4) == al
    assert lin(dm, fin=W + 8) == al and lin_back(dm, dfin=W + 8) == al and lin_back(dm, dst=W + 8) == al
    empty = (0, 1, 4, 64, 64, 0.5)
    assert lin(dm, shape=empty, t=[None] * 4) == dm.OK and lin_back(dm, shape=empty, t=[None] * 7) == dm.OK
    for i in range(3):
        assert lin(dm, t=(0, 1, 2, i)) == bad
    for i, j in itertools.product(range(4, 7), range(7)):
        t = list(range(7))
        if i != j:
            t[i] = j
            assert lin_back(dm, t=t) == bad, (i, j)


def test_step_refuses_bad_arguments(dm):
    bad, al = dm.ERR_INVALID_ARG, dm.ERR_ALIGNMENT

    def step(shape=(4, 1, 4, 64, 64, 0.5), t=(0, 1, 2, 3), g=W, slot=None, slots=4, st=W, new=W):
        h = [place(x) if isinstance(x, int) else x for x in t]
        return dm.lib().dmuon_linattn_step(ctypes.byref(dm.LinattnShape(*shape)), ref(h[0]), ref(h[1]),
                                           ref(h[2]), g, slot, slots, st, new, ref(h[3]), None)

    for s in BAD_SHAPES:
        assert step(shape=s) == bad, s
    assert step() not in ARGUMENT
    for i in range(4):
        t = [0, 1, 2, 3]
        t[i] = None
        assert step(t=t) == bad
        t[i] = place(i, off=1)
        assert step(t=t) == al
        t[i] = place(i, off=2)
        assert step(t=t) not in ARGUMENT
        t[i] = place(i, 0)
        assert step(t=t) == bad
    assert step(g=None) == bad and step(st=None) == bad and step(new=None) == bad
    assert step(slots=3) == bad and step(slots=3, slot=W) not in ARGUMENT and step(slots=-1, slot=W) == bad
    assert step(st=W + 4) == al and step(new=W + 8) == al and step(slot=W + 2) == al and step(g=W + 1) == al
    state = 4 * 4 * 64 * 64 * 4
    assert step(new=W + 16) == bad and step(new=W + state - 16) == bad and step(new=W + state) not in ARGUMENT
    assert step(t=(0, 1, 2, 0)) == bad
    assert step(shape=(0, 1, 4, 64, 64, 0.5), t=[None] * 4, st=None, new=None) == dm.OK
    assert step(shape=(1 << 22, 1, 1 << 12, 64, 64, 0.5), t=[place(i << 14, 1 << 18) for i in range(4)],
                slots=1 << 22, new=1 << 60) == dm.ERR_UNSUPPORTED


def test_states_lie_apart_from_what_is_written(dm):
    """States that are written may be the ones read, or lie apart from them and from every tensor."""
    bad = dm.ERR_INVALID_ARG
    n = 4 * 64 * 64 * 4                    # bytes of a sequence's states; tensors take 2048 here
    assert lin(dm, st=W, fin=W) not in ARGUMENT and lin_back(dm, dfin=W, dst=W) not in ARGUMENT
    for off in (16, n - 16, 16 - n):
        assert lin(dm, st=W, fin=W + off) == bad and lin_back(dm, dfin=W, dst=W + off) == bad
        # dstate is written after the last read of state
        assert lin_back(dm, st=W, dst=W + off) not in ARGUMENT
    empty = (0, 1, 4, 64, 64, 0.5)
    assert lin(dm, shape=empty, t=[None] * 4, st=W, fin=W + 16) == bad
    for off in (n, -n):
        assert lin(dm, st=W, fin=W + off) not in ARGUMENT
        assert lin_back(dm, dfin=W, dst=W + off) not in ARGUMENT
    for off in (0, 1024, 16 - n, 2032):
        for i in range(4):
            assert lin(dm, fin=P + i * GAP + off) == bad
            assert (lin(dm, st=P + i * GAP + off) == bad) == (i == 3)
        for i in range(7):
            assert lin_back(dm, dst=P + i * GAP + off) == bad
            assert (lin_back(dm, dfin=P + i * GAP + off) == bad) == (i > 3)
            assert (lin_back(dm, st=P + i * GAP + off) == bad) == (i > 3)
    for off in (2048, -n):
        assert lin(dm, fin=P + 3 * GAP + off) not in ARGUMENT
        assert lin_back(dm, dst=P + 6 * GAP + off) not in ARGUMENT


def test_step_states_lie_apart_from_what_is_written(dm):
    n = 4 * 4 * 64 * 64 * 4

    def step(st, new):
        h = [place(i) for i in range(4)]
        return dm.lib().dmuon_linattn_step(ctypes.byref(dm.LinattnShape(4, 1, 4, 64, 64, 0.5)),
                                           *(ref(x) for x in h[:3]), W, None, 4, st, new, ref(h[3]), None)

    for off in (0, 1024, 16 - n, 2032):
        for i in range(4):
            assert step(W, P + i * GAP + off) == dm.ERR_INVALID_ARG
            assert (step(P + i * GAP + off, W) == dm.ERR_INVALID_ARG) == (i == 3)
    for off in (2048, -n):
        assert step(P + 3 * GAP + off, P + 3 * GAP + off) not in ARGUMENT


def test_scales_whose_inverse_overflows_are_refused(dm):
    """The gradients' sweeps take the final states' gradient divided by the scale."""
    for scale, ok in ((1e-38, True), (-1e-38, True), (3e38, True), (2e-39, False), (1e-45, False)):
        s = (4, 1, 4, 64, 64, scale)
        assert (dm.lib().dmuon_linattn_workspace_bytes(ctypes.byref(dm.LinattnShape(*s)), 1) > 0) == ok
        assert (lin(dm, shape=s) == dm.ERR_INVALID_ARG) == (not ok)


def test_workspaces_stay_bounded(dm):
    """Sequences are shared among CTAs only where there are few of them."""
    one = lambda *s: dm.lib().dmuon_linattn_workspace_bytes(ctypes.byref(dm.LinattnShape(*s)), 1)
    assert 0 < one(1 << 20, 1, 1, 128, 128, 1.0) < one(1 << 20, 1, 32, 128, 128, 1.0) < 1 << 26
    assert one(1 << 20, 1 << 16, 64, 128, 128, 1.0) < 1 << 26


def test_overlap_is_found_as_element_sets_have_it(dm):
    """A step's output against its query, both parts of one buffer, at every distance: refused
    exactly where they share an element."""
    for tokens, heads, ts, hs in [(3, 2, 40, 16), (3, 2, 16, 48), (1, 2, 0, 24), (2, 1, 24, 0),
                                  (4, 3, 56, 16), (2, 3, 8, 16)]:
        cells = {t * ts + h * hs + x for t in range(tokens) for h in range(heads) for x in range(8)}
        for apart in range(-220, 221, 4):
            h = [Heads(P + GAP + i, ts, hs) for i in (0, GAP, 2 * GAP, 2 * apart)]
            s = dm.LinattnShape(tokens, 1, heads, 8, 8, 1.0)
            got = dm.lib().dmuon_linattn_step(ctypes.byref(s), ref(h[0]), ref(h[1]), ref(h[2]), W, None,
                                              tokens, W, W, ref(h[3]), None)
            share = any(c + apart in cells for c in cells)
            assert (got == dm.ERR_INVALID_ARG) == share, (tokens, heads, ts, hs, apart)


def test_overlap_of_unequal_head_sizes_is_found_as_element_sets_have_it(dm):
    """The same with keys wider or narrower than values, the output against the query (and the query
    against the output: the one that lies first changes with the sign of the distance) and, for
    gradients, those of queries and values against one another."""
    for tokens, heads, ts, hs in [(1, 1, 0, 0), (3, 1, 40, 0), (3, 1, 24, 0), (1, 2, 0, 32),
                                  (3, 2, 72, 24), (3, 2, 24, 80)]:
        for dk, dv in [(8, 24), (24, 8), (16, 24), (24, 16)]:
            def cells(d):
                return {t * ts + h * hs + x for t in range(tokens) for h in range(heads) for x in range(d)}
            s = dm.LinattnShape(tokens, 1, heads, dk, dv, 1.0)
            need = dm.lib().dmuon_linattn_workspace_bytes(ctypes.byref(s), 1)
            for apart in range(-240, 241, 8):
                h = [Heads(P + GAP + i, ts, hs) for i in (0, GAP, 2 * GAP, 2 * apart)]
                step = dm.lib().dmuon_linattn_step(ctypes.byref(s), ref(h[0]), ref(h[1]), ref(h[2]), W, None,
                                                   tokens, W, W, ref(h[3]), None)
                fwd = dm.lib().dmuon_linattn_forward(ctypes.byref(s), ref(h[0]), ref(h[1]), ref(h[2]), W, None,
                                                     None, None, ref(h[3]), W, need, None)
                t = [place(i + 4, ts, hs) for i in range(7)]           # dout, q, k, v, dq, dk, dv
                t[4], t[6] = h[0], h[3]
                back = dm.lib().dmuon_linattn_backward(ctypes.byref(s), *(ref(x) for x in t[:4]), W, None,
                                                       None, None, *(ref(x) for x in t[4:]), None, W, need,
                                                       None)
                at = cells(dk)
                share = any(c + apart in at for c in cells(dv))
                for got in (step, fwd, back):
                    assert (got == dm.ERR_INVALID_ARG) == share, (tokens, heads, ts, hs, dk, dv, apart)


def test_binding_refuses_bad_tensors(dm):
    """Types, shapes, devices and handles, as far as they show without a GPU."""
    with pytest.raises(dm.DMuonError):
        dm.LinearAttention(4, 2, 60, device="cpu")
    with pytest.raises(dm.DMuonError):
        dm.QKNormRope(4, 2, 2, 300, device="cpu")
    op, rope = dm.LinearAttention(4, 2, 64, device="cpu"), dm.QKNormRope(4, 2, 2, 64, device="cpu")
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    g = torch.zeros(2)
    for call in (lambda: op.forward(x, x, x, g, x), lambda: op.step(x, x, x, g, torch.zeros(4, 2, 64, 64), x),
                 lambda: op.backward(x, x, x, x, g, x, x, x),
                 lambda: rope.forward(x, x, None, None, torch.zeros(32), torch.zeros(4).int(), x, x)):
        with pytest.raises(ValueError):       # not on a GPU
            call()
    big = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        op.forward(big, big, big, g, big)
    with pytest.raises(ValueError):
        rope.forward(big, big, None, None, g, g, big, big)
    with pytest.raises(ValueError):
        op.forward(x[0], x, x, g, x)
    with pytest.raises(ValueError):
        dm.LinearAttention(4, 2, 64, backward=False, device="cpu").backward(x, x, x, x, g, x, x, x)
    with pytest.raises(ValueError):
        dm.QKNormRope(4, 2, 2, 64, backward=False, device="cpu").backward(x, x, x, x, None, None, g, g, x, x)


def test_shapes_of_a_call_follow_the_attributes(dm, monkeypatch):
    """A handle keeps the shapes of its last call, and makes new ones once it says something else."""
    monkeypatch.setattr(dm, "_launch_device", lambda t, what: 0)
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    rope, mix = dm.QKNormRope(4, 2, 2, 64, device="cpu"), dm.LinearAttention(4, 2, 64, device="cpu")
    same = rope._begin(q)[1], mix._begin(q)[2]
    assert rope._begin(q)[1] is same[0] and mix._begin(q)[2] is same[1]
    for name, value in (("eps", 0.25), ("interleaved", True), ("rotary_dim", 32), ("head_dim", 32),
                        ("q_heads", 3), ("k_heads", 1)):
        setattr(rope, name, value)
        t, shape, qs, ks, _ = rope._begin(q)
        assert getattr(shape, name) == value and t == 4, name
        assert qs == (4, rope.q_heads, rope.head_dim) and ks == (4, rope.k_heads, rope.head_dim)
    for name, value in (("scale", 0.25), ("key_dim", 32), ("value_dim", 16), ("heads", 3)):
        setattr(mix, name, value)
        t, n, shape, ks, vs, _, _ = mix._begin(q)
        assert getattr(shape, name) == value and (t, n) == (4, 1), name
        assert ks == (4, mix.heads, mix.key_dim) and vs == (4, mix.heads, mix.value_dim)


def test_gradients_of_states_refuse_far_scales(dm):
    """With states' gradients the scale is a factor of operands."""
    for scale, ok in ((2.0 ** -64, True), (-2.0 ** 64, True), (2.0 ** -65, False), (-2.0 ** 65, False),
                      (1e-38, False), (3e38, False)):
        s = (4, 1, 4, 64, 64, scale)
        assert lin_back(dm, shape=s) not in ARGUMENT
        for states in (dict(dfin=W), dict(dst=W), dict(dfin=W, dst=W)):
            assert (lin_back(dm, shape=s, **states) == dm.ERR_UNSUPPORTED) == (not ok), (scale, states)


def test_required_tensors_may_not_be_none(dm, monkeypatch):
    """Every tensor that a call cannot do without is refused by its name."""
    monkeypatch.setattr(dm, "_launch_device", lambda t, what: -1)
    monkeypatch.setattr(dm, "_launch_stream", lambda stream, dev: 0)
    x, g, f, pos = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(2), torch.zeros(32), torch.zeros(4).int()
    rope, mix = dm.QKNormRope(4, 2, 2, 64, device="cpu"), dm.LinearAttention(4, 2, 64, device="cpu")
    calls = [(rope.forward, [("q", x), ("k", x), (None, None), (None, None), ("inv_freq", f), ("position", pos),
                             ("q_out", x), ("k_out", x)]),
             (rope.backward, [("dq_out", x), ("dk_out", x), ("q", x), ("k", x), (None, None), (None, None),
                              ("inv_freq", f), ("position", pos), ("dq", x), ("dk", x)]),
             (mix.forward, [("q", x), ("k", x), ("v", x), ("log_decay", g), ("out", x)]),
             (mix.backward, [("dout", x), ("q", x), ("k", x), ("v", x), ("log_decay", g), ("dq", x), ("dk", x),
                             ("dv", x)]),
             (mix.step, [("q", x), ("k", x), ("v", x), ("log_decay", g), ("state", torch.zeros(4, 2, 64, 64)),
                         ("out", x)])]
    for call, args in calls:
        for i, (name, _) in enumerate(args):
            if name is not None:
                with pytest.raises(TypeError, match=f"^{name}: expected a tensor, got None"):
                    call(*(None if j == i else v for j, (_, v) in enumerate(args)))
