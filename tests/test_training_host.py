"""Host-side tests of the training-side operators' C ABI: workspace sizes, and bad
arguments refused before anything touches a GPU (addresses here are never read)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def dm():
    import os
    from newton_schulz_owner_gb300 import build_lib
    if not os.path.exists(build_lib.LIB):
        build_lib.build()
    from newton_schulz_owner_gb300 import dmuon
    return dmuon


P, W = 1 << 20, 1 << 30


def ffn_bytes(dm, *a, backward=0):
    return dm.lib().dmuon_ffn_workspace_bytes(ctypes.byref(dm.FfnShape(*a)), backward)


def xent_bytes(dm, *a, grads=1):
    return dm.lib().dmuon_xent_workspace_bytes(ctypes.byref(dm.XentShape(*a)), grads)


def test_workspaces_grow_with_tokens_and_refuse_bad_shapes(dm):
    for back in (0, 1):
        sizes = [ffn_bytes(dm, t, 1537, 8961, dm.ACT_SILU, dm.SAVE_BF16, backward=back)
                 for t in (0, 1, 2, 63, 64, 65, 300, 4096, 1 << 22)]
        assert sizes[0] > 0 and sizes == sorted(sizes)
        sizes = [xent_bytes(dm, t, 1537, 151936, grads=back)
                 for t in (0, 1, 255, 256, 257, 7000, 8000, 20000, 1 << 22)]
        assert sizes[0] > 0 and sizes == sorted(sizes)
    # the logits of a long batch are not kept: the workspace stays far below them
    assert xent_bytes(dm, 1 << 17, 4096, 128256) < (1 << 17) * 128256 * 2 / 4
    for bad in [(-1, 8, 8, 0, 1), (1, 0, 8, 0, 1), (1, 8, 0, 0, 1), (1, 8, 8, 3, 1), (1, 8, 8, 0, 3),
                (1, 8, 8, -1, 1), ((1 << 22) + 1, 8, 8, 0, 1), (1, (1 << 19) + 1, 8, 0, 1)]:
        assert ffn_bytes(dm, *bad) == 0, bad
    for bad in [(-1, 8, 8), (1, 0, 8), (1, 8, 0), (1, 8, (1 << 22) + 1), ((1 << 22) + 1, 8, 8)]:
        assert xent_bytes(dm, *bad) == 0, bad
    assert dm.lib().dmuon_ffn_workspace_bytes(None, 0) == 0
    assert dm.lib().dmuon_xent_workspace_bytes(None, 0) == 0


def test_ffn_refuses_bad_arguments(dm):
    lib = dm.lib()
    two = (ctypes.c_void_p * 4)(P, P, P, P)
    hole = (ctypes.c_void_p * 4)(P, None, P, P)

    def fwd(shape=(4, 64, 96, 0, 1), x=P, x_ld=64, wg=P, wu=P, wd=P, y=P, y_ld=64, saved=two, ws=W,
            nb=None):
        s = dm.FfnShape(*shape)
        need = lib.dmuon_ffn_workspace_bytes(ctypes.byref(s), 0)
        return lib.dmuon_ffn_forward(ctypes.byref(s), x, x_ld, wg, wu, wd, y, y_ld, saved, ws,
                                     need if nb is None else need + nb, None)

    def bwd(shape=(4, 64, 96, 0, 1), dy=P, x=P, wg=P, saved=two, dx=P, dx_ld=64, dwg=P, dwd=P, ws=W,
            nb=None):
        s = dm.FfnShape(*shape)
        need = lib.dmuon_ffn_workspace_bytes(ctypes.byref(s), 1)
        return lib.dmuon_ffn_backward(ctypes.byref(s), dy, 64, x, 64, wg, P, P, saved, dx, dx_ld,
                                      dwg, P, dwd, ws, need if nb is None else need + nb, None)

    bad = dm.ERR_INVALID_ARG
    assert lib.dmuon_ffn_forward(None, P, 64, P, P, P, P, 64, two, W, 1 << 40, None) == bad
    assert fwd(shape=(4, 64, 96, 5, 1)) == bad
    assert fwd(shape=(4, 64, 96, 0, 9)) == bad
    assert fwd(shape=(-1, 64, 96, 0, 1)) == bad
    assert fwd(x=None) == bad and fwd(y=None) == bad and fwd(wu=None) == bad and fwd(ws=None) == bad
    assert fwd(x_ld=63) == bad and fwd(y_ld=63) == bad
    assert fwd(saved=None) == bad and fwd(saved=hole) == bad
    assert fwd(wg=P + 2) == dm.ERR_ALIGNMENT and fwd(wd=P + 8) == dm.ERR_ALIGNMENT
    assert fwd(ws=W + 16) == dm.ERR_ALIGNMENT
    odd = (ctypes.c_void_p * 4)(P + 1, P, P, P)
    assert fwd(x=P + 1) == dm.ERR_ALIGNMENT and fwd(y=P + 1) == dm.ERR_ALIGNMENT
    assert fwd(saved=odd) == dm.ERR_ALIGNMENT and bwd(saved=odd) == dm.ERR_ALIGNMENT
    assert fwd(shape=(4, 65, 96, 0, 1), x_ld=65, y_ld=65, wg=P + 1) == dm.ERR_ALIGNMENT
    scale = (ctypes.c_void_p * 4)(P, P + 1, P, P)
    assert fwd(shape=(4, 64, 96, 0, 2), saved=scale) == dm.ERR_ALIGNMENT
    assert bwd(dy=P + 1) == dm.ERR_ALIGNMENT and bwd(dwd=P + 1) == dm.ERR_ALIGNMENT
    assert fwd(nb=-1) == dm.ERR_WORKSPACE
    assert fwd(shape=(0, 64, 96, 0, 0), x=None, y=None) == dm.OK       # no tokens, nothing to do
    assert bwd(shape=(4, 64, 96, 0, 0)) == bad                          # nothing was kept
    assert bwd(dy=None) == bad and bwd(dx=None) == bad and bwd(dwg=None) == bad and bwd(dwd=None) == bad
    assert bwd(dx_ld=10) == bad and bwd(saved=hole) == bad
    assert bwd(wg=P + 2) == dm.ERR_ALIGNMENT
    assert bwd(nb=-1) == dm.ERR_WORKSPACE


def test_xent_refuses_bad_arguments(dm):
    lib = dm.lib()

    def call(shape=(4, 64, 96), h=P, ld=64, w=P, t=P, gl=P, loss=P, lse=P, dh=P, dh_ld=64, dw=P, ws=W,
             nb=None):
        s = dm.XentShape(*shape)
        need = lib.dmuon_xent_workspace_bytes(ctypes.byref(s), 1)
        return lib.dmuon_xent(ctypes.byref(s), h, ld, w, t, gl, loss, lse, dh, dh_ld, dw, ws,
                              need if nb is None else need + nb, None)

    bad = dm.ERR_INVALID_ARG
    assert lib.dmuon_xent(None, P, 64, P, P, P, P, P, P, 64, P, W, 1 << 40, None) == bad
    assert call(shape=(4, 64, 0)) == bad
    for k in ("h", "w", "t", "gl", "loss", "lse", "dh", "dw", "ws"):
        assert call(**{k: None}) == bad, k
    assert call(ld=63) == bad and call(dh_ld=63) == bad
    assert call(w=P + 2) == dm.ERR_ALIGNMENT and call(ws=W + 128) == dm.ERR_ALIGNMENT
    for k, v in {"h": P + 1, "t": P + 4, "gl": P + 2, "loss": P + 2, "lse": P + 1, "dh": P + 1,
                 "dw": P + 1}.items():
        assert call(**{k: v}) == dm.ERR_ALIGNMENT, k
    assert call(nb=-1) == dm.ERR_WORKSPACE
    assert call(shape=(0, 64, 96), gl=None, dh=None, dw=None, h=None) == dm.OK


def test_act8_refuses_bad_arguments(dm):
    lib = dm.lib()
    bad = dm.ERR_INVALID_ARG
    for f, a, b in [(lib.dmuon_act8_save, 2, (3, 3)), (lib.dmuon_act8_load, 4, (3, 3))]:
        save = f is lib.dmuon_act8_save

        def call(rows=3, cols=40, x=P, ld=40, dt=dm.BF16, codes=P, scales=P):
            if save:
                return f(rows, cols, x, ld, dt, codes, scales, None)
            return f(rows, cols, codes, scales, x, ld, dt, None)

        assert call(rows=-1) == bad and call(cols=-1) == bad and call(dt=2) == bad
        assert call(x=None) == bad and call(codes=None) == bad and call(scales=None) == bad
        assert call(ld=39) == bad
        assert call(x=P + 1) == dm.ERR_ALIGNMENT and call(scales=P + 1) == dm.ERR_ALIGNMENT
        assert call(x=P + 2, dt=dm.F32) == dm.ERR_ALIGNMENT
        assert call(rows=1 << 31, cols=2049, ld=2049) == dm.ERR_UNSUPPORTED
        assert call(rows=0, x=None) == dm.OK and call(cols=0, x=None) == dm.OK


def test_binding_refuses_wrong_tensors(dm):
    import torch
    with pytest.raises(TypeError):
        dm._bf16_rows(torch.zeros(2, 3), 2, 3, "x")
    with pytest.raises(ValueError):
        dm._bf16_rows(torch.zeros(2, 3, dtype=torch.bfloat16), 2, 4, "x")
    with pytest.raises(ValueError):      # not on a GPU
        dm._bf16_rows(torch.zeros(2, 3, dtype=torch.bfloat16), 2, 3, "x")
    with pytest.raises(TypeError):
        dm.act8_save(torch.zeros(2, 3, dtype=torch.float16), torch.zeros(2, 3, dtype=torch.int8),
                     torch.zeros(2, 1, dtype=torch.bfloat16))
    with pytest.raises(dm.DMuonError):
        dm.GatedFFN(4, 0, 8, device="cpu")
    with pytest.raises(dm.DMuonError):
        dm.LinearXent(4, 8, 0, device="cpu")
    op = dm.GatedFFN(4, 8, 8, save=dm.SAVE_NONE, device="cpu")
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        op.backward(x, x, x, x, x, (), x, x, x, x)
    with pytest.raises(ValueError):
        op.forward(torch.zeros(5, 8, dtype=torch.bfloat16), x, x, x, x)
    head = dm.LinearXent(4, 8, 8, grads=False, device="cpu")
    with pytest.raises(ValueError):
        head.loss_and_grads(x, x, x, x, x, x, x, x)


def test_binding_refuses_gradients_without_their_tensors(dm):
    """A missing grad_loss is not a call for the loss alone: the gradients would stay as they were."""
    import torch
    head = dm.LinearXent(4, 8, 8, device="cpu")
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    each = torch.zeros(4)
    args = dict(hidden=x, weight=x, target=torch.zeros(4, dtype=torch.int64), grad_loss=each, loss=each,
                lse=each, dhidden=x, dweight=x)
    for name in ("grad_loss", "dhidden", "dweight"):
        with pytest.raises(TypeError, match=name):
            head.loss_and_grads(**{**args, name: None})


class OnDevice:
    """As much of a contiguous CUDA tensor as the binding looks at."""

    is_cuda = True

    def __init__(self, shape, dtype, index):
        import torch
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[1], 1)

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return P


def test_binding_refuses_tensors_on_other_devices(dm, monkeypatch):
    """A launch goes to the current device: the workspace and every tensor have to lie there."""
    import torch
    bf, f32, i8 = torch.bfloat16, torch.float32, torch.int8
    calls = []
    monkeypatch.setattr(dm, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(dm, "_raw_stream", None)
    for name in ("dmuon_ffn_forward", "dmuon_ffn_backward", "dmuon_xent", "dmuon_act8_save",
                 "dmuon_act8_load"):
        monkeypatch.setattr(dm._lib, name, lambda *a, name=name: calls.append(name) or 0)

    block = dm.GatedFFN(4, 8, 16, save=dm.SAVE_ACT8, device="cpu")
    head = dm.LinearXent(4, 8, 32, device="cpu")
    x = lambda: OnDevice((4, 8), bf, 0)
    ws = dict(w_gate=((16, 8), bf), w_up=((16, 8), bf), w_down=((8, 16), bf))
    saved = [OnDevice((4, 16), i8, 0), OnDevice((4, 1), bf, 0)] * 2
    cases = [
        (block.forward, dict(x=x(), y=x(), saved=saved, **{k: OnDevice(*v, 0) for k, v in ws.items()})),
        (block.backward, dict(x=x(), dy=x(), dx=x(), saved=saved,
                              **{k: OnDevice(*v, 0) for k, v in ws.items()},
                              **{"d" + k: OnDevice(*v, 0) for k, v in ws.items()})),
        (head.loss_and_grads, dict(hidden=x(), dhidden=x(), weight=OnDevice((32, 8), bf, 0),
                                   dweight=OnDevice((32, 8), bf, 0),
                                   target=OnDevice((4,), torch.int64, 0),
                                   **{k: OnDevice((4,), f32, 0) for k in ("grad_loss", "loss", "lse")})),
        (dm.act8_save, dict(x=OnDevice((4, 40), bf, 0), codes=OnDevice((4, 40), i8, 0),
                            scales=OnDevice((4, 2), bf, 0))),
        (dm.act8_load, dict(out=OnDevice((4, 40), f32, 0), codes=OnDevice((4, 40), i8, 0),
                            scales=OnDevice((4, 2), bf, 0)))]
    for op in (block, head):
        op.workspace = OnDevice((op.workspace.numel(),), torch.uint8, 0)
    for f, args in cases:
        f(**args, stream=1)
        assert len(calls) == 1 and calls.pop()          # all on the current device: launched
        for name, v in args.items():
            parts = range(4) if name == "saved" else [None]
            for i in parts:
                t = v if i is None else v[i]
                away = OnDevice(t.shape, t.dtype, 1)
                moved = away if i is None else [away if j == i else s for j, s in enumerate(v)]
                with pytest.raises(ValueError, match="cuda:1"):
                    f(**{**args, name: moved}, stream=1)
    for op, (f, args) in ((block, cases[0]), (block, cases[1]), (head, cases[2])):
        here = op.workspace
        op.workspace = OnDevice(here.shape, torch.uint8, 1)
        with pytest.raises(ValueError, match="workspace is on cuda:1"):
            f(**args, stream=1)
        op.workspace = here
    assert not calls


def test_a_workspace_for_gradients_serves_the_loss_alone(dm):
    for t in (1, 300, 1024, 16384, 1 << 18):
        for d in (8, 64, 65, 4096):
            for v in (1, 1000, 151936, 1 << 20, 1 << 22):
                assert xent_bytes(dm, t, d, v, grads=1) >= xent_bytes(dm, t, d, v, grads=0), (t, d, v)


def test_ffn_backward_refuses_dx_over_its_inputs(dm):
    """The weight gradients read x and dy after dx is written (and while it is)."""
    lib, t, d, f = dm.lib(), 4, 64, 96
    at = {n: (i + 2) << 24 for i, n in enumerate(("dy", "x", "dx", "wg", "wu", "wd", "gate", "up", "gg",
                                                  "gu", "gd"))}

    def call(dy_ld=d, x_ld=d, dx_ld=d, shape=(t, d, f, 0, 1), **move):
        a = {**at, **move}
        s = dm.FfnShape(*shape)
        need = lib.dmuon_ffn_workspace_bytes(ctypes.byref(s), 1)
        saved = (ctypes.c_void_p * 4)(a["gate"], a["up"], None, None)
        return lib.dmuon_ffn_backward(ctypes.byref(s), a["dy"], dy_ld, a["x"], x_ld, a["wg"], a["wu"],
                                      a["wd"], saved, a["dx"], dx_ld, a["gg"], a["gu"], a["gd"], W,
                                      need, None)

    import torch
    if torch.cuda.is_available():       # these addresses must not reach one
        pytest.skip("needs a machine without a GPU")
    fine = call()
    assert fine not in (dm.OK, dm.ERR_INVALID_ARG)          # past the checks, and no GPU
    size = t * d * 2
    for name in ("dy", "x"):
        for shift in (0, 2, -2, 16, size - 2, 2 - size):
            assert call(dx=at[name] + shift) == dm.ERR_INVALID_ARG, (name, shift)
        for shift in (size, -size, size + 16):
            assert call(dx=at[name] + shift) == fine, (name, shift)
        # columns side by side in rows of one pitch share nothing
        wide = dict(dy_ld=3 * d, x_ld=3 * d, dx_ld=3 * d)
        for shift in (d, 2 * d, -d, -2 * d):
            assert call(dx=at[name] + 2 * shift, **wide) == fine, (name, shift)
        for shift in (d - 1, 2 * d + 1, 1 - d, 3 * d, -3 * d):
            assert call(dx=at[name] + 2 * shift, **wide) == dm.ERR_INVALID_ARG, (name, shift)
    one = dict(shape=(1, d, f, 0, 1))
    assert call(dx=at["x"] + 2 * d, dx_ld=1 << 20, **one) == fine      # one row has no pitch
    assert call(dx=at["x"] + 2 * d - 2, dx_ld=1 << 20, **one) == dm.ERR_INVALID_ARG
