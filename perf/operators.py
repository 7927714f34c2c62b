"""Measured cases of the training-side operators next to the owner's step.

Five passes, each a user's call (or pair of calls) of one operator:

  ffn_fwd    gated feed-forward block, y = (act(x Wg^T) * (x Wu^T)) Wd^T, keeping
             nothing, or the two projections in bf16 or in 8 bits, for backward
  ffn_bwd    its backward pass: gradients of x and of the three weights, from the
             kept projections
  xent_loss  per-token softmax cross entropy of h W^T against one target per token
             (scoring, evaluation)
  xent_grad  the same with the gradients of h and W (training)
  act8       an activation kept in 8 bits and brought back

``own`` is set by whoever measures: false runs the plain form in elementary fp32
operations, true makes the framework's calls.  Activations, weights and their
gradients are bf16, as the owner's step takes them; losses and log-sum-exps fp32.
"""
import math

import torch

own = False

ACT_BLOCK = 32          # elements that share a scale in an 8-bit activation
IGNORE = -100           # target of a masked token


# ---------------------------------------------------------------- cases
def listed():
    # hidden / ffn / vocab sizes are those of the projection sets in the
    # package's workloads.py: 1536/8960/151936, 3584/18944/152064, 4096/14336/128256
    return [
        # one decoded token: three weight matrices read once, latency counts
        dict(name="ffn decode 1", op="ffn_fwd", tokens=1, hidden=4096, ffn=14336, act="silu",
             save="none"),
        # a serving batch of a few dozen streams
        dict(name="ffn serve 37", op="ffn_fwd", tokens=37, hidden=1536, ffn=8960, act="silu",
             save="none"),
        # a ragged micro-batch of a fine-tuning run, 8-bit activations kept
        dict(name="ffn train 515", op="ffn_fwd", tokens=515, hidden=3584, ffn=18944,
             act="gelu_tanh", save="act8"),
        # a full training micro-batch
        dict(name="ffn train 8192", op="ffn_fwd", tokens=8192, hidden=4096, ffn=14336, act="silu",
             save="bf16"),
        # backward of a small ragged micro-batch: writing the weight gradients dominates
        dict(name="ffn back 301", op="ffn_bwd", tokens=301, hidden=1536, ffn=8960, act="silu",
             save="bf16"),
        # backward of the full micro-batch from 8-bit activations
        dict(name="ffn back 8192", op="ffn_bwd", tokens=8192, hidden=4096, ffn=14336, act="silu",
             save="act8"),
        # log-probability of one token
        dict(name="loss 1", op="xent_loss", tokens=1, hidden=4096, vocab=128256),
        # scoring a ragged evaluation batch
        dict(name="loss 777", op="xent_loss", tokens=777, hidden=3584, vocab=152064),
        # loss and gradients of a short answer in a fine-tuning run
        dict(name="loss+grad 129", op="xent_grad", tokens=129, hidden=1536, vocab=151936),
        # loss and gradients of a training micro-batch
        dict(name="loss+grad 4096", op="xent_grad", tokens=4096, hidden=4096, vocab=128256),
        # one token's activation
        dict(name="act8 1", op="act8", tokens=1, cols=4096),
        # a micro-batch's feed-forward activation
        dict(name="act8 8192", op="act8", tokens=8192, cols=14336),
    ]


_MOST_FLOPS = 6 * 4096 * 4096 * 128256      # the largest listed case


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn_fwd", "ffn_fwd", "ffn_bwd", "xent_loss", "xent_grad", "act8"])
    tokens = _log_int(rng, 1, 8192)
    if op == "act8":
        return dict(op=op, tokens=tokens,
                    cols=rng.choice([1536, 3584, 4096, 8960, 14336, _log_int(rng, 33, 14336)]))
    if op in ("ffn_fwd", "ffn_bwd"):
        hidden, ffn = rng.choice([(1536, 8960), (3584, 18944), (4096, 14336),
                                  (_log_int(rng, 64, 4096), _log_int(rng, 128, 14336))])
        return dict(op=op, tokens=tokens, hidden=hidden, ffn=ffn,
                    act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]),
                    save=rng.choice(["none", "bf16", "act8"] if op == "ffn_fwd" else
                                    ["bf16", "act8"]))
    hidden, vocab = rng.choice([(1536, 151936), (3584, 152064), (4096, 128256),
                                (_log_int(rng, 64, 4096), _log_int(rng, 1000, 150000))])
    tokens = max(1, min(tokens, _MOST_FLOPS // (6 * hidden * vocab)))
    return dict(op=op, tokens=tokens, hidden=hidden, vocab=vocab)


def work(case):
    """Bytes: every input read once, every output written once (an 8-bit
    activation costs 1 + 2/32 bytes an element).  Flops: the matrix products."""
    t, act8 = case["tokens"], 1 + 2 / ACT_BLOCK
    if case["op"] == "act8":
        n = t * case["cols"]
        return {"bytes": n * (4 + 2 * act8), "flops": 0}
    d = case["hidden"]
    if case["op"].startswith("ffn"):
        f = case["ffn"]
        kept = {"none": 0, "bf16": 2, "act8": act8}[case["save"]] * 2 * t * f
        if case["op"] == "ffn_fwd":
            return {"bytes": 4 * t * d + 6 * d * f + kept, "flops": 6 * t * d * f}
        return {"bytes": 6 * t * d + 12 * d * f + kept, "flops": 12 * t * d * f}
    v = case["vocab"]
    if case["op"] == "xent_loss":
        return {"bytes": 2 * t * d + 2 * v * d + 16 * t, "flops": 2 * t * d * v}
    return {"bytes": 4 * t * d + 4 * v * d + 20 * t, "flops": 6 * t * d * v}


# ---------------------------------------------------------------- inputs
def _normal(gen, shape, std, dtype=torch.bfloat16):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return t.mul_(std).to(dtype)


def _channels(gen, tokens, cols):
    """A normalised activation: unit rows times a per-channel gain, with a few
    channels tens of times larger than the rest, as trained models have."""
    gain = torch.rand(cols, generator=gen, device="cuda").mul_(1.5).add_(0.25)
    big = torch.rand(cols, generator=gen, device="cuda") < 0.003
    gain = torch.where(big, gain * 20, gain)
    x = torch.randn((tokens, cols), generator=gen, device="cuda", dtype=torch.float32)
    return x.mul_(gain).to(torch.bfloat16)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    t, s = case["tokens"], {}
    if case["op"] == "act8":
        s["x"] = _channels(gen, t, case["cols"])
        return s
    d = case["hidden"]
    if case["op"].startswith("ffn"):
        f = case["ffn"]
        s["x"] = _normal(gen, (t, d), 1.0)
        s["w_gate"] = _normal(gen, (f, d), 0.02)
        s["w_up"] = _normal(gen, (f, d), 0.02)
        s["w_down"] = _normal(gen, (d, f), 0.02)
        if case["op"] == "ffn_bwd":
            s["dy"] = _normal(gen, (t, d), 1e-3)
            # the kept projections have the spread that x Wg^T and x Wu^T have
            for name in ("gate", "up"):
                p = _normal(gen, (t, f), 0.02 * math.sqrt(d))
                if case["save"] == "act8":
                    codes, scales = _codes(p.float())
                    s[name], s[name + "_scale"] = codes.to(torch.int8), scales.to(torch.bfloat16)
                else:
                    s[name] = p
        return s
    v = case["vocab"]
    s["weight"] = _normal(gen, (v, d), 0.02)
    # frequent tokens are frequent targets; some tokens are masked; the model is
    # sure of some answers, which pulls their hidden state towards the target's row
    u = torch.rand(t, generator=gen, device="cuda")
    target = (float(v) ** u - 1).long().clamp_(0, v - 1)
    sure = torch.rand(t, generator=gen, device="cuda").mul_(20.0)
    h = torch.randn((t, d), generator=gen, device="cuda", dtype=torch.float32)
    rows = s["weight"][target].float()
    h += rows * (sure / rows.square().sum(1).clamp_min(1e-6)).unsqueeze(1)
    s["hidden"] = h.to(torch.bfloat16)
    masked = torch.rand(t, generator=gen, device="cuda") < 0.06
    masked[0] = False
    s["target"] = torch.where(masked, torch.full_like(target, IGNORE), target)
    n = int((~masked).sum())
    s["grad_loss"] = torch.full((t,), 1.0 / n, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    if own:
        _keep(s)
    return s


def _keep(s):
    """What a program keeps between calls: the operator's handle (its workspace)
    and the tensors that receive results."""
    from newton_schulz_owner_gb300 import dmuon

    c = s["case"]
    if c["op"] == "act8":
        s["kept"] = dmuon.act8_empty(c["tokens"], c["cols"])
        s["out"] = torch.empty_like(s["x"])
        return
    if c["op"].startswith("ffn"):
        act = {"silu": dmuon.ACT_SILU, "gelu": dmuon.ACT_GELU,
               "gelu_tanh": dmuon.ACT_GELU_TANH}[c["act"]]
        save = {"none": dmuon.SAVE_NONE, "bf16": dmuon.SAVE_BF16,
                "act8": dmuon.SAVE_ACT8}[c["save"]]
        s["op"] = dmuon.GatedFFN(c["tokens"], c["hidden"], c["ffn"], activation=act, save=save)
        if c["op"] == "ffn_fwd":
            s["y"] = torch.empty_like(s["x"])
            s["saved"] = s["op"].empty_saved(c["tokens"])
            if c["save"] == "act8":
                s["values"] = [torch.empty((c["tokens"], c["ffn"]), dtype=torch.bfloat16,
                                           device="cuda") for _ in range(2)]
        else:
            s["saved"] = ((s["gate"], s["up"]) if c["save"] == "bf16" else
                          (s["gate"], s["gate_scale"], s["up"], s["up_scale"]))
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = [torch.empty_like(s[k]) for k in ("w_gate", "w_up", "w_down")]
        return
    grads = c["op"] == "xent_grad"
    s["op"] = dmuon.LinearXent(c["tokens"], c["hidden"], c["vocab"], grads=grads)
    s["loss"] = torch.empty(c["tokens"], device="cuda")
    s["lse"] = torch.empty(c["tokens"], device="cuda")
    if grads:
        s["dhidden"] = torch.empty_like(s["hidden"])
        s["dweight"] = torch.empty_like(s["weight"])


# ---------------------------------------------------------------- the passes
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from newton_schulz_owner_gb300 import dmuon

    op = s["case"]["op"]
    if op == "act8":
        codes, scales = s["kept"]
        dmuon.act8_save(s["x"], codes, scales)
        dmuon.act8_load(codes, scales, s["out"])
        return {"x": s["out"]}
    if op == "ffn_fwd":
        s["op"].forward(s["x"], s["w_gate"], s["w_up"], s["w_down"], s["y"], s["saved"])
        if s["case"]["save"] == "none":
            return {"y": s["y"]}
        if s["case"]["save"] == "bf16":
            return {"y": s["y"], "gate": s["saved"][0], "up": s["saved"][1]}
        dmuon.act8_load(s["saved"][0], s["saved"][1], s["values"][0])
        dmuon.act8_load(s["saved"][2], s["saved"][3], s["values"][1])
        return {"y": s["y"], "gate": s["values"][0], "up": s["values"][1]}
    if op == "ffn_bwd":
        s["op"].backward(s["dy"], s["x"], s["w_gate"], s["w_up"], s["w_down"], s["saved"],
                         s["dx"], *s["dw"])
        return {"dx": s["dx"], "dw_gate": s["dw"][0], "dw_up": s["dw"][1], "dw_down": s["dw"][2]}
    if op == "xent_loss":
        s["op"].loss(s["hidden"], s["weight"], s["target"], s["loss"], s["lse"])
        return {"loss": s["loss"], "lse": s["lse"]}
    s["op"].loss_and_grads(s["hidden"], s["weight"], s["target"], s["grad_loss"], s["loss"],
                           s["lse"], s["dhidden"], s["dweight"])
    return {"loss": s["loss"], "lse": s["lse"], "dhidden": s["dhidden"], "dweight": s["dweight"]}


def _blocks(v):
    """(rows, blocks, ACT_BLOCK) view of v, its columns padded with zeros."""
    pad = -v.shape[1] % ACT_BLOCK
    if pad:
        v = torch.nn.functional.pad(v, (0, pad))
    return v.reshape(v.shape[0], -1, ACT_BLOCK)


def _codes(v):
    """8-bit codes and block scales of fp32 values: the scale is the smallest bf16
    number >= max|v| / 127 (at least 2^-126), the code the nearest integer to v / scale."""
    b = _blocks(v)
    top = b.abs().amax(dim=2)
    bits = (top / 127.0).clamp_min(2.0 ** -126).view(torch.int32)
    scale = ((bits + 0xFFFF) & -0x10000).view(torch.float32)
    scale = torch.where(top == 0, torch.zeros_like(scale), scale)
    safe = torch.where(top == 0, torch.ones_like(scale), scale)
    codes = torch.round(b / safe.unsqueeze(2))
    return codes.reshape(v.shape[0], -1)[:, :v.shape[1]].contiguous(), scale


def _values(codes, scale):
    b = _blocks(codes.float()) * scale.float().unsqueeze(2)
    return b.reshape(codes.shape[0], -1)[:, :codes.shape[1]]


def _act(kind, g):
    """act(g) and its derivative."""
    if kind == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return g * sg, sg * (1 + g * (1 - sg))
    if kind == "gelu":
        phi = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    th = torch.tanh(k * (g + 0.044715 * g * g * g))
    return (0.5 * g * (1 + th),
            0.5 * (1 + th) + 0.5 * g * (1 - th * th) * k * (1 + 3 * 0.044715 * g * g))


def _run_plain(s):
    c, bf = s["case"], torch.bfloat16
    if c["op"] == "act8":
        return {"x": _values(*_codes(s["x"].float())).to(bf)}
    if c["op"] == "ffn_fwd":
        x = s["x"].float()
        g, u = x @ s["w_gate"].float().t(), x @ s["w_up"].float().t()
        out = {"y": ((_act(c["act"], g)[0] * u) @ s["w_down"].float().t()).to(bf)}
        if c["save"] == "bf16":
            out["gate"], out["up"] = g.to(bf), u.to(bf)
        elif c["save"] == "act8":
            out["gate"], out["up"] = _values(*_codes(g)).to(bf), _values(*_codes(u)).to(bf)
        return out
    if c["op"] == "ffn_bwd":
        x, dy = s["x"].float(), s["dy"].float()
        if c["save"] == "act8":
            g, u = _values(s["gate"], s["gate_scale"]), _values(s["up"], s["up_scale"])
        else:
            g, u = s["gate"].float(), s["up"].float()
        a, da = _act(c["act"], g)
        dh = dy @ s["w_down"].float()
        dg, du = dh * u * da, dh * a
        return {"dx": (dg @ s["w_gate"].float() + du @ s["w_up"].float()).to(bf),
                "dw_gate": (dg.t() @ x).to(bf), "dw_up": (du.t() @ x).to(bf),
                "dw_down": (dy.t() @ (a * u)).to(bf)}
    h, w, target = s["hidden"].float(), s["weight"].float(), s["target"]
    valid = (target >= 0) & (target < w.shape[0])
    at = torch.where(valid, target, torch.zeros_like(target)).unsqueeze(1)
    z = h @ w.t()
    zt = z.gather(1, at).squeeze(1)
    top = z.amax(dim=1, keepdim=True)
    z.sub_(top).exp_()
    total = z.sum(dim=1)
    lse = torch.log(total) + top.squeeze(1)
    zero = torch.zeros_like(lse)
    out = {"loss": torch.where(valid, lse - zt, zero), "lse": torch.where(valid, lse, zero)}
    if c["op"] == "xent_loss":
        return out
    gl = torch.where(valid, s["grad_loss"], zero)
    z.mul_((gl / total).unsqueeze(1))
    z.scatter_add_(1, at, -gl.unsqueeze(1))
    out["dhidden"] = (z @ w).to(bf)
    out["dweight"] = (z.t() @ torch.where(valid.unsqueeze(1), h, torch.zeros_like(h))).to(bf)
    return out


# ---------------------------------------------------------------- in 64 bits
def _exact_round_trip(v):
    r, n = v.shape
    width = -(-n // ACT_BLOCK) * ACT_BLOCK
    b = torch.zeros((r, width), dtype=torch.float64, device=v.device)
    b[:, :n] = v
    b = b.view(r, width // ACT_BLOCK, ACT_BLOCK)
    peak = b.abs().max(dim=2, keepdim=True).values
    mant, expo = torch.frexp((peak / 127).clamp(min=2.0 ** -126))
    scale = torch.ldexp(torch.ceil(mant * 256) / 256, expo)
    codes = torch.where(peak > 0, torch.round(b / scale), torch.zeros_like(b))
    return (codes * scale).view(r, width)[:, :n].contiguous()


def exact(case, seed):
    """The outputs of run() for these inputs in 64 bits, straight from the formulas."""
    s = _inputs(case, seed)
    t, op = case["tokens"], case["op"]
    if op == "act8":
        return {"x": _exact_round_trip(s["x"].double())}
    if op in ("ffn_fwd", "ffn_bwd"):
        x, wg, wu, wd = (s[k].double() for k in ("x", "w_gate", "w_up", "w_down"))
        if op == "ffn_fwd":
            gate, up = torch.mm(x, wg.T), torch.mm(x, wu.T)
        elif case["save"] == "bf16":
            gate, up = s["gate"].double(), s["up"].double()
        else:
            gate, up = (
                s[k].double() * s[k + "_scale"].double().repeat_interleave(ACT_BLOCK, 1)[:, :case["ffn"]]
                for k in ("gate", "up"))
        if case["act"] == "silu":
            slope = torch.sigmoid(gate)
            dact = slope + gate * slope * (1 - slope)
        elif case["act"] == "gelu":
            slope = torch.special.ndtr(gate)
            dact = slope + gate * torch.exp(-gate ** 2 / 2) / math.sqrt(2 * math.pi)
        else:
            inner = math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)
            slope = torch.sigmoid(2 * inner)
            dact = slope + gate * 2 * slope * (1 - slope) * math.sqrt(2 / math.pi) * (
                1 + 0.134145 * gate ** 2)
        act = gate * slope
        if op == "ffn_fwd":
            out = {"y": torch.mm(act * up, wd.T)}
            if case["save"] == "bf16":
                out.update(gate=gate, up=up)
            elif case["save"] == "act8":
                out.update(gate=_exact_round_trip(gate), up=_exact_round_trip(up))
            return out
        dy = s["dy"].double()
        dprod = torch.mm(dy, wd)
        dgate, dup = dprod * up * dact, dprod * act
        return {"dx": torch.mm(dgate, wg) + torch.mm(dup, wu), "dw_gate": torch.mm(dgate.T, x),
                "dw_up": torch.mm(dup.T, x), "dw_down": torch.mm(dy.T, act * up)}
    h, w, target = s["hidden"].double(), s["weight"].double(), s["target"]
    keep = torch.nonzero((target >= 0) & (target < case["vocab"])).squeeze(1)
    h, target = h[keep], target[keep]
    logp = torch.mm(h, w.T)
    norm = torch.logsumexp(logp, dim=1)
    logp -= norm[:, None]
    row = torch.arange(len(keep), device="cuda")
    out = {k: torch.zeros(t, dtype=torch.float64, device="cuda") for k in ("loss", "lse")}
    out["loss"][keep] = -logp[row, target]
    out["lse"][keep] = norm
    if op == "xent_loss":
        return out
    p = logp.exp_()
    p[row, target] -= 1
    p *= s["grad_loss"].double()[keep][:, None]
    out["dhidden"] = torch.zeros((t, case["hidden"]), dtype=torch.float64, device="cuda")
    out["dhidden"][keep] = torch.mm(p, w)
    out["dweight"] = torch.mm(p.T, h)
    return out
