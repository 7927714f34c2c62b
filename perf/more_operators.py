"""Measured cases of the operators that mix tokens, next to the training-side ones.

Five passes, each a user's call of one operator:

  rope_fwd   root-mean-square norm of every query and key head with a gain per element,
             then the rotation by position, in one pass
  rope_bwd   its backward pass: gradients of the queries, the keys and both gains
  mix_fwd    linear attention with a decay for each head over packed sequences (prompts and
             training micro-batches), from a state and to a state where serving keeps one:
               S_t = exp(log_decay) S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t
  mix_bwd    its backward pass: gradients of queries, keys and values
  mix_step   one token for each of many streams, every one with a state of its own

``own`` is set by whoever measures: false runs the plain form in elementary fp32
operations, true makes the framework's calls.  Activations, gains and gradients are bf16,
states, decays and frequencies fp32.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 500000.0          # of the rotation's frequencies
CHUNK = 128              # tokens that the plain form takes at a time


# ---------------------------------------------------------------- cases
def listed():
    # 12, 28 and 32 heads of 128 are the attention of the projection sets in the package's
    # workloads.py (hidden 1536, 3584, 4096; 2, 4 and 8 key heads)
    return [
        # one decoded token's heads: latency counts
        dict(name="rope decode 1", op="rope_fwd", tokens=1, q_heads=32, k_heads=8, dim=128,
             rotary=128, interleaved=False),
        # a ragged prompt
        dict(name="rope prompt 777", op="rope_fwd", tokens=777, q_heads=28, k_heads=4, dim=128,
             rotary=64, interleaved=True),
        # a training micro-batch, as many key heads as query heads
        dict(name="rope train 8192", op="rope_fwd", tokens=8192, q_heads=32, k_heads=32, dim=128,
             rotary=128, interleaved=False),
        # backward of a short ragged micro-batch
        dict(name="rope back 515", op="rope_bwd", tokens=515, q_heads=12, k_heads=2, dim=128,
             rotary=128, interleaved=False),
        # backward of the training micro-batch
        dict(name="rope back 8192", op="rope_bwd", tokens=8192, q_heads=32, k_heads=32, dim=128,
             rotary=128, interleaved=False),
        # a prompt of odd length that continues a conversation: state in, state out
        dict(name="mix prompt 1001", op="mix_fwd", tokens=1001, sequences=1, heads=12, key=128,
             value=128, states=True),
        # a training micro-batch of packed documents
        dict(name="mix train 8192", op="mix_fwd", tokens=8192, sequences=5, heads=32, key=128,
             value=128, states=False),
        # a long prompt into a cache
        dict(name="mix prompt 65536", op="mix_fwd", tokens=65536, sequences=1, heads=32, key=128,
             value=128, states=True),
        # backward of a short ragged micro-batch with narrow heads
        dict(name="mix back 515", op="mix_bwd", tokens=515, sequences=3, heads=24, key=64,
             value=64, states=False),
        # backward of the training micro-batch
        dict(name="mix back 8192", op="mix_bwd", tokens=8192, sequences=5, heads=32, key=128,
             value=128, states=False),
        # one stream's next token: latency counts
        dict(name="mix step 1", op="mix_step", rows=1, heads=32, key=128, value=128),
        # the next token of a serving batch
        dict(name="mix step 250", op="mix_step", rows=250, heads=32, key=128, value=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_bwd", "mix_fwd", "mix_fwd", "mix_bwd", "mix_step"])
    if op.startswith("rope"):
        q_heads = rng.choice([12, 28, 32, rng.randint(1, 40)])
        k_heads = rng.choice([q_heads, {12: 2, 28: 4, 32: 8}.get(q_heads, rng.randint(1, q_heads))])
        dim = rng.choice([64, 128, 128, 8 * rng.randint(2, 32)])
        return dict(op=op, tokens=_log_int(rng, 1, 8192), q_heads=q_heads, k_heads=k_heads, dim=dim,
                    rotary=rng.choice([dim, dim, dim // 16 * 8]), interleaved=rng.random() < 0.4)
    heads = rng.choice([12, 28, 32, rng.randint(1, 40)])
    key = rng.choice([64, 128, 128, 8 * rng.randint(2, 16)])
    value = rng.choice([key, key, 64, 128, 8 * rng.randint(2, 16)])
    if op == "mix_step":
        return dict(op=op, rows=_log_int(rng, 1, 250 * 32 // max(32, heads)), heads=heads, key=key,
                    value=value)
    tokens = _log_int(rng, 1, 32768 if op == "mix_fwd" else 8192)
    return dict(op=op, tokens=tokens, sequences=rng.choice([1, 1, 2, 5, min(64, 1 + tokens // 20)]),
                heads=heads, key=key, value=value, states=rng.random() < 0.5)


def work(case):
    """Bytes: every input read once, every output written once.  Flops of the mixing: with
    chunks of 64 tokens, the scores and their product with the values up to the diagonal, the
    state's update and its product with the queries."""
    op = case["op"]
    if op.startswith("rope"):
        n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        small = 4 * case["tokens"] + 2 * case["rotary"] + 4 * case["dim"]
        if op == "rope_fwd":
            return {"bytes": 4 * n + small, "flops": 10 * n}
        return {"bytes": 6 * n + small + 4 * case["dim"], "flops": 20 * n}
    h, dk, dv = case["heads"], case["key"], case["value"]
    if op == "mix_step":
        n = case["rows"] * h
        return {"bytes": n * (8 * dk * dv + 4 * dk + 4 * dv) + 4 * h, "flops": n * 5 * dk * dv}
    n = case["tokens"] * h
    state = 4 * case["sequences"] * h * dk * dv if case["states"] else 0
    one = 64 * (dk + dv) + 4 * dk * dv
    if op == "mix_fwd":
        return {"bytes": n * 4 * (dk + dv) + 2 * state, "flops": n * one}
    return {"bytes": n * 2 * (4 * dk + 3 * dv) + 3 * state, "flops": n * (128 * (dk + dv) + one + 4 * dk * dv)}


# ---------------------------------------------------------------- inputs
def _normal(gen, shape, std=1.0, dtype=torch.bfloat16):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return t.mul_(std).to(dtype)


def _unit(gen, shape):
    """Heads as the norm leaves them: a mean square of one, times a gain."""
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    t *= torch.rsqrt(t.square().mean(dim=-1, keepdim=True))
    return (t * (0.75 + 0.5 * torch.rand(shape[-1], generator=gen, device="cuda"))).to(torch.bfloat16)


def _lengths(case, seed):
    """Documents of a packed batch, longer and shorter ones, some empty or of one token."""
    rng = random.Random("%d %d %d" % (seed, case["tokens"], case["sequences"]))
    cuts = sorted(rng.randint(0, case["tokens"]) for _ in range(case["sequences"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": dict(case)}
    if case["op"].startswith("rope"):
        t, d = case["tokens"], case["dim"]
        s["q"] = _normal(gen, (t, case["q_heads"], d), 2.0)
        s["k"] = _normal(gen, (t, case["k_heads"], d), 2.0)
        s["w_q"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        s["w_k"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        at = torch.arange(case["rotary"] // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (BASE ** (-2 * at / max(1, case["rotary"]))).float()
        # a batch continues somewhere in a long context
        first = int(torch.randint(0, 100000, (), generator=gen, device="cuda"))
        s["position"] = torch.arange(first, first + t, device="cuda", dtype=torch.int32)
        if case["op"] == "rope_bwd":
            s["dq_out"] = _normal(gen, s["q"].shape, 1e-3)
            s["dk_out"] = _normal(gen, s["k"].shape, 1e-3)
        return s
    h, dk, dv = case["heads"], case["key"], case["value"]
    # the heads remember from a token or two to a few hundred
    s["log_decay"] = -torch.exp2(-8 * torch.arange(1, h + 1, device="cuda").float() / h)
    s["scale"] = dk ** -0.5
    rows = case.get("rows") or case["tokens"]
    s["q"], s["k"] = _unit(gen, (rows, h, dk)), _unit(gen, (rows, h, dk))
    s["v"] = _normal(gen, (rows, h, dv))
    if case["op"] == "mix_step":
        s["state"] = _normal(gen, (rows, h, dk, dv), 3.0, torch.float32)
        return s
    lengths = _lengths(case, seed)
    s["chunks"] = sum(-(-n // CHUNK) for n in lengths)
    ends = torch.tensor([0] + lengths, dtype=torch.int64).cumsum(0)
    s["offsets"] = ends.to(device="cuda", dtype=torch.int32)
    if case["states"]:
        s["state"] = _normal(gen, (case["sequences"], h, dk, dv), 3.0, torch.float32)
    if case["op"] == "mix_bwd":
        s["dout"] = _normal(gen, (rows, h, dv), 1e-3)
        if case["states"]:
            s["dfinal"] = _normal(gen, (case["sequences"], h, dk, dv), 1e-3, torch.float32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _keep(s)
    return s


def _keep(s):
    """What a program keeps between calls: the operator's handle (its workspace)
    and the tensors that receive results."""
    from newton_schulz_owner_gb300 import dmuon

    c = s["case"]
    if c["op"].startswith("rope"):
        s["op"] = dmuon.QKNormRope(c["tokens"], c["q_heads"], c["k_heads"], c["dim"], c["rotary"],
                                   eps=EPS, interleaved=c["interleaved"],
                                   backward=c["op"] == "rope_bwd")
        s["out"] = [torch.empty_like(s["q"]), torch.empty_like(s["k"])]
        if c["op"] == "rope_bwd":
            s["dw"] = [torch.empty_like(s["w_q"]), torch.empty_like(s["w_k"])]
        return
    n = c.get("rows") or c["tokens"]
    s["op"] = dmuon.LinearAttention(n, c["heads"], c["key"], c["value"],
                                    max_sequences=c.get("sequences", 1), scale=s["scale"],
                                    backward=c["op"] == "mix_bwd")
    s["out"] = ([torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])]
                if c["op"] == "mix_bwd" else torch.empty_like(s["v"]))
    s["state_out"] = torch.empty_like(s["state"]) if "state" in s else None


# ---------------------------------------------------------------- the passes
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    op = s["case"]["op"]
    if op == "rope_fwd":
        s["op"].forward(s["q"], s["k"], s["w_q"], s["w_k"], s["inv_freq"], s["position"], *s["out"])
        return {"q": s["out"][0], "k": s["out"][1]}
    if op == "rope_bwd":
        s["op"].backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["w_q"], s["w_k"], s["inv_freq"],
                         s["position"], *s["out"], *s["dw"])
        return {"dq": s["out"][0], "dk": s["out"][1], "dw_q": s["dw"][0], "dw_k": s["dw"][1]}
    if op == "mix_step":
        s["op"].step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["out"],
                     new_state=s["state_out"])
        return {"out": s["out"], "state": s["state_out"]}
    if op == "mix_fwd":
        s["op"].forward(s["q"], s["k"], s["v"], s["log_decay"], s["out"], offsets=s["offsets"],
                        state=s.get("state"), final_state=s["state_out"])
        out = {"out": s["out"]}
    else:
        s["op"].backward(s["dout"], s["q"], s["k"], s["v"], s["log_decay"], *s["out"],
                         offsets=s["offsets"], state=s.get("state"), dfinal_state=s.get("dfinal"),
                         dstate=s["state_out"])
        out = {"dq": s["out"][0], "dk": s["out"][1], "dv": s["out"][2]}
    if s["case"]["states"]:
        out["state"] = s["state_out"]
    return out


def _turn(x, cos, sin, interleaved):
    """The first 2 * cos.shape[-1] elements of each head rotated in pairs."""
    n = cos.shape[-1]
    rot, rest = x[..., :2 * n], x[..., 2 * n:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        pair = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = rot[..., :n], rot[..., n:]
        pair = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((pair, rest), dim=-1)


def _norm_back(x, w, g):
    """Gradients of x and w, given that of (x / rms(x)) * w."""
    r = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
    n = x * r
    gw = g * w
    return r * (gw - n * (gw * n).mean(dim=-1, keepdim=True)), (g * n).sum(dim=(0, 1))


def _powers(log_decay, n):
    """exp(log_decay * n) for whole n >= 0, the heads first; 0 where n < 0."""
    g = log_decay.double().reshape((-1,) + (1,) * n.dim())
    return torch.where(n >= 0, torch.exp(g * n.clamp_min(0)), torch.zeros_like(g)).float()


def _mix(q, k, v, log_decay, offsets, chunks, scale, state, before):
    """Linear attention of packed sequences, all chunks at once: within a chunk by scores,
    across chunks by the decayed sum of the earlier chunks' states of the sequence.  `before`:
    how many decays a token's own arrival is behind the state that it reads (1: the state is
    of the token before, 0: it is decayed already, as a gradient's running sum is)."""
    h, dk, dv, dev = q.shape[1], q.shape[2], v.shape[2], q.device
    ends = offsets.long()
    n_chunks = (ends[1:] - ends[:-1] + CHUNK - 1) // CHUNK
    seq = torch.repeat_interleave(torch.arange(len(n_chunks), device=dev), n_chunks,
                                  output_size=chunks)
    first = n_chunks.cumsum(0) - n_chunks
    start = ends[seq] + (torch.arange(chunks, device=dev) - first[seq]) * CHUNK
    stop = torch.minimum(start + CHUNK, ends[seq + 1])
    i = torch.arange(CHUNK, device=dev)
    row = start[:, None] + i
    live = row < stop[:, None]
    at = torch.where(live, row, torch.zeros_like(row))

    def cut(x):                                              # (heads, chunks, CHUNK, width)
        return torch.where(live[None, :, :, None], x.float()[at].permute(2, 0, 1, 3),
                           torch.zeros((), device=dev))

    qc, kc, vc = cut(q), cut(k), cut(v)
    score = (qc @ kc.transpose(-1, -2)) * _powers(log_decay, i[:, None] - i)[:, None]
    o = score @ vc
    size = stop - start
    kv = (kc * _powers(log_decay, size[:, None] - 1 - i + (1 - before))[..., None]).transpose(-1, -2) @ vc
    # decays from the end of each earlier chunk of the sequence to the start of this one
    apart = torch.where(seq[:, None] == seq, start[:, None] - stop, torch.full((), -1, device=dev))
    entry = (_powers(log_decay, apart) @ kv.reshape(h, chunks, dk * dv)).view(h, chunks, dk, dv)
    if state is not None:
        entry += _powers(log_decay, start - ends[seq])[..., None, None] * state.transpose(0, 1)[:, seq]
    o += (qc * _powers(log_decay, i + before)[:, None, :, None]) @ entry
    out = torch.zeros((q.shape[0], h, dv), device=dev)
    out[row[live]] = scale * o.permute(1, 2, 0, 3)[live]
    if state is None:
        return out, None
    # what every chunk still weighs at the end of its sequence, and the state before the first
    last = _powers(log_decay, ends[seq + 1] - stop)[..., None, None] * kv
    final = _powers(log_decay, ends[1:] - ends[:-1])[..., None, None] * state.transpose(0, 1)
    final = final.index_add(1, seq, last)
    return out, final.transpose(0, 1).contiguous()


def _run_plain(s):
    c, bf = s["case"], torch.bfloat16
    if c["op"].startswith("rope"):
        angle = (s["position"].double()[:, None] * s["inv_freq"].double())[:, None]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        q, k, w_q, w_k = (s[x].float() for x in ("q", "k", "w_q", "w_k"))
        if c["op"] == "rope_bwd":
            dq, dw_q = _norm_back(q, w_q, _turn(s["dq_out"].float(), cos, -sin, c["interleaved"]))
            dk, dw_k = _norm_back(k, w_k, _turn(s["dk_out"].float(), cos, -sin, c["interleaved"]))
            return {"dq": dq.to(bf), "dk": dk.to(bf), "dw_q": dw_q.to(bf), "dw_k": dw_k.to(bf)}
        q = q * torch.rsqrt(q.square().mean(dim=-1, keepdim=True) + EPS) * w_q
        k = k * torch.rsqrt(k.square().mean(dim=-1, keepdim=True) + EPS) * w_k
        return {"q": _turn(q, cos, sin, c["interleaved"]).to(bf),
                "k": _turn(k, cos, sin, c["interleaved"]).to(bf)}
    q, k, v, g, scale = (s[x] for x in ("q", "k", "v", "log_decay", "scale"))
    if c["op"] == "mix_step":
        state = torch.exp(g)[None, :, None, None] * s["state"] + \
            k.float().unsqueeze(-1) * v.float().unsqueeze(-2)
        return {"out": (scale * (q.float().unsqueeze(-1) * state).sum(dim=-2)).to(bf), "state": state}
    off, n = s["offsets"], s["chunks"]
    if c["op"] == "mix_fwd":
        o, final = _mix(q, k, v, g, off, n, scale, s.get("state"), 1)
        return {"out": o.to(bf), "state": final} if c["states"] else {"out": o.to(bf)}
    # the gradients are mixtures too: of dq along time from the entering state, of dk and dv
    # against time from the leaving state's gradient
    do = s["dout"]
    state, dfinal = s.get("state"), s.get("dfinal")
    across = (lambda x: None if x is None else x.transpose(-1, -2))  # noqa: E731
    dq, _ = _mix(do, v, k, g, off, n, scale, across(state), 1)
    back = q.shape[0] - off.flip(0)
    turned = [x.flip(0) for x in (q, k, v, do)]
    end = None if dfinal is None else dfinal.flip(0)
    ratio = None if end is None else end / scale
    dv, dstate = _mix(turned[1], turned[0], turned[3], g, back, n, scale, ratio, 0)
    dk, _ = _mix(turned[2], turned[3], turned[0], g, back, n, scale, across(ratio), 0)
    out = {"dq": dq.to(bf), "dk": dk.flip(0).to(bf), "dv": dv.flip(0).to(bf)}
    if c["states"]:
        out["state"] = scale * dstate.flip(0)
    return out


# ---------------------------------------------------------------- in 64 bits
def _exact_rotation(position, inv_freq, dim, interleaved):
    """(tokens, dim, dim) rotations would be large: pairs of element numbers, and their angles."""
    n = inv_freq.numel()
    i = torch.arange(n, device=inv_freq.device)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    return first, second, torch.outer(position.double(), inv_freq.double())[:, None, :]


def _exact_rope(x, w, position, inv_freq, interleaved):
    first, second, angle = _exact_rotation(position, inv_freq, x.shape[-1], interleaved)
    y = x / torch.sqrt((x * x).sum(dim=-1, keepdim=True) / x.shape[-1] + EPS) * w
    z = y.clone()
    z[..., first] = y[..., first] * torch.cos(angle) - y[..., second] * torch.sin(angle)
    z[..., second] = y[..., second] * torch.cos(angle) + y[..., first] * torch.sin(angle)
    return z


def _exact_sequence(q, k, v, lam_log, scale, state, span=64):
    """One sequence, (heads, tokens, width), a few tokens at a time after one another."""
    n, outs = q.shape[1], []
    for a in range(0, n, span):
        b = min(n, a + span)
        t = torch.arange(b - a, device=q.device, dtype=torch.float64)
        gap = t[:, None] - t
        weight = torch.exp(lam_log[:, None, None] * gap.clamp(min=0)) * (gap >= 0)
        qs, ks, vs = q[:, a:b], k[:, a:b], v[:, a:b]
        inner = torch.bmm(torch.bmm(qs, ks.mT) * weight, vs)
        outer = torch.bmm(qs, state) * torch.exp(lam_log[:, None] * (t + 1))[..., None]
        outs.append(scale * (inner + outer))
        left = torch.exp(lam_log[:, None] * (b - a - 1 - t))[..., None]
        state = state * torch.exp(lam_log * (b - a))[:, None, None] + torch.bmm((ks * left).mT, vs)
    return (torch.cat(outs, dim=1) if outs else v), state


def exact(case, seed):
    """The outputs of run() for these inputs in 64 bits, straight from the formulas; gradients
    by differentiating them."""
    s = _inputs(case, seed)
    op = case["op"]
    if op.startswith("rope"):
        x = [s[n].double().requires_grad_(op == "rope_bwd") for n in ("q", "k", "w_q", "w_k")]
        y = [_exact_rope(x[i], x[i + 2], s["position"], s["inv_freq"], case["interleaved"])
             for i in (0, 1)]
        if op == "rope_fwd":
            return {"q": y[0], "k": y[1]}
        d = torch.autograd.grad(y, x, [s["dq_out"].double(), s["dk_out"].double()])
        return {"dq": d[0], "dk": d[1], "dw_q": d[2], "dw_k": d[3]}
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    lam = s["log_decay"].double()
    if op == "mix_step":
        state = s["state"].double()
        state *= torch.exp(lam)[:, None, None]
        state += torch.einsum("rhi,rhj->rhij", k, v)
        return {"out": s["scale"] * torch.einsum("rhi,rhij->rhj", q, state), "state": state}
    back = op == "mix_bwd"
    shape = (case["sequences"], case["heads"], case["key"], case["value"])
    start = s["state"].double() if case["states"] else q.new_zeros(shape)
    leaves = [t.requires_grad_(back) for t in (q, k, v, start)]
    ends = s["offsets"].tolist()
    outs, finals = [], []
    for i, (a, b) in enumerate(zip(ends, ends[1:])):
        o, f = _exact_sequence(*(t[a:b].transpose(0, 1) for t in leaves[:3]), lam, s["scale"],
                               start[i])
        outs.append(o.transpose(0, 1))
        finals.append(f)
    out, final = torch.cat(outs), torch.stack(finals)
    if not back:
        return {"out": out, "state": final} if case["states"] else {"out": out}
    dfinal = s["dfinal"].double() if case["states"] else torch.zeros_like(final)
    d = torch.autograd.grad([out, final], leaves, [s["dout"].double(), dfinal])
    res = {"dq": d[0], "dk": d[1], "dv": d[2]}
    if case["states"]:
        res["state"] = d[3]
    return res
