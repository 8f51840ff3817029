"""Cases of the block operators: activation checkpoints in 8 bits, layer norm
with its input held in one, and the gated feed-forward block, whose backward
pass reads its projections from one.

A data-parallel training step keeps activations between its forward and its
backward pass; in 8 bits they take half the memory of a 16-bit type.  `run`
computes one operator, in plain torch operations or, with `own` set, through
the library's calls.

Case fields
  op        "ckpt": pack and unpack | "ln": layer norm, forward with a
            checkpoint of its input and backward from it | "ff": the gated
            feed-forward block's forward pass | "ff_train": forward and
            backward
  dtype     type of the activations (ff: and weights): f32, f16, bf16
  out       ckpt: "same" unpacks to the activations' type, "f32" to f32
  wdtype    ln: type of the weights and their gradients
  act       "silu" | "gelu" (erf) | "gelu_tanh"
  saved     ff_train: the projections kept for the backward pass, "same" in the
            activations' type or "8bit" as checkpoints

A checkpoint holds blocks of 32 columns of a row: with e the exponent of the
block's largest absolute value (at least -126), each value is the multiple of
2^(e-6) nearest to it (ties to even), at most 127 of them.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-5
_BLOCK = 32


def listed():
    return [
        # One short sequence's activations of odd width: every row of the
        # input starts off a 16-byte boundary.
        dict(name="ckpt_odd", op="ckpt", rows=67, dim=1001, dtype="f32", out="same"),
        # A training batch's residual stream.
        dict(name="ckpt_batch", op="ckpt", rows=16384, dim=4096, dtype="bf16", out="same"),
        # A short sequence of a small model.
        dict(name="ln_short", op="ln", rows=509, dim=512, dtype="f32", wdtype="f32"),
        # A training batch.
        dict(name="ln_batch", op="ln", rows=16384, dim=4096, dtype="bf16", wdtype="f32"),
        # One token of a serving step.
        dict(name="ff_token", op="ff", tokens=1, dim=4096, hidden=11264, dtype="bf16", act="silu"),
        # A serving step of 24 sequences.
        dict(name="ff_tokens", op="ff", tokens=24, dim=4096, hidden=11264, dtype="f16", act="silu"),
        # A prompt whose length is no multiple of anything.
        dict(name="ff_prompt", op="ff", tokens=511, dim=2048, hidden=5632, dtype="bf16", act="gelu_tanh"),
        # A batch of prompts.
        dict(name="ff_batch", op="ff", tokens=8192, dim=4096, hidden=11264, dtype="bf16", act="silu"),
        # A training step in binary32.
        dict(name="ff_train_f32", op="ff_train", tokens=513, dim=1024, hidden=2816, dtype="f32", act="gelu",
             saved="same"),
        # Odd widths: rows of activations and weights start off 16-byte
        # boundaries.
        dict(name="ff_train_odd", op="ff_train", tokens=1021, dim=1001, hidden=2731, dtype="f16", act="silu",
             saved="8bit"),
        # A training step that keeps the projections as they are.
        dict(name="ff_train_same", op="ff_train", tokens=2048, dim=2048, hidden=5632, dtype="bf16", act="gelu_tanh",
             saved="same"),
        # A training batch of a wide block.
        dict(name="ff_train_batch", op="ff_train", tokens=8192, dim=4096, hidden=11264, dtype="bf16", act="silu",
             saved="8bit"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(2.0 ** rng.uniform(math.log2(lo), math.log2(hi + 1)))))


def _width(rng, lo, hi):
    """Half of them any number, half multiples of 64."""
    d = _log_int(rng, lo, hi)
    return d if rng.random() < 0.5 else max(64, d // 64 * 64)


def draw(rng):
    op = rng.choice(["ckpt", "ln", "ff", "ff_train"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op in ("ckpt", "ln"):
        dim = _width(rng, 64, 8192)
        case = dict(op=op, rows=min(_log_int(rng, 1, 65536), (16384 * 4096) // dim), dim=dim, dtype=dtype)
        if op == "ckpt":
            case["out"] = rng.choice(["same", "same", "f32"])
        else:
            case["wdtype"] = rng.choice([dtype, "f32"])
        return case
    case = dict(op=op, tokens=_log_int(rng, 1, 1024 if dtype == "f32" else 8192), dim=_width(rng, 64, 4096),
                hidden=_width(rng, 64, 11264), dtype=dtype, act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]))
    if op == "ff_train":
        # in binary32 a value next to a border of two codes can fall on either
        # side of it, by the order of a sum alone
        case["saved"] = "same" if dtype == "f32" else rng.choice(["same", "8bit"])
    return case


def work(case):
    op, e = case["op"], _ES[case["dtype"]]
    if op in ("ckpt", "ln"):
        r, d = case["rows"], case["dim"]
        blocks = -(-d // _BLOCK)
        held = r * (d + blocks)
        if op == "ckpt":
            return {"bytes": r * d * (e + (e if case["out"] == "same" else 4)) + 2 * held, "flops": 4 * r * d}
        w = _ES[case["wdtype"]]
        return {"bytes": 4 * r * d * e + 2 * held + 16 * r + 5 * d * w, "flops": 24 * r * d}
    t, d, f = case["tokens"], case["dim"], case["hidden"]
    forward = {"bytes": (t * d + 2 * f * d + t * f) * e, "flops": 4 * t * d * f}
    if op == "ff":
        return forward
    saved = 2 * t * f * e if case["saved"] == "same" else 2 * t * (f + -(-f // _BLOCK))
    back = (t * f + 2 * t * d + 4 * f * d) * e  # dh; x and dx; both weights and their gradients
    return {"bytes": forward["bytes"] + back + 2 * saved, "flops": 12 * t * d * f}


# ------------------------------------------------------------------ inputs

def _stream(rows, dim, gen):
    """A residual stream: channels of different size and offset, rows of
    different size."""
    x = torch.randn(rows, dim, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(dim, generator=gen, device="cuda"))
    x += 0.3 * torch.randn(dim, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    return x


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, dim = _DT[case["dtype"]], case["dim"]
    if case["op"] in ("ckpt", "ln"):
        rows = case["rows"]
        out = {"x": _stream(rows, dim, gen).to(dt)}
        if case["op"] == "ln":
            wt = _DT[case["wdtype"]]
            out["weight"] = (1.0 + 0.1 * torch.randn(dim, generator=gen, device="cuda")).to(wt)
            out["bias"] = (0.1 * torch.randn(dim, generator=gen, device="cuda")).to(wt)
            out["dout"] = torch.randn(rows, dim, generator=gen, device="cuda").mul_(0.1).to(dt)
        return out
    t, f = case["tokens"], case["hidden"]
    # a norm's output, channels of different size, and weights that keep the size
    x = torch.randn(t, dim, generator=gen, device="cuda")
    x *= torch.exp(0.3 * torch.randn(dim, generator=gen, device="cuda"))
    out = {"x": x.to(dt)}
    for name in ("wgate", "wup"):
        out[name] = torch.randn(f, dim, generator=gen, device="cuda").mul_(dim ** -0.5).to(dt)
    if case["op"] == "ff_train":
        # of a scaled loss, as binary16 needs it
        out["dout"] = torch.randn(t, f, generator=gen, device="cuda").mul_(0.1).to(dt)
    return out


def prepare(case, seed):
    s = dict(case=case, **_inputs(case, seed))
    if not own:
        return s
    import ring_all_reduce_scatter_amd as rar
    op, dt = case["op"], _DT[case["dtype"]]

    def empty(*shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def held(rows, dim):
        return empty(rar.checkpoint_bytes(rows, dim), dtype=torch.uint8)

    if op == "ckpt":
        s["held"] = held(case["rows"], case["dim"])
        s["out"] = empty(case["rows"], case["dim"], dtype=dt if case["out"] == "same" else torch.float32)
    elif op == "ln":
        r, d, wt = case["rows"], case["dim"], _DT[case["wdtype"]]
        s.update(held=held(r, d), out=empty(r, d), mean=empty(r, dtype=torch.float32),
                 rstd=empty(r, dtype=torch.float32), dx=empty(r, d), dweight=empty(d, dtype=wt),
                 dbias=empty(d, dtype=wt), ws=empty(rar.layernorm_workspace_bytes(r, d), dtype=torch.uint8))
    else:
        t, d, f = case["tokens"], case["dim"], case["hidden"]
        s["out"] = empty(t, f)
        s["act"] = {"silu": rar.ACT_SILU, "gelu": rar.ACT_GELU, "gelu_tanh": rar.ACT_GELU_TANH}[case["act"]]
        if op == "ff_train":
            for name in ("gate", "up"):
                s[name] = empty(t, f) if case["saved"] == "same" else held(t, f)
            s.update(dx=empty(t, d), dwgate=empty(f, d), dwup=empty(f, d),
                     ws=empty(rar.gated_ff_workspace_bytes(t, d, f, s["x"].dtype), dtype=torch.uint8))
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import ring_all_reduce_scatter_amd as rar
    op = s["case"]["op"]
    if op == "ckpt":
        rar.checkpoint_pack(s["x"], s["held"])
        rar.checkpoint_unpack(s["held"], s["out"])
        return [s["out"]]
    if op == "ln":
        rar.layernorm_forward_checkpoint(s["x"], s["weight"], s["bias"], s["out"], s["held"], eps=_EPS, mean=s["mean"],
                                         rstd=s["rstd"])
        rar.layernorm_backward_checkpoint(s["dout"], s["held"], s["weight"], s["mean"], s["rstd"], s["dx"],
                                          s["dweight"], s["dbias"], s["ws"])
        return [s["out"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"]]
    if op == "ff":
        rar.gated_ff_forward(s["x"], s["wgate"], s["wup"], s["out"], act=s["act"])
        return [s["out"]]
    rar.gated_ff_forward(s["x"], s["wgate"], s["wup"], s["out"], act=s["act"], gate=s["gate"], up=s["up"])
    rar.gated_ff_backward(s["dout"], s["x"], s["wgate"], s["wup"], s["gate"], s["up"], s["dx"], s["dwgate"], s["dwup"],
                          s["ws"], act=s["act"])
    kept = [s["gate"], s["up"]] if s["case"]["saved"] == "same" else []
    return [s["out"], s["dx"], s["dwgate"], s["dwup"]] + kept


def _power(k):
    """2^k in binary64, k a tensor of whole numbers in -1022 ... 1023."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _held_plain(x):
    """What a checkpoint of x (binary32 values) stands for, in binary32."""
    rows, dim = x.shape
    blocks = torch.nn.functional.pad(x, (0, -dim % _BLOCK)).view(rows, -1, _BLOCK)
    top = blocks.abs().amax(2, keepdim=True)
    e = ((top.view(torch.int32) >> 23).clamp(min=1) - 127)
    q = (blocks.double() * _power(6 - e)).round().clamp(-127.0, 127.0)
    value = (q * _power(e - 6)).float()
    value = torch.where(torch.isfinite(top), value, float("nan"))
    return value.view(rows, -1)[:, :dim]


def _act_plain(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    x = s["x"].float()
    if op == "ckpt":
        return [_held_plain(x).to(dt if case["out"] == "same" else torch.float32)]
    if op == "ln":
        wt = _DT[case["wdtype"]]
        w = s["weight"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = (xc.square().mean(1, keepdim=True) + _EPS).rsqrt()
        y = (xc * rstd * w + s["bias"].float()).to(dt)
        h = (_held_plain(x) - mean) * rstd
        dy = s["dout"].float()
        g = dy * w
        dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
        return [y, mean[:, 0], rstd[:, 0], dx.to(dt), (dy * h).sum(0).to(wt), dy.sum(0).to(wt)]
    wg, wu = s["wgate"].float(), s["wup"].float()
    gate, up = x @ wg.t(), x @ wu.t()
    h = (_act_plain(gate, case["act"])[0] * up).to(dt)
    if op == "ff":
        return [h]
    kept = [gate.to(dt), up.to(dt)] if case["saved"] == "same" else []
    gate, up = (k.float() for k in kept) if kept else (_held_plain(gate), _held_plain(up))
    a, da = _act_plain(gate, case["act"])
    dh = s["dout"].float()
    dg, du = dh * up * da, dh * a
    dx = dg @ wg + du @ wu
    return [h, dx.to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)] + kept


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _held_exact(x):
    """The values a checkpoint of x stands for: the largest of each block of
    columns is m 2^p with m in [1/2, 1), so its exponent is p - 1."""
    parts = []
    for b in torch.split(x, _BLOCK, dim=1):
        largest = b.abs().max(dim=1, keepdim=True).values.clamp(min=2.0 ** -126)
        step = largest / torch.frexp(largest).mantissa / 128.0  # a power of two, without a rounding
        parts.append(torch.round(b / step).clamp(min=-127, max=127) * step)
    return torch.cat(parts, 1)


def _act_exact(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return 0.5 * g * torch.erfc(-g / math.sqrt(2.0))
    # (1 + tanh z) / 2 is the logistic function of 2 z
    return g * torch.sigmoid(math.sqrt(8.0 / math.pi) * (g + 0.044715 * g ** 3))


def exact(case, seed):
    s = _inputs(case, seed)
    op, f64 = case["op"], torch.float64
    x = s["x"].to(f64)
    if op == "ckpt":
        return [_held_exact(x)]
    if op == "ln":
        n = case["dim"]
        w = s["weight"].to(f64)
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + _EPS)
        y = torch.addcmul(s["bias"].to(f64), (x - mean[:, None]) * rstd[:, None], w)
        # the transposed Jacobian of the normalisation, at the kept input
        h = (_held_exact(x) - mean[:, None]) * rstd[:, None]
        dy = s["dout"].to(f64)
        db, dw = torch.sum(dy, 0), torch.sum(dy * h, 0)
        g = dy * w
        g -= torch.sum(g, 1, keepdim=True) / n + h * (torch.sum(g * h, 1, keepdim=True) / n)
        return [y, mean, rstd, g * rstd[:, None], dw, db]
    wg, wu = s["wgate"].to(f64), s["wup"].to(f64)
    gate, up = torch.mm(x, wg.T), torch.mm(x, wu.T)
    h = _act_exact(gate, case["act"]) * up
    if op == "ff":
        return [h]
    kept = []
    if case["saved"] == "same":
        kept = [gate, up]
        gate, up = gate.to(s["x"].dtype).to(f64), up.to(s["x"].dtype).to(f64)
    else:
        gate, up = _held_exact(gate), _held_exact(up)
    # the product's gradients at the kept projections
    gate, up = gate.requires_grad_(), up.requires_grad_()
    with torch.enable_grad():
        dg, du = torch.autograd.grad(_act_exact(gate, case["act"]) * up, (gate, up), s["dout"].to(f64))
    dx = torch.addmm(torch.mm(dg, wg), du, wu)
    return [h, dx, torch.mm(dg.T, x), torch.mm(du.T, x)] + [k.detach() for k in kept]
