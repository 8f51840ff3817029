"""Cases of the gradient-path operators: embedding lookup and its gradient,
layer norm forward and backward, the global gradient norm and clipping.

A data-parallel training step makes gradients out of a batch of tokens
(embedding, layer norm), sums them over the ranks (the library's rings) and
then clips them by their global norm.  `run` computes one operator, in plain
torch operations or, with `own` set, through the library's calls.

Case fields
  op        "norm" | "clip" | "embed" | "embed_grad" | "ln" | "ln_grad"
  dtype     type of the gradients, embeddings or activations: f32, f16, bf16,
            or (norm, clip) "mixed": tensors under 65,536 elements in f32, the
            others in bf16
  out       clip: "same" writes each tensor's own type, "f32" writes f32
  align     clip: each clipped tensor starts on a multiple of so many elements
            of one flat buffer per type (the optimizer's)
  wdtype    type of the weights and their gradients (embed: of the table)
"""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}
_MIXED_BORDER = 65536
_EPS = 1e-5
_CLIP_EPS = 1e-6


def listed():
    return [
        # The gradients of one small block (biases, norm weights, a small
        # projection) logged after a backward pass: latency counts.
        dict(name="norm_small", op="norm", kind="l2", tensors=16, lo=256, hi=32768, size_seed=1, dtype="f32",
             scale=1.0),
        # The bucketed all-reduce's tensor list, 200 tensors of 1K to 16M
        # elements in bf16, monitored by its norm; 1/16 makes the sum of 16
        # ranks their mean.
        dict(name="norm_buckets", op="norm", kind="l2", tensors=200, lo=1024, hi=1 << 24, size_seed=3, dtype="bf16",
             scale=0.0625),
        # A reduced set of f32 gradients of a few layers, clipped into the
        # optimizer's own buffers.
        dict(name="clip_layers", op="clip", kind="l2", tensors=40, lo=4096, hi=1 << 21, size_seed=5, dtype="f32",
             out="same", align=64, scale=0.125, max_norm=1.0),
        # The whole bucketed list, matrices in bf16 and vectors in f32.
        dict(name="clip_buckets", op="clip", kind="l2", tensors=200, lo=1024, hi=1 << 24, size_seed=3, dtype="mixed",
             out="same", align=64, scale=0.0625, max_norm=1.0),
        # One decoding step of four sequences.
        dict(name="embed_token", op="embed", tokens=4, vocab=32768, dim=4096, dtype="bf16", wdtype="bf16", scale=1.0,
             invalid=0.0),
        # A training batch whose length is no multiple of anything, scaled
        # by sqrt(dim).
        dict(name="embed_batch", op="embed", tokens=16383, vocab=65536, dim=4096, dtype="bf16", wdtype="bf16",
             scale=64.0, invalid=0.02),
        # A short sequence's gradient for a small table.
        dict(name="embed_grad_small", op="embed_grad", tokens=509, vocab=8192, dim=512, dtype="f32", wdtype="f32",
             scale=1.0, invalid=0.02),
        # A batch of natural text (a few tokens make up most of it), reduced
        # into a f32 gradient of the table.
        dict(name="embed_grad_batch", op="embed_grad", tokens=32768, vocab=50021, dim=2048, dtype="bf16", wdtype="f32",
             scale=1.0, invalid=0.02),
        # One token of a serving step.
        dict(name="ln_token", op="ln", rows=1, dim=4096, dtype="bf16", wdtype="bf16"),
        # A training batch in binary16 with f32 weights.
        dict(name="ln_batch", op="ln", rows=16384, dim=4096, dtype="f16", wdtype="f32"),
        # Odd rows of odd length: every row starts off a 16-byte boundary.
        dict(name="ln_grad_odd", op="ln_grad", rows=2047, dim=1001, dtype="f32", wdtype="f32"),
        # A training batch of a wide model.
        dict(name="ln_grad_batch", op="ln_grad", rows=16384, dim=8192, dtype="bf16", wdtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(2.0 ** rng.uniform(math.log2(lo), math.log2(hi + 1)))))


def _dim(rng, lo, hi):
    d = _log_int(rng, lo, hi)
    return d if rng.random() < 0.5 else max(64, d // 64 * 64)


def draw(rng):
    op = rng.choice(["norm", "clip", "embed", "embed_grad", "ln", "ln_grad"])
    if op in ("norm", "clip"):
        case = dict(op=op, kind=rng.choice(["l2", "l2", "max"]), tensors=_log_int(rng, 1, 200),
                    lo=_log_int(rng, 1, 4096), hi=_log_int(rng, 1 << 14, 1 << 23), size_seed=rng.randrange(1 << 20),
                    dtype=rng.choice(["f32", "f16", "bf16", "mixed"]), scale=rng.choice([1.0, 0.5, 0.125, 1.0 / 3.0]))
        if op == "clip":
            case.update(max_norm=rng.choice([0.1, 1.0, 1.0, 10.0]), out=rng.choice(["same", "same", "f32"]),
                        align=rng.choice([1, 64, 64]))
        return case
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    wdtype = rng.choice([dtype, "f32"])
    if op in ("embed", "embed_grad"):
        dim = _dim(rng, 64, 4096)
        return dict(op=op, tokens=min(_log_int(rng, 1, 32768), (32768 * 1024) // dim),
                    vocab=min(_log_int(rng, 256, 65536), (65536 * 1024) // dim), dim=dim, dtype=dtype, wdtype=wdtype,
                    scale=rng.choice([1.0, math.sqrt(dim)]), invalid=rng.choice([0.0, 0.02, 0.3]))
    dim = _dim(rng, 64, 8192)
    return dict(op=op, rows=min(_log_int(rng, 1, 65536), (16384 * 4096) // dim), dim=dim, dtype=dtype, wdtype=wdtype)


# ------------------------------------------------------------------ sizes

def _sizes(case):
    """Log-uniform tensor sizes in [lo, hi], from the case alone."""
    r = random.Random(case["size_seed"])
    lo, hi = math.log2(case["lo"]), math.log2(case["hi"])
    return [int(2.0 ** r.uniform(lo, hi)) for _ in range(case["tensors"])]


def _types(case):
    """Type of each tensor of a norm or clip case."""
    if case["dtype"] == "mixed":
        return ["f32" if n < _MIXED_BORDER else "bf16" for n in _sizes(case)]
    return [case["dtype"]] * case["tensors"]


def _flat(case, dtype):
    """The clipped gradients' flat buffers, one per type, and each tensor's
    place in its buffer."""
    names = [t if case["out"] == "same" else "f32" for t in _types(case)]
    used = {t: 0 for t in sorted(set(names))}
    places = []
    for t, n in zip(names, _sizes(case)):
        places.append((t, used[t], n))
        used[t] += -(-n // case["align"]) * case["align"]
    flat = {t: torch.zeros(n, dtype=dtype or _DT[t], device="cuda") for t, n in used.items()}
    return [flat[t] for t in flat], [flat[t][a:a + n] for t, a, n in places]


def _distinct(case):
    """Expected number of distinct table rows among the tokens (id k, before
    they are mixed, has the probability ln((k+2)/(k+1)) / ln(V+1))."""
    t = case["tokens"] * (1.0 - case["invalid"])
    k = torch.arange(case["vocab"], dtype=torch.float64)
    p = torch.log((k + 2.0) / (k + 1.0)) / math.log(case["vocab"] + 1.0)
    return float((1.0 - torch.exp(t * torch.log1p(-p))).sum())


def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        sizes, types = _sizes(case), _types(case)
        n = sum(sizes)
        nbytes = 4 + sum(s * _ES[t] for s, t in zip(sizes, types))
        if op == "clip":
            nbytes += sum(s * (_ES[t] if case["out"] == "same" else 4) for s, t in zip(sizes, types))
        return {"bytes": nbytes, "flops": (3 if op == "clip" else 2) * n}
    e = _ES[case["dtype"]]
    w = _ES[case["wdtype"]]
    d = case["dim"]
    if op == "embed":
        return {"bytes": 8 * case["tokens"] + int(_distinct(case)) * d * w + case["tokens"] * d * e,
                "flops": case["tokens"] * d}
    if op == "embed_grad":
        return {"bytes": 8 * case["tokens"] + case["tokens"] * d * e + case["vocab"] * d * w,
                "flops": case["tokens"] * d}
    r = case["rows"]
    if op == "ln":
        return {"bytes": 2 * r * d * e + 2 * d * w + 8 * r, "flops": 8 * r * d}
    return {"bytes": 3 * r * d * e + 3 * d * w + 8 * r, "flops": 14 * r * d}


# ------------------------------------------------------------------ inputs

def _gradient(n, gen):
    """N(0, 1e-3) with one element in a hundred a hundred times larger."""
    g = torch.randn(n, generator=gen, device="cuda")
    big = torch.rand(n, generator=gen, device="cuda") < 0.01
    return g * torch.where(big, 0.1, 0.001)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("norm", "clip"):
        return {"grads": [_gradient(n, gen).to(_DT[t]) for n, t in zip(_sizes(case), _types(case))]}
    dt, wt, d = _DT[case["dtype"]], _DT[case["wdtype"]], case["dim"]
    if op in ("embed", "embed_grad"):
        t, v = case["tokens"], case["vocab"]
        u = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64)
        rank = (torch.exp(u * math.log(v + 1.0)) - 1.0).long().clamp_(0, v - 1)
        ids = torch.randperm(v, generator=gen, device="cuda")[rank]
        # positions that carry no token
        ids = torch.where(torch.rand(t, generator=gen, device="cuda") < case["invalid"], -1, ids)
        if op == "embed":
            w = torch.randn(v, d, generator=gen, device="cuda").mul_(0.02).to(wt)
            return {"ids": ids, "weight": w}
        return {"ids": ids, "dout": _gradient(t * d, gen).view(t, d).to(dt)}
    r = case["rows"]
    # a residual stream: channels of different size and offset, rows of different size
    x = torch.randn(r, d, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(d, generator=gen, device="cuda"))
    x += 0.3 * torch.randn(d, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(r, 1, generator=gen, device="cuda"))
    w = (1.0 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(wt)
    out = {"x": x.to(dt), "weight": w}
    if op == "ln":
        out["bias"] = (0.1 * torch.randn(d, generator=gen, device="cuda")).to(wt)
        return out
    del x
    out["dout"] = _gradient(r * d, gen).view(r, d).to(dt)
    # the statistics that the forward pass left
    x64 = out["x"].double()
    mean = x64.mean(1, keepdim=True)
    out["rstd"] = ((x64 - mean).square().mean(1) + _EPS).rsqrt().float()
    out["mean"] = mean[:, 0].float()
    return out


def prepare(case, seed):
    state = dict(case=case, **_inputs(case, seed))
    if case["op"] == "clip":
        state["flat"], state["outs"] = _flat(case, None)
    if not own:
        return state
    import ring_all_reduce_scatter_amd as rar
    op, dev = case["op"], "cuda"
    if op in ("norm", "clip"):
        grads = state["grads"]
        ws = torch.empty(rar.grad_clip_workspace_bytes([g.numel() for g in grads]), dtype=torch.uint8, device=dev)
        state.update(clip=rar.GradClip(grads, ws, outs=state.get("outs")),
                     norm=torch.empty(1, dtype=torch.float32, device=dev))
        return state
    dt, wt, d = _DT[case["dtype"]], _DT[case["wdtype"]], case["dim"]
    if op == "embed":
        state["out"] = torch.empty(case["tokens"], d, dtype=dt, device=dev)
    elif op == "embed_grad":
        state["dweight"] = torch.empty(case["vocab"], d, dtype=wt, device=dev)
        state["ws"] = torch.empty(rar.embedding_workspace_bytes(case["tokens"], case["vocab"], d), dtype=torch.uint8,
                                  device=dev)
    elif op == "ln":
        state["out"] = torch.empty_like(state["x"])
        state["mean"] = torch.empty(case["rows"], dtype=torch.float32, device=dev)
        state["rstd"] = torch.empty(case["rows"], dtype=torch.float32, device=dev)
    else:
        state["dx"] = torch.empty_like(state["x"])
        state["dweight"] = torch.empty(d, dtype=wt, device=dev)
        state["dbias"] = torch.empty(d, dtype=wt, device=dev)
        state["ws"] = torch.empty(rar.layernorm_workspace_bytes(case["rows"], d), dtype=torch.uint8, device=dev)
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import ring_all_reduce_scatter_amd as rar
    case = s["case"]
    op = case["op"]
    if op in ("norm", "clip"):
        kind = rar.NORM_L2 if case["kind"] == "l2" else rar.NORM_MAX
        if op == "norm":
            s["clip"].norm(s["norm"], norm_type=kind, scale=case["scale"])
            return [s["norm"]]
        s["clip"].clip(case["max_norm"], s["norm"], norm_type=kind, scale=case["scale"])
        return [s["norm"]] + s["flat"]
    if op == "embed":
        rar.embedding_forward(s["weight"], s["ids"], s["out"], scale=case["scale"])
        return [s["out"]]
    if op == "embed_grad":
        rar.embedding_backward(s["dout"], s["ids"], s["dweight"], s["ws"], scale=case["scale"])
        return [s["dweight"]]
    if op == "ln":
        rar.layernorm_forward(s["x"], s["weight"], s["bias"], s["out"], eps=_EPS, mean=s["mean"], rstd=s["rstd"])
        return [s["out"], s["mean"], s["rstd"]]
    rar.layernorm_backward(s["dout"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                           s["ws"])
    return [s["dx"], s["dweight"], s["dbias"]]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("norm", "clip"):
        if case["kind"] == "l2":
            parts = [g.float().square().sum(dtype=torch.float64) for g in s["grads"]]
            norm = torch.stack(parts).sum().sqrt() * abs(case["scale"])
        else:
            parts = [g.float().abs().max() for g in s["grads"]]
            norm = torch.stack(parts).max() * abs(case["scale"])
        norm = norm.float().view(1)
        if op == "norm":
            return [norm]
        factor = (case["max_norm"] / (norm + _CLIP_EPS)).clamp(max=1.0) * case["scale"]
        for out, g in zip(s["outs"], s["grads"]):
            out.copy_(g.float() * factor)
        return [norm] + s["flat"]
    if op in ("embed", "embed_grad"):
        ids, v, dt, wt = s["ids"], case["vocab"], _DT[case["dtype"]], _DT[case["wdtype"]]
        valid = (ids >= 0) & (ids < v)
        if op == "embed":
            rows = s["weight"][torch.where(valid, ids, 0)].float() * case["scale"]
            return [(rows * valid[:, None]).to(dt)]
        dw = torch.zeros(v + 1, case["dim"], device=ids.device)  # the last row takes the positions without a token
        dw.index_add_(0, torch.where(valid, ids, v), s["dout"].float() * case["scale"])
        return [dw[:v].to(wt)]
    x = s["x"].float()
    w = s["weight"].float()
    if op == "ln":
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = (xc.square().mean(1, keepdim=True) + _EPS).rsqrt()
        return [(xc * rstd * w + s["bias"].float()).to(s["x"].dtype), mean[:, 0], rstd[:, 0]]
    dy = s["dout"].float()
    rstd = s["rstd"][:, None]
    h = (x - s["mean"][:, None]) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return [dx.to(s["x"].dtype), (dy * h).sum(0).to(s["weight"].dtype), dy.sum(0).to(s["weight"].dtype)]


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op in ("norm", "clip"):
        scale = case["scale"]
        if case["kind"] == "l2":
            norm = math.sqrt(math.fsum(float(torch.dot(g.to(f64), g.to(f64))) for g in s["grads"])) * abs(scale)
        else:
            norm = max(float(torch.max(torch.abs(g)).to(f64)) for g in s["grads"]) * abs(scale)
        first = torch.tensor([norm], dtype=f64)
        if op == "norm":
            return [first]
        factor = scale * min(1.0, case["max_norm"] / (norm + _CLIP_EPS))
        flat, outs = _flat(case, f64)
        for out, g in zip(outs, s["grads"]):
            torch.mul(g.to(f64), factor, out=out)
        return [first] + flat
    if op == "embed":
        # a table with one more row, of zeros, for the positions without a token
        table = torch.cat([s["weight"].to(f64) * case["scale"],
                           torch.zeros(1, case["dim"], dtype=f64, device="cuda")])
        ids = s["ids"].clone()
        ids[(ids < 0) | (ids >= case["vocab"])] = case["vocab"]
        return [table.index_select(0, ids)]
    if op == "embed_grad":
        # sums of runs of equal tokens, as differences of running sums over the sorted tokens
        key, order = torch.sort(s["ids"], stable=True)
        edges = torch.searchsorted(key, torch.arange(case["vocab"] + 1, device="cuda"))
        parts = []
        for c in range(0, case["dim"], 512):
            d = s["dout"][:, c:c + 512].to(f64)[order]
            total = torch.cat([torch.zeros(1, d.shape[1], dtype=f64, device="cuda"), torch.cumsum(d, 0)])[edges]
            parts.append((total[1:] - total[:-1]) * case["scale"])
        return [torch.cat(parts, 1)]
    x = s["x"].to(f64)
    n = case["dim"]
    w = s["weight"].to(f64)
    if op == "ln":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + _EPS)
        y = torch.addcmul(s["bias"].to(f64), (x - mean[:, None]) * rstd[:, None], w)
        return [y, mean, rstd]
    # the transposed Jacobian of the normalisation, row by row, with the
    # statistics that the backward pass is given
    r = s["rstd"].to(f64)[:, None]
    h = x.sub_(s["mean"].to(f64)[:, None]).mul_(r)
    dy = s["dout"].to(f64)
    db = torch.sum(dy, 0)
    dw = torch.sum(dy * h, 0)
    g = dy.mul_(w)
    along_one = torch.sum(g, 1, keepdim=True) / n
    along_h = torch.sum(g * h, 1, keepdim=True) / n
    dx = g.sub_(along_one).sub_(h.mul_(along_h)).mul_(r)
    return [dx, dw, db]
