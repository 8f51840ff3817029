"""64-bit references of the operators next to the rings, with bounds on what
the kernels' roundings can add up to.

u = 2^-24 is half a step of binary32 and half_step(t) half a step of the
output type.  A binary32 sum of n terms is off by at most depth * u times
the sum of their absolute values, depth being the longest chain of additions
a term goes through (n at most); each product or further operation adds one
u of its result.  Second-order terms are covered by the factor SLACK.  Below
the smallest normal number a rounding is off by at most half the smallest
subnormal, `tiny`.
"""
import torch

U = 2.0 ** -24
SLACK = 1.0 + 2.0 ** -10
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dt) -> float:
    return torch.finfo(dt).eps / 2


def tiny(dt) -> float:
    f = torch.finfo(dt)
    return f.tiny * f.eps / 2


def assert_within(got, ref, tol, what):
    """|got - ref| <= tol element by element; NaN and infinities must agree.
    A reference beyond the type's largest value may come back as infinity."""
    g = got.double().cpu()
    ref, tol = ref.double().cpu(), tol.double().cpu().expand_as(ref)
    assert g.shape == ref.shape, f"{what}: shape {tuple(g.shape)} != {tuple(ref.shape)}"
    finite = torch.isfinite(ref)
    same = torch.where(torch.isnan(ref), torch.isnan(g), g == ref)
    ok = torch.where(finite, (g - ref).abs() <= tol, same)
    ok |= finite & torch.isinf(g) & (g.sign() == ref.sign()) & (ref.abs() + tol >= torch.finfo(got.dtype).max)
    if not bool(ok.all()):
        i = int((~ok).flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} off; first at {i}: got "
                             f"{g.flatten()[i].item()!r}, expected {ref.flatten()[i].item()!r} within "
                             f"{tol.flatten()[i].item()!r}")


def rounded(ref, err, dt):
    """Bound after the result, off by err, is rounded to dt."""
    return (err + (ref.abs() + err) * half_step(dt)) * SLACK + tiny(dt)


# ------------------------------------------------------------------ norm and clip

def norm(grads, kind, scale):
    if not sum(g.numel() for g in grads):
        return 0.0
    flat = torch.cat([g.double().flatten().cpu() for g in grads])
    n = flat.square().sum().sqrt() if kind == 0 else flat.abs().max()
    return float(n) * abs(scale)


def clipped(g, total, max_norm, scale, dt):
    """(reference, bound): the factor is rounded to binary32, then the
    product, then (to a shorter type) the output."""
    c = max_norm / (total + 1e-6)
    f = scale * (1.0 if c > 1.0 else c)
    ref = g.double().cpu() * f
    err = ref.abs() * (U if dt == torch.float32 else 2 * U) + tiny(torch.float32) * 2
    return ref, rounded(ref, err, dt)


# ------------------------------------------------------------------ embedding

def valid_ids(ids, vocab, padding=None):
    ok = (ids >= 0) & (ids < vocab)
    return ok if padding is None else ok & (ids != padding)


def embedding(weight, ids, scale, dt):
    ids = ids.cpu().flatten().long()
    ok = valid_ids(ids, weight.shape[0])
    w = weight.double().cpu()
    ref = torch.zeros(ids.numel(), w.shape[1], dtype=torch.float64)
    ref[ok] = w[ids[ok]] * scale
    err = ref.abs() * (0 if dt == torch.float32 else U)
    return ref, rounded(ref, err, dt)


def embedding_grad(dout, ids, vocab, scale, dt, padding=None, old=None):
    ids = ids.cpu().flatten().long()
    ok = valid_ids(ids, vocab, padding)
    d = dout.double().cpu().reshape(ids.numel(), -1)
    dim = d.shape[1]
    ref = torch.zeros(vocab, dim, dtype=torch.float64)
    mag = torch.zeros(vocab, dim, dtype=torch.float64)
    ref.index_add_(0, ids[ok], d[ok])
    mag.index_add_(0, ids[ok], d[ok].abs())
    count = torch.bincount(ids[ok], minlength=vocab).double()[:, None]
    err = mag * abs(scale) * (count + 1) * U
    ref = ref * scale
    touched = (count > 0).expand_as(ref)
    if old is not None:
        o = old.double().cpu()
        err = torch.where(touched, err + ((ref + o).abs() + err) * U, torch.zeros_like(err))
        ref = ref + o
    return ref, torch.where(touched, rounded(ref, err, dt), torch.zeros_like(err))


# ------------------------------------------------------------------ layer norm

def _depth(dim):
    """Additions on the longest way of a row's element into its sum: a lane
    of a wavefront or workgroup adds at least every 64th element, then the
    lanes are joined in a tree."""
    return dim // 64 + 24


def layernorm(x, weight, bias, eps, dt):
    """(y, bound), (mean, bound), (rstd, bound)"""
    x = x.double().cpu()
    dim = x.shape[-1]
    w = torch.ones(dim, dtype=torch.float64) if weight is None else weight.double().cpu()
    b = torch.zeros(dim, dtype=torch.float64) if bias is None else bias.double().cpu()
    mu = x.mean(-1, keepdim=True)
    xc = x - mu
    var = xc.square().mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    d = _depth(dim)
    e_mu = (d + 2) * U * x.abs().mean(-1, keepdim=True) * SLACK + tiny(torch.float32)
    # the squares about a mean that is off by e_mu: each difference is
    # rounded (u of itself), and the shift adds e_mu^2 to their mean
    e_var = (d + 6) * U * var + (e_mu + U * xc.abs().amax(-1, keepdim=True)).square() * 4 + tiny(torch.float32)
    rel = e_var / (var + eps) / 2 * (1 + 2.0 ** -4) + 4 * U
    e_rstd = rstd * rel
    h = xc * rstd
    e_h = h.abs() * (rel + 3 * U) + e_mu * rstd * (1 + rel)
    y = h * w + b
    e_y = e_h * w.abs() + U * ((h * w).abs() + y.abs())
    return ((y, rounded(y, e_y, dt)), (mu[..., 0], e_mu[..., 0]), (rstd[..., 0], e_rstd[..., 0] * SLACK))


def layernorm_grad(dy, x, weight, mean, rstd, dt, wdt, old_w=None, old_b=None):
    """(dx, bound), (dw, bound), (db, bound) for the given statistics."""
    x, dy = x.double().cpu(), dy.double().cpu()
    rows, dim = x.shape
    w = torch.ones(dim, dtype=torch.float64) if weight is None else weight.double().cpu()
    mu, r = mean.double().cpu()[:, None], rstd.double().cpu()[:, None]
    h = (x - mu) * r
    g = dy * w
    mg, mgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    d = _depth(dim)
    e_mg = (d + 3) * U * g.abs().mean(1, keepdim=True) * SLACK + tiny(torch.float32)
    e_mgh = (d + 6) * U * (g * h).abs().mean(1, keepdim=True) * SLACK + tiny(torch.float32)
    dx = r * (g - mg - h * mgh)
    parts = g.abs() + mg.abs() + (h * mgh).abs()
    e_dx = r * (e_mg + h.abs() * e_mgh + 6 * U * parts) + U * dx.abs()
    res = [(dx, rounded(dx, e_dx, dt))]
    for terms, old in ((dy * h, old_w), (dy, old_b)):
        s = terms.sum(0)
        err = (rows + 8) * U * terms.abs().sum(0)
        if old is not None:
            o = old.double().cpu()
            err = err + U * ((s + o).abs() + err)
            s = s + o
        res.append((s, rounded(s, err, wdt)))
    return res
