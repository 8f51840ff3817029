"""64-bit references of the activation checkpoints and the gated feed-forward
block, with bounds on what the kernels' roundings can add up to (operator_ref
has the notation).

A checkpoint is exact arithmetic, so its bytes and values are compared as
they are.  The matrix instructions add in binary32 in an order of their own;
each of a sum's additions is taken to be off by at most one step, 2u, of the
sum of absolute values.
"""
import math

import torch

from operator_ref import SLACK, U, half_step, rounded, tiny


# ------------------------------------------------------------------ checkpoints

def held(x):
    """(codes int8 (rows, 32 nb), exponents uint8 (rows, nb), values float64
    (rows, dim)) of the checkpoint of x, on the CPU."""
    x = x.cpu().float()
    rows, dim = x.shape
    blocks = torch.nn.functional.pad(x, (0, -dim % 32)).view(rows, -1, 32)
    top = blocks.abs().amax(2)
    e = top.view(torch.int32) >> 23
    bad = e == 255  # also where the largest is NaN
    bad |= blocks.isnan().any(2)
    k = 6 - (e.clamp(min=1) - 127)
    scale = ((k.long() + 1023) << 52).view(torch.float64)[..., None]
    q = (blocks.double() * scale).round().clamp(-127, 127)
    q = torch.where(bad[..., None], 0.0, q) + 0.0
    values = torch.where(bad[..., None], math.nan, q / scale)
    return (q.to(torch.int8).view(rows, -1), torch.where(bad, 255, e).to(torch.uint8),
            values.view(rows, -1)[:, :dim])


def held_bytes(x):
    """The checkpoint's buffer."""
    codes, exps, _ = held(x)
    return torch.cat([codes.flatten().view(torch.uint8), exps.flatten()])


# ------------------------------------------------------------------ gated feed-forward

def act(g, kind):
    """act(g) and its derivative in binary64."""
    if kind == 0:
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    if kind == 1:
        p = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) / 2 * c * (1 + 3 * 0.044715 * g * g)


# The activations' slopes stay below 1.13, their second derivatives below
# 1.13 too.  An activation is g times a factor in [0, 1] that a dozen roundings
# make, the largest of them the exponent's, 8 |z| u s (1 - s) <= 2.3 u: 12 u of
# |g| in all.  A derivative adds products of the same kind, up to 2.5 times as
# large: 100 u of 1 + |g|.
SLOPE = 1.13


def forward(x, wg, wu, kind, dt):
    """(gate, bound), (up, bound) unrounded, (h, bound) rounded to dt."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    n = x.shape[1]
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = ((n + 2) * 2 * U * SLACK * (x.abs() @ w.abs().t()) + tiny(torch.float32) for w in (wg, wu))
    a = act(g, kind)[0]
    ea = SLOPE * eg + 12 * U * (g.abs() + eg)
    h = a * u
    eh = ea * (u.abs() + eu) + a.abs() * eu + U * h.abs()
    return (g, eg), (u, eu), (h, rounded(h, eh, dt))


def backward(dh, x, wg, wu, gate, up, kind, dt, wdt, old=None):
    """(dx, bound), (dwgate, bound), (dwup, bound) for the given projections."""
    dh, x, wg, wu, gate, up = (t.double() for t in (dh, x, wg, wu, gate, up))
    a, d = act(gate, kind)
    dg, du = dh * up * d, dh * a
    ed = 100 * U * (1 + gate.abs())
    eg = (dh * up).abs() * (ed + 3 * U * d.abs())
    eu = dh.abs() * (12 * U * gate.abs() + 2 * U * a.abs())
    if dt != torch.float32:
        eg, eu = ((e + (v.abs() + e) * half_step(dt)) * SLACK + tiny(dt) for e, v in ((eg, dg), (eu, du)))
    dx = dg @ wg + du @ wu
    size = (dg.abs() + eg) @ wg.abs() + (du.abs() + eu) @ wu.abs()
    ex = eg @ wg.abs() + eu @ wu.abs() + (2 * gate.shape[1] + 8) * 2 * U * SLACK * size + tiny(torch.float32)
    res = [(dx, rounded(dx, ex, dt))]
    for v, e, o in ((dg, eg, old and old[0]), (du, eu, old and old[1])):
        w = v.t() @ x
        ew = e.t() @ x.abs() + (x.shape[0] + 8) * 2 * U * SLACK * ((v.abs() + e).t() @ x.abs()) + tiny(torch.float32)
        if o is not None:
            w = w + o.double()
            ew = ew + U * (w.abs() + ew)
        res.append((w, rounded(w, ew, wdt)))
    return res
