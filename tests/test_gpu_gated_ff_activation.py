"""Activations of the gated feed-forward block in binary32, value by value: a
width of one and an x of ones make the projections the weights themselves.

Bounds, in roundings u = 2^-24.  exp is off by at most 3 steps (6 u), erfc by 16
(32 u), the reciprocal by 2 u, each product and sum by u; where a value is
subnormal, by 2^-149 at each step, times the gate behind it.
  silu       s of exp, sum, reciprocal, product: 10 u, with g and u 12 u
  gelu       x = g / sqrt 2 by 2 u, of which erfc makes x^2 * 2 + 1 times as
             much (its slope over its value): (2 g^2 + 2 + 32 + 2) u
  gelu_tanh  z by 7 u, of which exp(-|z|) makes |z| times as much, and 12 u
A derivative adds two terms, s and g times the slope (of the logistic function
t / (1 + t)^2: 2 (6 u) + 8 u and, of z, 21 u |z| at most; of the density g^2 / 2
+ 9 u), with three more products and one sum.
"""
import math

import pytest
import torch

import block_ref
import ring_all_reduce_scatter_amd as rar

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
FAR = torch.linspace(-104.0, 104.0, 4159, dtype=torch.float64)
NEAR = torch.linspace(-14.5, 14.5, 2327, dtype=torch.float64)
GATES = torch.cat([FAR, NEAR, torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-41, 700.0, -700.0, 3e38, -3e38])]).float()


def _value(g, kind):
    """act(g) in binary64 and the bound of its error."""
    a = g.abs()
    if kind == rar.ACT_SILU:
        s = torch.exp(-a) / (1 + torch.exp(-a))
        v, k = g * torch.where(g < 0, s, 1 / (1 + torch.exp(-a))), 12.0
    elif kind == rar.ACT_GELU:
        v, k = g * torch.special.erfc(-g / math.sqrt(2)) / 2, 2 * g.clamp(-40, 40) ** 2 + 36
    else:
        z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
        s = torch.exp(-z.abs()) / (1 + torch.exp(-z.abs()))
        v, k = g * torch.where(g < 0, s, 1 / (1 + torch.exp(-z.abs()))), 7 * z.abs().clamp(max=200) + 12
    # second-order terms: k u is below 2^-12 throughout
    return v, v.abs() * k * U * (1 + 2.0 ** -10) + a * 2.0 ** -144 + 2.0 ** -149


def _slope(g, kind):
    a = g.abs()
    if kind == rar.ACT_GELU:
        p = torch.special.erfc(-g / math.sqrt(2)) / 2
        q = g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        c = g.clamp(-40, 40) ** 2
        bound = p * (2 * c + 35) + q.abs() * (c / 2 + 12)
    else:
        z, f = g, torch.ones_like(g)
        if kind == rar.ACT_GELU_TANH:
            z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
            f = math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
        t = torch.exp(-z.abs())
        p, q = torch.where(z < 0, t / (1 + t), 1 / (1 + t)), g * f * t / (1 + t) ** 2
        zu = z.abs().clamp(max=200) * (21 if kind == rar.ACT_GELU_TANH else 0)
        bound = p * (zu + 11) + q.abs() * (zu + 32)
    # a sum that cancels keeps the terms' errors; the products that make the
    # weight's gradient may lose what is subnormal
    return p + q, bound * U * (1 + 2.0 ** -10) + U * (p + q).abs() + 2.0 ** -125


def _within(got, want, bound, what):
    off = (got.double().cpu() - want).abs()
    bad = ~(off <= bound)
    i = int(bad.float().argmax())
    assert not bool(bad.any()), f"{what}: gate {float(GATES[i])!r} gives {float(got.flatten()[i])!r}, {float(want[i])!r}"


@pytest.mark.parametrize("kind", [rar.ACT_SILU, rar.ACT_GELU, rar.ACT_GELU_TANH])
@pytest.mark.parametrize("rows", [1, 9, 20, 40, 70])
def test_binary32_values(rows, kind):
    w, one = GATES.to(DEV)[:, None].contiguous(), torch.ones(GATES.numel(), 1, device=DEV)
    x, out = torch.ones(rows, 1, device=DEV), torch.empty(rows, GATES.numel(), device=DEV)
    rar.gated_ff_forward(x, w, one, out, act=kind)
    v, bound = _value(GATES.double(), kind)
    assert bool((out == out[0]).all())
    _within(out[0], v, bound, f"act {kind}")


@pytest.mark.parametrize("kind", [rar.ACT_SILU, rar.ACT_GELU, rar.ACT_GELU_TANH])
def test_binary32_slopes(kind):
    """One token, so that the weights' gradients are dg and du themselves."""
    n = GATES.numel()
    w, one = GATES.to(DEV)[:, None].contiguous(), torch.ones(n, 1, device=DEV)
    x, ones = torch.ones(1, 1, device=DEV), torch.ones(1, n, device=DEV)
    dwg, dwu = torch.empty(n, 1, device=DEV), torch.empty(n, 1, device=DEV)
    ws = torch.empty(rar.gated_ff_workspace_bytes(1, 1, n, torch.float32), dtype=torch.uint8, device=DEV)
    rar.gated_ff_backward(ones, x, w, one, GATES.to(DEV)[None], ones, None, dwg, dwu, ws, act=kind)
    _within(dwg[:, 0], *_slope(GATES.double(), kind), f"slope {kind}")
    v, bound = _value(GATES.double(), kind)
    _within(dwu[:, 0], v, bound + 2.0 ** -125, f"act {kind}")


def test_bounds_hold_for_the_reference():
    """The forms above are the reference's, where that does not lose digits."""
    g = NEAR
    for kind in (rar.ACT_SILU, rar.ACT_GELU, rar.ACT_GELU_TANH):
        a, d = block_ref.act(g, kind)
        assert torch.allclose(_value(g, kind)[0], a, rtol=1e-9, atol=1e-15)
        assert torch.allclose(_slope(g, kind)[0], d, rtol=1e-9, atol=1e-14)


@pytest.mark.parametrize("dtype,finite", [(torch.float16, False), (torch.bfloat16, True), (torch.float32, True)])
def test_gradients_beyond_binary16(dtype, finite):
    """dg of 10^5 at one place is infinite in binary16 only, and spoils its row
    of dx and its row of dwgate, no others."""
    rows, dim, hidden, r, c = 150, 72, 96, 5, 40
    g = torch.Generator(device=DEV).manual_seed(1)
    x, wg, wu, dh, gate, up = (torch.randn(*s, generator=g, device=DEV).to(dtype) for s in (
        (rows, dim), (hidden, dim), (hidden, dim), (rows, hidden), (rows, hidden), (rows, hidden)))
    dh[r, c], gate[r, c] = 1000.0, 20.0
    ws = torch.empty(rar.gated_ff_workspace_bytes(rows, dim, hidden, dtype), dtype=torch.uint8, device=DEV)
    runs = []
    for u in (1.0, 100.0):
        up[r, c] = u
        out = torch.empty_like(x), *(torch.empty(hidden, dim, device=DEV) for _ in range(2))
        rar.gated_ff_backward(dh, x, wg, wu, gate, up, *out, ws)
        runs.append(out)
    (dx0, dg0, du0), (dx, dg, du) = runs
    assert bool(dx[r].isfinite().all()) == bool(dg[c].isfinite().all()) == finite
    others = [torch.arange(n, device=DEV) != i for n, i in ((rows, r), (hidden, c))]
    assert torch.equal(dx[others[0]], dx0[others[0]]) and torch.equal(dg[others[1]], dg0[others[1]])
    assert torch.equal(du, du0) and all(bool(t.isfinite().all()) for t in (dx0, dg0, du0))
