"""Layer norm forward and backward on the GPU against the 64-bit formulas."""
import math

import pytest
import torch

import operator_ref as ref
import ring_all_reduce_scatter_amd as rar
from operator_ref import DTYPES, U, assert_within

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
EPS = 1e-5


def _forward(x, w, b, eps=EPS, out=None):
    rows = x.numel() // x.shape[-1]
    out = torch.full(x.shape, 7.0, device=DEV, dtype=x.dtype) if out is None else out
    mean, rstd = torch.full((rows,), 9.0, device=DEV), torch.full((rows,), 9.0, device=DEV)
    rar.layernorm_forward(x, w, b, out, eps=eps, mean=mean, rstd=rstd)
    return out, mean, rstd


def _check_forward(x, w, b, got, eps=EPS, what=""):
    want = ref.layernorm(x.reshape(-1, x.shape[-1]), w, b, eps, x.dtype)
    for g, (r, tol), name in zip(got, want, ("y", "mean", "rstd")):
        assert_within(g.reshape(r.shape), r, tol, f"{what} {name}")


def _backward(dy, x, w, mean, rstd, wdt, old=None):
    rows, dim = x.numel() // x.shape[-1], x.shape[-1]
    dx = torch.full(x.shape, 7.0, device=DEV, dtype=x.dtype)
    dw, db = [torch.full((dim,), 3.0, device=DEV, dtype=wdt) if old is None else o.clone() for o in (old or (0, 0))]
    ws = torch.empty(rar.layernorm_workspace_bytes(rows, dim), dtype=torch.uint8, device=DEV)
    rar.layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, ws, accumulate=old is not None)
    return dx, dw, db


def _check_backward(dy, x, w, mean, rstd, got, wdt, old=(None, None), what=""):
    dim = x.shape[-1]
    want = ref.layernorm_grad(dy.reshape(-1, dim), x.reshape(-1, dim), w, mean, rstd, x.dtype, wdt, *old)
    for g, (r, tol), name in zip(got, want, ("dx", "dw", "db")):
        assert_within(g.reshape(r.shape), r, tol, f"{what} {name}")


SHAPES = [(1, 1), (3, 2), (1, 64), (5, 63), (70, 129), (4, 512), (33, 513), (257, 768), (1, 1000), (130, 1024),
          (9, 1025), (65, 2048), (3, 2049), (1, 4096), (40, 4096), (17, 4097), (5, 8192), (11, 8191), (3, 16384),
          (2, 16391), (3, 40_003), (2000, 96), (9000, 33), (37, 2561),
          (20, 1300), (600, 40), (700, 250), (513, 2570), (1, 300)]


@pytest.mark.parametrize("dts", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_forward_and_backward_match_formula(rows, dim, dts):
    xt, wt = DTYPES[dts[0]], DTYPES[dts[1]]
    g = torch.Generator(device=DEV).manual_seed(rows + dim)
    x = (torch.randn(rows, dim, generator=g, device=DEV) * 2 + 0.5).to(xt)
    w = (1 + 0.2 * torch.randn(dim, generator=g, device=DEV)).to(wt)
    b = torch.randn(dim, generator=g, device=DEV).to(wt)
    dy = torch.randn(rows, dim, generator=g, device=DEV).to(xt)
    got = _forward(x, w, b)
    _check_forward(x, w, b, got, what="affine")
    _, mean, rstd = got
    _check_backward(dy, x, w, mean, rstd, _backward(dy, x, w, mean, rstd, wt), wt, what="affine")
    _check_forward(x, None, None, _forward(x, None, None), what="plain")
    _check_backward(dy, x, None, mean, rstd, _backward(dy, x, None, mean, rstd, wt), wt, what="plain")
    old = (torch.randn(dim, generator=g, device=DEV).to(wt), torch.randn(dim, generator=g, device=DEV).to(wt))
    res = _backward(dy, x, w, mean, rstd, wt, old)
    _check_backward(dy, x, w, mean, rstd, res, wt, old, what="accumulated")
    assert all(torch.equal(p, q) for p, q in zip(res, _backward(dy, x, w, mean, rstd, wt, old))), "bits differ"


def test_parts_of_the_backward_pass():
    """dx, dweight and dbias alone and in pairs equal the whole call's."""
    x = torch.randn(50, 700, device=DEV).to(torch.bfloat16)
    dy, w = torch.randn_like(x), torch.randn(700, device=DEV)
    _, mean, rstd = _forward(x, w, None)
    whole = _backward(dy, x, w, mean, rstd, torch.float32)
    ws = torch.empty(rar.layernorm_workspace_bytes(50, 700), dtype=torch.uint8, device=DEV)
    for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1)):
        out = [torch.full_like(t, 5.0) if k else None for t, k in zip(whole, want)]
        rar.layernorm_backward(dy, x, w, mean, rstd, *out, ws if any(want[1:]) else None)
        for t, o in zip(whole, out):
            assert o is None or torch.equal(t, o), want
    y1, y2 = torch.empty_like(x), torch.empty_like(x)
    rar.layernorm_forward(x, w, None, y1)
    rar.layernorm_forward(x, w, None, y2, mean=mean, rstd=rstd)
    assert torch.equal(y1, y2)


@pytest.mark.parametrize("dim", [100, 3001, 40_000])
def test_in_place(dim):
    x = torch.randn(7, dim, device=DEV)
    w, b, dy = torch.randn(dim, device=DEV), torch.randn(dim, device=DEV), torch.randn(7, dim, device=DEV)
    y, mean, rstd = _forward(x, w, b)
    dx, dw, db = _backward(dy, x, w, mean, rstd, torch.float32)
    ws = torch.empty(rar.layernorm_workspace_bytes(7, dim), dtype=torch.uint8, device=DEV)
    for over in ("dy", "x"):
        a, c = dy.clone(), x.clone()
        d = a if over == "dy" else c
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        rar.layernorm_backward(a, c, w, mean, rstd, d, dw2, db2, ws)
        assert torch.equal(d, dx) and torch.equal(dw2, dw) and torch.equal(db2, db), over
    rar.layernorm_forward(x, w, b, x)
    assert torch.equal(x, y)


def test_no_rows():
    x = torch.empty(0, 30, device=DEV)
    w, s = torch.ones(30, device=DEV), torch.empty(0, device=DEV)
    _forward(x, w, w)
    _, dw, db = _backward(x, x, w, s, s, torch.float32)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    old = torch.randn(30, device=DEV), torch.randn(30, device=DEV)
    _, dw, db = _backward(x, x, w, s, s, torch.float32, old)
    assert torch.equal(dw, old[0]) and torch.equal(db, old[1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [65, 1000, 4099, 40_001])
def test_strided_unaligned_and_broadcast_rows(dt, dim):
    t = DTYPES[dt]
    store = torch.randn(6, 5, dim + 12, device=DEV).to(t)
    x = store[:, :, 1:1 + dim]
    w, b = torch.randn(dim + 1, device=DEV).to(t)[1:], torch.randn(dim + 1, device=DEV).to(t)[1:]
    out_store = torch.full((6, 5, dim + 5), 4.0, device=DEV, dtype=t)
    y = out_store[:, :, 3:3 + dim]
    got = _forward(x, w, b, out=y)
    _check_forward(x, w, b, got, what="strided")
    assert bool((out_store[:, :, :3] == 4.0).all()) and bool((out_store[:, :, 3 + dim:] == 4.0).all())
    _, mean, rstd = got
    dy = torch.randn(dim, device=DEV).to(t).expand(6, 5, dim)  # one row for all
    _check_backward(dy, x, w, mean, rstd, _backward(dy, x, w, mean, rstd, t), t, what="broadcast dy")
    same = x[0, 0].expand(30, dim)
    got = _forward(same, w, b)
    _check_forward(same, w, b, got, what="broadcast x")


@pytest.mark.parametrize("dim", [7, 1024, 5000])
def test_constant_rows_and_large_offsets(dim):
    """No variance: h is 0 and rstd 1/sqrt(eps); and a mean far above the spread."""
    x = torch.full((3, dim), 100.0, device=DEV)
    x[1] = 0.0
    w, b = torch.randn(dim, device=DEV), torch.randn(dim, device=DEV)
    got = _forward(x, w, b)
    _check_forward(x, w, b, got, what="constant")
    y, mean, rstd = _forward(x, w, b, eps=0.0)  # 0 * inf, as the formula has it
    assert bool(torch.isinf(rstd[1])) and bool(y[1].isnan().all())
    far = 1000.0 + torch.randn(4, dim, device=DEV)
    _check_forward(far, w, b, _forward(far, w, b), what="far")


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_non_finite_rows_stay_apart(bad):
    x = torch.randn(20, 600, device=DEV)
    w, b = torch.randn(600, device=DEV), torch.randn(600, device=DEV)
    clean, *_ = _forward(x, w, b)
    x[7, 599] = bad
    y, mean, rstd = _forward(x, w, b)
    assert bool(y[7].isnan().all())
    keep = [r for r in range(20) if r != 7]
    assert torch.equal(y[keep], clean[keep])


def test_offsets_beyond_32_bits():
    stride = (1 << 32) // 2 + 9
    big = torch.empty(2 * stride + 600, dtype=torch.bfloat16, device=DEV)
    x = big.as_strided((3, 515), (stride, 1))
    x.copy_(torch.randn(3, 515, device=DEV))
    w, b = torch.randn(515, device=DEV), torch.randn(515, device=DEV)
    near = x.clone()
    y, mean, rstd = _forward(x, w, b)
    y2, *_ = _forward(near, w, b)
    assert torch.equal(y, y2)
    dy = torch.randn(3, 515, device=DEV).to(torch.bfloat16)
    want = _backward(dy, near, w, mean, rstd, torch.float32)
    got = _backward(dy, x, w, mean, rstd, torch.float32)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    ws = torch.empty(rar.layernorm_workspace_bytes(3, 515), dtype=torch.uint8, device=DEV)
    rar.layernorm_backward(dy, near, w, mean, rstd, x, None, None, ws)  # dx into the far rows
    assert torch.equal(x, want[0])
    rar.layernorm_forward(near, w, b, x)
    assert torch.equal(x, y)


def test_gradient_against_differences():
    """f = sum(y * dy): central differences along random directions of x, w
    and b.  y is rounded within its bound; the difference quotient's own
    error is taken from the quotients at two distances (it shrinks with the
    square of the distance, so at the shorter one it is a third of their gap)."""
    x, dy = torch.randn(30, 200, device=DEV), torch.randn(30, 200, device=DEV)
    w, b = 1 + 0.2 * torch.randn(200, device=DEV), torch.randn(200, device=DEV)
    _, mean, rstd = _forward(x, w, b)
    dx, dw, db = _backward(dy, x, w, mean, rstd, torch.float32)
    want = ref.layernorm_grad(dy, x, w, mean, rstd, torch.float32, torch.float32)
    # the statistics themselves are off by their bounds: relative to dx, twice each
    (_, ey), (_, em), (r64, er) = ref.layernorm(x, w, b, EPS, torch.float32)
    for name, var, grad in (("x", 0, dx), ("w", 1, dw), ("b", 2, db)):
        args = [x, w, b]
        v = torch.randn_like(args[var])

        def f(h):
            a = list(args)
            a[var] = a[var] + h * v
            return float((_forward(*a)[0].double() * dy.double()).sum())

        h = 2.0 ** -7
        q1, q2 = (f(h) - f(-h)) / (2 * h), (f(2 * h) - f(-2 * h)) / (4 * h)
        along = float((grad.double() * v.double()).sum())
        step = U * float((args[var].abs() + 2 * h * v.abs()).max())  # the shifted argument is rounded
        slope = float((grad.double().abs()).sum())
        rounding = (float((ey.to(DEV) * dy.double().abs()).sum()) * 2 + step * slope * 2) / h
        bound = float((want[var][1].to(DEV) * v.double().abs()).sum())
        stats = float((er / r64).max() + (em.to(DEV) * rstd.double()).max().cpu()) * 8 * slope * float(v.abs().max())
        tol = abs(q1 - q2) + rounding + bound + stats
        assert abs(q1 - along) <= tol, (name, q1, along, tol)
        assert tol < 0.05 * float((grad.double().square().sum() * v.double().square().sum()).sqrt()), (name, tol)


def test_replays_in_a_graph():
    x, dy = torch.randn(300, 1500, device=DEV).to(torch.bfloat16), torch.randn(300, 1500, device=DEV).to(torch.bfloat16)
    w, b = torch.randn(1500, device=DEV), torch.randn(1500, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(300, device=DEV), torch.empty(300, device=DEV)
    dw, db = torch.empty(1500, device=DEV), torch.empty(1500, device=DEV)
    ws = torch.empty(rar.layernorm_workspace_bytes(300, 1500), dtype=torch.uint8, device=DEV)

    def step():
        rar.layernorm_forward(x, w, b, y, mean=mean, rstd=rstd)
        rar.layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(4):
        x.mul_(-1.25)
        dy.copy_(dy.roll(1, 0))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, mean, rstd, dx, dw, db)]
        step()
        assert all(torch.equal(p, q) for p, q in zip(got, (y, mean, rstd, dx, dw, db))), f"replay {k}"
