"""Refusals of the activation checkpoints, layer norm from them and the gated
feed-forward block, by the binding and by the C entry points, before any
launch.  CPU only: host tensors reach the binding's own checks, and the C
calls get addresses that are never read."""
import math

import pytest
import torch

import block_ref
import ring_all_reduce_scatter_amd as rar

OK, EINVAL, EDTYPE, EALIGN, EWORKSPACE, ENOTSUP, EOVERLAP = 0, 1, 2, 3, 4, 6, 7
G = 1 << 32
B = 1 << 40  # base addresses; calls that would touch them must be refused first


def _raises(match, fn, *a, **k):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*a, **k)


# ------------------------------------------------------------------ binding

def test_checkpoint_binding_refusals():
    x, buf = torch.zeros(4, 40), torch.zeros(4 * 66, dtype=torch.uint8)

    def unpack(out, held):
        return rar.checkpoint_unpack(held, out)

    for f in (rar.checkpoint_pack, unpack):
        def call(x=x, buf=buf, f=f):
            return f(x, buf)
        _raises("at least one element", call, torch.zeros(4, 0))
        _raises("264 are needed", call, x, buf[:-1])
        _raises("contiguous bytes", call, x, torch.zeros(600, dtype=torch.uint8)[::2])
        _raises("contiguous bytes", call, x, torch.zeros(264, dtype=torch.float32))
        _raises("last dimension", call, torch.zeros(4, 80)[:, ::2])
        _raises("equally far apart", call, torch.zeros(4, 4, 40)[:2, :3])
        _raises("unsupported dtype", call, x.double())
        _raises("GPU tensor", call)
    _raises("overlap", rar.checkpoint_unpack, buf, torch.zeros(1, 40).expand(4, 40))


def test_layernorm_checkpoint_binding_refusals():
    x, w, s = torch.zeros(4, 6), torch.zeros(6), torch.zeros(4)
    buf = torch.zeros(rar.checkpoint_bytes(4, 6), dtype=torch.uint8)
    f = rar.layernorm_forward_checkpoint
    _raises("132 are needed", f, x, w, w, x, buf[1:])
    _raises("out must have x's type", f, x, w, w, x.half(), buf)
    _raises("rows of 6", f, x, w, w, torch.zeros(4, 7), buf)
    _raises("contiguous with 4", f, x, w, w, torch.zeros(4, 6), buf, rstd=torch.zeros(5))
    _raises("GPU tensor", f, x, w, w, x, buf)
    bw = rar.layernorm_backward_checkpoint
    ws = torch.zeros(rar.layernorm_workspace_bytes(4, 6), dtype=torch.uint8)
    _raises("132 are needed", bw, x, buf[1:], w, s, s, x, w, w, ws)
    _raises("dout's type", bw, x, buf, w, s, s, x.half(), w, w, ws)
    _raises("one type", bw, x, buf, w, s, s, x, w.half(), w, ws)
    _raises("mean must be float32", bw, x, buf, w, s.half(), s, x, w, w, ws)
    _raises("GPU tensor", bw, x, buf, w, s, s, x, w, w, ws)


def test_gated_ff_binding_refusals():
    x, w, h = torch.zeros(4, 6), torch.zeros(10, 6), torch.zeros(4, 10)
    buf = torch.zeros(rar.checkpoint_bytes(4, 10), dtype=torch.uint8)
    f = rar.gated_ff_forward
    _raises("must both be", f, x, w, torch.zeros(9, 6), h)
    _raises("must both be", f, x, w[0], w[0], h)
    _raises("must both be", f, x, w[:0], w[:0], h)
    _raises("rows of 6", f, x, torch.zeros(10, 5), torch.zeros(10, 5), h)
    _raises("x's type", f, x, w.half(), w, h)
    _raises("x's type", f, x, w, w, h.half())
    _raises("rows of 10", f, x, w, w, torch.zeros(4, 9))
    _raises("3 rows, 4 are needed", f, x, w, w, torch.zeros(3, 10))
    _raises("overlap", f, x, w, w, torch.zeros(1, 10).expand(4, 10))
    _raises("of one kind", f, x, w, w, h, gate=h)
    _raises("of one kind", f, x, w, w, h, gate=h, up=buf)
    _raises("gate must be contiguous bytes", f, x, w, w, h, gate=h.half(), up=h.half())
    _raises("132 are needed", f, x, w, w, h, gate=buf, up=buf[1:])
    _raises("rows of 10", f, x, w, w, h, gate=h, up=torch.zeros(4, 9))
    _raises("GPU tensor", f, x, w, w, h)
    _raises("GPU tensor", f, x, w, w, h, gate=buf, up=buf)
    bw = rar.gated_ff_backward
    ws = torch.zeros(rar.gated_ff_workspace_bytes(4, 6, 10, torch.float32), dtype=torch.uint8)
    _raises("gate and up are needed", bw, h, x, w, w, None, None, x, w, w, ws)
    _raises("dout has 3 rows", bw, h[:3], x, w, w, h, h, x, w, w, ws)
    _raises("up has 3 rows", bw, h, x, w, w, h, h[:3], x, w, w, ws)
    _raises("x's type", bw, h.half(), x, w, w, h, h, x, w, w, ws)
    _raises("x's type", bw, h, x, w, w, h, h, x.half(), w, w, ws)
    _raises("of one kind", bw, h, x, w, w, h, h, x, w, None, ws)
    _raises("of one kind", bw, h, x, w, w, h, h, x, w, w.half(), ws)
    _raises("or be float32", bw, h, x, w, w, h, h, x, w.half(), w.half(), ws)
    _raises("10 are needed", bw, h, x, w, w, h, h, x, w[:9], w, ws)
    _raises("weights' shape", bw, h, x, w, w, h, h, x, w.view(2, 5, 6), w, ws)
    _raises("workspace must be contiguous", bw, h, x, w, w, h, h, x, w, w, ws[::2])
    _raises("unsupported dtype", rar.gated_ff_workspace_bytes, 4, 6, 10, torch.float64)
    _raises("GPU tensor", bw, h, x, w, w, h, h, x, w, w, ws)


# ------------------------------------------------------------------ C entry points

def test_checkpoint_c_refusals():
    L = rar.lib()
    assert rar.checkpoint_bytes(3, 33) == 3 * 66 and rar.checkpoint_bytes(0, 33) == 0
    assert rar.checkpoint_bytes(3, 0) == 0 and rar.checkpoint_bytes(3, 1 << 31) == 0
    assert rar.checkpoint_bytes(1 << 60, 1 << 20) == 0

    def pack(x=B, xs=40, rows=4, dim=40, dt=0, ck=B + G, n=1 << 20):
        return L.rar_checkpoint_pack(x, xs, rows, dim, dt, ck, n, None)

    def unpack(x=B, xs=40, rows=4, dim=40, dt=0, ck=B + G, n=1 << 20):
        return L.rar_checkpoint_unpack(ck, n, rows, dim, x, xs, dt, None)

    for f in (pack, unpack):
        assert f(dt=3) == EDTYPE
        assert f(dim=0) == EINVAL
        assert f(dim=1 << 31) == ENOTSUP
        assert f(rows=1 << 60) == EINVAL
        assert f(x=0) == EOVERLAP and f(ck=0) == EOVERLAP
        assert f(x=B + 2) == EALIGN and f(x=B + 1, dt=1) == EALIGN and f(ck=B + G + 8) == EALIGN
        assert f(n=4 * 66 - 1) == EWORKSPACE
        assert f(ck=B + 16) == EOVERLAP and f(ck=B - 4 * 66 + 16 + 8) in (EOVERLAP, EALIGN)
        assert f(rows=0, x=0, ck=0, n=0) == OK
    assert unpack(xs=39) == EINVAL


def test_layernorm_checkpoint_c_refusals():
    L = rar.lib()

    def fwd(x=B, y=B + G, mean=B + 2 * G, rstd=B + 3 * G, ck=B + 4 * G, n=1 << 20, rows=4, dim=40, dt=0, w=0):
        return L.rar_layernorm_forward_checkpoint(x, dim, w, 0, rows, dim, dt, 0, 1e-5, y, dim, mean, rstd, ck, n, None)

    assert fwd(ck=0) == EOVERLAP and fwd(ck=B + 4 * G + 4) == EALIGN and fwd(n=4 * 66 - 1) == EWORKSPACE
    for at in (B, B + G, B + 2 * G, B + 3 * G, B + 5 * G):
        assert fwd(ck=at, w=B + 5 * G) == EOVERLAP
    assert fwd(rows=1 << 60) == EINVAL and fwd(dt=7) == EDTYPE
    assert fwd(rows=0, ck=0, n=0) == OK

    def bwd(dy=B, ck=B + G, n=1 << 20, mean=B + 2 * G, rstd=B + 3 * G, dx=B + 4 * G, dw=B + 5 * G, db=B + 6 * G,
            ws=B + 7 * G, nb=1 << 30, rows=4, dim=40):
        return L.rar_layernorm_backward_checkpoint(dy, dim, ck, n, 0, mean, rstd, rows, dim, 0, 0, dx, dim, dw, db, 0,
                                                   ws, nb, None)

    assert bwd(ck=0) == EOVERLAP and bwd(ck=B + G + 2) == EALIGN and bwd(n=4 * 66 - 1) == EWORKSPACE
    for at in (B + 4 * G, B + 5 * G, B + 6 * G, B + 7 * G):
        assert bwd(ck=at) == EOVERLAP
    assert bwd(nb=64) == EWORKSPACE and bwd(mean=0) == EOVERLAP


def _forward(x=B, xs=48, wg=B + G, wgs=48, wu=B + 2 * G, wus=48, rows=70, dim=48, hidden=80, dt=2, act=0, h=B + 3 * G,
             hs=80, keep=1, g=B + 4 * G, gs=80, u=B + 5 * G, us=80):
    return rar.lib().rar_gated_ff_forward(x, xs, wg, wgs, wu, wus, rows, dim, hidden, dt, act, h, hs, keep, g, gs, u,
                                          us, None)


def _backward(dh=B, dhs=80, x=B + G, xs=48, wg=B + 2 * G, wgs=48, wu=B + 3 * G, wus=48, keep=1, g=B + 4 * G, gs=80,
              u=B + 5 * G, us=80, rows=70, dim=48, hidden=80, dt=2, act=0, dx=B + 6 * G, dxs=48, dg=B + 7 * G, dgs=48,
              du=B + 8 * G, dus=48, wdt=2, ws=B + 9 * G, n=1 << 30):
    return rar.lib().rar_gated_ff_backward(dh, dhs, x, xs, wg, wgs, wu, wus, keep, g, gs, u, us, rows, dim, hidden, dt,
                                           act, dx, dxs, dg, dgs, du, dus, wdt, 0, ws, n, None)


def test_gated_ff_forward_c_refusals():
    f = _forward
    assert f(dt=3) == EDTYPE and f(act=3) == EINVAL and f(act=-1) == EINVAL and f(keep=3) == EINVAL
    assert f(dim=0) == EINVAL and f(hidden=0) == EINVAL
    big = dict(xs=1 << 21, wgs=1 << 21, wus=1 << 21, hs=1 << 21, gs=1 << 21, us=1 << 21)
    assert f(dim=(1 << 20) + 1, **big) == ENOTSUP and f(hidden=(1 << 20) + 1, **big) == ENOTSUP
    for name in ("xs", "wgs", "wus"):
        assert f(**{name: (1 << 21) + 1}) == ENOTSUP and f(dt=0, **{name: (1 << 20) + 1}) == ENOTSUP
    assert f(rows=(1 << 30) + 1) == ENOTSUP
    assert f(rows=1 << 20, hidden=1 << 20, hs=1 << 20, gs=1 << 20, us=1 << 20) == ENOTSUP
    assert f(hs=79) == EINVAL and f(gs=79) == EINVAL and f(us=79) == EINVAL
    assert f(xs=1 << 50) == EINVAL and f(wus=1 << 50) == EINVAL
    for name in ("x", "wg", "wu", "h", "g", "u"):
        assert f(**{name: 0}) == EOVERLAP
        assert f(**{name: B + 1}) == EALIGN
    # outputs over inputs and one another
    for out in ("h", "g", "u"):
        for other in (B, B + G, B + 2 * G, *(B + k * G for k, n in ((3, "h"), (4, "g"), (5, "u")) if n != out)):
            assert f(**{out: other}) == EOVERLAP, (out, other)
    n = 70 * 99
    assert f(keep=2, gs=n - 1, us=n) == EWORKSPACE and f(keep=2, gs=n, us=n - 1) == EWORKSPACE
    assert f(keep=2, gs=n, us=n, g=B + 4 * G + 8) == EALIGN and f(keep=2, gs=n, us=n, u=0) == EOVERLAP
    assert f(keep=2, gs=n, us=n, u=B + 4 * G + 16) == EOVERLAP
    assert f(rows=0, x=0, h=0, g=0, u=0) == OK


def test_gated_ff_backward_c_refusals():
    f = _backward
    assert f(dt=3) == EDTYPE and f(act=3) == EINVAL and f(keep=0) == EINVAL and f(wdt=1) == EDTYPE
    assert f(dim=0) == EINVAL and f(hidden=0) == EINVAL and f(rows=(1 << 30) + 1) == ENOTSUP
    for name in ("xs", "wgs", "wus"):
        assert f(**{name: (1 << 21) + 1}) == ENOTSUP
    assert f(dg=0) == EINVAL and f(du=0) == EINVAL
    assert f(dxs=47) == EINVAL and f(dgs=47) == EINVAL and f(dus=47) == EINVAL
    for name in ("dh", "x", "wg", "wu", "g", "u"):
        assert f(**{name: 0}) == EOVERLAP
        assert f(**{name: B + 1}) == EALIGN
    assert f(dx=B + 6 * G + 1) == EALIGN and f(dg=B + 7 * G + 2, wdt=0) == EALIGN
    need = rar.gated_ff_workspace_bytes(70, 48, 80, torch.bfloat16)
    assert f(n=need - 1) == EWORKSPACE and f(ws=0) == EWORKSPACE and f(ws=B + 9 * G + 8) == EALIGN
    outs = {"dx": 6, "dg": 7, "du": 8, "ws": 9}
    for out, at in outs.items():
        for other in range(10):
            if other != at:
                assert f(**{out: B + other * G}) == EOVERLAP, (out, other)
    m = 70 * 99
    assert f(keep=2, gs=m - 1, us=m) == EWORKSPACE and f(keep=2, gs=m, us=m, dx=B + 4 * G) == EOVERLAP
    assert f(dx=0, dg=0, du=0) == OK  # nothing asked for
    assert f(rows=0, dh=0, x=0, g=0, u=0, dx=0, dg=0, du=0, ws=0, n=0) == OK


def test_workspace_sizes():
    f = rar.gated_ff_workspace_bytes
    assert f(0, 48, 80, torch.float32) == 0 and f(5, 0, 80, torch.float32) == 0
    for t, es in ((torch.float32, 4), (torch.bfloat16, 2)):
        # the two gradients of the projections, rows of whole blocks
        assert f(8192, 4096, 11264, t) == 2 * 8192 * 11264 * es
        assert f(100, 48, 80, t) >= 2 * 100 * 96 * es


def test_reference_checkpoint():
    """The reference itself, on values whose codes are plain."""
    x = torch.zeros(2, 33)
    x[0, :4] = torch.tensor([1.0, -0.5, 1 / 64, 1 / 128])
    x[0, 32] = 3.0
    x[1, 5] = math.nan
    codes, exps, values = block_ref.held(x)
    assert codes[0, :4].tolist() == [64, -32, 1, 0] and exps[0].tolist() == [127, 128]
    assert codes[0, 32] == 96 and values[0, 32] == 3.0 and values[0, 0] == 1.0
    assert exps[1].tolist() == [255, 0] and bool(values[1, :32].isnan().all()) and values[1, 32] == 0.0
    assert block_ref.held(torch.full((1, 32), 255.0))[0][0, 0] == 127  # 127.5 steps of 2 would be 128


def test_reference_gradients_against_autograd():
    x, wg, wu, dh = (torch.randn(*s, dtype=torch.float64) for s in ((5, 7), (9, 7), (9, 7), (5, 9)))
    for kind, f in enumerate((torch.nn.functional.silu, torch.nn.functional.gelu,
                              lambda t: torch.nn.functional.gelu(t, approximate="tanh"))):
        a, b, c = (t.clone().requires_grad_() for t in (x, wg, wu))
        ((f(a @ b.t()) * (a @ c.t())) * dh).sum().backward()
        res = block_ref.backward(dh, x, wg, wu, x @ wg.t(), x @ wu.t(), kind, torch.float32, torch.float32)
        for (r, _), t in zip(res, (a, b, c)):
            assert torch.allclose(r, t.grad, rtol=1e-10, atol=1e-12)
