"""Gated feed-forward block on the GPU against the 64-bit formulas, and bit by
bit on whole numbers, whose sums are exact in any order."""
import math

import pytest
import torch

import block_ref
import ring_all_reduce_scatter_amd as rar
from operator_ref import DTYPES, assert_within, rounded

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ACTS = {"silu": rar.ACT_SILU, "gelu": rar.ACT_GELU, "gelu_tanh": rar.ACT_GELU_TANH}


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV)


def _backward(dh, x, wg, wu, gate, up, kind, wdt, old=None, want_dx=True, want_dw=True):
    rows, dim, hidden = x.numel() // x.shape[-1], x.shape[-1], wg.shape[0]
    dx = torch.full(x.shape, 7.0, device=DEV, dtype=x.dtype) if want_dx else None
    dw = [None, None]
    if want_dw:
        dw = [torch.full((hidden, dim), 3.0, device=DEV, dtype=wdt) if old is None else o.clone()
              for o in (old or (0, 0))]
    ws = _bytes(rar.gated_ff_workspace_bytes(rows, dim, hidden, x.dtype))
    rar.gated_ff_backward(dh, x, wg, wu, gate, up, dx, *dw, ws, act=kind, accumulate=old is not None)
    return dx, *dw


def _normal(rows, dim, hidden, dt, seed=0):
    g = torch.Generator(device=DEV).manual_seed(rows * 7 + dim * 3 + hidden + seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return (rand(rows, dim).to(dt), (rand(hidden, dim) * dim ** -0.5).to(dt), (rand(hidden, dim) * dim ** -0.5).to(dt),
            rand(rows, hidden).to(dt))


def _check_all(x, wg, wu, dh, kind, wdt):
    """Forward with every way of keeping, backward from both, the formula's
    values within their bounds."""
    dt, rows, dim, hidden = x.dtype, x.numel() // x.shape[-1], x.shape[-1], wg.shape[0]
    flat = x.reshape(rows, dim)
    (g, eg), (u, eu), (h, eh) = block_ref.forward(flat, wg, wu, kind, dt)
    out = torch.full((*x.shape[:-1], hidden), 7.0, dtype=dt, device=DEV)
    rar.gated_ff_forward(x, wg, wu, out, act=kind)
    assert_within(out.reshape(rows, hidden), h, eh, "h")
    gate, up, out2 = torch.full_like(out, 5.0), torch.full_like(out, 5.0), torch.full_like(out, 5.0)
    rar.gated_ff_forward(x, wg, wu, out2, act=kind, gate=gate, up=up)
    assert torch.equal(out, out2), "h beside kept rows"
    assert_within(gate.reshape(rows, hidden), g, rounded(g, eg, dt), "gate")
    assert_within(up.reshape(rows, hidden), u, rounded(u, eu, dt), "up")
    n = rar.checkpoint_bytes(rows, hidden)
    cg, cu = (torch.full((n + 16,), 0xA5, dtype=torch.uint8, device=DEV) for _ in range(2))
    rar.gated_ff_forward(x, wg, wu, out2, act=kind, gate=cg, up=cu)
    assert_within(out2.reshape(rows, hidden), h, eh, "h beside checkpoints")
    kept = []
    for buf, v, e in ((cg, g, eg), (cu, u, eu)):
        assert bool((buf[n:] == 0xA5).all()), "bytes past the checkpoint"
        val = torch.empty(rows, hidden, device=DEV)
        rar.checkpoint_unpack(buf, val)
        # within half a step of the block (a whole one at the clamp), the
        # largest value being off by its own error
        top = torch.nn.functional.pad(v.abs() + e, (0, -hidden % 32)).view(rows, -1, 32).amax(2, keepdim=True)
        step = (top * 2.0 ** -7).expand(-1, -1, 32).reshape(rows, -1)[:, :hidden]
        assert_within(val, v, step + e, "kept in 8 bits")
        kept.append(val)
        # packing the values again changes nothing: the bytes are a checkpoint's
        again = torch.empty_like(buf)
        rar.checkpoint_pack(val, again)
        back = torch.empty_like(val)
        rar.checkpoint_unpack(again, back)
        assert torch.equal(back, val)
    old = None
    for gt, ut, gv, uv in ((gate, up, gate, up), (cg, cu, *kept)):
        res = _backward(dh, x, wg, wu, gt, ut, kind, wdt, old)
        want = block_ref.backward(dh.reshape(rows, hidden), flat, wg, wu, gv.reshape(rows, hidden),
                                  uv.reshape(rows, hidden), kind, dt, wdt, old)
        for r, (v, tol), name in zip(res, want, ("dx", "dwgate", "dwup")):
            assert_within(r.reshape(v.shape), v, tol, name)
        again = _backward(dh, x, wg, wu, gt, ut, kind, wdt, old)
        assert all(torch.equal(p, q) for p, q in zip(res, again)), "bits differ"
        alone = _backward(dh, x, wg, wu, gt, ut, kind, wdt, old, want_dw=False)[0]
        assert torch.equal(alone, res[0])
        alone = _backward(dh, x, wg, wu, gt, ut, kind, wdt, old, want_dx=False)[1:]
        assert all(torch.equal(p, q) for p, q in zip(alone, res[1:]))
        old = [torch.randn(hidden, dim, device=DEV).to(wdt) for _ in range(2)]


SHAPES = [(1, 1, 1), (1, 8, 32), (2, 3, 5), (1, 128, 96), (16, 64, 64), (17, 100, 33), (31, 200, 70), (64, 64, 130),
          (65, 64, 130), (70, 129, 67), (128, 256, 128), (129, 264, 200), (200, 1001, 77), (3, 1000, 1000),
          (300, 40, 520), (513, 72, 96), (5, 520, 1100), (1, 4099, 45), (2, 2565, 67), (3, 4099, 33),
          (31, 4099, 20)]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dts", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,dim,hidden", SHAPES)
def test_matches_formula(rows, dim, hidden, dts, act):
    dt = DTYPES[dts[0]]
    x, wg, wu, dh = _normal(rows, dim, hidden, dt)
    _check_all(x, wg, wu, dh, ACTS[act], DTYPES[dts[1]])


# Both tile sizes of each product, in whole and partial tiles, with several
# stages of terms, and the splits of a long sum over few tiles.
EXACT = [(5, 300, 70), (130, 136, 200), (256, 128, 256), (700, 520, 264), (2100, 72, 4104), (4100, 4104, 40),
         (70, 2056, 4104), (257, 257, 129), (1000, 33, 31), (3000, 64, 64), (65, 4096, 96), (2048, 2048, 2048)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,dim,hidden", EXACT)
def test_whole_numbers_bit_by_bit(rows, dim, hidden, dt):
    """Small whole numbers: the projections are exact, and with gates of 0 and
    64 the gelu's value (0, 64) and slope (1/2, 1) too, so that every sum is
    exact in binary32 and only the outputs are rounded."""
    t = DTYPES[dt]
    g = torch.Generator(device=DEV).manual_seed(rows + dim + hidden)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device=DEV).float()

    x, wg, wu = ints(-2, 2, rows, dim), ints(-1, 1, hidden, dim), ints(-1, 1, hidden, dim)
    gate, up, out = (torch.full((rows, hidden), 9.0, dtype=t, device=DEV) for _ in range(3))
    rar.gated_ff_forward(x.to(t), wg.to(t), wu.to(t), out, act=rar.ACT_GELU, gate=gate, up=up)
    assert torch.equal(gate, (x.double() @ wg.double().t()).to(t)), "gate"
    assert torch.equal(up, (x.double() @ wu.double().t()).to(t)), "up"
    kept_g, kept_u, dh = ints(0, 1, rows, hidden) * 64, ints(-2, 2, rows, hidden), ints(-1, 1, rows, hidden)
    a, d = kept_g, torch.where(kept_g > 0, 1.0, 0.5)
    dg, du = (dh * kept_u * d).double(), (dh * a / 64).double()  # du in units of 64
    dx = dg @ wg.double() + 64 * (du @ wu.double())
    for wdt in {torch.float32, t}:
        res = _backward(dh.to(t), x.to(t), wg.to(t), wu.to(t), kept_g.to(t), kept_u.to(t), rar.ACT_GELU, wdt)
        assert torch.equal(res[0], dx.to(t)), "dx"
        assert torch.equal(res[1], (dg.t() @ x.double()).to(wdt)), "dwgate"
        assert torch.equal(res[2], (64 * (du.t() @ x.double())).to(wdt)), "dwup"
    # the same from checkpoints, whose steps these values are multiples of
    n = rar.checkpoint_bytes(rows, hidden)
    cg, cu = _bytes(n), _bytes(n)
    rar.checkpoint_pack(kept_g, cg)
    rar.checkpoint_pack(kept_u, cu)
    again = _backward(dh.to(t), x.to(t), wg.to(t), wu.to(t), cg, cu, rar.ACT_GELU, t)
    assert torch.equal(again[0], res[0]) and torch.equal(again[1], (dg.t() @ x.double()).to(t))
    # forward into checkpoints: the bytes that packing the exact projections gives
    if float((x.double() @ wg.double().t()).abs().max()) < 2 ** 24:
        rar.gated_ff_forward(x.to(t), wg.to(t), wu.to(t), out, act=rar.ACT_GELU, gate=cg, up=cu)
        want = _bytes(n)
        for buf, w in ((cg, wg), (cu, wu)):
            rar.checkpoint_pack((x.double() @ w.double().t()).float(), want)
            assert torch.equal(buf, want)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,hidden", [(12, 40, 72), (130, 200, 150), (300, 136, 72)])
def test_strided_unaligned_and_broadcast(rows, dim, hidden, dt):
    """Columns of wider matrices, off 16-byte boundaries, the weights as halves
    of one matrix, one row for all, and what lies beside the outputs."""
    t = DTYPES[dt]
    big = torch.randn(rows, dim + 11, device=DEV).to(t)
    both = (torch.randn(2 * hidden, dim + 3, device=DEV) * dim ** -0.5).to(t)
    x, wg, wu = big[:, 5:5 + dim], both[:hidden, 1:1 + dim], both[hidden:, 1:1 + dim]
    dh = torch.randn(rows, 2 * hidden + 1, device=DEV).to(t)[:, 3:3 + hidden]
    _check_all(x, wg, wu, dh, rar.ACT_SILU, t)
    # outputs as columns of one matrix
    wide = torch.full((rows, 3 * hidden + 5), 4.0, device=DEV, dtype=t)
    out, gate, up = (wide[:, 1 + i * (hidden + 1):1 + i * (hidden + 1) + hidden] for i in range(3))
    rar.gated_ff_forward(x, wg, wu, out, gate=gate, up=up)
    plain = [torch.empty(rows, hidden, device=DEV, dtype=t) for _ in range(3)]
    rar.gated_ff_forward(x.contiguous(), wg.contiguous(), wu.contiguous(), plain[0], gate=plain[1], up=plain[2])
    for a, b in zip((out, gate, up), plain):
        assert torch.equal(a, b)
    beside = torch.ones(wide.shape[1], dtype=torch.bool)
    for i in range(3):
        beside[1 + i * (hidden + 1):1 + i * (hidden + 1) + hidden] = False
    assert bool((wide[:, beside.to(DEV)] == 4.0).all())
    grads = torch.full((2 * hidden, dim + 5), 4.0, device=DEV, dtype=t)
    dxs = torch.full((rows, dim + 4), 4.0, device=DEV, dtype=t)
    ws = _bytes(rar.gated_ff_workspace_bytes(rows, dim, hidden, t))
    rar.gated_ff_backward(dh, x, wg, wu, gate, up, dxs[:, 3:3 + dim], grads[:hidden, 2:2 + dim],
                          grads[hidden:, 2:2 + dim], ws)
    want = _backward(dh.contiguous(), x.contiguous(), wg.contiguous(), wu.contiguous(), plain[1], plain[2],
                     rar.ACT_SILU, t)
    assert torch.equal(dxs[:, 3:3 + dim], want[0])
    assert torch.equal(grads[:hidden, 2:2 + dim], want[1]) and torch.equal(grads[hidden:, 2:2 + dim], want[2])
    assert bool((dxs[:, :3] == 4.0).all()) and bool((dxs[:, 3 + dim:] == 4.0).all())
    assert bool((grads[:, :2] == 4.0).all()) and bool((grads[:, 2 + dim:] == 4.0).all())
    one = torch.randn(dim, device=DEV).to(t).expand(rows, dim)
    dh1 = torch.randn(hidden, device=DEV).to(t).expand(rows, hidden)
    _check_all(one, wg, wu, dh1, rar.ACT_GELU_TANH, t)


def test_leading_dimensions():
    x, wg, wu, dh = _normal(24, 48, 80, torch.bfloat16)
    flat = torch.empty(24, 80, device=DEV, dtype=x.dtype)
    rar.gated_ff_forward(x, wg, wu, flat)
    out = torch.empty(2, 3, 4, 80, device=DEV, dtype=x.dtype)
    rar.gated_ff_forward(x.view(2, 3, 4, 48), wg, wu, out)
    assert torch.equal(out.view(24, 80), flat)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,dim,hidden", [(5, 40, 48), (150, 72, 90), (150, 71, 91)])
def test_infinite_and_nan_values_stay_in_their_rows(rows, dim, hidden, dt):
    """A token with an infinity or NaN spoils its own row and the weights'
    gradients, never another row, nor another row's checkpoint."""
    t = DTYPES[dt]
    x, wg, wu, dh = _normal(rows, dim, hidden, t)
    clean = torch.empty(rows, hidden, device=DEV, dtype=t)
    n = rar.checkpoint_bytes(rows, hidden)
    bufs = [_bytes(n) for _ in range(4)]
    rar.gated_ff_forward(x, wg, wu, clean, gate=bufs[0], up=bufs[1])
    bad = x.clone()
    bad[1, dim - 1], bad[3, 0] = math.nan, math.inf
    out = torch.empty_like(clean)
    rar.gated_ff_forward(bad, wg, wu, out, gate=bufs[2], up=bufs[3])
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[[1, 3]] = False
    assert torch.equal(out[keep], clean[keep]) and bool(out[1].isnan().all())
    vals = [torch.empty(rows, hidden, device=DEV) for _ in range(4)]
    for b, v in zip(bufs, vals):
        rar.checkpoint_unpack(b, v)
    for a, b in ((0, 2), (1, 3)):
        assert torch.equal(vals[a][keep], vals[b][keep]) and bool(vals[b][[1, 3]].isnan().all())
    dx0 = _backward(dh, x, wg, wu, bufs[0], bufs[1], 0, t)[0]
    dx, dwg, dwu = _backward(dh, bad, wg, wu, bufs[2], bufs[3], 0, t)
    assert torch.equal(dx[keep], dx0[keep]) and bool(dx[[1, 3]].isnan().all())
    assert bool(dwg.isnan().all()) and bool(dwu.isnan().all())


def test_large_gates():
    """Activations far out: no NaN from an overflowing exponential."""
    gates = torch.tensor([-1e30, -2000.0, -100.0, -89.0, -88.0, -20.0, -0.0, 0.0, 20.0, 89.0, 100.0, 2000.0, 1e30])
    wg, wu = gates[:, None].to(DEV), torch.ones(13, 1, device=DEV)
    x = torch.ones(70, 1, device=DEV)
    for kind in range(3):
        _check = torch.empty(70, 13, device=DEV)
        g, u = torch.empty_like(_check), torch.empty_like(_check)
        rar.gated_ff_forward(x, wg, wu, _check, act=kind, gate=g, up=u)
        want = block_ref.act(gates.double(), kind)[0].expand(70, 13)
        assert_within(_check, want, want.abs() * 2.0 ** -20 + 2.0 ** -100 * 0 + gates.abs().double() * 2.0 ** -126 * 4,
                      f"activation {kind}")
        dx, dwg, _ = _backward(torch.ones(70, 13, device=DEV), x, wg, wu, g, u, kind, torch.float32)
        d = block_ref.act(gates.double(), kind)[1]
        assert_within(dwg[:, 0], 70 * d, 70 * (d.abs() * 2.0 ** -18 + 2.0 ** -100) + 70 * 100 * 2.0 ** -24, "slope")


def test_no_rows():
    x, wg, wu, dh = _normal(0, 24, 40, torch.bfloat16)
    out = torch.empty(0, 40, dtype=x.dtype, device=DEV)
    rar.gated_ff_forward(x, wg, wu, out, gate=out.clone(), up=out.clone())
    dx, dwg, dwu = _backward(dh, x, wg, wu, out, out.clone(), 0, x.dtype)
    assert bool((dwg == 0).all()) and bool((dwu == 0).all())
    old = [torch.randn(40, 24, device=DEV).to(x.dtype) for _ in range(2)]
    dx, dwg, dwu = _backward(dh, x, wg, wu, out, out.clone(), 0, x.dtype, old)
    assert torch.equal(dwg, old[0]) and torch.equal(dwu, old[1])


def test_gradients_against_differences():
    """dx and dw against central differences of the library's own forward."""
    rows, dim, hidden, eps = 6, 20, 24, 2.0 ** -7
    x, wg, wu, dh = _normal(rows, dim, hidden, torch.float32)
    for kind in range(3):
        gate, up, out = (torch.empty(rows, hidden, device=DEV) for _ in range(3))

        def loss(a, b, c):
            o = torch.empty(rows, hidden, device=DEV)
            rar.gated_ff_forward(a, b, c, o, act=kind)
            return float((o.double() * dh.double()).sum())

        rar.gated_ff_forward(x, wg, wu, out, act=kind, gate=gate, up=up)
        grads = _backward(dh, x, wg, wu, gate, up, kind, torch.float32)
        for which, (t, gr) in enumerate(zip((x, wg, wu), grads)):
            for i in (0, 7, t.numel() - 1):
                vals = []
                for sign in (1, -1):
                    args = [x.clone(), wg.clone(), wu.clone()]
                    args[which].view(-1)[i] += sign * eps
                    vals.append(loss(*args))
                # third derivatives stay below 4 per term: eps^2 of a sum of at
                # most 24 terms, and binary32 forward values over 2 eps
                size = float(dh.abs().sum())
                tol = eps ** 2 * 24 * 8 + 2.0 ** -20 * size / eps
                assert abs((vals[0] - vals[1]) / (2 * eps) - float(gr.view(-1)[i])) < tol, (kind, which, i)


@pytest.mark.parametrize("rows", [7, 300])
def test_replays_in_a_graph_and_other_streams(rows):
    """Two graphs that share a workspace, replayed in turn with eager steps."""
    dim, hidden, t = 264, 200, torch.bfloat16
    x, wg, wu, dh = _normal(rows, dim, hidden, t)
    out, dx = torch.empty(rows, hidden, device=DEV, dtype=t), torch.empty_like(x)
    n = rar.checkpoint_bytes(rows, hidden)
    held = [_bytes(n), _bytes(n)]
    kept = [torch.empty_like(out), torch.empty_like(out)]
    dwg, dwu = torch.empty(hidden, dim, device=DEV), torch.empty(hidden, dim, device=DEV)
    ws = _bytes(rar.gated_ff_workspace_bytes(rows, dim, hidden, t))

    def step(keep, stream=None):
        rar.gated_ff_forward(x, wg, wu, out, gate=keep[0], up=keep[1], stream=stream)
        rar.gated_ff_backward(dh, x, wg, wu, keep[0], keep[1], dx, dwg, dwu, ws, stream=stream)

    outs = (out, dx, dwg, dwu)
    for keep in (held, kept):
        step(keep)
    torch.cuda.synchronize()
    graphs = []
    for keep in (held, kept):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(keep)
    side = torch.cuda.Stream()
    for k in range(6):
        x.copy_(_normal(rows, dim, hidden, t, seed=k + 1)[0])
        keep = (held, kept)[k % 2]
        step(keep)
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        if k < 4:
            graphs[k % 2].replay()
        else:
            step(keep, side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs)), k


def _whole(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV).to(torch.bfloat16)


def _kept_gradients(dh, kept_g, kept_u):
    """dg and du (64 bits) of gates of 0 and 64 through the gelu, exact."""
    return dh.double() * kept_u.double() * torch.where(kept_g > 0, 1.0, 0.5), dh.double() * kept_g.double()


def test_rows_past_four_gib():
    """x and dx of 4.2 GiB: the first and the last rows hold whole numbers, the
    others zeros, so that both gradients of the weights are exact."""
    rows, dim, hidden, ends = 1_100_003, 2048, 40, 300
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device=DEV)
    dh, up, gate, out = (torch.zeros(rows, hidden, dtype=torch.bfloat16, device=DEV) for _ in range(4))
    wg, wu = _whole(g, -1, 1, hidden, dim), _whole(g, -1, 1, hidden, dim)
    for part in (slice(0, ends), slice(rows - ends, rows)):
        x[part] = _whole(g, -2, 2, ends, dim)
    rar.gated_ff_forward(x, wg, wu, out, act=rar.ACT_GELU, gate=gate, up=up)
    for part in (slice(0, ends), slice(rows - ends, rows)):
        assert torch.equal(gate[part], (x[part].double() @ wg.double().t()).bfloat16()), part
        assert torch.equal(up[part], (x[part].double() @ wu.double().t()).bfloat16()), part
    assert not bool(gate[ends:-ends].any()) and not bool(out[ends:-ends].any())
    want = [torch.zeros(hidden, dim, dtype=torch.float64, device=DEV) for _ in range(2)]
    pieces = []
    for part in (slice(0, ends), slice(rows - ends, rows)):
        dh[part], gate[part], up[part] = (_whole(g, -1, 1, ends, hidden), 64 * _whole(g, 0, 1, ends, hidden),
                                          _whole(g, -2, 2, ends, hidden))
        dg, du = _kept_gradients(dh[part], gate[part], up[part])
        want[0] += dg.t() @ x[part].double()
        want[1] += du.t() @ x[part].double()
        pieces.append((part, (dg @ wg.double() + du @ wu.double()).bfloat16()))
    dx, dwg, dwu = _backward(dh, x, wg, wu, gate, up, rar.ACT_GELU, torch.float32)
    for part, value in pieces:
        assert torch.equal(dx[part], value), part
    assert not bool(dx[ends:-ends].any())
    assert torch.equal(dwg, want[0].float()) and torch.equal(dwu, want[1].float())


@pytest.mark.parametrize("rows", [2, 5, 40, 70])
def test_weights_past_four_gib(rows):
    """Weights and their gradients of 4.3 GiB each, with whole numbers in the
    first and the last rows and zeros between them."""
    hidden, dim, ends = 1_048_576, 2200, 200
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = _whole(g, -2, 2, rows, dim)
    wg, wu = (torch.zeros(hidden, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dh, gate, up, out = (torch.zeros(rows, hidden, dtype=torch.bfloat16, device=DEV) for _ in range(4))
    parts = (slice(0, ends), slice(hidden - ends, hidden))
    for part in parts:
        wg[part], wu[part] = _whole(g, -1, 1, ends, dim), _whole(g, -1, 1, ends, dim)
    rar.gated_ff_forward(x, wg, wu, out, act=rar.ACT_GELU, gate=gate, up=up)
    for part in parts:
        assert torch.equal(gate[:, part], (x.double() @ wg[part].double().t()).bfloat16()), part
        assert torch.equal(up[:, part], (x.double() @ wu[part].double().t()).bfloat16()), part
    assert not bool(gate[:, ends:-ends].any()) and not bool(out[:, ends:-ends].any())
    want_dx, want_dw = 0, []
    for part in parts:
        dh[:, part], gate[:, part], up[:, part] = (_whole(g, -1, 1, rows, ends), 64 * _whole(g, 0, 1, rows, ends),
                                                   _whole(g, -2, 2, rows, ends))
        dg, du = _kept_gradients(dh[:, part], gate[:, part], up[:, part])
        want_dx = want_dx + dg @ wg[part].double() + du @ wu[part].double()
        want_dw.append((part, (dg.t() @ x.double()).bfloat16(), (du.t() @ x.double()).bfloat16()))
    dx, dwg, dwu = _backward(dh, x, wg, wu, gate, up, rar.ACT_GELU, torch.bfloat16)
    assert torch.equal(dx, want_dx.bfloat16())
    for part, value_g, value_u in want_dw:
        assert torch.equal(dwg[part], value_g) and torch.equal(dwu[part], value_u), part
    assert not bool(dwg[ends:-ends].any()) and not bool(dwu[ends:-ends].any())
