"""Activation checkpoints in 8 bits on the GPU: their bytes and values against
the definition, and layer norm with its input held in one."""
import math

import pytest
import torch

import block_ref
import operator_ref as ref
import ring_all_reduce_scatter_amd as rar
from operator_ref import DTYPES, assert_within

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
GUARD = 64


def _buffer(rows, dim):
    """A checkpoint's bytes with a guard after them."""
    return torch.full((rar.checkpoint_bytes(rows, dim) + GUARD,), 0xA5, dtype=torch.uint8, device=DEV)


def _check_bytes(buf, x, what=""):
    want = block_ref.held_bytes(x)
    got = buf.cpu()
    n = want.numel()
    assert got.numel() == n + GUARD and bool((got[n:] == 0xA5).all()), f"{what}: bytes past the checkpoint"
    bad = (got[:n] != want).nonzero()
    assert not bad.numel(), f"{what}: {bad.numel()} bytes differ, first at {int(bad[0])}"


def _values(rows, dim, dt, seed=0):
    """Rows and blocks of very different size, zeros among them."""
    g = torch.Generator(device=DEV).manual_seed(seed + rows * 131 + dim)
    x = torch.randn(rows, dim, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-12, 12, (rows, dim), generator=g, device=DEV).float())
    x[torch.rand(rows, dim, generator=g, device=DEV) < 0.1] = 0.0
    return x.to(dt)


SHAPES = [(1, 1), (1, 31), (1, 32), (2, 33), (3, 64), (5, 7), (70, 129), (257, 200), (33, 513), (9, 1001), (4, 4096),
          (3, 8192), (2, 16391), (1000, 40), (4099, 65)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_bytes_and_values(rows, dim, dt):
    x = _values(rows, dim, DTYPES[dt])
    buf = _buffer(rows, dim)
    rar.checkpoint_pack(x, buf)
    _check_bytes(buf, x)
    values = block_ref.held(x)[2]
    for out in DTYPES.values():
        y = torch.full((rows + 1, dim), 7.0, dtype=out, device=DEV)
        rar.checkpoint_unpack(buf, y[:rows])
        assert torch.equal(y[:rows].cpu(), values.to(out)) and bool((y[rows] == 7.0).all()), out
    # half a step, or what the clamp at 127 takes (a value that rounds to 128)
    err = (values - x.cpu().double()).abs()
    top = torch.nn.functional.pad(x.cpu().double().abs(), (0, -dim % 32)).view(rows, -1, 32).amax(2, keepdim=True)
    assert bool((torch.nn.functional.pad(err, (0, -dim % 32)).view(rows, -1, 32) <= top * 2.0 ** -7).all())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_special_values(dt):
    t = DTYPES[dt]
    info = torch.finfo(t)
    x = torch.randn(14, 96).to(t)
    x[0, 5], x[1, 40], x[2, 95] = math.inf, -math.inf, math.nan
    x[3] = 0.0
    x[4] = -0.0
    x[5, :32], x[5, 3] = info.tiny / 8, -info.tiny  # subnormals
    x[6] = info.tiny * info.eps  # the smallest value
    x[7] = info.max
    x[8] = -info.max
    x[9, ::2] = info.max
    x[10, 32:64] = 1.0  # a whole power of two
    x[11, :32] = torch.tensor([127.5, 126.5, 1.5, 0.5, 2.5, -0.5, -1.5, 127.4375] * 4).to(t)  # ties, and one at the clamp
    x[12, 0], x[12, 33] = math.inf, math.nan
    x[13, :] = torch.tensor([1e-30, 1.0, 2.0 ** -7, 2.0 ** -8 * 1.0] * 24).to(t)
    x = x.to(DEV)
    buf = _buffer(14, 96)
    rar.checkpoint_pack(x, buf)
    _check_bytes(buf, x)
    y = torch.empty(14, 96, device=DEV)
    rar.checkpoint_unpack(buf, y)
    want = block_ref.held(x)[2].float()
    assert torch.equal(y.cpu().nan_to_num(nan=-1e38), want.nan_to_num(nan=-1e38))
    assert bool(y[0, :32].isnan().all()) and bool(torch.isfinite(y[0, 32:]).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [33, 100, 1000])
def test_strided_unaligned_and_broadcast_rows(dt, dim):
    t = DTYPES[dt]
    store = _values(30, dim + 9, t).view(6, 5, dim + 9)
    x = store[:, :, 1:1 + dim]
    buf = _buffer(30, dim)
    rar.checkpoint_pack(x, buf)
    _check_bytes(buf, x.reshape(30, dim), "strided")
    out = torch.full((6, 5, dim + 5), 4.0, device=DEV, dtype=t)
    rar.checkpoint_unpack(buf, out[:, :, 3:3 + dim])
    assert torch.equal(out[:, :, 3:3 + dim].reshape(30, dim).cpu(), block_ref.held(x.reshape(30, dim))[2].to(t))
    assert bool((out[:, :, :3] == 4.0).all()) and bool((out[:, :, 3 + dim:] == 4.0).all())
    same = x[0, 0].expand(30, dim)
    rar.checkpoint_pack(same, buf)
    _check_bytes(buf, same, "broadcast")


def test_no_rows():
    x = torch.empty(0, 40, device=DEV)
    buf = torch.empty(0, dtype=torch.uint8, device=DEV)
    rar.checkpoint_pack(x, buf)
    rar.checkpoint_unpack(buf, x)
    w, s = torch.ones(40, device=DEV), torch.empty(0, device=DEV)
    rar.layernorm_forward_checkpoint(x, w, w, torch.empty_like(x), buf, mean=s, rstd=s)
    dw, db = torch.full((40,), 3.0, device=DEV), torch.full((40,), 3.0, device=DEV)
    ws = torch.empty(rar.layernorm_workspace_bytes(0, 40), dtype=torch.uint8, device=DEV)
    rar.layernorm_backward_checkpoint(x, buf, w, s, s, torch.empty_like(x), dw, db, ws)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_large_matrix():
    """Offsets past 32 bits: 4.3 billion bytes of bf16, 2.2 billion codes."""
    rows, dim = 2 ** 19 + 3, 4100
    x = torch.empty(rows, dim, dtype=torch.bfloat16, device=DEV)
    part = _values(1027, dim, torch.bfloat16)
    for i in range(0, rows, 1027):
        x[i:i + 1027] = part[:min(1027, rows - i)]
    buf = torch.empty(rar.checkpoint_bytes(rows, dim), dtype=torch.uint8, device=DEV)
    rar.checkpoint_pack(x, buf)
    y = torch.empty_like(x)
    rar.checkpoint_unpack(buf, y)
    want = block_ref.held(part)[2].to(torch.bfloat16).to(DEV)
    for i in list(range(0, rows, 1027 * 97)) + [rows // 1027 * 1027]:
        n = min(1027, rows - i)
        assert torch.equal(y[i:i + n], want[:n]), i


# ------------------------------------------------------------------ layer norm

LN_SHAPES = [(1, 1), (3, 2), (1, 64), (5, 63), (70, 129), (4, 512), (33, 513), (257, 768), (1, 1000), (130, 1024),
             (9, 1025), (65, 2048), (3, 2049), (40, 4096), (17, 4097), (5, 8192), (11, 8191), (3, 16384), (2, 16391),
             (3, 20_003), (2000, 96), (9000, 33), (37, 2561), (20, 1300), (600, 40), (513, 2570), (1, 300), (64, 1056)]


@pytest.mark.parametrize("dts", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("rows,dim", LN_SHAPES)
def test_layernorm_from_a_checkpoint(rows, dim, dts):
    """Forward: the bits of layernorm_forward and of checkpoint_pack.
    Backward: dx has the bits of layernorm_backward on the checkpoint's values
    (which binary32 and bfloat16 hold exactly), and everything is the formula's
    within its bound."""
    xt, wt = DTYPES[dts[0]], DTYPES[dts[1]]
    g = torch.Generator(device=DEV).manual_seed(rows + dim)
    x = (torch.randn(rows, dim, generator=g, device=DEV) * 2 + 0.5).to(xt)
    w = (1 + 0.2 * torch.randn(dim, generator=g, device=DEV)).to(wt)
    b = torch.randn(dim, generator=g, device=DEV).to(wt)
    dy = torch.randn(rows, dim, generator=g, device=DEV).to(xt)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    mean, rstd, mean2, rstd2 = (torch.empty(rows, device=DEV) for _ in range(4))
    buf = _buffer(rows, dim)
    rar.layernorm_forward(x, w, b, y, mean=mean, rstd=rstd)
    rar.layernorm_forward_checkpoint(x, w, b, y2, buf, mean=mean2, rstd=rstd2)
    assert torch.equal(y, y2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    _check_bytes(buf, x)
    held = torch.empty_like(x)
    rar.checkpoint_unpack(buf, held)
    if xt == torch.float16:
        assert torch.equal(held.double().cpu(), block_ref.held(x)[2])  # exact in this range too
    ws = torch.empty(rar.layernorm_workspace_bytes(rows, dim), dtype=torch.uint8, device=DEV)
    for accumulate in (False, True):
        old = [torch.randn(dim, generator=g, device=DEV).to(wt) for _ in range(2)]
        res = []
        for from_checkpoint in (False, True):
            dx = torch.full_like(x, 7.0)
            dw, db = old[0].clone(), old[1].clone()
            if from_checkpoint:
                rar.layernorm_backward_checkpoint(dy, buf, w, mean, rstd, dx, dw, db, ws, accumulate=accumulate)
            else:
                rar.layernorm_backward(dy, held, w, mean, rstd, dx, dw, db, ws, accumulate=accumulate)
            res.append((dx, dw, db))
        # (the sums over rows are formed in groups whose size may differ)
        assert torch.equal(res[0][0], res[1][0]), f"accumulate={accumulate}"
        want = ref.layernorm_grad(dy, block_ref.held(x)[2], w, mean, rstd, xt, wt, *(old if accumulate else ()))
        for got, (r, tol), name in zip(res[1], want, ("dx", "dw", "db")):
            assert_within(got.reshape(r.shape), r, tol, name)
    only = torch.empty_like(x)
    rar.layernorm_backward_checkpoint(dy, buf, w, mean, rstd, only, None, None, None)
    assert torch.equal(only, res[1][0])


@pytest.mark.parametrize("dim", [100, 3001, 20_001])
def test_layernorm_in_place(dim):
    x = _values(7, dim, torch.float32)
    w, b, dy = torch.randn(dim, device=DEV), torch.randn(dim, device=DEV), torch.randn(7, dim, device=DEV)
    y, mean, rstd = torch.empty_like(x), torch.empty(7, device=DEV), torch.empty(7, device=DEV)
    rar.layernorm_forward(x, w, b, y, mean=mean, rstd=rstd)
    buf, z = _buffer(7, dim), x.clone()
    rar.layernorm_forward_checkpoint(z, w, b, z, buf)
    assert torch.equal(z, y)
    _check_bytes(buf, x)
    ws = torch.empty(rar.layernorm_workspace_bytes(7, dim), dtype=torch.uint8, device=DEV)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    rar.layernorm_backward_checkpoint(dy, buf, w, mean, rstd, dx, dw, db, ws)
    over, dw2, db2 = dy.clone(), torch.empty_like(w), torch.empty_like(w)
    rar.layernorm_backward_checkpoint(over, buf, w, mean, rstd, over, dw2, db2, ws)
    assert torch.equal(over, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_layernorm_with_infinite_and_nan_inputs(dt):
    x = torch.randn(6, 200, device=DEV).to(DTYPES[dt])
    x[1, 3], x[2, 64], x[4, 199] = math.inf, math.nan, -math.inf
    buf, y = _buffer(6, 200), torch.empty_like(x)
    rar.layernorm_forward_checkpoint(x, None, None, y, buf)
    _check_bytes(buf, x)
    assert all(bool(y[r].isnan().any()) == (r in (1, 2, 4)) for r in range(6))


def test_replays_in_a_graph_and_other_streams():
    rows, dim = 300, 520
    x = _values(rows, dim, torch.bfloat16)
    w, dy = torch.ones(dim, device=DEV), torch.randn(rows, dim, device=DEV).to(torch.bfloat16)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dw, db = torch.empty(dim, device=DEV), torch.empty(dim, device=DEV)
    buf = _buffer(rows, dim)
    ws = torch.empty(rar.layernorm_workspace_bytes(rows, dim), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        rar.layernorm_forward_checkpoint(x, w, None, y, buf, mean=mean, rstd=rstd, stream=stream)
        rar.layernorm_backward_checkpoint(dy, buf, w, mean, rstd, dx, dw, db, ws, stream=stream)
        rar.checkpoint_pack(x, buf, stream=stream)
        rar.checkpoint_unpack(buf, y, stream=stream)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    side = torch.cuda.Stream()
    for k in range(4):
        x.copy_(_values(rows, dim, torch.bfloat16, seed=k))
        step()
        want = [t.clone() for t in (dx, dw, db, y, buf)]
        for t in (dx, dw, db, y):
            t.zero_()
        buf[:-GUARD].zero_()
        torch.cuda.synchronize()
        if k % 2:
            graph.replay()
        else:
            step(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (dx, dw, db, y, buf))), k
        _check_bytes(buf, x)
