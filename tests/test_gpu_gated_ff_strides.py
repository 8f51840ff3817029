"""Gated feed-forward block with weights whose rows lie differently far apart,
bit by bit on whole numbers, whose sums are exact in any order."""
import pytest
import torch

import ring_all_reduce_scatter_amd as rar
from operator_ref import DTYPES

pytestmark = pytest.mark.gpu

DEV = "cuda:0"

# dx in large tiles, whole and in splits of which one holds the end of gate's
# terms and the start of up's; in small tiles, whole and likewise split; of
# odd width, where both weights are copied; forward and dx of few tokens
SHAPES = [(4096, 4096, 136), (2048, 2048, 2100), (2048, 2048, 200), (130, 264, 1030), (70, 129, 67), (20, 520, 72),
          (1, 64, 40)]
# elements between the rows beyond dim of wgate and of wup; None: one row for all
STEPS = [(0, 8), (24, 0), (0, 3), (5, 0), (16, 48), (None, 0), (0, None), (None, 8), (3, None)]


def _matrix(values, step, first, room):
    """The values as rows dim + step elements apart from element `first` on, in
    a buffer of `room` elements of 77 that holds either matrix's steps."""
    hidden, dim = values.shape
    buf = torch.full((room,), 77.0, dtype=values.dtype, device=DEV)
    if step is None:
        view = buf.as_strided((1, dim), (dim, 1), first)
        view.copy_(values[:1])
        return view.expand(hidden, dim)
    view = buf.as_strided((hidden, dim), (dim + step, 1), first)
    view.copy_(values)
    return view


@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("steps", STEPS)
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,dim,hidden", SHAPES)
def test_weights_of_different_strides(rows, dim, hidden, dt, steps, first):
    """Gates of 0 and 64 make the gelu's value (0, 64) and slope (1/2, 1) exact,
    so that only the outputs are rounded."""
    t = DTYPES[dt]
    g = torch.Generator(device=DEV).manual_seed(rows + dim + hidden)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device=DEV).to(t)

    room = hidden * (dim + max(s or 0 for s in steps)) + first + 64
    x = ints(-2, 2, rows, dim)
    wg, wu = (_matrix(ints(-1, 1, hidden, dim), s, first, room) for s in steps)
    gate, up, out = (torch.full((rows, hidden), 9.0, dtype=t, device=DEV) for _ in range(3))
    rar.gated_ff_forward(x, wg, wu, out, act=rar.ACT_GELU, gate=gate, up=up)
    assert torch.equal(gate, (x.double() @ wg.double().t()).to(t)), "gate"
    assert torch.equal(up, (x.double() @ wu.double().t()).to(t)), "up"
    gate, up, dh = 64 * ints(0, 1, rows, hidden), ints(-2, 2, rows, hidden), ints(-1, 1, rows, hidden)
    dg = dh.double() * up.double() * torch.where(gate > 0, 1.0, 0.5)
    du = dh.double() * gate.double()
    dx = torch.full((rows, dim), 7.0, dtype=t, device=DEV)
    dwg, dwu = (torch.full((hidden, dim), 3.0, device=DEV) for _ in range(2))
    ws = torch.empty(rar.gated_ff_workspace_bytes(rows, dim, hidden, t), dtype=torch.uint8, device=DEV)
    rar.gated_ff_backward(dh, x, wg, wu, gate, up, dx, dwg, dwu, ws, act=rar.ACT_GELU)
    assert torch.equal(dx, (dg @ wg.double() + du @ wu.double()).to(t)), "dx"
    assert torch.equal(dwg, (dg.t() @ x.double()).float()), "dwgate"
    assert torch.equal(dwu, (du.t() @ x.double()).float()), "dwup"


# products of which large tiles, had they been taken, would be split more often
# than the small ones that rows off 16 bytes take: dx unsplit and in two splits,
# the weights' gradients in two
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows,dim,hidden", [(1024, 4096, 2056), (16384, 104, 2100), (4100, 104, 8192)])
def test_rows_off_16_bytes_in_small_tiles(rows, dim, hidden, dt):
    t = DTYPES[dt]
    g = torch.Generator(device=DEV).manual_seed(rows + dim + hidden)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device=DEV).to(t)

    aligned = ints(-2, 2, rows, dim), ints(-1, 1, hidden, dim), ints(-1, 1, hidden, dim)
    off = [_matrix(m, 0, 1, m.numel() + 8) for m in aligned]
    gate, up, dh = 64 * ints(0, 1, rows, hidden), ints(-2, 2, rows, hidden), ints(-1, 1, rows, hidden)
    dg = dh.double() * up.double() * torch.where(gate > 0, 1.0, 0.5)
    du = dh.double() * gate.double()
    x, wg, wu = (m.double() for m in aligned)
    old = [ints(-8, 8, hidden, dim).float() for _ in range(2)]
    want = [(dg @ wg + du @ wu).to(t), (old[0].double() + dg.t() @ x).float(), (old[1].double() + du.t() @ x).float()]
    ws = torch.empty(rar.gated_ff_workspace_bytes(rows, dim, hidden, t), dtype=torch.uint8, device=DEV)
    for operands in (aligned, off):
        dx = torch.full((rows, dim), 7.0, dtype=t, device=DEV)
        dw = [o.clone() for o in old]
        rar.gated_ff_backward(dh, *operands, gate, up, dx, *dw, ws, act=rar.ACT_GELU, accumulate=True)
        for got, value, name in zip((dx, *dw), want, ("dx", "dwgate", "dwup")):
            assert torch.equal(got, value), name
