"""Gated feed-forward block at sizes that one launch, or 32 bits, cannot hold."""
import pytest
import torch

import ring_all_reduce_scatter_amd as rar
from operator_ref import DTYPES

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("hidden,dim", [(40, 72), (1 << 20, 1 << 14)])
def test_no_rows_and_many_weights(hidden, dim):
    """Without rows the weights' gradients become zeros: of the larger size 2^34
    elements each, four to a thread more threads than a launch has."""
    t = torch.bfloat16
    w = torch.ones(1, dim, dtype=t, device=DEV).expand(hidden, dim)
    x, none = torch.empty(0, dim, dtype=t, device=DEV), torch.empty(0, hidden, dtype=t, device=DEV)
    dw = [torch.full((hidden, dim), 3.0, dtype=t, device=DEV) for _ in range(2)]
    rar.gated_ff_backward(none, x, w, w, none, none.clone(), None, *dw, None, accumulate=True)
    assert all(bool((d[i] == 3.0).all()) for d in dw for i in (0, hidden // 2, hidden - 1))
    rar.gated_ff_backward(none, x, w, w, none, none.clone(), None, *dw, None)
    for d in dw:
        for part in d.view(torch.int16).split(1 << 16):
            assert not bool(part.any())


def _whole(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV).float()


# unsplit large tiles of the weights' gradients, small ones, and splits
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,dim,hidden", [(70, 2056, 4104), (2100, 72, 4104), (2048, 2048, 2048), (700, 520, 264),
                                             (1000, 33, 31), (3000, 64, 64), (4100, 2056, 1032)])
def test_accumulates_bit_by_bit(rows, dim, hidden, dt):
    """Whole numbers in the weights' gradients before the call, from kept rows
    and from checkpoints, into both types: the sums are exact and rounded once."""
    t = DTYPES[dt]
    g = torch.Generator(device=DEV).manual_seed(rows + dim + hidden)
    x, wg, wu = _whole(g, -2, 2, rows, dim), _whole(g, -1, 1, hidden, dim), _whole(g, -1, 1, hidden, dim)
    # gates of 0 and 64 make the gelu's value (0, 64) and slope (1/2, 1) exact
    gate, up, dh = 64 * _whole(g, 0, 1, rows, hidden), _whole(g, -2, 2, rows, hidden), _whole(g, -1, 1, rows, hidden)
    dg, du = (dh * up * torch.where(gate > 0, 1.0, 0.5)).double(), (dh * gate).double()
    dx = (dg @ wg.double() + du @ wu.double()).to(t)
    held = [torch.empty(rar.checkpoint_bytes(rows, hidden), dtype=torch.uint8, device=DEV) for _ in range(2)]
    rar.checkpoint_pack(gate, held[0])
    rar.checkpoint_pack(up, held[1])
    ws = torch.empty(rar.gated_ff_workspace_bytes(rows, dim, hidden, t), dtype=torch.uint8, device=DEV)
    for wdt in {torch.float32, t}:
        old = [_whole(g, -100, 100, hidden, dim).to(wdt) for _ in range(2)]
        want = [(o.double() + p.t() @ x.double()).to(wdt) for o, p in zip(old, (dg, du))]
        for kept in ((gate.to(t), up.to(t)), held):
            got = [torch.full((rows, dim), 7.0, dtype=t, device=DEV), *(o.clone() for o in old)]
            rar.gated_ff_backward(dh.to(t), x.to(t), wg.to(t), wu.to(t), *kept, *got, ws, act=rar.ACT_GELU,
                                  accumulate=True)
            for a, b, name in zip(got, (dx, *want), ("dx", "dwgate", "dwup")):
                assert torch.equal(a, b), name


def test_projections_past_four_gib():
    """Projections of 4.6 thousand million elements, so that h, the kept rows,
    the checkpoints' codes and the workspace's dg and du all pass 4 GiB: whole
    numbers in the first and the last rows of x and of the weights, zeros
    between them."""
    rows, dim, hidden, ends, t = 70_003, 40, 65_600, 300, torch.bfloat16
    g = torch.Generator(device=DEV).manual_seed(5)
    row_ends, col_ends = ((slice(0, ends), slice(n - ends, n)) for n in (rows, hidden))
    x, wg, wu = (torch.zeros(n, dim, dtype=t, device=DEV) for n in (rows, hidden, hidden))
    for r in row_ends:
        x[r] = _whole(g, -2, 2, ends, dim).to(t)
    for c in col_ends:
        wg[c], wu[c] = _whole(g, -1, 1, ends, dim).to(t), _whole(g, -1, 1, ends, dim).to(t)

    def corners_only(m):
        assert not any(bool(p.view(torch.int16).any()) for p in m[ends:-ends].split(4096))
        assert not bool(m[:, ends:-ends][:ends].any()) and not bool(m[:, ends:-ends][-ends:].any())

    gate, up, out = (torch.full((rows, hidden), 9.0, dtype=t, device=DEV) for _ in range(3))
    rar.gated_ff_forward(x, wg, wu, out, act=rar.ACT_GELU, gate=gate, up=up)
    for m, w in ((gate, wg), (up, wu)):
        for r in row_ends:
            for c in col_ends:
                assert torch.equal(m[r, c], (x[r].double() @ w[c].double().t()).to(t))
    held = [torch.empty(rar.checkpoint_bytes(rows, hidden), dtype=torch.uint8, device=DEV) for _ in range(2)]
    again = torch.empty_like(out)
    rar.gated_ff_forward(x, wg, wu, again, act=rar.ACT_GELU, gate=held[0], up=held[1])
    assert torch.equal(again, out)
    # sums of at most 80, of which a block's step is 1 at most
    for buf, m in zip(held, (gate, up)):
        rar.checkpoint_unpack(buf, again)
        assert torch.equal(again, m)
        again.copy_(m)
        corners_only(again.abs_())  # without the sign of a zero
    dh = out.zero_()
    gate.zero_()
    up.zero_()
    want_dx, want_dw = {}, {}
    for i, r in enumerate(row_ends):
        for j, c in enumerate(col_ends):
            dh[r, c], gate[r, c], up[r, c] = (_whole(g, -1, 1, ends, ends).to(t), 64 * _whole(g, 0, 1, ends, ends).to(t),
                                              _whole(g, -2, 2, ends, ends).to(t))
            dg = dh[r, c].double() * up[r, c].double() * torch.where(gate[r, c] > 0, 1.0, 0.5)
            du = dh[r, c].double() * gate[r, c].double()
            want_dx[i] = want_dx.get(i, 0) + dg @ wg[c].double() + du @ wu[c].double()
            for k, d in enumerate((dg, du)):
                want_dw[j, k] = want_dw.get((j, k), 0) + d.t() @ x[r].double()
    rar.checkpoint_pack(gate, held[0])
    rar.checkpoint_pack(up, held[1])
    ws = torch.empty(rar.gated_ff_workspace_bytes(rows, dim, hidden, t), dtype=torch.uint8, device=DEV)
    for kept in ((gate, up), held):
        dx = torch.full((rows, dim), 7.0, dtype=t, device=DEV)
        dw = [torch.full((hidden, dim), 3.0, device=DEV) for _ in range(2)]
        rar.gated_ff_backward(dh, x, wg, wu, *kept, dx, *dw, ws, act=rar.ACT_GELU)
        for i, r in enumerate(row_ends):
            assert torch.equal(dx[r], want_dx[i].to(t)), i
        assert not bool(dx[ends:-ends].any())
        for j, c in enumerate(col_ends):
            for k, name in enumerate(("dwgate", "dwup")):
                assert torch.equal(dw[k][c], want_dw[j, k].float()), (name, j)
        assert not any(bool(d[ends:-ends].any()) for d in dw)
