"""Embedding lookup and gradient on the GPU against the 64-bit formulas."""
import math

import pytest
import torch

import operator_ref as ref
import ring_all_reduce_scatter_amd as rar
from operator_ref import DTYPES, assert_within

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _ids(kind, tokens, vocab, seed=0, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed + 17 * tokens + vocab)
    if kind == "uniform":
        ids = torch.randint(0, vocab, (tokens,), generator=g)
    elif kind == "one":
        ids = torch.full((tokens,), vocab - 1)
    elif kind == "few":
        ids = torch.randint(0, min(vocab, 3), (tokens,), generator=g)
    elif kind == "skew":
        u = torch.rand(tokens, generator=g, dtype=torch.float64)
        ids = (torch.exp(u * math.log(vocab + 1.0)) - 1).long().clamp_(0, vocab - 1)
        ids[torch.rand(tokens, generator=g) < 0.2] = -1
    else:  # none
        ids = torch.where(torch.rand(tokens, generator=g) < 0.5, -1, vocab)
    return ids.to(dtype).to(DEV)


def _grad(dout, ids, vocab, dt, scale=1.0, padding=None, old=None):
    dim = dout.shape[-1]
    dw = torch.full((vocab, dim), 7.0, device=DEV, dtype=dt) if old is None else old.clone()
    ws = torch.empty(rar.embedding_workspace_bytes(ids.numel(), vocab, dim), dtype=torch.uint8, device=DEV)
    rar.embedding_backward(dout, ids, dw, ws, scale=scale, padding_id=padding, accumulate=old is not None)
    return dw


SHAPES = [(1, 1, 1), (1, 5, 64), (2, 300, 7), (63, 17, 33), (64, 64, 512), (65, 1000, 513), (500, 40, 1001),
          (3001, 4099, 96), (5000, 33_000, 40)]


@pytest.mark.parametrize("dts", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("tokens,vocab,dim", SHAPES)
def test_lookup_and_gradient_match_formula(tokens, vocab, dim, dts):
    act, wt = DTYPES[dts[0]], DTYPES[dts[1]]
    g = torch.Generator(device=DEV).manual_seed(tokens)
    w = torch.randn(vocab, dim, generator=g, device=DEV).to(wt)
    dout = torch.randn(tokens, dim, generator=g, device=DEV).to(act)
    scale = float(torch.tensor(math.sqrt(dim)))  # a binary32 number
    for k, kind in enumerate(("uniform", "one", "few", "skew", "none")):
        ids = _ids(kind, tokens, vocab, dtype=torch.int32 if k % 2 else torch.int64)
        out = torch.full((tokens, dim), 5.0, device=DEV, dtype=act)
        rar.embedding_forward(w, ids, out, scale=scale)
        assert_within(out, *ref.embedding(w, ids, scale, act), f"lookup {kind}")
        dw = _grad(dout, ids, vocab, wt, scale)
        assert_within(dw, *ref.embedding_grad(dout, ids, vocab, scale, wt), f"gradient {kind}")
        old = torch.randn(vocab, dim, generator=g, device=DEV).to(wt)
        dw = _grad(dout, ids, vocab, wt, scale, padding=int(ids[0]), old=old)
        assert_within(dw, *ref.embedding_grad(dout, ids, vocab, scale, wt, int(ids[0]), old), f"accumulated {kind}")


@pytest.mark.parametrize("tokens,vocab,dim,kind", [(40_000, 50_021, 256, "skew"), (30_000, 7, 64, "uniform"),
                                                   (20_000, 1, 136, "one"), (9000, 600_000, 16, "uniform"),
                                                   (70_000, 3, 24, "one")])
def test_long_batches_and_large_tables(tokens, vocab, dim, kind):
    ids = _ids(kind, tokens, vocab)
    dout = torch.randn(tokens, dim, device=DEV).to(torch.bfloat16)
    for dt in (torch.float32, torch.bfloat16):
        dw = _grad(dout, ids, vocab, dt, 0.5)
        assert_within(dw, *ref.embedding_grad(dout, ids, vocab, 0.5, dt), f"{dt}")
        assert torch.equal(dw, _grad(dout, ids, vocab, dt, 0.5)), "not the same bits twice"


def test_no_tokens():
    ids = torch.empty(0, dtype=torch.int64, device=DEV)
    w = torch.ones(10, 8, device=DEV)
    out = torch.empty(0, 8, device=DEV)
    rar.embedding_forward(w, ids, out)
    assert bool((_grad(out, ids, 10, torch.float32) == 0).all())
    old = torch.randn(10, 8, device=DEV)
    assert torch.equal(_grad(out, ids, 10, torch.float32, old=old), old)


def test_ids_that_would_wrap_are_outside():
    """64-bit ids keep their upper half: 2^32 + 1 is not row 1."""
    ids = torch.tensor([1, (1 << 32) + 1, -1, -(1 << 40), (1 << 63) - 1, 9, 10, 1 << 31], device=DEV)
    w = torch.arange(1.0, 11.0, device=DEV)[:, None].repeat(1, 20)
    out = torch.full((8, 20), 3.0, device=DEV)
    rar.embedding_forward(w, ids, out)
    assert out[:, 0].tolist() == [2, 0, 0, 0, 0, 10, 0, 0]
    dw = _grad(torch.ones(8, 20, device=DEV), ids, 10, torch.float32)
    assert dw[:, 3].tolist() == [0, 1, 0, 0, 0, 0, 0, 0, 0, 1]


def test_rows_of_ignored_tokens_are_not_read_into_sums():
    """NaN and infinity in ignored tokens' gradients and in unused table rows."""
    ids = torch.tensor([3, -1, 5, 3, 99, 7], device=DEV)
    dout = torch.ones(6, 70, device=DEV)
    dout[1], dout[4], dout[5] = math.nan, math.inf, -math.inf
    dw = _grad(dout, ids, 8, torch.float32, padding=7)
    assert dw[:, 0].tolist() == [0, 0, 0, 2, 0, 1, 0, 0] and bool(torch.isfinite(dw).all())
    w = torch.full((8, 70), math.nan, device=DEV)
    w[3], w[5], w[7] = 1.0, 2.0, 3.0
    out = torch.empty(6, 70, device=DEV)
    rar.embedding_forward(w, ids, out)
    assert out[:, 69].tolist() == [1, 0, 2, 1, 0, 3]
    dout[0] = math.nan  # a used token's NaN goes to its own row only
    dw = _grad(dout, ids, 8, torch.float32, padding=7)
    assert bool(dw[3].isnan().all()) and bool(torch.isfinite(dw[:3]).all()) and bool(torch.isfinite(dw[4:]).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strided_and_unaligned_rows(dt):
    t = DTYPES[dt]
    store = torch.randn(50, 300, device=DEV).to(t)
    w = store[:, 3:3 + 129]
    ids = _ids("uniform", 4 * 31, 50).view(4, 31)
    out_store = torch.full((4, 31, 200), 4.0, device=DEV, dtype=t)
    out = out_store[:, :, 1:130]
    rar.embedding_forward(w, ids, out, scale=2.0)
    r, tol = ref.embedding(w, ids, 2.0, t)
    assert_within(out.reshape(124, 129), r, tol, "lookup")
    assert bool((out_store[:, :, 0] == 4.0).all()) and bool((out_store[:, :, 130:] == 4.0).all())
    dw_store = torch.full((50, 131), 6.0, device=DEV, dtype=t)
    dw = dw_store[:, 1:130]
    ws = torch.empty(rar.embedding_workspace_bytes(124, 50, 129), dtype=torch.uint8, device=DEV)
    rar.embedding_backward(out, ids, dw, ws)
    r, tol = ref.embedding_grad(out.reshape(124, 129), ids, 50, 1.0, t)
    assert_within(dw, r, tol, "gradient")
    assert bool((dw_store[:, 0] == 6.0).all()) and bool((dw_store[:, 130] == 6.0).all())
    # one gradient row for all tokens (the gradient of a sum over tokens)
    row = torch.randn(129, device=DEV).to(t)
    rar.embedding_backward(row.expand(4, 31, 129), ids, dw, ws)
    r, tol = ref.embedding_grad(row.expand(124, 129), ids, 50, 1.0, t)
    assert_within(dw, r, tol, "broadcast gradient")


def test_offsets_beyond_32_bits():
    """Table, outputs and gradients whose rows lie past 2^32 elements."""
    stride = (1 << 32) // 3 + 5
    big = torch.empty(3 * stride + 64, dtype=torch.bfloat16, device=DEV)
    w = big.as_strided((4, 48), (stride, 1))
    w.copy_(torch.arange(4 * 48, device=DEV).view(4, 48))
    ids = torch.tensor([3, 0, 3, 2], device=DEV)
    out = torch.empty(4, 48, dtype=torch.bfloat16, device=DEV)
    rar.embedding_forward(w, ids, out)
    assert torch.equal(out, w[ids])
    ws = torch.empty(rar.embedding_workspace_bytes(4, 4, 48), dtype=torch.uint8, device=DEV)
    dw = torch.empty(4, 48, device=DEV)
    rar.embedding_backward(w, ids, dw, ws)  # the far rows as gradients
    want = torch.zeros(4, 48, device=DEV).index_add_(0, ids, w.float())
    assert torch.equal(dw, want)
    src = w.clone()
    rar.embedding_backward(src, ids, w, ws)  # the far rows as the table's gradient
    assert torch.equal(w.float(), want.to(torch.bfloat16).float())


def test_more_tokens_than_one_wavefront_each():
    """2^25 wavefronts fill the largest launch; the lookup goes round."""
    tokens = (1 << 25) + 70
    ids = torch.randint(-1, 17, (tokens,), device=DEV, dtype=torch.int32)
    w = torch.randn(17, 8, device=DEV).to(torch.bfloat16)
    w[16] = 0
    out = torch.full((tokens, 8), 3.0, device=DEV, dtype=torch.bfloat16)
    rar.embedding_forward(w[:16], ids, out)
    want = w[torch.where(ids < 0, 16, ids).long()]
    assert torch.equal(out, want)


def test_many_tokens():
    ids = _ids("skew", 400_000, 3000, dtype=torch.int32)
    dout = torch.randn(400_000, 24, device=DEV)
    dw = _grad(dout, ids, 3000, torch.float32)
    assert_within(dw, *ref.embedding_grad(dout, ids, 3000, 1.0, torch.float32), "gradient")


def test_gradient_against_differences():
    """The lookup is linear in the table: for f = sum(out * dout) the change
    along a direction is the gradient's product with it, up to roundings."""
    w = torch.randn(40, 100, device=DEV)
    ids = _ids("skew", 200, 40)
    dout, v = torch.randn(200, 100, device=DEV), torch.randn(40, 100, device=DEV)
    dw = _grad(dout, ids, 40, torch.float32, 3.0)
    outs = []
    for s in (1.0, -1.0):
        out = torch.empty(200, 100, device=DEV)
        rar.embedding_forward(w + s * v, ids, out, scale=3.0)
        outs.append(out.double())
    diff = float(((outs[0] - outs[1]) * dout.double()).sum() / 2)
    along = float((dw.double() * v.double()).sum())
    # w +- v and the scaled outputs are rounded once each (u of at most |w| + |v|), dw by its bound
    mag = (outs[0].abs() + outs[1].abs()) * dout.double().abs()
    tol = 2 * ref.U * float(mag.sum()) + float((ref.embedding_grad(dout, ids, 40, 3.0, torch.float32)[1].to(DEV)
                                                * v.double().abs()).sum())
    assert abs(diff - along) <= tol, (diff, along, tol)


def test_replays_in_a_graph():
    ids = _ids("skew", 3000, 2000)
    dout = torch.randn(3000, 130, device=DEV)
    dw = torch.empty(2000, 130, device=DEV)
    out = torch.empty(3000, 130, device=DEV)
    ws = torch.empty(rar.embedding_workspace_bytes(3000, 2000, 130), dtype=torch.uint8, device=DEV)

    def step():
        rar.embedding_backward(dout, ids, dw, ws)
        rar.embedding_forward(dw, ids, out)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(4):
        dout.mul_(1.5)
        ids.copy_(ids.roll(k + 1))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = dw.clone(), out.clone()
        step()
        assert torch.equal(got[0], dw) and torch.equal(got[1], out), f"replay {k}"
