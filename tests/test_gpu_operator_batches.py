"""The loops that batches run in: workgroups that take several rows or tiles,
table gradients of several column segments, partial sums joined on every
level.

Sums are made of small integers (times powers of two) whose partial sums
binary32 holds exactly in any order, so one lost, doubled or stale part of a
sum shows as a difference, however long the sum is.  What is formed row by
row must not depend on the batch that a row is in, so a batch is compared bit
by bit with calls of so few rows that no workgroup takes a second one."""
import math

import pytest
import torch

import operator_ref as ref
import ring_all_reduce_scatter_amd as rar
from operator_ref import DTYPES, U, assert_within

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(shape, dt, gen, top=3):
    return torch.randint(-top, top + 1, shape, generator=gen, device=DEV).to(dt)


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device=DEV)


def _same(got, want, what):
    if not torch.equal(got, want):
        bad = (got != want).nonzero()
        raise AssertionError(f"{what}: {bad.shape[0]} of {got.numel()} differ, first at {bad[0].tolist()}")


# ------------------------------------------------------------------ embedding gradient

def _ids(kind, tokens, vocab, gen):
    if kind == "one":
        return torch.full((tokens,), vocab - 1, device=DEV)
    if kind == "two":  # two long runs that meet anywhere in a piece
        return (torch.rand(tokens, generator=gen, device=DEV) < 0.37).long() * (vocab - 1)
    u = torch.rand(tokens, generator=gen, device=DEV, dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1.0)) - 1).long().clamp_(0, vocab - 1)
    return torch.where(torch.rand(tokens, generator=gen, device=DEV) < 0.1, -1, ids)


BATCHES = [(1025, 3, 513, "one"), (1500, 700, 1001, "two"), (3001, 900, 2048, "skew"), (5000, 40, 520, "one"),
           (20_000, 5000, 1536, "skew"), (70_000, 3, 600, "one"), (70_000, 3, 24, "two"), (400_000, 3000, 24, "skew"),
           (32_768, 50_021, 2048, "skew"), (2000, 300, 4100, "two"),
          (3, 2, 512 * 65_535 + 3, "two")]  # more segments than a grid dimension of the few-token launch


@pytest.mark.parametrize("dts", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("tokens,vocab,dim,kind", BATCHES)
def test_sorted_gradient_is_exact_in_every_segment(tokens, vocab, dim, kind, dts):
    act, wt = DTYPES[dts[0]], DTYPES[dts[1]]
    gen = _gen(tokens + dim)
    ids = _ids(kind, tokens, vocab, gen)
    dout = _ints((tokens, dim), act, gen)
    old = _ints((vocab, dim), wt, gen, 60)
    pad = int(ids[0]) if kind == "skew" else None
    ok = (ids >= 0) if pad is None else (ids >= 0) & (ids != pad)
    want = torch.zeros(vocab, dim, dtype=torch.float64, device=DEV)
    step = max(1024, (1 << 26) // tokens)  # columns in binary64 at a time
    for c in range(0, dim, step):
        want[:, c:c + step].index_add_(0, ids[ok], dout[ok, c:c + step].double())
    assert float(want.abs().max()) < 2.0 ** 22  # a sum is exact in binary32, whatever its order
    ws = _bytes(rar.embedding_workspace_bytes(tokens, vocab, dim))
    ws.fill_(0x5A)
    dw = torch.full((vocab, dim), 7.0, device=DEV, dtype=wt)
    rar.embedding_backward(dout, ids, dw, ws, scale=0.5, padding_id=pad)
    _same(dw, (want * 0.5).to(wt), "gradient")
    dw = old.clone()
    rar.embedding_backward(dout, ids, dw, ws, scale=2.0, padding_id=pad, accumulate=True)
    _same(dw, (want * 2.0 + old.double()).to(wt), "accumulated")


# ------------------------------------------------------------------ layer norm

# Whole vectors of a row (4 binary32 or 8 16-bit elements) and rows that are
# more than two turns of every workgroup forward (768 groups of 16, 4, 2 or 1
# rows, or 256) and backward (256 groups of 64 rows to 1), by no multiple.
WIDTHS = [(11, 32_805), (27, 32_805), (61, 24_613), (101, 6185), (201, 6185), (331, 3091), (501, 1541), (901, 1541),
          (1601, 601), (3001, 601)]
FEW = 200  # rows of a call in which no workgroup takes a second one
# The reference's bounds count a sum's additions as dim / 64 + 24; sixteen
# lanes a row make up to dim / 16 + 5 of them, at most 37 where it has 31.
DEPTH = 1.25


def _sample(rows, gen):
    some = torch.randint(0, rows, (40,), generator=gen, device=DEV)
    return torch.cat([torch.tensor([0, 1, rows - 2, rows - 1], device=DEV), some])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vecs,rows", WIDTHS)
def test_layernorm_forward_takes_rows_in_turns(vecs, rows, dt):
    t = DTYPES[dt]
    dim = vecs * (4 if dt == "f32" else 8) + vecs % 4
    gen = _gen(dim)
    x = (torch.randn(rows, dim, generator=gen, device=DEV) * 2 + 0.5).to(t)
    w, b = 1 + 0.2 * torch.randn(dim, generator=gen, device=DEV), torch.randn(dim, generator=gen, device=DEV)
    y, mean, rstd = torch.full_like(x, 7.0), torch.full((rows,), 9.0, device=DEV), torch.full((rows,), 9.0, device=DEV)
    rar.layernorm_forward(x, w, b, y, mean=mean, rstd=rstd)
    y2, mean2, rstd2 = torch.full_like(x, 5.0), torch.empty_like(mean), torch.empty_like(rstd)
    for r in range(0, rows, FEW):
        s = slice(r, r + FEW)
        rar.layernorm_forward(x[s], w, b, y2[s], mean=mean2[s], rstd=rstd2[s])
    _same(mean, mean2, "mean")
    _same(rstd, rstd2, "rstd")
    _same(y, y2, "y")
    at = _sample(rows, gen)
    for g, (r, tol), name in zip((y, mean, rstd), ref.layernorm(x[at], w, b, 1e-5, t), ("y", "mean", "rstd")):
        assert_within(g[at], r, tol * DEPTH, name)
    rar.layernorm_forward(x, w, b, x)
    _same(x, y, "in place")


def test_layernorm_forward_of_more_long_rows_than_workgroups():
    """Rows too long for the registers, each one element further into a buffer."""
    rows, dim = 65_536 + 70, 16_400
    gen = _gen(3)
    base = torch.randn(rows + dim, generator=gen, device=DEV).to(torch.bfloat16)
    x = base.as_strided((rows, dim), (1, 1))
    y = torch.full((rows, dim), 7.0, device=DEV, dtype=torch.bfloat16)
    mean, rstd = torch.full((rows,), 9.0, device=DEV), torch.full((rows,), 9.0, device=DEV)
    rar.layernorm_forward(x, None, None, y, mean=mean, rstd=rstd)
    at = torch.tensor([0, 1, 65_534, 65_535, 65_536, 65_537, rows - 1], device=DEV)
    for g, (r, tol), name in zip((y, mean, rstd), ref.layernorm(x[at], None, None, 1e-5, torch.bfloat16),
                                 ("y", "mean", "rstd")):
        assert_within(g[at], r, tol, name)
    # unit variance and at most sqrt(dim) of it in one element, of every row
    assert float(y.abs().max()) < 8 and float((y.float().square().mean(1) - 1).abs().max()) < 2.0 ** -6


def _check_grad_batch(rows, dim, dt, wdt, seed):
    """Everything that layernorm_backward makes of integer x and dy and
    statistics that are powers of two: dw and db exact, dx as in calls of few
    rows, and the same written over dy or x."""
    t, wt = DTYPES[dt], DTYPES[wdt]
    gen = _gen(seed)
    x, dy = _ints((rows, dim), t, gen), _ints((rows, dim), t, gen)
    mean = _ints((rows,), torch.float32, gen, 1)
    rstd = torch.tensor([0.5, 1.0, 2.0], device=DEV)[torch.randint(0, 3, (rows,), generator=gen, device=DEV)]
    w = (1 + 0.2 * torch.randn(dim, generator=gen, device=DEV)).to(wt)
    old = _ints((dim,), wt, gen, 60), _ints((dim,), wt, gen, 60)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    want = (dy.double() * h).sum(0), dy.double().sum(0)
    assert rows * 3 * 8 < 2 ** 22  # in halves: exact in binary32, whatever the order
    del h
    ws = _bytes(rar.layernorm_workspace_bytes(rows, dim))

    def call(dy, x, dx, accumulate=False, s=slice(None), sums=True):
        dw, db = (o.clone() if accumulate else torch.full_like(o, 7.0) for o in old) if sums else (None, None)
        rar.layernorm_backward(dy[s], x[s], w, mean[s], rstd[s], dx[s], dw, db, ws if sums else None, accumulate)
        return dw, db

    dx = torch.full_like(x, 9.0)
    for name, got, sums in zip(("dw", "db"), call(dy, x, dx), want):
        _same(got, sums.to(wt), name)
    dx2 = torch.full_like(x, 8.0)
    for name, got, sums, o in zip(("dw", "db"), call(dy, x, dx2, True), want, old):
        _same(got, (sums + o.double()).to(wt), f"accumulated {name}")
    _same(dx, dx2, "dx of the accumulated call")
    dx2.fill_(8.0)
    call(dy, x, dx2, sums=False)
    _same(dx, dx2, "dx alone")
    dx2.fill_(8.0)
    for r in range(0, rows, FEW):
        call(dy, x, dx2, s=slice(r, r + FEW))
    _same(dx, dx2, "dx by few rows")
    at = _sample(rows, gen)
    r, tol = ref.layernorm_grad(dy[at], x[at], w, mean[at], rstd[at], t, wt)[0]
    assert_within(dx[at], r, tol * DEPTH, "dx")
    for over in ("dy", "x"):
        a, c = dy.clone(), x.clone()
        d = a if over == "dy" else c
        for name, got, sums in zip(("dw", "db"), call(a, c, d), want):
            _same(got, sums.to(wt), f"{name} with dx over {over}")
        _same(d, dx, f"dx over {over}")
    dw, db = torch.full_like(old[0], 7.0), torch.full_like(old[1], 7.0)
    rar.layernorm_backward(dy, x, w, mean, rstd, None, dw, db, ws)
    _same(dw, want[0].to(wt), "dw without dx")
    _same(db, want[1].to(wt), "db without dx")


@pytest.mark.parametrize("dts", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("vecs,rows", WIDTHS)
def test_layernorm_backward_takes_rows_in_turns(vecs, rows, dts):
    dim = vecs * (4 if dts[0] == "f32" else 8) + vecs % 4
    _check_grad_batch(rows, dim, *dts, seed=dim)


@pytest.mark.parametrize("rows,dim,dts", [(200, 16_400, ("bf16", "bf16")), (200, 8200, ("f32", "f32")),
                                          (131, 20_001, ("f16", "f32")), (700, 9001, ("f32", "f32"))])
def test_layernorm_backward_of_long_rows_in_row_groups(rows, dim, dts):
    _check_grad_batch(rows, dim, *dts, seed=rows)


@pytest.mark.parametrize("dim", [(1 << 28) - 1, (1 << 28) + 70])
def test_layernorm_backward_of_rows_past_one_grid_dimension(dim):
    """2^28 columns are 2^32 threads of the launch that adds partial rows."""
    rows = 2
    gen = _gen(9)
    pattern = torch.randint(-3, 4, (rows, dim), generator=gen, device=DEV, dtype=torch.int8)
    x, dy = pattern.to(torch.bfloat16), pattern.roll(1, 1).to(torch.bfloat16)
    mean, rstd = torch.tensor([1.0, -1.0], device=DEV), torch.tensor([0.5, 2.0], device=DEV)
    dw = torch.full((dim,), 7.0, device=DEV, dtype=torch.bfloat16)
    db = torch.full_like(dw, 7.0)
    ws = _bytes(rar.layernorm_workspace_bytes(rows, dim))
    rar.layernorm_backward(dy, x, None, mean, rstd, None, dw, db, ws)
    h = (x.float() - mean[:, None]) * rstd[:, None]
    _same(dw, (dy.float() * h).sum(0).to(torch.bfloat16), "dw")
    _same(db, dy.float().sum(0).to(torch.bfloat16), "db")


# ------------------------------------------------------------------ norm and clip

def _norm_of(grads, kind):
    """The norm in binary64, on the GPU."""
    if kind == rar.NORM_MAX:
        return max(float(g.abs().max()) for g in grads if g.numel())
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def _check_norm(got, want, what):
    assert_within(got, torch.tensor([want], dtype=torch.float64), torch.tensor(abs(want) * U * (1 + 2.0 ** -20)), what)


@pytest.mark.parametrize("kind", [rar.NORM_L2, rar.NORM_MAX])
@pytest.mark.parametrize("dt,n", [("f32", 9_000_001), ("bf16", 17_000_001), ("f16", 17_000_001), ("f32", 34_000_003)])
def test_norm_groups_take_tiles_in_turns(dt, n, kind):
    """More than two turns of the 1024 tile groups, and more tiles (8192) than
    a clip leaves in the caches."""
    t = DTYPES[dt]
    gen = _gen(n)
    grads = [torch.randn(n, generator=gen, device=DEV).to(t), torch.randn(4097, generator=gen, device=DEV),
             torch.randn(70_001, generator=gen, device=DEV).to(torch.bfloat16)]
    ws, norm = _bytes(rar.grad_clip_workspace_bytes([g.numel() for g in grads])), torch.zeros(1, device=DEV)
    outs = [torch.full_like(g, 3.0) for g in grads]
    plan = rar.GradClip(grads, ws, outs=outs)
    tile = 16_384 // grads[0].element_size()
    # the largest value wherever a turn begins or ends
    for at in (0, 1023 * tile, 1024 * tile + tile - 1, 2047 * tile + 1, 2048 * tile, n - 1):
        keep = grads[0][at].clone()
        grads[0][at] = -50.0
        want = _norm_of(grads, kind)
        plan.norm(norm, kind)
        _check_norm(norm, want, f"norm, {at}")
        plan.clip(want / 4, norm, kind, scale=0.5)
        _check_norm(norm, want * 0.5, f"clip, {at}")
        grads[0][at] = keep
    # the last clip: the factor is rounded, then the product, then the output
    grads[0][n - 1] = -50.0
    f = 0.5 * min(1.0, want / 4 / (want * 0.5 + 1e-6))
    for i, (g, o) in enumerate(zip(grads, outs)):
        r = g.double() * f
        tol = ref.rounded(r, r.abs() * 2 * U + 2.0 ** -148, o.dtype)
        assert bool(((o.double() - r).abs() <= tol).all()), f"tensor {i}"


@pytest.mark.parametrize("kind", [rar.NORM_L2, rar.NORM_MAX])
@pytest.mark.parametrize("n", [3000, 300_001])  # one launch, and two
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_infinite_max_norm_only_scales(dt, n, kind):
    """One overflowed element of a set that is unscaled: the others keep their
    values.  A NaN still makes everything NaN, and so does zero times infinity."""
    gen = _gen(n)
    g = torch.randn(n, generator=gen, device=DEV).to(DTYPES[dt])
    g[n // 2] = -math.inf
    ws, norm, out = _bytes(rar.grad_clip_workspace_bytes([n])), torch.zeros(1, device=DEV), torch.empty_like(g)
    plan = rar.GradClip([g], ws, outs=[out])
    for scale in (1.0, -0.25):
        out.fill_(3.0)
        plan.clip(math.inf, norm, kind, scale=scale)
        assert norm.item() == math.inf
        _same(out, (g.float() * scale).to(g.dtype), f"scale {scale}")
    plan.clip(math.inf, norm, kind, scale=0.0)
    assert math.isnan(norm.item()) and bool(out.isnan().all())
    plan.clip(1e30, norm, kind)  # a finite limit: the factor is zero
    assert norm.item() == math.inf and int((out != 0).sum()) == 1 and bool(out[n // 2].isnan())
    g[0] = math.nan
    plan.clip(math.inf, norm, kind)
    assert math.isnan(norm.item()) and bool(out.isnan().all())


@pytest.mark.parametrize("kind", [rar.NORM_L2, rar.NORM_MAX])
def test_norm_of_tensors_that_overlap(kind):
    """A norm writes no tensor, so one may be held twice or overlap another."""
    flat = torch.randn(40_000, generator=_gen(1), device=DEV)
    grads = [flat[:30_000], flat[:30_000], flat[10_000:], flat]
    ws, norm = _bytes(rar.grad_clip_workspace_bytes([g.numel() for g in grads])), torch.zeros(1, device=DEV)
    rar.grad_norm(grads, ws, norm, norm_type=kind, scale=0.5)
    _check_norm(norm, _norm_of(grads, kind) * 0.5, "overlapping")
    plan = rar.GradClip(grads, ws, norm_only=True)
    with pytest.raises(rar.RarError):
        plan.clip(1.0, norm)
    with pytest.raises(rar.RarError):
        rar.clip_grad_norm(grads, 1.0, ws, norm)


# ------------------------------------------------------------------ columns of one matrix

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(5, 40), (700, 129), (1300, 1000), (70, 9000)])
def test_layernorm_between_columns_of_one_matrix(rows, dim, dt):
    """Inputs and outputs as columns of one buffer, in either order."""
    t, gen = DTYPES[dt], _gen(dim)
    w, b = torch.randn(dim, generator=gen, device=DEV), torch.randn(dim, generator=gen, device=DEV)
    x, dy = _ints((rows, dim), t, gen), _ints((rows, dim), t, gen)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    rar.layernorm_forward(x, w, b, y, mean=mean, rstd=rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    ws = _bytes(rar.layernorm_workspace_bytes(rows, dim))
    rar.layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
    for order in ((0, 1, 2, 3), (3, 2, 1, 0)):
        m = torch.full((rows, 4 * dim + 1), 9.0, device=DEV, dtype=t)
        xs, ys, dys, dxs = (m[:, i * dim:(i + 1) * dim] for i in order)
        xs.copy_(x)
        dys.copy_(dy)
        rar.layernorm_forward(xs, w, b, ys)
        dw2, db2 = torch.full_like(dw, 7.0), torch.full_like(db, 7.0)
        rar.layernorm_backward(dys, xs, w, mean, rstd, dxs, dw2, db2, ws)
        for name, got, want in (("x", xs, x), ("y", ys, y), ("dy", dys, dy), ("dx", dxs, dx), ("dw", dw2, dw),
                                ("db", db2, db), ("gap", m[:, -1], torch.full_like(m[:, -1], 9.0))):
            _same(got, want, name)


@pytest.mark.parametrize("tokens,dim", [(300, 40), (2000, 700)])
def test_embedding_between_columns_of_one_matrix(tokens, dim):
    gen = _gen(dim)
    ids = torch.randint(-1, tokens, (tokens,), generator=gen, device=DEV)
    m = torch.full((tokens, 2 * dim + 3), 9.0, device=DEV)
    a, c = m[:, :dim], m[:, dim + 1:2 * dim + 1]
    a.copy_(_ints((tokens, dim), torch.float32, gen))
    want = torch.where(ids[:, None] < 0, 0.0, a[ids.clamp(min=0)])
    rar.embedding_forward(a, ids, c)  # the table beside its output
    _same(c, want, "lookup")
    grad = torch.zeros(tokens, dim, device=DEV).index_add_(0, ids.clamp(min=0), torch.where(ids[:, None] < 0, 0.0, c))
    ws = _bytes(rar.embedding_workspace_bytes(tokens, tokens, dim))
    rar.embedding_backward(c, ids, a, ws)
    _same(a, grad, "gradient")
    assert bool((m[:, dim] == 9.0).all()) and bool((m[:, 2 * dim + 1:] == 9.0).all())


def test_norm_among_the_tensors_is_refused():
    flat, out = torch.ones(64, device=DEV), torch.zeros(32, dtype=torch.float16, device=DEV)
    grads = [flat[:32], torch.empty(0, device=DEV)]
    plan = rar.GradClip(grads, _bytes(rar.grad_clip_workspace_bytes([32, 0])), outs=[out, torch.empty(0, device=DEV)])
    for bad in (flat[:1], flat[31:32], out[:2].view(torch.float32), out[30:].view(torch.float32)):
        for call in (lambda: plan.norm(bad), lambda: plan.clip(1.0, bad)):
            with pytest.raises(rar.RarError, match="overlap"):
                call()
    plan.norm(flat[32:33])
    _check_norm(flat[32:33], 32 ** 0.5, "beside the tensors")
    assert bool((flat[:32] == 1).all()) and bool((out == 0).all())
