"""Layer norm, forward and backward, against its formula in binary64.

Tolerances, derived: u = 2^-24 is half an fp32 step.  A sum of n terms in
any order is off by at most n u times the sum of their magnitudes; a
thread's own chain here is at most 64 long before the sums meet in trees
(cols / 512 in the streaming kernels), so a mean over a row is off by at most
(64 + cols / 512 + 32) u times the mean magnitude.  The output is rounded
once more to its type: eps / 2 relative.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import bit_nf4_quantized_21_b200 as q
import oracle.tail as OT

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
EPS = 1e-5


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _inputs(rows, cols, dtype, seed, shift=0.3):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) + shift).to(dtype)
    dy = torch.randn(rows, cols, generator=g).to(dtype)
    w = (torch.randn(cols, generator=g) * 0.2 + 1.0)
    b = torch.randn(cols, generator=g) * 0.2
    return x, dy, w, b


def _check_fwd(x, w, b, y, mean, rstd, eps=EPS):
    cols = x.shape[1]
    chain = 96 + cols / 512
    X = f64(x)
    ry, rm, rr = OT.layernorm_fwd(X, None if w is None else f64(w), None if b is None else f64(b), eps)
    W = np.ones(cols) if w is None else np.abs(f64(w))
    B = np.zeros(cols) if b is None else np.abs(f64(b))
    big = np.abs(X).max(1)
    dm = chain * U * np.abs(X).mean(1) + U * np.abs(rm)          # the mean's own error
    assert np.all(np.abs(f64(mean) - rm) <= dm)
    # variance: chain, a few roundings, and the mean's error squared
    # plus the rounding of each difference x - mean, relative to |x| + |mean|
    dx = dm + 2 * U * (big + np.abs(rm))
    var = 1.0 / rr ** 2 - eps
    dvar = chain * U * var + 2 * np.sqrt(var) * dx + dx ** 2 + 4 * U * (var + eps)
    drel = 0.5 * dvar / (var + eps) + 4 * U
    assert np.all(np.abs(f64(rstd) - rr) <= drel * rr)
    xh = np.abs(X - rm[:, None]) * rr[:, None]
    slack = ((dx * rr)[:, None] + xh * (drel[:, None] + 4 * U)) * W[None] + 4 * U * (xh * W[None] + B[None])
    assert np.all(np.abs(f64(y) - ry) <= half_step(y.dtype) * (np.abs(ry) + slack) + slack)
    return rm, rr


def _check_bwd(x, dy, w, mean, rstd, dx, dw, db):
    rows, cols = x.shape
    X, D = f64(x), f64(dy)
    W = np.ones(cols) if w is None else f64(w)
    m, r = f64(mean), f64(rstd)
    rdx, rdw, rdb = OT.layernorm_bwd(D, X, W, m, r)
    chain = 96 + cols / 512
    xh = np.abs(X - m[:, None]) * r[:, None]
    dxh = 3 * U * (np.abs(X) + np.abs(m)[:, None]) * r[:, None]      # xh itself: a difference and a product
    g = np.abs(D * W)
    m1 = chain * U * g.mean(1)
    m2 = chain * U * (g * xh).mean(1) + (g * dxh).mean(1)
    c2 = (g * xh).mean(1)
    slack = r[:, None] * (4 * U * g + m1[:, None] + xh * m2[:, None] + dxh * c2[:, None] + 6 * U * (g.mean(1)[:, None] + xh * c2[:, None]))
    assert np.all(np.abs(f64(dx) - rdx) <= half_step(dx.dtype) * (np.abs(rdx) + slack) + slack)
    # column sums: rows terms in whatever order
    n = rows + 8
    if dw is not None:
        slack = n * U * (np.abs(D) * xh).sum(0) + (np.abs(D) * dxh).sum(0)
        assert np.all(np.abs(f64(dw) - rdw) <= half_step(dw.dtype) * (np.abs(rdw) + slack) + slack)
    if db is not None:
        slack = n * U * np.abs(D).sum(0)
        assert np.all(np.abs(f64(db) - rdb) <= half_step(db.dtype) * (np.abs(rdb) + slack) + slack)


# every plan: a warp, 128 .. 1024 threads a row, element by element, streaming
SHAPES = [(1, 1), (3, 8), (5, 64), (2, 257), (7, 512), (9, 1000), (33, 1024), (6, 1500), (4, 2048), (300, 2051),
          (37, 4096), (5, 6000), (1300, 768), (3, 8192), (2, 8191), (3, 16384), (2, 16392), (2, 20001),
          # rows through the ring: enough of them, a ragged last round
          (2401, 1032), (4801, 1032), (4740, 2048), (1333, 4096), (2402, 4096), (1190, 5120), (1200, 8192), (600, 16384)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_matches_formula(rows, cols, dtype):
    x, dy, w, b = _inputs(rows, cols, dtype, rows * 7 + cols)
    w, b = w.to(dtype), b.to(dtype)
    xd, dyd, wd, bd = (t.to(DEV) for t in (x, dy, w, b))
    y, mean, rstd = q.qlora_layernorm_fwd(xd, wd, bd, EPS)
    _check_fwd(x, w, b, y, mean, rstd)
    dx, dw, db = q.qlora_layernorm_bwd(dyd, xd, wd, mean, rstd)
    _check_bwd(x, dy, w, mean, rstd, dx, dw, db)


@pytest.mark.parametrize("cols", [512, 515])
def test_parameter_types_and_absent_parameters(cols):
    x, dy, w, b = _inputs(11, cols, torch.bfloat16, 3)
    xd, dyd = x.to(DEV), dy.to(DEV)
    for ww, bb in ((w, b), (None, b), (w, None), (None, None)):
        y, mean, rstd = q.qlora_layernorm_fwd(xd, None if ww is None else ww.to(DEV), None if bb is None else bb.to(DEV))
        _check_fwd(x, ww, bb, y, mean, rstd)
    for ww in (w, None):
        dx, dw, db = q.qlora_layernorm_bwd(dyd, xd, None if ww is None else ww.to(DEV), mean, rstd,
                                           grad_dtype=torch.bfloat16)
        assert dw.dtype == torch.bfloat16
        _check_bwd(x, dy, ww, mean, rstd, dx, dw, db)
    frozen, nw, nb = q.qlora_layernorm_bwd(dyd, xd, w.to(DEV), mean, rstd, want_params=False)
    assert nw is None and nb is None
    assert torch.equal(frozen, q.qlora_layernorm_bwd(dyd, xd, w.to(DEV), mean, rstd)[0])


@pytest.mark.parametrize("cols", [640, 4096, 20001])
def test_large_mean_keeps_the_variance(cols):
    x, _, w, b = _inputs(4, cols, torch.float32, 8, shift=1000.0)
    y, mean, rstd = q.qlora_layernorm_fwd(x.to(DEV), w.to(DEV), b.to(DEV))
    _check_fwd(x, w, b, y, mean, rstd)
    c = torch.full((2, cols), 7.0)                    # no spread at all: rstd = 1 / sqrt(eps), y = bias
    y, mean, rstd = q.qlora_layernorm_fwd(c.to(DEV), w.to(DEV), b.to(DEV))
    assert torch.equal(mean.cpu(), torch.full((2,), 7.0))
    assert torch.equal(y.cpu(), b.expand(2, cols))


@pytest.mark.parametrize("rows,cols,ld,off", [(6, 512, 768, 0), (6, 512, 515, 0), (6, 512, 600, 1), (6, 33, 40, 3),
                                              (6, 17000, 17001, 1), (4800, 2048, 2064, 8)])
def test_strided_and_offset_rows_leave_the_rest_alone(rows, cols, ld, off):
    x, dy, w, b = _inputs(rows, cols, torch.bfloat16, cols + ld)

    def spread(t):
        base = torch.full((rows, ld), 99.0, dtype=t.dtype, device=DEV)
        v = base[:, off:off + cols] if off + cols <= ld else base[:, :cols]
        v.copy_(t)
        return base, v
    _, xd = spread(x)
    _, dyd = spread(dy)
    ybase, y = spread(torch.zeros_like(x))
    dbase, dx = spread(torch.zeros_like(x))
    w, b = w.bfloat16(), b.bfloat16()
    _, mean, rstd = q.qlora_layernorm_fwd(xd, w.to(DEV), b.to(DEV), Y=y)
    _check_fwd(x, w, b, y, mean, rstd)
    dx, dw, db = q.qlora_layernorm_bwd(dyd, xd, w.to(DEV), mean, rstd, dX=dx)
    _check_bwd(x, dy, w, mean, rstd, dx, dw, db)
    for base, v in ((ybase, y), (dbase, dx)):
        v.fill_(99.0)
        assert torch.all(base == 99.0)


@pytest.mark.parametrize("rows,cols", [(40, 96), (40, 4096), (40, 4099), (40, 18000), (2400, 2048)])
def test_in_place(rows, cols):
    x, dy, w, b = _inputs(rows, cols, torch.float32, 5)
    xd, dyd, wd, bd = (t.to(DEV) for t in (x, dy, w, b))
    y, mean, rstd = q.qlora_layernorm_fwd(xd, wd, bd)
    z = xd.clone()
    q.qlora_layernorm_fwd(z, wd, bd, Y=z)
    assert torch.equal(z, y)
    dx, dw, db = q.qlora_layernorm_bwd(dyd, xd, wd, mean, rstd)
    for which in (0, 1):
        bufs = [dyd.clone(), xd.clone()]
        got = q.qlora_layernorm_bwd(bufs[0], bufs[1], wd, mean, rstd, dX=bufs[which])
        assert all(torch.equal(a, e) for a, e in zip(got, (dx, dw, db)))


def test_nan_stays_in_its_row_and_infinity_too():
    x, _, w, b = _inputs(5, 1024, torch.float32, 6)
    x[1, 7] = float("nan")
    x[3, 9] = float("inf")
    y, _, _ = q.qlora_layernorm_fwd(x.to(DEV), w.to(DEV), b.to(DEV))
    y = y.cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    assert torch.isfinite(y[[0, 2, 4]]).all()


def test_no_rows():
    x = torch.empty((0, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    y, mean, rstd = q.qlora_layernorm_fwd(x, w)
    assert y.shape == (0, 64)
    _, dw, db = q.qlora_layernorm_bwd(x, x, w, mean, rstd, dweight=torch.full((64,), 3.0, device=DEV),
                                      dbias=torch.full((64,), 3.0, device=DEV))
    assert torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


def test_gradient_against_differences():
    # <dL/dx, v> against (L(x + h v) - L(x - h v)) / 2h for L = <c, y>: the
    # remainder is h^2 / 6 times a third derivative of order |c| |v|^3 (unit
    # spread rows), the rounding of L about cols * 2^-22 |c| / h
    x, c, w, b = _inputs(3, 768, torch.float32, 12)
    v = torch.randn(3, 768, generator=torch.Generator().manual_seed(13))
    wd, bd = w.to(DEV), b.to(DEV)
    _, mean, rstd = q.qlora_layernorm_fwd(x.to(DEV), wd, bd)
    dx, dw, _ = q.qlora_layernorm_bwd(c.to(DEV), x.to(DEV), wd, mean, rstd)
    h = 1e-2
    L = lambda xx: (q.qlora_layernorm_fwd(xx.to(DEV), wd, bd)[0].double().cpu() * c.double()).sum()
    fd = ((L(x + h * v) - L(x - h * v)) / (2 * h)).item()
    an = (dx.double().cpu() * v.double()).sum().item()
    scale = (c.abs() * v.abs()).sum().item()
    assert abs(fd - an) <= 2e-4 * scale
    u = torch.randn(768, generator=torch.Generator().manual_seed(14))
    Lw = lambda ww: (q.qlora_layernorm_fwd(x.to(DEV), ww.to(DEV), bd)[0].double().cpu() * c.double()).sum()
    fd = ((Lw(w + h * u) - Lw(w - h * u)) / (2 * h)).item()      # linear in w: no remainder
    assert abs(fd - (dw.double().cpu() * u.double()).sum().item()) <= 2e-4 * scale


@pytest.mark.parametrize("rows,cols", [(900, 1536), (2500, 2560), (50, 999)])
def test_repeats_bit_for_bit_and_replays_from_a_graph(rows, cols):
    x, dy, w, b = (t.to(DEV) for t in _inputs(rows, cols, torch.bfloat16, 20))
    ws = torch.empty(q.qlora_layernorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    y, mean, rstd = q.qlora_layernorm_fwd(x, w, b)
    first = q.qlora_layernorm_bwd(dy, x, w, mean, rstd, workspace=ws)
    ws.fill_(255)                                               # nothing is kept in the workspace between calls
    again = q.qlora_layernorm_bwd(dy, x, w, mean, rstd, workspace=ws)
    assert all(torch.equal(a, e) for a, e in zip(first, again))
    out = [torch.empty_like(t) for t in (y, mean, rstd, *first)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        q.qlora_layernorm_fwd(x, w, b, Y=out[0], mean=out[1], rstd=out[2])
        q.qlora_layernorm_bwd(dy, x, w, out[1], out[2], dX=out[3], dweight=out[4], dbias=out[5], workspace=ws)
    for _ in range(2):
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(out, (y, mean, rstd, *first)))
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    third = q.qlora_layernorm_bwd(dy, x, w, mean, rstd, stream=s2)
    s2.synchronize()
    assert all(torch.equal(a, e) for a, e in zip(first, third))
