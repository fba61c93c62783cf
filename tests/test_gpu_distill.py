"""Distillation from a teacher's top logits, loss and gradient, against the
formula in binary64 (oracle/tail.py).

Tolerances, derived (u = 2^-24): ex2.approx is within 2^-22 relative; its
argument (z - m) log2(e) / tau carries 2.5 roundings of its size, A =
max |z - m| / tau over what matters (terms below e^-30 do not: A <= 30 u
each).  The sum's chain per thread is vocab / 512 terms at most before trees
and merges, so log-sum-exp is off by at most
  E = (vocab / 512 + 64) u + 2^-21 + 4 u 30 + 2 u |m| / tau
and q = exp((z - m) / tau - log s) by E + 2^-21 + 4 u 30 relative (the last
where q matters at all; below e^-30 the absolute error is nothing).  The
gradient is rounded once to its type: eps / 2.
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


def f64(t):
    return t.detach().double().cpu().numpy()


def _inputs(rows, vocab, top, dtype, seed, ids_dtype=torch.int32, t_dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, vocab, generator=g) * 2.5
    noisy = z + torch.randn(rows, vocab, generator=g)
    t, ids = torch.topk(noisy, min(top, vocab), dim=1)
    if top > vocab:                                    # longer lists than the vocabulary: ids repeat
        ids = torch.cat([ids, torch.randint(0, vocab, (rows, top - vocab), generator=g)], 1)
        t = torch.cat([t, torch.randn(rows, top - vocab, generator=g)], 1)
    w = torch.rand(rows, generator=g) + 0.25
    return z.to(dtype), ids.to(ids_dtype).contiguous(), t.to(t_dtype).contiguous(), w


def _bounds(z, t, tau):
    Z, T = f64(z), f64(t)
    fin = np.where(np.abs(Z) < 1e30, np.abs(Z), 0).max(1)
    tin = np.where(np.abs(T) < 1e30, np.abs(T), 0).max(1)
    E = (Z.shape[1] / 512 + 64) * U + 2.0 ** -21 + 120 * U + 2 * U * fin / tau
    return E, fin, tin


def _check(z, ids, t, tau, w, loss=None, lse=None, dz=None, grad=None, from_lse=None):
    E, fin, tin = _bounds(z, t, tau)
    W = np.ones(z.shape[0]) if w is None else f64(w)
    G = np.ones(z.shape[0]) if grad is None else f64(grad)
    rl, rlse, rdz = OT.distill(f64(z), ids.cpu().numpy(), f64(t), tau, W, None if grad is None else G,
                               None if from_lse is None else f64(from_lse))
    if lse is not None:
        assert np.all(np.abs(f64(lse) - rlse) <= E + 2 * U * np.abs(rlse))
    if loss is not None:
        # |log p|, |log q| <= (spread of the entries + log of the sums): 2 (tin + fin) / tau + 20
        size = 2 * (tin + fin) / tau + 20
        tol = np.abs(W) * tau * tau * (E + 2.0 ** -20 * 1 + (ids.shape[1] / 512 + 64) * U * size)
        ok = np.isfinite(rl)
        assert np.array_equal(ok, np.isfinite(f64(loss)))
        assert np.all(np.abs(f64(loss) - rl)[ok] <= tol[ok])
    if dz is not None:
        fac = np.abs(G * W) * tau
        E2 = E + 2.0 ** -21 + 120 * U + (0 if from_lse is None else 4 * U * np.abs(f64(from_lse)))
        # p: a sum of ids.shape[1] exponentials (expf: 2 ulp) of t / tau
        Ep = (ids.shape[1] / 512 + 64) * U + 4 * U * (tin / tau + 4)
        extra = np.zeros_like(rdz)
        p_sum = np.zeros_like(rdz)
        idn, T = ids.cpu().numpy(), f64(t)
        for i in range(z.shape[0]):
            for j in range(idn.shape[1]):
                if 0 <= idn[i, j] < z.shape[1]:
                    p_sum[i, idn[i, j]] = 1.0
        q_part = np.abs(rdz) + p_sum * fac[:, None]
        extra = E2[:, None] * q_part + p_sum * (Ep * fac)[:, None] + fac[:, None] * 1e-13
        hs = torch.finfo(dz.dtype).eps / 2
        got = f64(dz)
        assert np.all(np.isfinite(got) == np.isfinite(rdz))
        tol = hs * (np.abs(rdz) + extra) + extra + torch.finfo(dz.dtype).tiny
        ok = np.isfinite(rdz)
        assert np.all(np.abs(got - rdz)[ok] <= tol[ok])


def _all(z, ids, t, tau, w):
    zd, idd, td = z.to(DEV), ids.to(DEV), t.to(DEV)
    wd = None if w is None else w.to(DEV)
    loss, lse = q.qlora_distill_topk_fwd(zd, idd, td, tau, row_weight=wd)
    _check(z, ids, t, tau, w, loss, lse)
    dz = torch.full_like(zd, float("nan"))
    loss2, lse2 = q.qlora_distill_topk_fwd(zd, idd, td, tau, row_weight=wd, dZ=dz)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    _check(z, ids, t, tau, w, dz=dz)
    g = torch.rand(z.shape[0], generator=torch.Generator().manual_seed(1)) + 0.5
    bz = q.qlora_distill_topk_bwd(zd, idd, td, tau, lse, row_weight=wd, grad_loss=g.to(DEV))
    _check(z, ids, t, tau, w, dz=bz, grad=g, from_lse=lse)
    return loss, lse, dz, bz


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,top", [
    (1, 1, 1), (2, 3, 2), (5, 7, 7), (3, 17, 40), (4, 1000, 1), (9, 4099, 33), (3, 32768, 64), (2, 50021, 1024),
    (700, 129, 5), (1, 131077, 256), (30, 9001, 17), (160, 16384, 8)])
def test_matches_formula(rows, vocab, top, dtype):
    z, ids, t, w = _inputs(rows, vocab, top, dtype, rows + vocab + top)
    _all(z, ids, t, 1.5, w)


@pytest.mark.parametrize("tau", [0.5, 1.0, 4.0])
@pytest.mark.parametrize("ids_dtype,t_dtype", [(torch.int32, torch.bfloat16), (torch.int64, torch.float32)])
def test_types_temperatures_and_no_weights(ids_dtype, t_dtype, tau):
    z, ids, t, _ = _inputs(6, 5000, 12, torch.bfloat16, 4, ids_dtype, t_dtype)
    _all(z, ids, t, tau, None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [40, 40003])
def test_masked_logits(vocab, dtype):
    z, ids, t, w = _inputs(6, vocab, 8, dtype, 9)
    low = torch.finfo(dtype).min
    mask = torch.rand(z.shape, generator=torch.Generator().manual_seed(2)) < 0.7
    mask.scatter_(1, ids.long(), False)
    z[0][mask[0]] = float("-inf")
    z[1][mask[1]] = low
    t[2, 3] = float("-inf")                 # p = 0 there, whatever the student holds
    z[2, ids[2, 3]] = float("-inf")
    z[3] = low                              # a row masked whole: a uniform softmax
    zd, idd, td, wd = z.to(DEV), ids.to(DEV), t.to(DEV), w.to(DEV)
    dz = torch.empty_like(zd)
    loss, lse = q.qlora_distill_topk_fwd(zd, idd, td, 1.0, row_weight=wd, dZ=dz)
    _check(z, ids, t, 1.0, w, loss, lse, dz)
    keep = torch.tensor([0, 1, 2, 4, 5])    # (fp32 cannot hold -3e38 + log n: the backward's rows are the others)
    bz = q.qlora_distill_topk_bwd(zd[keep], idd[keep], td[keep], 1.0, lse[keep], row_weight=wd[keep])
    _check(z[keep], ids[keep], t[keep], 1.0, w[keep], dz=bz, from_lse=lse[keep])
    # the teacher wants what the student has ruled out
    z[4, ids[4, 0]] = float("-inf")
    loss, _ = q.qlora_distill_topk_fwd(z.to(DEV), idd, td, 1.0, row_weight=wd)
    assert torch.isposinf(loss[4]).item() and torch.isfinite(loss[[0, 1, 2, 3, 5]]).all()


@pytest.mark.parametrize("vocab", [64, 33333])
def test_rows_with_nothing_to_learn(vocab):
    z, ids, t, w = _inputs(6, vocab, 5, torch.float32, 11)
    ids[0] = -1                             # no entry at all
    t[1] = float("-inf")                    # no entry with weight
    w[2] = 0.0                              # a padded position ...
    z[2] = float("nan")                     # ... that holds anything
    ids[3, 1:] = -7
    zd, idd, td, wd = z.to(DEV), ids.to(DEV), t.to(DEV), w.to(DEV)
    dz = torch.full_like(zd, float("nan"))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    loss, lse = q.qlora_distill_topk_fwd(zd, idd, td, 2.0, row_weight=wd, dZ=dz, d_status=st)
    assert st.item() == 0
    assert torch.count_nonzero(loss[:3]) == 0 and torch.count_nonzero(dz[:3]) == 0
    live = torch.tensor([3, 4, 5])
    _check(z[live], ids[live], t[live], 2.0, w[live], loss[live], lse[live], dz[live])
    bz = torch.full_like(zd, float("nan"))
    g = torch.tensor([1.0, 1, 1, 1, 0, 1], device=DEV)
    q.qlora_distill_topk_bwd(zd, idd, td, 2.0, lse, row_weight=wd, grad_loss=g, dZ=bz)
    assert torch.count_nonzero(bz[[0, 1, 2, 4]]) == 0 and torch.count_nonzero(bz[3]) > 0


@pytest.mark.parametrize("vocab", [50, 40001])
def test_repeated_and_foreign_ids(vocab):
    z, ids, t, w = _inputs(4, vocab, 9, torch.float32, 15)
    ids[0, 1:4] = ids[0, 0]                 # one index four times
    ids[1] = ids[1, 0]                      # nothing but one index
    _all(z, ids, t, 1.0, w)
    ids[2, 5] = vocab                       # past the end: left out, and said
    ids[3, 0] = 2 ** 31 - 1
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dz = torch.empty(z.shape, device=DEV)
    loss, lse = q.qlora_distill_topk_fwd(z.to(DEV), ids.to(DEV), t.to(DEV), 1.0, row_weight=w.to(DEV), dZ=dz, d_status=st)
    assert st.item() == q.qlora.DEV_INDEX
    _check(z, ids, t, 1.0, w, loss, lse, dz)


def test_nan_and_hopeless_rows_are_nan():
    z, ids, t, w = _inputs(4, 3000, 4, torch.float32, 17)
    z[0, 1234] = float("nan")
    z[1] = float("-inf")
    z[2, 5] = float("inf")
    dz = torch.empty(z.shape, device=DEV)
    loss, _ = q.qlora_distill_topk_fwd(z.to(DEV), ids.to(DEV), t.to(DEV), 1.0, dZ=dz)
    assert torch.isnan(loss[:3]).all() and torch.isfinite(loss[3])
    assert torch.isfinite(dz[3]).all() and torch.isnan(dz[0]).any()


@pytest.mark.parametrize("vocab,ld,off", [(1000, 1003, 0), (1001, 1024, 5), (33000, 33001, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_offset_and_in_place(vocab, ld, off, dtype):
    z, ids, t, w = _inputs(5, vocab, 20, dtype, 19)
    idd, td, wd = ids.to(DEV), t.to(DEV), w.to(DEV)

    def spread(fill):
        base = torch.full((5, ld), fill, dtype=dtype, device=DEV)
        return base, (base[:, off:off + vocab] if off + vocab <= ld else base[:, :vocab])
    zb, zv = spread(77.0)
    zv.copy_(z)
    db, dv = spread(77.0)
    loss, lse = q.qlora_distill_topk_fwd(zv, idd, td, 1.0, row_weight=wd, dZ=dv)
    _check(z, ids, t, 1.0, w, loss, lse, dv)
    packed = torch.empty_like(z, device=DEV)          # another alignment than Z's
    q.qlora_distill_topk_fwd(zv, idd, td, 1.0, row_weight=wd, dZ=packed)
    _check(z, ids, t, 1.0, w, dz=packed)
    before = dv.clone()
    l2, _ = q.qlora_distill_topk_fwd(zv, idd, td, 1.0, row_weight=wd, dZ=zv)      # in place
    assert torch.equal(l2, loss) and torch.equal(zv, before)
    zv.copy_(z)
    q.qlora_distill_topk_bwd(zv, idd, td, 1.0, lse, row_weight=wd, dZ=zv)
    _check(z, ids, t, 1.0, w, dz=zv, from_lse=lse)
    for base, v in ((zb, zv), (db, dv)):
        v.fill_(77.0)
        assert torch.all(base == 77.0)


def test_gradient_against_differences():
    # <dL/dz, v> against a central difference of the loss: the remainder is
    # h^2 / 6 of a third derivative of order tau^2 |v|^3 / tau^3, the loss is
    # known to about 1e-6
    z, ids, t, w = _inputs(3, 800, 10, torch.float32, 23)
    v = torch.randn(z.shape, generator=torch.Generator().manual_seed(3))
    tau, h = 2.0, 2e-2
    idd, td, wd = ids.to(DEV), t.to(DEV), w.to(DEV)
    dz = torch.empty(z.shape, device=DEV)
    q.qlora_distill_topk_fwd(z.to(DEV), idd, td, tau, row_weight=wd, dZ=dz)
    L = lambda zz: q.qlora_distill_topk_fwd(zz.to(DEV), idd, td, tau, row_weight=wd)[0].double().cpu()
    fd = (L(z + h * v) - L(z - h * v)) / (2 * h)
    an = (dz.double().cpu() * v.double()).sum(1)
    assert torch.all((fd - an).abs() <= 1e-3 * w.double() * tau)


def test_no_rows():
    z = torch.empty((0, 10), device=DEV)
    loss, lse = q.qlora_distill_topk_fwd(z, torch.empty((0, 2), dtype=torch.int32, device=DEV),
                                         torch.empty((0, 2), device=DEV))
    assert loss.shape == (0,) and lse.shape == (0,)


def test_repeats_bit_for_bit_and_replays_from_a_graph():
    for rows, vocab in ((40, 70001), (600, 5000)):
        z, ids, t, w = (x.to(DEV) for x in _inputs(rows, vocab, 30, torch.bfloat16, 29))
        dz = torch.empty_like(z)
        loss, lse = q.qlora_distill_topk_fwd(z, ids, t, 2.0, row_weight=w, dZ=dz)
        for _ in range(3):
            d2 = torch.empty_like(z)
            l2, s2 = q.qlora_distill_topk_fwd(z, ids, t, 2.0, row_weight=w, dZ=d2)
            assert torch.equal(l2, loss) and torch.equal(s2, lse) and torch.equal(d2, dz)
        bz = q.qlora_distill_topk_bwd(z, ids, t, 2.0, lse, row_weight=w)
        out = [torch.empty_like(x) for x in (loss, lse, dz, bz)]
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            q.qlora_distill_topk_fwd(z, ids, t, 2.0, row_weight=w, loss=out[0], lse=out[1], dZ=out[2])
            q.qlora_distill_topk_bwd(z, ids, t, 2.0, out[1], row_weight=w, dZ=out[3])
        for x in out:
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(out, (loss, lse, dz, bz)))
