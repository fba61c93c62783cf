"""The distillation loss at the edges of its temperature and of its teacher's
list, against the formula in binary64 with the maximum subtracted before the
temperature divides."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import bit_nf4_quantized_21_b200 as q

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def _formula(z, ids, t, tau):
    """(loss, dz) of weights of one; every id is listed once and inside the vocabulary."""
    z, t, ids = z.double().numpy(), t.double().numpy(), ids.numpy()
    e = (t - t.max(1, keepdims=True)) / tau
    logp = e - np.log(np.exp(e).sum(1, keepdims=True))
    p = np.exp(logp)
    u = (z - z.max(1, keepdims=True)) / tau
    logq = u - np.log(np.exp(u).sum(1, keepdims=True))
    at = np.take_along_axis(logq, ids, 1)
    loss = tau * tau * np.where(p > 0, p * (logp - at), 0.0).sum(1)
    dz = np.exp(logq)
    np.put_along_axis(dz, ids, np.take_along_axis(dz, ids, 1) - p, 1)
    return loss, dz * tau


# A list masked whole by its type's lowest value stands for p = 1 / top, at any temperature.
# Bounds: p and q are exponentials (2^-21 relative) of arguments below 40, each rounded three
# times (40 * 3 u), over sums of at most `vocab` / 256 + 64 roundings in a chain: E.  The loss
# adds terms of at most 2 |log q| <= 80 with that error; the gradient is tau times a difference
# of two values of at most one.
@pytest.mark.parametrize("t_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tau", [0.25, 0.5, 0.99, 1.0, 3.0])
@pytest.mark.parametrize("vocab,top", [(50, 3), (40003, 40)])
def test_teachers_lists_of_the_lowest_value(vocab, top, tau, t_dtype):
    g = torch.Generator().manual_seed(vocab + top)
    z = torch.randn(4, vocab, generator=g)
    ids = torch.stack([torch.randperm(vocab, generator=g)[:top] for _ in range(4)])
    t = torch.randn(4, top, generator=g).to(t_dtype)
    low = torch.finfo(t_dtype).min
    t[0] = low                          # masked whole
    t[1, 1:] = low                      # one entry left: p = 1 there
    t[2, 0] = -low                      # the type's highest: everything else vanishes beside it
    zd, idd, td = z.to(DEV), ids.to(DEV), t.to(DEV)
    dz = torch.empty_like(zd)
    loss, lse = q.qlora_distill_topk_fwd(zd, idd, td, tau, dZ=dz)
    bz = q.qlora_distill_topk_bwd(zd, idd, td, tau, lse)
    rl, rdz = _formula(z, ids, t, tau)
    E = 2.0 ** -21 + 120 * U + (vocab / 256 + 64) * U
    spread = float(z.max() - z.min()) / tau + np.log(vocab)
    assert np.all(np.abs(loss.double().cpu().numpy() - rl) <= tau * tau * (2 * E + E * spread))
    for got, more in ((dz, 0.0), (bz, 4 * U * float(lse.abs().max()))):
        err = np.abs(got.double().cpu().numpy() - rdz)
        assert np.all(err <= tau * (2 * E + more) + np.abs(rdz) * U)
    assert loss[0].item() > 0 and torch.count_nonzero(dz[0]).item() > vocab // 2


# The student holds its type's lowest value, L, at listed entries.  The loss is then w tau sum p_j |L|
# but for what the sum's rounding swallows: finite where that is, and +inf where it passes fp32's largest
# number.  Bounds: p_j and the sum as above (E), the products and the sum of the list's terms one
# rounding each, the weight's and tau's products two more.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tau", [0.25, 0.5, 0.99, 1.0, 3.0])
@pytest.mark.parametrize("vocab,top", [(50, 3), (40003, 40)])
def test_students_logits_of_the_lowest_value_at_listed_entries(vocab, top, tau, dtype):
    g = torch.Generator().manual_seed(vocab + top + 1)
    z = torch.randn(3, vocab, generator=g).to(dtype)
    ids = torch.stack([torch.randperm(vocab, generator=g)[:top] for _ in range(3)])
    t = torch.randn(3, top, generator=g)
    w = torch.tensor([0.5, 0.25, 1.0])
    z[0, ids[0]] = torch.finfo(dtype).min
    z[1, ids[1, 1]] = torch.finfo(dtype).min
    zd, idd, td, wd = z.to(DEV), ids.to(DEV), t.to(DEV), w.to(DEV)
    dz = torch.empty_like(zd)
    loss, _ = q.qlora_distill_topk_fwd(zd, idd, td, tau, row_weight=wd, dZ=dz)
    rl, rdz = _formula(z, ids, t, tau)
    rl, rdz = rl * w.double().numpy(), rdz * w.double().numpy()[:, None]
    assert (rl[0] > 1e37) and (rl[1] > 1e24)        # (of the formula: one entry's p may be 1e-9 at tau = 0.25)
    E = 2.0 ** -21 + 120 * U + (vocab / 256 + 64) * U
    spread = float(z[2].double().max() - z[2].double().min()) / tau + np.log(vocab)
    got = loss.double().cpu().numpy()
    tol = np.array([(E + 8 * U) * rl[0], (E + 8 * U) * rl[1], tau * tau * (2 * E + E * spread)])
    largest = torch.finfo(torch.float32).max
    inside = rl + tol < largest
    assert np.all(np.abs(got - rl)[inside] <= tol[inside])
    assert np.all(np.isposinf(got)[rl - tol > largest])
    assert np.all(np.abs(dz.double().cpu().numpy() - rdz) <= tau * 2 * E + np.abs(rdz) * torch.finfo(dtype).eps / 2)
