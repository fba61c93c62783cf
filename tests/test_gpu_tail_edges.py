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
