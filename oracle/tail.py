"""Binary64 statements of the operators around the frozen products -- TEST
INFRASTRUCTURE ONLY: the FP8 frozen layer, the layer norm and the
distillation loss, written from their formulas with numpy, row by row where
that is the plainer form."""
from __future__ import annotations

import numpy as np

from .oracle import e4m3_encode, e4m3_values

FLT_MIN = np.float32(np.finfo(np.float32).tiny)


# ------------------------------------------------------------------ FP8 blocks

def fp8_quantize(x: np.ndarray, block_rows: int):
    """(codes uint8 [rows, cols], scale fp32) of fp32 x: the format's fp32
    steps s = absmax / 448, r = 1 / s, code = E4M3(x r)."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    nb, kb = -(-rows // block_rows), -(-cols // 128)
    codes = np.zeros((rows, cols), np.uint8)
    scale = np.zeros((nb, kb), np.float32)
    for i in range(nb):
        for j in range(kb):
            at = (slice(i * block_rows, (i + 1) * block_rows), slice(j * 128, (j + 1) * 128))
            b = x[at]
            s = np.float32(np.abs(b).max() / np.float32(448.0))
            if s < FLT_MIN:
                continue
            r = np.float32(1.0) / s
            v = (b * r).astype(np.float32)
            # the encoder takes magnitudes; the sign is the top bit
            mag = e4m3_encode(np.abs(v).ravel()).reshape(v.shape).astype(np.uint8)
            codes[at] = mag | (np.signbit(v).astype(np.uint8) << 7)
            scale[i, j] = s
    return codes, (scale.T.copy() if block_rows == 1 else scale)


def fp8_values(codes: np.ndarray, scale: np.ndarray, block_rows: int) -> np.ndarray:
    """Binary64 values of a matrix in the format."""
    table = np.asarray(e4m3_values(), np.float64)
    c = codes.astype(np.int64)
    v = np.where(c & 0x80, -1.0, 1.0) * table[c & 0x7F]
    s = np.asarray(scale, np.float64)
    if block_rows == 1:
        s = s.T
    s = np.repeat(np.repeat(s, block_rows, 0)[:codes.shape[0]], 128, 1)[:, :codes.shape[1]]
    return v * s


# ------------------------------------------------------------------ layer norm

def layernorm_fwd(x, w=None, b=None, eps=1e-5):
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1.0 / np.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if b is not None:
        y = y + np.asarray(b, np.float64)
    return y, mean, rstd


def layernorm_bwd(dy, x, w, mean, rstd):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    xh = (x - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    g = dy if w is None else dy * np.asarray(w, np.float64)
    dx = np.asarray(rstd, np.float64)[:, None] * (g - g.mean(1)[:, None] - xh * (g * xh).mean(1)[:, None])
    return dx, (dy * xh).sum(0), dy.sum(0)


# ---------------------------------------------------------------- distillation

def distill(z, ids, t, tau, weight=None, grad=None, lse=None):
    """(loss, lse, dz): loops over rows; an entry is used when 0 <= id < vocab."""
    z, t = np.asarray(z, np.float64), np.asarray(t, np.float64)
    rows, vocab = z.shape
    w = np.ones(rows) if weight is None else np.asarray(weight, np.float64)
    g = np.ones(rows) if grad is None else np.asarray(grad, np.float64)
    loss, out_lse, dz = np.zeros(rows), np.zeros(rows), np.zeros((rows, vocab))
    with np.errstate(all="ignore"):
        for i in range(rows):
            u = z[i] / tau
            top = u.max()
            top = top if np.isfinite(top) else 0.0
            total = np.log(np.exp(u - top).sum())       # of the shifted logits: -1e38 + log n is -1e38
            out_lse[i] = top + total
            used = [j for j in range(ids.shape[1]) if 0 <= ids[i, j] < vocab]
            e = np.array([t[i, j] / tau for j in used])
            if len(used) == 0 or np.all(e == -np.inf) or w[i] == 0 or g[i] == 0:
                if not (len(used) == 0 or np.all(e == -np.inf) or w[i] == 0):
                    raise ValueError("a zero upstream gradient is for the backward alone")
                continue
            shift = e.max()
            p = np.exp(e - shift)
            logp = (e - shift) - np.log(p.sum())
            p = p / p.sum()
            logq = (u - top) - total if lse is None else u - lse[i]
            for j, pj, lp in zip(used, p, logp):
                if pj != 0:
                    loss[i] += w[i] * tau * tau * pj * (lp - logq[ids[i, j]])
            dz[i] = np.exp(logq)
            for j, pj in zip(used, p):
                dz[i, ids[i, j]] -= pj
            dz[i] *= g[i] * w[i] * tau
    return loss, out_lse, dz
