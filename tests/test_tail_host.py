"""Host-side checks, without a GPU, of the FP8 layer, the layer norm and the
distillation loss: sizes, refusals before anything is enqueued, and the
binary64 statements against differences of themselves."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import bit_nf4_quantized_21_b200 as q
import oracle.tail as OT
from bit_nf4_quantized_21_b200 import qlora as binding

# Fake, aligned, never-dereferenced device addresses: every call below must
# fail validation on the host, before anything is enqueued.
FAKE = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6


def _m(rows, cols, block_rows, /, **kw):
    m = binding.FP8MatrixC(rows, cols, -(-cols // 128) * 128, block_rows, 0, FAKE, FAKE)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


# ------------------------------------------------------------------ FP8 layer

def test_fp8_sizes():
    assert q.qlora_fp8_sizes(256, 512) == (256 * 512, 2 * 4 * 4)
    assert q.qlora_fp8_sizes(300, 130) == (300 * 256, 3 * 2 * 4)
    assert q.qlora_fp8_sizes(7, 130, 1) == (7 * 256, 7 * 2 * 4)
    assert q.qlora_fp8_sizes(0, 130, 1) == (0, 0)
    for bad in ((-1, 128, 1), (4, 0, 1), (4, 128, 64)):
        with pytest.raises(q.QloraError):
            q.qlora_fp8_sizes(*bad)


@pytest.mark.parametrize("field,value,expect", [
    ("rows", -1, INVALID), ("cols", 0, INVALID), ("ld", 500, INVALID), ("ld", 520, INVALID), ("block_rows", 64, INVALID),
    ("reserved", 1, INVALID), ("codes", None, INVALID), ("codes", FAKE + 8, INVALID), ("scale", None, INVALID),
    ("scale", FAKE + 2, INVALID), ("ld", 1 << 31, UNSUPPORTED), ("rows", 1 << 31, UNSUPPORTED)])
def test_fp8_refuses_bad_descriptors(field, value, expect):
    L = q.lib()
    W, X = _m(256, 512, 128), _m(16, 512, 1)
    bad = _m(256, 512, 128, **{field: value})
    assert L.qlora_fp8_quantize(FAKE, 1, 512, ctypes.byref(bad), None, None) == expect
    if field != "rows":
        assert L.qlora_fp8_linear_fwd(FAKE, 1, 512, ctypes.byref(bad), ctypes.byref(X), FAKE, 1, 256, None, None) == expect
    badx = _m(16, 512, 1, **{field: value})
    assert L.qlora_fp8_linear_fwd(FAKE, 1, 512, ctypes.byref(W), ctypes.byref(badx), FAKE, 1, 256, None, None) == expect


def test_fp8_refuses_bad_calls():
    L = q.lib()
    W, X, G = _m(256, 512, 128), _m(16, 512, 1), _m(16, 256, 1)
    r = ctypes.byref
    good = [FAKE, 1, 512, r(W), r(X), FAKE, 1, 256, None, None]

    def f(i, v, fn=L.qlora_fp8_linear_fwd, base=good):
        a = list(base)
        a[i] = v
        return fn(*a)
    assert f(0, FAKE + 1) == INVALID            # misaligned bf16
    assert f(1, 7) == INVALID and f(6, 7) == INVALID
    assert f(2, 511) == INVALID                 # rows overlap
    assert f(7, 255) == INVALID
    assert f(5, None) == INVALID and f(5, FAKE + 1) == INVALID
    assert f(3, None) == INVALID and f(4, None) == INVALID
    assert f(3, r(_m(256, 512, 1))) == INVALID  # activations' blocks as a weight
    assert f(4, r(_m(16, 512, 128))) == INVALID
    assert f(4, r(G)) == INVALID                # another width
    assert f(3, r(_m(0, 512, 128))) == INVALID
    bwd = [FAKE, 1, 256, r(W), r(G), FAKE, 1, 512, None, None]
    assert f(4, r(X), L.qlora_fp8_linear_bwd, bwd) == INVALID
    assert f(7, 511, L.qlora_fp8_linear_bwd, bwd) == INVALID
    assert f(2, 255, L.qlora_fp8_linear_bwd, bwd) == INVALID
    assert L.qlora_fp8_quantize(None, 1, 512, r(X), None, None) == INVALID
    assert L.qlora_fp8_quantize(FAKE, 1, 100, r(X), None, None) == INVALID
    # no rows: nothing to do, nothing looked at
    assert L.qlora_fp8_linear_fwd(None, 1, 512, r(W), r(_m(0, 512, 1, codes=None, scale=None)), None, 1, 256, None, None) == 0


# ------------------------------------------------------------------ layer norm

def test_layernorm_refusals():
    L = q.lib()
    fwd = [FAKE, 64, 4, 64, 1, FAKE, FAKE, 1, 1e-5, FAKE, 64, FAKE, FAKE, None, None]

    def f(i, v):
        a = list(fwd)
        a[i] = v
        return L.qlora_layernorm_fwd(*a)
    for i, v in ((0, None), (0, FAKE + 1), (1, 63), (2, -1), (3, 0), (4, 5), (7, 5), (8, -1.0), (8, float("nan")),
                 (9, None), (9, FAKE + 1), (10, 63), (5, FAKE + 1), (6, FAKE + 1), (11, FAKE + 2), (12, FAKE + 2)):
        assert f(i, v) == INVALID, (i, v)
    assert L.qlora_layernorm_fwd(FAKE, 64, 4, 64, 1, None, None, 1, 1e-5, FAKE, 72, None, None, None, None) == INVALID
    need = q.qlora_layernorm_workspace_bytes(4, 64)
    assert need > 0 and q.qlora_layernorm_workspace_bytes(0, 64) == 0
    assert q.qlora_layernorm_workspace_bytes(-1, 64) == 0 and q.qlora_layernorm_workspace_bytes(4, 0) == 0
    other = FAKE + 4096
    bwd = [FAKE, 64, other, 64, 4, 64, 1, FAKE, 1, FAKE, FAKE, FAKE, 64, FAKE, FAKE, 0, FAKE, need, None, None]

    def b(i, v):
        a = list(bwd)
        a[i] = v
        return L.qlora_layernorm_bwd(*a)
    for i, v in ((0, None), (2, None), (9, None), (10, None), (11, None), (1, 60), (3, 60), (12, 60), (4, -2), (5, 0),
                 (6, 9), (8, 9), (15, 9), (13, FAKE + 2), (14, FAKE + 2), (11, FAKE + 1), (12, 72)):   # in place, another stride
        assert b(i, v) == INVALID, (i, v)
    assert b(16, None) == WORKSPACE and b(16, FAKE + 8) == WORKSPACE and b(17, need - 1) == WORKSPACE


# ---------------------------------------------------------------- distillation

def test_distill_refusals():
    L = q.lib()
    fwd = [FAKE, 100, 4, 100, 1, FAKE, 32, FAKE, 0, 8, 1.0, FAKE, FAKE, FAKE, FAKE, 100, None, None]

    def f(i, v, also=()):
        a = list(fwd)
        a[i] = v
        for j, w in also:
            a[j] = w
        return L.qlora_distill_topk_fwd(*a)
    for i, v in ((0, None), (0, FAKE + 1), (1, 99), (2, -1), (3, 0), (4, 4), (5, None), (5, FAKE + 2), (6, 16), (7, None),
                 (7, FAKE + 2), (8, 4), (9, 0), (9, 1025), (10, 0.0), (10, -1.0), (10, float("nan")), (10, float("inf")),
                 (10, 1e-40), (11, FAKE + 2), (12, None), (12, FAKE + 2), (13, FAKE + 2), (14, FAKE + 1), (15, 99)):
        assert f(i, v) == INVALID, (i, v)
    assert f(6, 64, [(5, FAKE + 4)]) == INVALID
    assert f(15, 104, [(14, FAKE)]) == INVALID              # in place with another stride
    assert f(3, 1 << 31, [(1, 1 << 31), (15, 1 << 31)]) == UNSUPPORTED
    bwd = [FAKE, 100, 4, 100, 1, FAKE, 32, FAKE, 0, 8, 1.0, FAKE, FAKE, FAKE, FAKE, 100, None, None]
    for i, v in ((12, None), (12, FAKE + 2), (13, FAKE + 2), (14, None), (14, FAKE + 1), (9, 2000)):
        a = list(bwd)
        a[i] = v
        assert L.qlora_distill_topk_bwd(*a) == INVALID, (i, v)


def test_binding_refuses_what_it_cannot_pass_on():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        q.qlora_layernorm_fwd(x)                             # host tensors
    with pytest.raises(ValueError):
        q.qlora_distill_topk_fwd(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        q.qlora_fp8_quantize(x)
    with pytest.raises(ValueError):
        q.qlora_fp8_quantize(x.half())
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_fwd(x, q.empty_fp8(128, 64, "cpu"))


# ------------------------------------------------- the statements themselves

def _differences(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_layernorm_statement_against_differences():
    r = np.random.default_rng(1)
    x, c, w, b, v = r.normal(size=(3, 40)), r.normal(size=(3, 40)), r.normal(size=40), r.normal(size=40), r.normal(size=(3, 40))
    _, mean, rstd = OT.layernorm_fwd(x, w, b)
    dx, dw, db = OT.layernorm_bwd(c, x, w, mean, rstd)
    L = lambda xx=x, ww=w, bb=b: (OT.layernorm_fwd(xx, ww, bb)[0] * c).sum()
    assert abs(_differences(lambda xx: L(xx=xx), x, v) - (dx * v).sum()) < 1e-6
    assert abs(_differences(lambda ww: L(ww=ww), w, v[0]) - (dw * v[0]).sum()) < 1e-6
    assert abs(_differences(lambda bb: L(bb=bb), b, v[0]) - (db * v[0]).sum()) < 1e-6


def test_distill_statement_against_differences_and_special_cases():
    r = np.random.default_rng(2)
    z, t, v = r.normal(size=(3, 30)) * 2, r.normal(size=(3, 6)), r.normal(size=(3, 30))
    ids = r.integers(0, 30, size=(3, 6))
    ids[1, 2] = ids[1, 0]
    ids[2, 4] = -1
    w = np.array([0.5, 1.0, 2.0])
    loss, lse, dz = OT.distill(z, ids, t, 1.7, w)
    fd = _differences(lambda zz: OT.distill(zz, ids, t, 1.7, w)[0], z, v)
    assert np.all(np.abs(fd - (dz * v).sum(1)) < 1e-6)
    assert np.all(np.abs(dz.sum(1)) < 1e-12)                  # p and q both sum to one
    # a student that equals a teacher listed whole: no loss, no gradient
    full = np.argsort(-z, axis=1)
    loss, _, dz = OT.distill(z, full, np.take_along_axis(z, full, 1), 1.3)
    assert np.all(np.abs(loss) < 1e-12) and np.all(np.abs(dz) < 1e-12)


def test_fp8_statement_reconstructs_within_half_a_step():
    r = np.random.default_rng(3)
    x = r.normal(size=(130, 200)).astype(np.float32)
    for br in (1, 128):
        codes, scale = OT.fp8_quantize(x, br)
        v = OT.fp8_values(codes, scale, br)
        s = np.repeat(np.repeat((scale.T if br == 1 else scale).astype(np.float64), br, 0)[:130], 128, 1)[:, :200]
        # half a step: 2^-4 relative for normal values, 2^-10 scales below them
        assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) * (1 + 1e-6))
