"""Rows whose offsets pass 32 bits, and products of a single block of 128 over
many tiles: the FP8 layer, the layer norm and the distillation loss on rows of
much wider matrices give the bits that they give on compact ones."""
import pytest
import torch

import bit_nf4_quantized_21_b200 as q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _normal(shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def _far(x, ld):
    """x as rows of a matrix ld elements wide (the last row is not padded)."""
    rows, cols = x.shape
    base = torch.empty((rows - 1) * ld + cols, dtype=x.dtype, device=DEV)
    assert (rows - 1) * ld > 2 ** 31
    out = base.as_strided((rows, cols), (ld, 1))
    out.copy_(x)
    return out


@pytest.mark.parametrize("rows,cols,ld", [(3, 515, 2 ** 30 + 8), (3, 4096, 2 ** 30 + 8), (1200, 4096, 1900032),
                                          (3, 20000, 2 ** 30 + 8)])
def test_layer_norm_of_far_rows(rows, cols, ld):
    x, dy, w = _normal((rows, cols), 1), _normal((rows, cols), 2), _normal((cols,), 3)
    y, mean, rstd = q.qlora_layernorm_fwd(x, w, w)
    fx, fy = _far(x, ld), _far(torch.zeros_like(x), ld)
    _, m2, r2 = q.qlora_layernorm_fwd(fx, w, w, Y=fy)
    assert torch.equal(fy, y) and torch.equal(m2, mean) and torch.equal(r2, rstd)
    dx, dw, db = q.qlora_layernorm_bwd(dy, x, w, mean, rstd)
    fy.copy_(dy)
    _, dw2, db2 = q.qlora_layernorm_bwd(fy, fx, w, mean, rstd, dX=fy)      # in place of dY
    assert torch.equal(fy, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("rows,vocab,ld", [(3, 50021, 2 ** 30 + 8), (5, 8192, 2 ** 29 + 8)])
def test_distillation_of_far_rows(rows, vocab, ld):
    z, t = _normal((rows, vocab), 4), _normal((rows, 20), 5)
    ids = torch.randint(0, vocab, (rows, 20), generator=torch.Generator().manual_seed(6)).to(DEV)
    dz = torch.empty_like(z)
    loss, lse = q.qlora_distill_topk_fwd(z, ids, t, 2.0, dZ=dz)
    fz = _far(z, ld)
    back = _far(z, ld)
    l2, s2 = q.qlora_distill_topk_fwd(fz, ids, t, 2.0, dZ=fz)              # in place
    assert torch.equal(l2, loss) and torch.equal(s2, lse) and torch.equal(fz, dz)
    want = q.qlora_distill_topk_bwd(z, ids, t, 2.0, lse)
    assert torch.equal(q.qlora_distill_topk_bwd(back, ids, t, 2.0, lse, dZ=back), want)


@pytest.mark.parametrize("M", [3, 200])
def test_fp8_layer_over_far_rows(M):
    N, K = 300, 400
    W = q.qlora_fp8_quantize(_normal((N, K), 7, 0.05))
    ldw = 2 ** 31 // (N - 1) // 16 * 16 + 16
    codes = torch.zeros((N - 1) * ldw + 512, dtype=torch.uint8, device=DEV).as_strided((N, 512), (ldw, 1))
    far = q.FP8Matrix(N, K, 128, codes, torch.empty_like(W.scale))
    ldx = 2 ** 31 // (M - 1) // 8 * 8 + 8
    q.qlora_fp8_quantize(_normal((N, K), 7, 0.05), out=far)
    assert torch.equal(far.codes[:, :K], W.codes[:, :K]) and torch.equal(far.scale, W.scale)
    x, dy = _normal((M, K), 8), _normal((M, N), 9)
    want, dwant = q.qlora_fp8_linear_fwd(x, W), q.qlora_fp8_linear_bwd(dy, W)
    fx = _far(x, ldx)
    out = _far(torch.zeros((M, N), dtype=torch.bfloat16, device=DEV), ldx)
    assert torch.equal(q.qlora_fp8_linear_fwd(fx, far, Y=out), want) and torch.equal(out, want)
    del fx
    dout = _far(torch.zeros((M, K), dtype=torch.bfloat16, device=DEV), ldx)
    out.copy_(dy)
    assert torch.equal(q.qlora_fp8_linear_bwd(out, far, dX=dout), dwant)


# one block of the contraction, more tiles than run at once
@pytest.mark.parametrize("M,N,K", [(2600, 2600, 100), (2600, 100, 2600), (4200, 2600, 128), (5000, 4000, 16)])
def test_single_blocks_over_many_tiles(M, N, K):
    W = q.qlora_fp8_quantize(_normal((N, K), 10, 0.05))
    x, dy = _normal((M, K), 11), _normal((M, N), 12)
    y, dx = q.qlora_fp8_linear_fwd(x, W), q.qlora_fp8_linear_bwd(dy, W)
    # every slice of rows by itself (other tiles, other widths): the same sums in the same order
    for lo in range(0, M, 700):
        hi = min(M, lo + 700)
        if hi - lo <= 32:
            continue
        assert torch.equal(q.qlora_fp8_linear_fwd(x[lo:hi], W), y[lo:hi])
        assert torch.equal(q.qlora_fp8_linear_bwd(dy[lo:hi], W), dx[lo:hi])
