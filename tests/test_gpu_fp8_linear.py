"""The FP8 frozen layer: quantiser bit for bit against the oracle, forward
and dX against binary64 products of the quantised values.

Tolerances, derived: a block's 128 products (exact) are added by the tensor
core at fp32 precision or better, at worst truncating (2^-23 per addition),
then K / 128 scaled sums in fp32 (and 8 partial sums in the streaming
kernel), so an output is off by at most (128 + K / 128 + 12) 2^-23 times the
sum of its products' magnitudes; a bf16 output is rounded once more (2^-8
relative at most, 1.7e-3 in the mean: 2e-3 for the whole matrix).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import bit_nf4_quantized_21_b200 as q
import oracle as O
import oracle.tail as OT

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().double().cpu().numpy()


def _normal(shape, sigma, seed, dtype=torch.float32):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * sigma).to(dtype)


def _codes(m):
    return m.codes.view(torch.uint8)[:, :m.cols].cpu().numpy()


def _values(m):
    """Binary64 values of a quantised matrix on the GPU, decoded with torch's own table."""
    v = m.codes.view(torch.float8_e4m3fn)[:, :m.cols].double()
    s = m.scale.double()
    if m.block_rows == 1:
        s = s.t()
    s = s.repeat_interleave(m.block_rows, 0)[:m.rows].repeat_interleave(128, 1)[:, :m.cols]
    return v * s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,block_rows", [
    (1, 1, 1), (3, 127, 1), (5, 128, 1), (2, 300, 1), (40, 1000, 1), (1, 1, 128), (130, 257, 128), (128, 128, 128),
    (200, 384, 128)])
def test_quantiser_matches_oracle(rows, cols, block_rows, dtype):
    x = _normal((rows, cols), 0.5, rows + cols, dtype)
    if rows > 1:
        x[0, :min(cols, 128)] = 0.0
        x[1, 0] = 300.0
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m = q.qlora_fp8_quantize(x.to(DEV), block_rows=block_rows, d_status=st)
    assert st.item() == 0
    codes, scale = OT.fp8_quantize(x.float().numpy(), block_rows)
    assert np.array_equal(m.scale.cpu().numpy(), scale)
    got = _codes(m)
    assert np.array_equal(np.where(got == 0x80, 0, got), np.where(codes == 0x80, 0, codes))


def test_quantiser_ties_extremes_and_strides():
    # absmax 448 exactly: s = 1, so values land on E4M3 numbers, midpoints and their neighbours
    vals = O.e4m3_values()
    mid = (vals[1:] + vals[:-1]) / 2
    x = np.concatenate([vals, mid, np.nextafter(mid.astype(np.float32), np.float32(1e9)),
                        np.nextafter(mid.astype(np.float32), np.float32(0))]).astype(np.float32)
    x = np.concatenate([x, -x])
    rows = -(-x.size // 127)
    full = np.zeros((rows, 128), np.float32)
    full[:, 0] = 448.0
    full[:, 1:].reshape(-1)[:] = 0
    flat = np.zeros(rows * 127, np.float32)
    flat[:x.size] = x
    full[:, 1:] = flat.reshape(rows, 127)
    m = q.qlora_fp8_quantize(torch.tensor(full, device=DEV), block_rows=1)
    codes, scale = OT.fp8_quantize(full, 1)
    assert np.all(scale == 1.0) and np.array_equal(m.scale.cpu().numpy(), scale)
    assert np.array_equal(_codes(m), codes)
    # tiny and huge blocks: below the smallest scale zeros, at the top no overflow
    ext = np.zeros((4, 128), np.float32)
    ext[0, :3] = [1e-37, -5e-36, 3e-39]      # s = 1.1e-38 is below the smallest normal number
    ext[1, :3] = [6e-36, -1e-36, 1e-38]
    ext[2, :3] = [3.4e38, -1e38, 1.0]
    m = q.qlora_fp8_quantize(torch.tensor(ext, device=DEV), block_rows=1)
    codes, scale = OT.fp8_quantize(ext, 1)
    got = _codes(m)
    assert scale[0, 0] == 0 and scale[0, 1] > 0 and np.array_equal(m.scale.cpu().numpy(), scale)
    assert np.array_equal(np.where(got == 0x80, 0, got), np.where(codes == 0x80, 0, codes))
    # rows of a wider matrix, at an odd offset: same codes
    base = _normal((50, 400), 1.0, 5, torch.bfloat16).to(DEV)
    for lo, hi in ((3, 303), (0, 256), (8, 333)):
        a = q.qlora_fp8_quantize(base[:, lo:hi], block_rows=1)
        b = q.qlora_fp8_quantize(base[:, lo:hi].contiguous(), block_rows=1)
        assert torch.equal(a.codes[:, :hi - lo], b.codes[:, :hi - lo]) and torch.equal(a.scale, b.scale)


def test_quantiser_says_non_finite_and_the_row_turns_nan():
    W = q.qlora_fp8_quantize(_normal((256, 256), 0.1, 1).to(DEV))
    for m in (4, 40):
        for bad in (float("nan"), float("inf")):
            x = _normal((m, 256), 1.0, 2)
            x[1, 100] = bad
            st = torch.zeros(1, dtype=torch.int32, device=DEV)
            y = q.qlora_fp8_linear_fwd(x.to(DEV), W, d_status=st)
            assert st.item() == q.qlora.DEV_NONFINITE
            assert torch.isnan(y[1]).all()
            assert torch.isfinite(y[torch.arange(m) != 1]).all()


def _check(out, a, b, ctr):
    """out against a @ b^T (binary64 on the GPU)."""
    ref, mag = a @ b.t(), a.abs() @ b.abs().t()
    slack = (128 + ctr / 128 + 12) * 2.0 ** -23 * mag
    hs = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    err = (out.double() - ref).abs()
    assert torch.all(err <= hs * (ref.abs() + slack) + slack), f"worst {(err / (mag + 1e-300)).max().item():.3e}"
    if out.dtype == torch.bfloat16:
        assert (err.norm() / ref.norm()).item() <= 2e-3


# token counts on either side of every rule: one, the streaming kernel's tiles
# (8, 16, 32), the first of the tile kernel, one tile, several tiles
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 300, 200), (5, 17, 100), (8, 256, 512), (9, 1000, 1040), (16, 128, 1152), (31, 300, 2000),
    (32, 515, 129), (33, 64, 64), (64, 256, 256), (100, 500, 130), (256, 512, 1024), (257, 300, 2048), (700, 1030, 900),
    (2100, 520, 384)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_forward_and_backward_match_binary64(M, N, K, out_dtype):
    W = q.qlora_fp8_quantize(_normal((N, K), 0.05, N + K).to(DEV))
    x = _normal((M, K), 1.0, M + K, torch.bfloat16).to(DEV)
    dy = _normal((M, N), 1e-3, M + N, torch.float32).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    xq, gq = q.empty_fp8(M, K, DEV, 1), q.empty_fp8(M, N, DEV, 1)
    y = q.qlora_fp8_linear_fwd(x, W, out_dtype=out_dtype, Xq=xq, d_status=st)
    dx = q.qlora_fp8_linear_bwd(dy, W, out_dtype=out_dtype, dYq=gq, d_status=st)
    assert st.item() == 0
    Wv = _values(W)
    _check(y, _values(xq), Wv, K)
    _check(dx, _values(gq), Wv.t(), N)
    # the quantised activations alone give the same result
    assert torch.equal(q.qlora_fp8_linear_fwd(xq, W, out_dtype=out_dtype), y)
    assert torch.equal(q.qlora_fp8_linear_bwd(gq, W, out_dtype=out_dtype), dx)
    # against the unquantised layer: two roundings to E4M3 (2^-4 at most each, about 2.6 % rms each) per product
    full = x.double() @ Wv.t()
    assert ((y.double() - full).norm() / full.norm()).item() <= 2.0 ** -4


# both tile widths of the product, either side of the last count of narrow
# tiles that all run at once, and more tiles than run at once, in each
# direction; whole and broken scale blocks, aligned and odd rows
@pytest.mark.parametrize("M,N,K", [
    (256, 9472, 384), (256, 9473, 300), (300, 9500, 700), (300, 384, 9472), (256, 300, 9475), (300, 700, 9500),
    (2600, 2600, 300), (2500, 300, 2601), (1100, 5000, 640)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_every_tile_width_and_count_matches_binary64(M, N, K, out_dtype):
    test_forward_and_backward_match_binary64(M, N, K, out_dtype)


def test_padding_bytes_of_the_weight_never_matter():
    N, K = 300, 200
    W = q.qlora_fp8_quantize(_normal((N, K), 0.05, 3).to(DEV))
    Z = q.FP8Matrix(N, K, 128, W.codes.clone(), W.scale)
    Z.codes[:, K:] = 0x7F                    # NaN codes
    tight = q.FP8Matrix(N, K, 128, W.codes[:, :208].contiguous(), W.scale)      # ld = 208
    tight.codes[:, K:] = 0x7F
    for M in (3, 20, 90):
        x = _normal((M, K), 1.0, M, torch.bfloat16).to(DEV)
        dy = _normal((M, N), 1.0, M + 1, torch.bfloat16).to(DEV)
        for V in (Z, tight):
            assert torch.equal(q.qlora_fp8_linear_fwd(x, W), q.qlora_fp8_linear_fwd(x, V))
            assert torch.equal(q.qlora_fp8_linear_bwd(dy, W), q.qlora_fp8_linear_bwd(dy, V))


@pytest.mark.parametrize("M", [2, 70])
@pytest.mark.parametrize("N,ld,off", [(264, 300, 0), (256, 257, 1), (130, 136, 3)])
def test_strided_rows_leave_the_rest_alone(M, N, ld, off):
    K = 256
    W = q.qlora_fp8_quantize(_normal((N, K), 0.05, 7).to(DEV))
    xb = _normal((M, K + 5), 1.0, 8, torch.bfloat16).to(DEV)
    for dt in (torch.bfloat16, torch.float32):
        base = torch.full((M + 1, ld), 55.0, dtype=dt, device=DEV)
        y = base[:M, off:off + N]
        q.qlora_fp8_linear_fwd(xb[:, 3:3 + K], W, Y=y)
        assert torch.equal(y, q.qlora_fp8_linear_fwd(xb[:, 3:3 + K].contiguous(), W, out_dtype=dt))
        y.fill_(55.0)
        assert torch.all(base == 55.0)
        base = torch.full((M + 1, K + ld), 55.0, dtype=dt, device=DEV)
        dx = base[:M, off:off + K]
        dy = _normal((M, N), 1.0, 9, torch.bfloat16).to(DEV)
        q.qlora_fp8_linear_bwd(dy, W, dX=dx)
        assert torch.equal(dx, q.qlora_fp8_linear_bwd(dy, W, out_dtype=dt))
        dx.fill_(55.0)
        assert torch.all(base == 55.0)


def test_every_persistent_tile_is_written():
    # more tiles than pairs of SMs, ragged on both sides, and the group of tile rows cut
    M, N, K = 2600, 3000, 256
    W = q.qlora_fp8_quantize(_normal((N, K), 0.05, 11).to(DEV))
    x = _normal((M, K), 1.0, 12, torch.bfloat16).to(DEV)
    xq = q.empty_fp8(M, K, DEV, 1)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    q.qlora_fp8_linear_fwd(x, W, Y=y, Xq=xq)
    _check(y, _values(xq), _values(W), K)


def test_no_tokens():
    W = q.qlora_fp8_quantize(_normal((128, 128), 0.05, 1).to(DEV))
    assert q.qlora_fp8_linear_fwd(torch.empty((0, 128), device=DEV), W).shape == (0, 128)
    assert q.qlora_fp8_linear_bwd(torch.empty((0, 128), device=DEV), W).shape == (0, 128)


def test_gradient_against_differences():
    # dX is linear in dY and Y linear in the quantised X: <dY, Y(x + h v) - Y(x)> for a
    # step v that the quantiser represents exactly equals h <dX, v> up to the
    # quantisation of dY; take dY exact too (powers of two) and fp32 outputs
    N = K = 256
    W = q.qlora_fp8_quantize(_normal((N, K), 0.05, 13).to(DEV))
    x = torch.ones((40, K), device=DEV) * 448.0
    v = torch.zeros_like(x)
    v[:, ::3] = -448.0
    dy = torch.sign(_normal((40, N), 1.0, 14)).to(DEV)
    d = q.qlora_fp8_linear_fwd(x + v, W, out_dtype=torch.float32) - q.qlora_fp8_linear_fwd(x, W, out_dtype=torch.float32)
    dx = q.qlora_fp8_linear_bwd(dy, W, out_dtype=torch.float32)
    a, b = (d.double() * dy.double()).sum().item(), (dx.double() * v.double()).sum().item()
    mag = (v.abs().double() @ _values(W).abs().t()).sum().item()
    assert abs(a - b) <= 160 * 2.0 ** -22 * mag


def test_repeats_bit_for_bit_and_replays_from_a_graph():
    W = q.qlora_fp8_quantize(_normal((1024, 2048), 0.05, 15).to(DEV))
    for M in (7, 600):
        x = _normal((M, 2048), 1.0, 16, torch.bfloat16).to(DEV)
        dy = _normal((M, 1024), 1.0, 17, torch.bfloat16).to(DEV)
        y, dx = q.qlora_fp8_linear_fwd(x, W), q.qlora_fp8_linear_bwd(dy, W)
        for _ in range(3):
            assert torch.equal(q.qlora_fp8_linear_fwd(x, W), y) and torch.equal(q.qlora_fp8_linear_bwd(dy, W), dx)
        xq, gq = q.empty_fp8(M, 2048, DEV, 1), q.empty_fp8(M, 1024, DEV, 1)
        out = [torch.empty_like(y), torch.empty_like(dx)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q.qlora_fp8_linear_fwd(x, W, Y=out[0], Xq=xq)
            q.qlora_fp8_linear_bwd(dy, W, dX=out[1], dYq=gq)
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], y) and torch.equal(out[1], dx)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        z = q.qlora_fp8_linear_fwd(x, W, stream=side)
        side.synchronize()
        assert torch.equal(z, y)
