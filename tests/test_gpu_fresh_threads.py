"""Calls that are the first CUDA work of a host thread: the device's context is
current in no thread before the runtime has made it so there."""
from __future__ import annotations

import threading

import pytest
import torch

import bit_nf4_quantized_21_b200 as q

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _normal(shape, scale, seed):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(DEV).bfloat16()


def _calls():
    """name -> (call, the tensors it writes): everything is allocated here, so that the call itself comes first."""
    M, N, K, r = 300, 512, 768, 16
    w, x, dy = _normal((N, K), 0.05, 1), _normal((M, K), 1.0, 2), _normal((M, N), 1.0, 3)
    A, B = _normal((r, K), 0.05, 4), _normal((N, r), 0.05, 5)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    f32 = dict(dtype=torch.float32, device=DEV)
    W8, W4 = q.qlora_fp8_quantize(w), q.qlora_quantize_nf4(w)
    xq, gq = q.empty_fp8(M, K, DEV, 1), q.empty_fp8(M, N, DEV, 1)
    kept = q.qlora_fp8_quantize(x, block_rows=1)
    y, dx, T, ws = torch.empty(M, N, **bf), torch.empty(M, K, **bf), torch.empty(M, r, **f32), torch.empty(
        q.qlora_workspace_bytes(M, N, K, r), dtype=torch.uint8, device=DEV)
    dA, dB = torch.empty(r, K, **f32), torch.empty(N, r, **f32)
    g, b, ny, mean, rstd = _normal((K,), 1.0, 6), _normal((K,), 1.0, 7), torch.empty_like(x), torch.empty(M, **f32), torch.empty(M, **f32)
    return {
        "fp8_fwd": (lambda: q.qlora_fp8_linear_fwd(x, W8, y, Xq=xq), [y]),
        "fp8_fwd_quantised": (lambda: q.qlora_fp8_linear_fwd(kept, W8, y), [y]),
        "fp8_fwd_token": (lambda: q.qlora_fp8_linear_fwd(x[:1], W8, y[:1], Xq=q.FP8Matrix(
            1, K, 1, xq.codes[:1], xq.scale.view(-1)[:K // 128])), [y[:1]]),
        "fp8_bwd": (lambda: q.qlora_fp8_linear_bwd(dy, W8, dx, dYq=gq), [dx]),
        "nf4_fwd": (lambda: q.qlora_linear_fwd(x, W4, A, B, 32.0, Y=y, T_save=T, workspace=ws), [y, T]),
        "nf4_bwd": (lambda: q.qlora_linear_bwd(dy, x, W4, A, B, 32.0, T_saved=T, dX=dx, dA=dA, dB=dB, workspace=ws),
                    [dx, dA, dB]),
        "norm": (lambda: q.qlora_layernorm_fwd(x, g, b, Y=ny, mean=mean, rstd=rstd), [ny, mean, rstd]),
    }


@pytest.mark.parametrize("name", ["fp8_fwd", "fp8_fwd_quantised", "fp8_fwd_token", "fp8_bwd", "nf4_fwd", "nf4_bwd", "norm"])
def test_first_call_of_a_thread(name):
    calls = _calls()
    if name == "nf4_bwd":
        calls["nf4_fwd"][0]()
    call, out = calls[name]
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            call()
        except Exception as e:                       # noqa: BLE001
            errors.append(e)
    for _ in range(3):
        t = threading.Thread(target=work)
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert all(torch.equal(a, b) for a, b in zip(out, want))
