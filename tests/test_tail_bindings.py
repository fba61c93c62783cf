"""Host-side checks, without a GPU, of the compiled binding and of what the
library settles before it enqueues anything."""
from __future__ import annotations

import ctypes
import os
import sysconfig

import pytest
import torch

import bit_nf4_quantized_21_b200 as q
from bit_nf4_quantized_21_b200 import build, qlora as binding


def _matrix(dtype, rows=128, cols=64, block_rows=128):
    m = q.empty_fp8(rows, cols, "cpu", block_rows)
    m.codes = m.codes.view(dtype)
    return m


# Only the type is looked at before the device: codes of the right type are
# then refused as host tensors.
@pytest.mark.parametrize("dtype,wrong", [
    (torch.float8_e5m2, True), (torch.float8_e4m3fnuz, True), (torch.float8_e5m2fnuz, True), (torch.int8, True),
    (torch.bool, True), (torch.uint8, False), (torch.float8_e4m3fn, False)])
def test_fp8_codes_are_e4m3_or_bytes(dtype, wrong):
    message = "codes must be uint8 or float8_e4m3fn" if wrong else "CUDA tensors only"
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match=message):
        q.qlora_fp8_quantize(x, out=_matrix(dtype, 4, 64, 1))
    with pytest.raises(ValueError, match=message):
        q.qlora_fp8_linear_fwd(x, _matrix(dtype))
    with pytest.raises(ValueError, match=message):
        q.qlora_fp8_linear_bwd(torch.zeros(4, 128), _matrix(dtype))
    with pytest.raises(ValueError, match=message):           # the activations' codes, as scratch and as input
        q.qlora_fp8_linear_fwd(x, _matrix(torch.uint8), Xq=_matrix(dtype, 4, 64, 1))
    with pytest.raises(ValueError, match=message):
        q.qlora_fp8_linear_fwd(_matrix(dtype, 4, 64, 1), _matrix(torch.uint8))


# ------------------------------------------- nothing is enqueued by a call that is refused

FAKE = 1 << 40                      # an aligned device address that nothing reads
UNSUPPORTED = 2


def _c(rows, cols, block_rows):
    return binding.FP8MatrixC(rows, cols, -(-cols // 128) * 128, block_rows, 0, FAKE, FAKE)


@pytest.mark.skipif(torch.cuda.is_available(), reason="shown by a status that only a machine without a device gives")
@pytest.mark.parametrize("quantise", [True, False])
def test_fp8_products_with_too_many_tiles_are_refused_first(quantise):
    """2^22 rows of tiles by 2^8 columns of them: more than the product counts.  The
    quantiser alone would take these activations, so the refusal has to come before it;
    here its launch would fail, for want of a device, with another status."""
    L = q.lib()
    M, N, K = 1 << 30, 1 << 16, 128
    X = FAKE if quantise else None
    W, A = _c(N, K, 128), _c(M, K, 1)
    assert L.qlora_fp8_linear_fwd(X, 1, K, ctypes.byref(W), ctypes.byref(A), FAKE, 1, N, None, None) == UNSUPPORTED
    W, A = _c(K, N, 128), _c(M, K, 1)
    assert L.qlora_fp8_linear_bwd(X, 1, K, ctypes.byref(W), ctypes.byref(A), FAKE, 1, N, None, None) == UNSUPPORTED


def _body(source, head):
    """The text of a function, from its head to the brace that closes it."""
    at = source.index(head)
    return source[at:source.index("\n}\n", at)]


def test_the_nf4_layer_does_not_hang_on_the_fp8_kernels():
    """What readies the NF4 kernels looks at none of the FP8 ones: a build of those that the
    library will not launch (too few registers to share out) refuses FP8 calls, nothing else."""
    with open(os.path.join(os.path.dirname(binding.__file__), "csrc", "qlora.cu")) as f:
        source = f.read()
    old, new = _body(source, "bool ensure_smem_attrs() {"), _body(source, "bool ensure_fp8_attrs() {")
    assert "k_gemm_nf4" in old and "k_skinny" in old and "fp8" not in old.lower() and "f8" not in old.lower()
    assert "k_fp8_gemm" in new and "k_fp8_gemv" in new and "numRegs" in new
    for head in ("qlora_status plan_fp8_gemm(", "qlora_status fp8_linear("):
        body = _body(source, head)
        assert "ensure_fp8_attrs()" in body and "ensure_smem_attrs()" not in body


# ---------------------------------------------- the binary of the interpreter and torch at hand

def test_another_torch_or_python_does_not_take_a_binding_built_for_this_one(monkeypatch):
    path = build.build_calls()
    assert os.path.exists(path) and not build.calls_need_build()
    monkeypatch.setattr(binding, "_calls_mod", None)
    assert binding._calls().layernorm_fwd is not None
    for module, name, value in ((torch, "__version__", "2.99.0+cu999"),
                                (sysconfig, "get_config_var", lambda _: ".cpython-399-x86_64-linux-gnu.so")):
        with monkeypatch.context() as m:
            m.setattr(module, name, value)
            m.setattr(binding, "_calls_mod", None)
            assert build.calls_path() != path and build.calls_need_build()
            with pytest.raises(RuntimeError, match="build it with"):
                binding._calls()


# ------------------------------------------------------------------ temperatures

@pytest.mark.parametrize("tau,refused", [
    (1e-17, False), (1.1e-19, False), (1.0, False), (1.8e19, False),
    (1e-19, True), (1e-20, True), (1e-23, True), (4e-39, True), (1.9e19, True)])
def test_temperatures_whose_square_is_no_normal_number_are_refused(tau, refused):
    """The loss carries tau^2: where that is subnormal or 0 in fp32, the loss of a row
    (of the size of tau |z|) would come out short of bits, or as 0.  No rows: only looked at."""
    fwd = [FAKE, 100, 0, 100, 1, FAKE, 32, FAKE, 0, 8, tau, FAKE, FAKE, FAKE, FAKE, 100, None, None]
    expect = 1 if refused else 0
    assert q.lib().qlora_distill_topk_fwd(*fwd) == expect
    assert q.lib().qlora_distill_topk_bwd(*fwd) == expect


# ------------------------------------------------------------------ truth values

def test_a_flag_without_a_truth_value_raises_its_own_error():
    class Neither:
        def __bool__(self):
            raise OverflowError("neither")
    x, s = torch.zeros(4, 64), torch.zeros(4)
    with pytest.raises(OverflowError, match="neither"):
        q.qlora_layernorm_bwd(x, x, None, s, s, want_params=Neither())
