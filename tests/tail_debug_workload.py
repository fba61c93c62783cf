"""One pass over the kernels of the FP8 layer, the layer norm and the
distillation loss, for the debug-build test (as debug_build_workload.py): one
JSON line with the SHA-256 of every output and the range-failure word."""
from __future__ import annotations

import ctypes
import hashlib
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import bit_nf4_quantized_21_b200 as q  # noqa: E402

DEV = "cuda"


def normal(shape, sigma, seed, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * sigma).to(DEV).to(dtype)


def digest(t):
    return hashlib.sha256(t.detach().contiguous().cpu().view(torch.uint8).numpy().tobytes()).hexdigest()[:16]


def main():
    L = q.lib()
    site = ctypes.c_uint(0)
    assert L.qlora_debug_range_check(ctypes.byref(site)) == 0
    out = {"checks": int(L.qlora_debug_checks_enabled())}
    W = q.qlora_fp8_quantize(normal((1100, 900), 0.05, 1))
    out["codes"] = [digest(W.codes[:, :900]), digest(W.scale)]
    for M in (1, 9, 20, 33, 700):
        x, dy = normal((M, 900), 1.0, 2 + M), normal((M, 1100), 1.0, 3 + M)
        out[f"fp8_{M}"] = [digest(q.qlora_fp8_linear_fwd(x, W)), digest(q.qlora_fp8_linear_bwd(dy, W)),
                           digest(q.qlora_fp8_linear_fwd(x, W, out_dtype=torch.float32))]
    for rows, cols in ((5, 64), (40, 1000), (7, 2051), (1300, 1024), (1300, 4096), (3, 20001)):
        x, dy, w = normal((rows, cols), 1.0, 4 + cols), normal((rows, cols), 1.0, 5 + cols), normal((cols,), 0.1, 6) + 1
        y, mean, rstd = q.qlora_layernorm_fwd(x, w, w)
        out[f"norm_{rows}_{cols}"] = [digest(t) for t in (y, mean, rstd, *q.qlora_layernorm_bwd(dy, x, w, mean, rstd))]
    for rows, V in ((3, 70001), (800, 1000)):
        z, t = normal((rows, V), 2.0, 7 + V), normal((rows, 20), 1.0, 8, torch.float32)
        ids = torch.randint(0, V, (rows, 20), generator=torch.Generator().manual_seed(9)).to(DEV)
        dz = torch.empty_like(z)
        loss, lse = q.qlora_distill_topk_fwd(z, ids, t, 2.0, dZ=dz)
        out[f"distill_{rows}_{V}"] = [digest(x) for x in (loss, lse, dz, q.qlora_distill_topk_bwd(z, ids, t, 2.0, lse))]
    torch.cuda.synchronize()
    assert L.qlora_debug_range_check(ctypes.byref(site)) == 0
    out["range_site"] = int(site.value)
    print(json.dumps(out))


if __name__ == "__main__":
    main()
