"""FP8 products into rows that start on 16 bytes and end inside them: what lies
behind a row's last column stays as it was."""
from __future__ import annotations

import pytest
import torch

import bit_nf4_quantized_21_b200 as q

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _normal(shape, scale, seed):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(DEV).bfloat16()


# 33 and 300 tokens: tiles of 128 columns; 2600 with 2600 columns and more: of 256.  Widths that
# end 1, 3, 4, 5 and 7 elements past 16 bytes, inside the first box of a tile and in later ones,
# and one that ends on them.  Both products write the width: M x width from a contraction of 200.
@pytest.mark.parametrize("M,cols", [(33, 1), (33, 7), (33, 9), (300, 67), (300, 131), (300, 811), (300, 816), (300, 2604),
                                    (2600, 2603), (2600, 2693), (2600, 2820)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("backward", [False, True])
def test_what_lies_behind_a_row_stays(M, cols, dtype, backward):
    inner = 200
    W = q.qlora_fp8_quantize(_normal((inner, cols) if backward else (cols, inner), 0.05, cols))
    x = _normal((M, inner), 1.0, cols + 1)
    product = q.qlora_fp8_linear_bwd if backward else q.qlora_fp8_linear_fwd
    want = product(x, W, out_dtype=dtype)
    for ld in (-(-cols // 8) * 8, -(-cols // 8) * 8 + 24):
        base = torch.full((M + 1, ld), 55.0, dtype=dtype, device=DEV)      # (and a row behind the last)
        y = base[:M, :cols]
        assert torch.equal(product(x, W, y), want)
        assert torch.equal(y, want)
        y.fill_(55.0)
        assert torch.all(base == 55.0)
