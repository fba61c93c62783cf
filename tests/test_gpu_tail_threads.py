"""Layer norms of many rows from several host threads at once: widths whose
rows need different amounts of shared memory in the same kernel."""
from __future__ import annotations

import threading

import pytest
import torch

import bit_nf4_quantized_21_b200 as q

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DEV).bfloat16()


class _Norm:
    """One width's calls, on outputs that it keeps."""

    def __init__(self, rows, cols, seed):
        self.x, self.dy = _normal((rows, cols), seed), _normal((rows, cols), seed + 1)
        self.w, self.b = _normal((cols,), seed + 2), _normal((cols,), seed + 3)
        self.stream = torch.cuda.Stream()
        f32 = dict(dtype=torch.float32, device=DEV)
        self.mean, self.rstd = torch.empty(rows, **f32), torch.empty(rows, **f32)
        self.y, self.dx = torch.empty_like(self.x), torch.empty_like(self.x)
        self.dw, self.db = torch.empty(cols, **f32), torch.empty(cols, **f32)
        self.ws = torch.empty(q.qlora_layernorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)

    def forward(self):
        q.qlora_layernorm_fwd(self.x, self.w, self.b, Y=self.y, mean=self.mean, rstd=self.rstd)

    def backward(self):
        q.qlora_layernorm_bwd(self.dy, self.x, self.w, self.mean, self.rstd, dX=self.dx, dweight=self.dw, dbias=self.db,
                              workspace=self.ws)

    def outputs(self):
        return [t.clone() for t in (self.y, self.mean, self.rstd, self.dx, self.dw, self.db)]


# (the first two widths of a set share their kernels and differ in shared memory: 8 x 5120
# and 7 x 7168 bytes of rows forward, 8 x 10240 and 7 x 14336 backward; likewise 5120 and 6400)
@pytest.mark.parametrize("rows,widths", [(4096, (2560, 3584, 2560, 3584)), (1200, (5120, 6400, 5120, 6400))])
def test_widths_that_share_a_kernel(rows, widths):
    norms = [_Norm(rows, c, 10 * i) for i, c in enumerate(widths)]
    want = []
    for n in norms:
        n.forward()
        n.backward()
        want.append(n.outputs())
    torch.cuda.synchronize()
    start, errors = threading.Barrier(len(norms)), []

    def work(n, call):
        try:
            with torch.cuda.stream(n.stream):
                start.wait()
                for i in range(400):
                    call(n)
                    if i % 50 == 49:                 # (a full launch queue would hand the threads their turns)
                        n.stream.synchronize()
        except Exception as e:                       # noqa: BLE001
            errors.append(e)
    for call in (_Norm.forward, _Norm.backward):
        threads = [threading.Thread(target=work, args=(n, call)) for n in norms]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    torch.cuda.synchronize()
    assert not errors, errors[:2]
    for n, w in zip(norms, want):
        assert all(torch.equal(a, b) for a, b in zip(n.outputs(), w))
