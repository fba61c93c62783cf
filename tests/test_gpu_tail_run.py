"""The end of a fine-tuning step as it is used: norm, NF4 projection with its
adapter, norm, FP8 output head, distillation loss, and back through all of
them to the adapter's Adam step; against the same chain in binary64.

Tolerances: each stage's kernel is held to its own bound elsewhere; here the
chain's outputs are compared with the binary64 chain run on the kernels' own
intermediate inputs, stage by stage, by relative Frobenius error: 2e-3 for a
bf16 output (its rounding alone is 1.7e-3), 1e-4 for fp32 ones.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import bit_nf4_quantized_21_b200 as q
import oracle as O
import oracle.tail as OT
from gpu_util import bits

pytestmark = pytest.mark.gpu
DEV = "cuda"


def f64(t):
    return t.detach().double().cpu().numpy()


def _problem(M, H, V, r, top, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, sigma=1.0: torch.randn(*s, generator=g) * sigma
    p = dict(h=n(M, H).bfloat16(), g1=(1 + n(H, sigma=0.1)).bfloat16(), b1=n(H, sigma=0.1).bfloat16(),
             g2=(1 + n(H, sigma=0.1)).bfloat16(), b2=n(H, sigma=0.1).bfloat16(), W=n(H, H, sigma=0.05).bfloat16(),
             A=n(r, H, sigma=0.02).bfloat16(), B=n(H, r, sigma=0.02).bfloat16(), head=n(V, H, sigma=0.05).bfloat16(),
             ids=torch.randint(0, V, (M, top), generator=g, dtype=torch.int32), t=n(M, top, sigma=2.0),
             weight=torch.full((M,), 1.0 / M))
    p["weight"][0] = 0.0
    p["ids"][1] = -1
    return {k: v.to(DEV) for k, v in p.items()}


def _step(p, Wq, head, tau, alpha):
    s = {}
    M, r = p["h"].shape[0], p["A"].shape[0]
    s["x1"], s["m1"], s["r1"] = q.qlora_layernorm_fwd(p["h"], p["g1"], p["b1"])
    s["T"] = torch.empty((M, r), device=DEV)
    s["y"] = q.qlora_linear_fwd(s["x1"], Wq, p["A"], p["B"], alpha, T_save=s["T"])
    s["x2"], s["m2"], s["r2"] = q.qlora_layernorm_fwd(s["y"], p["g2"], p["b2"])
    s["xq"] = q.empty_fp8(M, head.cols, DEV, 1)
    s["z"] = q.qlora_fp8_linear_fwd(s["x2"], head, Xq=s["xq"])
    s["dz"] = s["z"].clone()
    s["loss"], s["lse"] = q.qlora_distill_topk_fwd(s["dz"], p["ids"], p["t"], tau, row_weight=p["weight"], dZ=s["dz"])
    s["dzq"] = q.empty_fp8(M, head.rows, DEV, 1)
    s["dx2"] = q.qlora_fp8_linear_bwd(s["dz"], head, dYq=s["dzq"])
    s["dy"], s["dg2"], s["db2"] = q.qlora_layernorm_bwd(s["dx2"], s["y"], p["g2"], s["m2"], s["r2"])
    s["dx1"], s["dA"], s["dB"] = q.qlora_linear_bwd(s["dy"], s["x1"], Wq, p["A"], p["B"], alpha, T_saved=s["T"])
    s["dh"], s["dg1"], s["db1"] = q.qlora_layernorm_bwd(s["dx1"], p["h"], p["g1"], s["m1"], s["r1"])
    return s


def _rel(got, want):
    return O.rel_fro(f64(got), want)


def _values(m):
    return OT.fp8_values(m.codes.view(torch.uint8)[:, :m.cols].cpu().numpy(), m.scale.cpu().numpy(), m.block_rows)


@pytest.mark.parametrize("M,H,V", [(5, 256, 600), (150, 512, 1111)])
def test_chain_matches_binary64_stage_by_stage(M, H, V):
    tau, alpha, r, top = 2.0, 16.0, 8, 12
    p = _problem(M, H, V, r, top, M + V)
    Wq, head = q.qlora_quantize_nf4(p["W"]), q.qlora_fp8_quantize(p["head"])
    s = _step(p, Wq, head, tau, alpha)
    torch.cuda.synchronize()
    got = lambda k: f64(s[k])
    par = lambda k: f64(p[k])
    y1, m1, r1 = OT.layernorm_fwd(par("h"), par("g1"), par("b1"))
    assert _rel(s["x1"], y1) <= 2e-3
    Wh = O.nf4_dequantize(O.nf4_quantize(p["W"].float().cpu().numpy()))
    Y, T = O.linear_fwd(bits(s["x1"]), Wh, bits(p["A"]), bits(p["B"]), alpha, r)
    assert _rel(s["y"], Y) <= 2e-3 and _rel(s["T"], T) <= 1e-4
    y2, _, _ = OT.layernorm_fwd(got("y"), par("g2"), par("b2"))
    assert _rel(s["x2"], y2) <= 2e-3
    HV = _values(head)
    assert _rel(s["z"], _values(s["xq"]) @ HV.T) <= 2e-3
    loss, lse, dz = OT.distill(got("z"), p["ids"].cpu().numpy(), par("t"), tau, par("weight"))
    assert np.allclose(got("loss"), loss, rtol=0, atol=1e-4 * np.abs(loss).max()) and _rel(s["lse"], lse) <= 1e-4
    assert _rel(s["dz"], dz) <= 2e-3
    assert _rel(s["dx2"], _values(s["dzq"]) @ HV) <= 2e-3
    dy, dg2, db2 = OT.layernorm_bwd(got("dx2"), got("y"), par("g2"), got("m2"), got("r2"))
    assert _rel(s["dy"], dy) <= 2e-3 and _rel(s["dg2"], dg2) <= 1e-4 and _rel(s["db2"], db2) <= 1e-4
    g = O.linear_bwd(bits(s["dy"]), bits(s["x1"]), Wh, bits(p["A"]), bits(p["B"]), alpha, r)
    assert _rel(s["dx1"], g["dX"]) <= 2e-3 and _rel(s["dA"], g["dA"]) <= 1e-4
    dh, dg1, db1 = OT.layernorm_bwd(got("dx1"), par("h"), par("g1"), got("m1"), got("r1"))
    assert _rel(s["dh"], dh) <= 2e-3 and _rel(s["dg1"], dg1) <= 1e-4
    # rows without a loss send nothing back
    assert torch.count_nonzero(s["dh"][:2]) == 0


def test_chain_replays_from_a_graph_and_steps_the_adapter():
    M, H, V, r = 40, 256, 700, 8
    p = _problem(M, H, V, r, 9, 3)
    Wq, head = q.qlora_quantize_nf4(p["W"]), q.qlora_fp8_quantize(p["head"])
    want = _step(p, Wq, head, 1.5, 16.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = _step(p, Wq, head, 1.5, 16.0)
    graph.replay()
    torch.cuda.synchronize()
    for k in ("z", "loss", "dz", "dx2", "dy", "dA", "dB", "dh", "dg1", "dg2"):
        assert torch.equal(s[k], want[k]), k
    master = p["A"].float().flatten()
    m, v, param = torch.zeros_like(master), torch.zeros_like(master), torch.empty_like(p["A"].flatten())
    q.qlora_adam_step(master, m, v, s["dA"].flatten(), 1, 1e-3, param=param)
    assert torch.isfinite(master).all() and not torch.equal(param, p["A"].flatten())
