"""How a program uses the FP8 layer, the layer norm and the distillation loss
beside other work: calls on several streams and host threads at once, graphs
that share a workspace, a wait that runs out, an allocator that hands a
call's scratch on."""
from __future__ import annotations

import threading

import pytest
import torch

import bit_nf4_quantized_21_b200 as q

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _normal(shape, sigma, seed, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * sigma).to(DEV).to(dtype)


def _problem(seed, M=300, H=512, V=1500, top=9):
    return dict(x=_normal((M, H), 1.0, seed), w=_normal((H,), 0.1, seed + 1) + 1, b=_normal((H,), 0.1, seed + 2),
                head=q.qlora_fp8_quantize(_normal((V, H), 0.05, seed + 3)), ids=torch.randint(0, V, (M, top), device=DEV),
                t=_normal((M, top), 2.0, seed + 4, torch.float32))


def _chain(p, stream=None):
    y, mean, rstd = q.qlora_layernorm_fwd(p["x"], p["w"], p["b"], stream=stream)
    z = q.qlora_fp8_linear_fwd(y, p["head"], stream=stream)
    loss, lse = q.qlora_distill_topk_fwd(z, p["ids"], p["t"], 1.5, dZ=z, stream=stream)
    dy = q.qlora_fp8_linear_bwd(z, p["head"], stream=stream)
    return (loss, lse, z, *q.qlora_layernorm_bwd(dy, p["x"], p["w"], mean, rstd, stream=stream))


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_streams_side_by_side():
    ps = [_problem(10 * i, M=200 + 150 * i) for i in range(4)]
    want = [_chain(p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = []
    for _ in range(3):
        got = [_chain(p, s) for p, s in zip(ps, streams)]
    torch.cuda.synchronize()
    assert all(_same(g, w) for g, w in zip(got, want))


def test_a_current_stream_context_is_followed():
    p = _problem(50)
    want = _chain(p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = _chain(p)
        # what the calls allocated for themselves is handed on here and overwritten
        junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
    s.synchronize()
    assert _same(got, want) and len(junk) == 8


def test_host_threads_at_once():
    ps = [_problem(100 + i, M=64 + i) for i in range(4)]
    want = [_chain(p) for p in ps]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i] = _chain(ps[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:                      # noqa: BLE001
            errors.append(e)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors and all(_same(g, w) for g, w in zip(got, want))


def test_two_graphs_that_share_a_workspace_and_a_scratch():
    p = _problem(200, M=400)
    q2 = _problem(210, M=400)
    rows, cols = 400, 512
    ws = torch.empty(q.qlora_layernorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    scratch = q.empty_fp8(rows, cols, DEV, 1)

    def call(p, out):
        q.qlora_layernorm_fwd(p["x"], p["w"], p["b"], Y=out[0], mean=out[1], rstd=out[2])
        q.qlora_fp8_linear_fwd(out[0], p["head"], Y=out[3], Xq=scratch)
        q.qlora_layernorm_bwd(out[0], p["x"], p["w"], out[1], out[2], dX=out[4], dweight=out[5], dbias=out[6], workspace=ws)

    def outputs():
        f = lambda *s, dt=torch.float32: torch.full(s, float("nan"), dtype=dt, device=DEV)
        return [f(rows, cols, dt=torch.bfloat16), f(rows), f(rows), f(rows, 1500, dt=torch.bfloat16),
                f(rows, cols, dt=torch.bfloat16), f(cols), f(cols)]
    want = []
    for prob in (p, q2):
        o = outputs()
        call(prob, o)
        torch.cuda.synchronize()
        want.append(o)
    graphs, outs = [], []
    for prob in (p, q2):
        o = outputs()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(prob, o)
        graphs.append(g)
        outs.append(o)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert _same(outs[0], want[0]) and _same(outs[1], want[1])


@pytest.mark.parametrize("which", ["fp8_fwd", "fp8_bwd", "norm_fwd", "norm_bwd"])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(which):
    L = q.lib()
    W = q.qlora_fp8_quantize(_normal((600, 768), 0.05, 400))
    x, dy = _normal((520, 768), 1.0, 401), _normal((520, 600), 1.0, 402)
    n, g = _normal((1300, 8192), 1.0, 403), _normal((1300, 8192), 1.0, 404)     # rows enough for the ring
    _, mean, rstd = q.qlora_layernorm_fwd(n)
    calls = {"fp8_fwd": lambda st: q.qlora_fp8_linear_fwd(x, W, d_status=st),
             "fp8_bwd": lambda st: q.qlora_fp8_linear_bwd(dy, W, d_status=st),
             "norm_fwd": lambda st: q.qlora_layernorm_fwd(n, d_status=st)[0],
             "norm_bwd": lambda st: q.qlora_layernorm_bwd(g, n, None, mean, rstd, d_status=st)[1]}
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = calls[which](st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert L.qlora_debug_set_wait_limit(1_000_000) == 0      # 1 ms
    assert L.qlora_debug_inject_stall(1) == 0
    try:
        calls[which](st)
        torch.cuda.synchronize()
    finally:
        assert L.qlora_debug_inject_stall(0) == 0
        assert L.qlora_debug_set_wait_limit(0) == 0
    assert st.item() & q.qlora.DEV_TIMEOUT
    st.zero_()
    for _ in range(2):
        assert torch.equal(calls[which](st), want)
    assert st.item() == 0


def test_refusals_of_the_binding_on_device_tensors():
    x = _normal((4, 256), 1.0, 500)
    W = q.qlora_fp8_quantize(_normal((128, 256), 0.05, 501))
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_fwd(x[:, :128], W)                       # another width
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_fwd(x, W, Y=torch.empty(4, 127, device=DEV))
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_fwd(x.half(), W)
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_fwd(x, W, Xq=q.empty_fp8(3, 256, DEV, 1))
    with pytest.raises(ValueError):
        q.qlora_fp8_linear_fwd(x.expand(4, 256)[:1].expand(4, 256), W)   # one row four times: stride 0
    with pytest.raises(q.QloraError):
        q.qlora_fp8_linear_fwd(x, q.qlora_fp8_quantize(x, block_rows=1))
    with pytest.raises(ValueError):
        q.qlora_layernorm_fwd(x.t())
    with pytest.raises(ValueError):
        q.qlora_layernorm_fwd(x, torch.ones(255, device=DEV))
    with pytest.raises(ValueError):
        q.qlora_layernorm_fwd(x, torch.ones(256, device=DEV), torch.ones(256, device=DEV).bfloat16())
    with pytest.raises(ValueError):
        q.qlora_layernorm_fwd(x, torch.ones(256))                   # a host tensor among them
    ids, t = torch.zeros((4, 3), dtype=torch.int32, device=DEV), torch.zeros((4, 3), device=DEV)
    with pytest.raises(ValueError):
        q.qlora_distill_topk_fwd(x, ids[:3], t)
    with pytest.raises(ValueError):
        q.qlora_distill_topk_fwd(x, ids.float(), t)
    with pytest.raises(ValueError):
        q.qlora_distill_topk_fwd(x, ids, t, dZ=torch.empty(4, 256, device=DEV))     # another type
    with pytest.raises(q.QloraError):
        q.qlora_distill_topk_fwd(x, ids, t, tau=0.0)
