"""The operators of a training step's tail, as cases to be measured.

Three operators and their gradients, as a fine-tuning program over a frozen
base calls them: the layer norm in front of a frozen projection, the frozen
projection itself held in 8-bit floating point with one scale per 128, and
the distillation loss against a teacher's top logits.

``own`` False: plain torch in fp32.  ``own`` True: the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
E4M3_MAX = 448.0
FLT_MIN = torch.finfo(torch.float32).tiny
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token through the widest projection of the decode workload: a stream of the weight
        {"name": "fp8_fwd_token", "op": "fp8_fwd", "m": 1, "n": 28672, "k": 8192},
        # a handful of sequences decoding together, an odd number of them: latency counts
        {"name": "fp8_fwd_tokens", "op": "fp8_fwd", "m": 7, "n": 4096, "k": 4096},
        # a training micro-batch through the gate projection
        {"name": "fp8_fwd_train", "op": "fp8_fwd", "m": 2048, "n": 11008, "k": 4096},
        # a packed batch of odd length and a projection whose sides end inside a scale block
        {"name": "fp8_fwd_ragged", "op": "fp8_fwd", "m": 1000, "n": 4100, "k": 4040},
        # the gradient of the same micro-batch back through the gate projection
        {"name": "fp8_bwd_train", "op": "fp8_bwd", "m": 2048, "n": 11008, "k": 4096},
        # the norm in front of a decode step: one small launch
        {"name": "norm_fwd_decode", "op": "norm_fwd", "rows": 16, "cols": 4096, "dtype": "bf16"},
        # the norm over the largest token count and width that the model workloads use
        {"name": "norm_fwd_wide", "op": "norm_fwd", "rows": 8192, "cols": 8192, "dtype": "bf16"},
        # a micro-batch's backward pass with the gradients of weight and bias
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 4096, "cols": 4096, "dtype": "bf16"},
        # fp32 activations, a width that no vector divides and a ragged number of rows
        {"name": "norm_bwd_odd", "op": "norm_bwd", "rows": 1237, "cols": 2051, "dtype": "f32"},
        # the loss alone for a few evaluated positions over a wide vocabulary
        {"name": "distill_loss_few", "op": "distill_fwd", "rows": 6, "vocab": 131072, "top": 32, "dtype": "bf16",
         "tau": 1.0},
        # a training micro-batch: loss and gradient of the logits in one call
        {"name": "distill_step", "op": "distill_step", "rows": 4096, "vocab": 32768, "top": 64, "dtype": "bf16",
         "tau": 2.0},
        # the gradient from the saved normaliser, fp32 logits, an odd vocabulary
        {"name": "distill_bwd_odd", "op": "distill_bwd", "rows": 777, "vocab": 50021, "top": 20, "dtype": "f32",
         "tau": 1.5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: token counts from one to a training batch, widths and vocabularies over the models' range."""
    op = rng.choice(["fp8_fwd", "fp8_fwd", "fp8_bwd", "norm_fwd", "norm_bwd", "distill_fwd", "distill_step",
                     "distill_bwd"])
    if op.startswith("fp8"):
        m = _log_int(rng, 1, 4096)
        k = _log_int(rng, 512, 8192)
        n = _log_int(rng, 512, 28672)
        if rng.random() < 0.7:   # most projections are whole scale blocks wide
            k, n = -(-k // BLOCK) * BLOCK, -(-n // BLOCK) * BLOCK
        while m * n * k > 2048 * 11008 * 4096:
            m = max(1, m // 2)
        return {"op": op, "m": m, "n": n, "k": k}
    if op.startswith("norm"):
        rows, cols = _log_int(rng, 1, 16384), _log_int(rng, 64, 12288)
        if rng.random() < 0.7:
            cols = -(-cols // 64) * 64
        while rows * cols > 8192 * 8192:
            rows //= 2
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    rows, vocab = _log_int(rng, 1, 8192), _log_int(rng, 1000, 160000)
    if rng.random() < 0.5:
        vocab = -(-vocab // 64) * 64
    while rows * vocab > 4096 * 32768:
        rows //= 2
    return {"op": op, "rows": rows, "vocab": vocab, "top": _log_int(rng, 1, 256),
            "dtype": rng.choice(["bf16", "bf16", "f32"]), "tau": rng.choice([1.0, 1.5, 2.0, 4.0])}


# ------------------------------------------------------------------ inputs

def _normal(shape, sigma, gen, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(sigma).to(dtype)


def _fp8_weight(w):
    """E4M3 codes [n, ld] (ld: k rounded up to 128) and the 128 x 128 scales of a weight, as a loader keeps them."""
    n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    pad = torch.zeros((nb * BLOCK, kb * BLOCK), device=DEV, dtype=torch.float32)
    pad[:n, :k] = w
    tiles = pad.view(nb, BLOCK, kb, BLOCK)
    scale = tiles.abs().amax((1, 3)) / E4M3_MAX
    codes = (tiles * (1.0 / scale)[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.reshape(nb * BLOCK, kb * BLOCK)[:n].contiguous(), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 13)
    op = case["op"]
    if op.startswith("fp8"):
        m, n, k = case["m"], case["n"], case["k"]
        codes, scale = _fp8_weight(_normal((n, k), 0.02, gen, torch.float32))
        s = {"op": op, "n": n, "k": k, "codes": codes, "scale": scale}
        # activations have a few channels far above the rest; gradients are small
        width = k if op == "fp8_fwd" else n
        gain = torch.ones(width, device=DEV)
        gain[torch.rand(width, generator=gen, device=DEV) < 0.002] = 20.0 if op == "fp8_fwd" else 1.0
        x = _normal((m, width), 1.0 if op == "fp8_fwd" else 1e-3, gen, torch.float32) * gain
        s["x"] = x.to(torch.bfloat16)
        return s
    dtype = DTYPES[case["dtype"]]
    if op.startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        x = (_normal((rows, cols), 1.0, gen, torch.float32) + 0.3).to(dtype)
        s = {"op": op, "x": x, "w": (_normal((cols,), 0.1, gen, torch.float32) + 1.0).to(dtype),
             "b": _normal((cols,), 0.1, gen, dtype)}
        if op == "norm_bwd":
            x64 = x.double()
            mean = x64.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = torch.rsqrt((x64 - mean[:, None]).square().mean(1) + EPS).float()
            s["dy"] = _normal((rows, cols), 1.0, gen, dtype)
        return s
    rows, vocab, top = case["rows"], case["vocab"], min(case["top"], case["vocab"])
    z = _normal((rows, vocab), 2.5, gen, torch.float32)
    teacher, ids = torch.topk(z + _normal((rows, vocab), 1.0, gen, torch.float32), top, dim=1)
    ids = ids.to(torch.int32)
    # a stored list is sometimes shorter than the others: the rest is marked by -1
    short = torch.rand((rows, top), generator=gen, device=DEV) < 0.02
    ids[short] = -1
    weight = torch.full((rows,), 1.0 / rows, device=DEV)
    if rows > 1:                       # padded positions carry no loss
        weight[torch.rand(rows, generator=gen, device=DEV) < 0.05] = 0.0
    s = {"op": op, "z": z.to(dtype), "ids": ids, "t": teacher, "weight": weight, "tau": case["tau"]}
    if op == "distill_bwd":
        s["lse"] = torch.logsumexp(s["z"].double() / case["tau"], 1).float()
        s["grad"] = torch.rand(rows, generator=gen, device=DEV) + 0.5
    return s


# ------------------------------------------------------------------ plain forms

def _plain_rows_fp8(x):
    """The values that 1 x 128 blocks of E4M3 codes stand for."""
    m, k = x.shape
    kb = -(-k // BLOCK)
    pad = torch.zeros((m, kb * BLOCK), device=x.device, dtype=torch.float32)
    pad[:, :k] = x
    blocks = pad.view(m, kb, BLOCK)
    top = blocks.abs().amax(2, keepdim=True)
    scale = top / torch.full_like(top, E4M3_MAX)   # a division: by a number it would be a product with 1/448
    scale = torch.where(scale < FLT_MIN, torch.zeros_like(scale), scale)
    recip = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
    values = (blocks * recip).to(torch.float8_e4m3fn).float() * scale
    return values.view(m, kb * BLOCK)[:, :k]


def _plain_weight(s):
    n, k = s["n"], s["k"]
    scale = s["scale"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return s["codes"][:, :k].float() * scale


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt(c.square().mean(1, keepdim=True) + EPS)
    y = c * rstd * s["w"].float() + s["b"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def _plain_teacher(s):
    """(listed ids with 0 for what is left out, log p, p) of each row's list."""
    listed_ = s["ids"] >= 0
    t = torch.where(listed_, s["t"] / s["tau"], torch.full_like(s["t"], -math.inf))
    top = t.amax(1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(t - top)
    total = e.sum(1, keepdim=True)
    p = torch.where(listed_ & (total > 0), e / total, torch.zeros_like(e))
    logp = torch.where(p > 0, t - top - torch.log(total), torch.zeros_like(t))
    return s["ids"].clamp(min=0).long(), logp, p


def _plain_loss(s):
    ids, logp, p = _plain_teacher(s)
    z = s["z"].float() / s["tau"]
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
    logq = torch.gather(z, 1, ids) - lse[:, None]
    kl = torch.where(p > 0, p * (logp - logq), torch.zeros_like(p)).sum(1)
    loss = s["weight"] * (s["tau"] * s["tau"]) * kl
    return loss, lse


def _plain_dlogits(s, lse, grad):
    ids, _, p = _plain_teacher(s)
    q = torch.exp(s["z"].float() / s["tau"] - lse[:, None])
    q = torch.where(p.sum(1, keepdim=True) > 0, q, torch.zeros_like(q)).scatter_add_(1, ids, -p)
    factor = s["weight"] * s["tau"] if grad is None else s["weight"] * s["tau"] * grad
    return (q * factor[:, None]).to(s["z"].dtype)


def _plain(s):
    op = s["op"]
    if op == "fp8_fwd":
        return {"y": (_plain_rows_fp8(s["x"].float()) @ _plain_weight(s).t()).to(torch.bfloat16)}
    if op == "fp8_bwd":
        return {"dx": (_plain_rows_fp8(s["x"].float()) @ _plain_weight(s)).to(torch.bfloat16)}
    if op == "norm_fwd":
        return _plain_norm_fwd(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "distill_fwd":
        loss, lse = _plain_loss(s)
        return {"loss": loss, "lse": lse}
    if op == "distill_step":
        loss, lse = _plain_loss(s)
        return {"loss": loss, "lse": lse, "dz": _plain_dlogits(s, lse, None)}
    return {"dz": _plain_dlogits(s, s["lse"], s["grad"])}


# ------------------------------------------------------------------ the library's calls

def _own(s):
    import bit_nf4_quantized_21_b200 as q
    op = s["op"]
    if op.startswith("fp8"):
        W = q.FP8Matrix(s["n"], s["k"], BLOCK, s["codes"].view(torch.uint8), s["scale"])
        if op == "fp8_fwd":
            return {"y": q.qlora_fp8_linear_fwd(s["x"], W)}
        return {"dx": q.qlora_fp8_linear_bwd(s["x"], W)}
    if op == "norm_fwd":
        y, mean, rstd = q.qlora_layernorm_fwd(s["x"], s["w"], s["b"], EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dx, dw, db = q.qlora_layernorm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "distill_fwd":
        loss, lse = q.qlora_distill_topk_fwd(s["z"], s["ids"], s["t"], s["tau"], row_weight=s["weight"])
        return {"loss": loss, "lse": lse}
    if op == "distill_step":
        dz = torch.empty_like(s["z"])
        loss, lse = q.qlora_distill_topk_fwd(s["z"], s["ids"], s["t"], s["tau"], row_weight=s["weight"], dZ=dz)
        return {"loss": loss, "lse": lse, "dz": dz}
    return {"dz": q.qlora_distill_topk_bwd(s["z"], s["ids"], s["t"], s["tau"], s["lse"], row_weight=s["weight"],
                                           grad_loss=s["grad"])}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op.startswith("fp8"):
        m, n, k = case["m"], case["n"], case["k"]
        blocks = -(-n // BLOCK) * -(-k // BLOCK)
        return {"bytes": 2 * m * k + n * k + 4 * blocks + 2 * m * n, "flops": 2 * m * n * k}
    size = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        if op == "norm_fwd":
            return {"bytes": 2 * rows * cols * size + 2 * cols * size + 8 * rows, "flops": 8 * rows * cols}
        return {"bytes": 3 * rows * cols * size + cols * size + 8 * rows + 8 * cols, "flops": 14 * rows * cols}
    rows, vocab, top = case["rows"], case["vocab"], min(case["top"], case["vocab"])
    passes = 1 if op == "distill_fwd" else 2
    return {"bytes": passes * rows * vocab * size + 8 * rows * top + 12 * rows, "flops": 4 * passes * rows * vocab}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_fp8_operand(x):
    """x [m, width] as codes times scales, both as the format defines them, widened to 64 bits."""
    m, width = x.shape
    parts = []
    for at in range(0, width, BLOCK):
        block = x[:, at:at + BLOCK].float()
        scale = (block.abs().max(1).values.double() / E4M3_MAX).float()
        recip = torch.where(scale >= FLT_MIN, 1.0 / scale, torch.zeros_like(scale))
        code = (block * recip[:, None]).to(torch.float8_e4m3fn)
        parts.append(code.double() * torch.where(scale >= FLT_MIN, scale, torch.zeros_like(scale)).double()[:, None])
    return torch.cat(parts, 1)


def _exact_fp8(s):
    n, k = s["n"], s["k"]
    w = torch.empty((n, k), device=DEV, dtype=torch.float64)
    for i in range(s["scale"].shape[0]):
        rows = slice(i * BLOCK, min(n, (i + 1) * BLOCK))
        col = torch.arange(k, device=DEV) // BLOCK
        w[rows] = s["codes"][rows, :k].double() * s["scale"][i].double()[col]
    x = _exact_fp8_operand(s["x"])
    return {"y": x @ w.T} if s["op"] == "fp8_fwd" else {"dx": x @ w}


def _exact_norm(s):
    x = s["x"].double()
    w = s["w"].double()
    cols = x.shape[1]
    if s["op"] == "norm_fwd":
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = (x - mean.unsqueeze(1)) / torch.sqrt(var + EPS).unsqueeze(1) * w + s["b"].double()
        return {"y": y, "mean": mean, "rstd": rstd}
    dy, mean, rstd = s["dy"].double(), s["mean"].double(), s["rstd"].double()
    xh = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
    a = (dy @ w) / cols
    c = ((dy * xh) @ w) / cols
    dx = rstd.unsqueeze(1) * (dy * w - a.unsqueeze(1) - xh * c.unsqueeze(1))
    return {"dx": dx, "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def _exact_distill(s):
    tau = s["tau"]
    keep = (s["ids"] >= 0)
    logp = torch.log_softmax((s["t"].double() / tau).masked_fill(~keep, -math.inf), 1)
    any_left = keep.any(1)
    p = torch.where(keep, logp.exp(), torch.zeros_like(logp)).masked_fill(~any_left[:, None], 0.0)
    ids = s["ids"].long().masked_fill(~keep, 0)
    out = {}
    weight = s["weight"].double()
    if s["op"] == "distill_bwd":
        logq = s["z"].double() / tau - s["lse"].double()[:, None]
        weight = weight * s["grad"].double()
    else:
        logq = torch.log_softmax(s["z"].double() / tau, 1)
        term = p * (logp - logq.gather(1, ids))
        out["loss"] = weight * tau ** 2 * torch.where(p > 0, term, torch.zeros_like(term)).sum(1)
        out["lse"] = torch.logsumexp(s["z"].double() / tau, 1)
    if s["op"] != "distill_fwd":
        q = logq.exp_()
        q[~any_left] = 0.0
        q.scatter_add_(1, ids, -p)
        out["dz"] = q.mul_((weight * tau)[:, None])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"].startswith("fp8"):
        return _exact_fp8(s)
    return _exact_norm(s) if s["op"].startswith("norm") else _exact_distill(s)
