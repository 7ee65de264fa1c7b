"""What is measured of the operators around the MoE layer, and their plain forms.

Five operators of the block that a routed layer sits in:

* ``norm``          layer norm or RMS norm of token rows, with the residual addition in front of it;
* ``norm_grad``     its backward pass: the rows' gradient (with the gradient that reaches the residual
                    stream from elsewhere) and the reductions of the weight's and the bias's gradients;
* ``ffn``           the dense gated feed-forward block  y = (act(x Wg^T) * (x Wu^T)) Wd^T;
* ``ffn_step``      one training step of it: the forward pass and every gradient;
* ``linear_fp8``    a linear layer in 8-bit floating point (e4m3): the activations quantised with one scale
                    per row and 128 columns, multiplied with weights of one scale per 128 x 128 block.

The plain forms compute in 32 bits with elementary torch operations and round once at the end.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FP8_MAX = 448.0   # largest finite e4m3 value
BLOCK = 128       # columns (and, for weights, rows) that share a scale


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step, width of the Mixtral-like layers: latency
        {"name": "norm_decode", "op": "norm", "T": 1, "d": 4096, "kind": "rms", "dtype": "bf16", "w_dtype": "bf16",
         "residual": True, "bias": False},
        # the tokens of a prefill, residual added on the way in
        {"name": "norm_prefill", "op": "norm", "T": 8192, "d": 4096, "kind": "rms", "dtype": "bf16", "w_dtype": "bf16",
         "residual": True, "bias": False},
        # an odd width in fp32, as a head or an adapter of odd size has it
        {"name": "norm_odd_f32", "op": "norm", "T": 2047, "d": 1411, "kind": "layer", "dtype": "f32", "w_dtype": "f32",
         "residual": False, "bias": True},
        # a training batch of the OLMoE-like width, fp32 norm weights
        {"name": "norm_grad_batch", "op": "norm_grad", "T": 8192, "d": 2048, "kind": "layer", "dtype": "bf16",
         "w_dtype": "f32", "residual": True, "bias": True},
        # many short rows: the Gemma-like width
        {"name": "norm_grad_narrow", "op": "norm_grad", "T": 30001, "d": 640, "kind": "rms", "dtype": "f16",
         "w_dtype": "f16", "residual": False, "bias": False},
        # one decoded token through the Mixtral-like dense block: every weight is read once
        {"name": "ffn_decode", "op": "ffn", "T": 1, "d": 4096, "h": 14336, "act": "silu", "dtype": "bf16"},
        # a small serving batch through the block of the Qwen-style shared expert's size
        {"name": "ffn_batch", "op": "ffn", "T": 57, "d": 2048, "h": 5632, "act": "gelu_tanh", "dtype": "f16"},
        # prefill through the Mixtral-like dense block: the tensor cores' rate
        {"name": "ffn_prefill", "op": "ffn", "T": 4096, "d": 4096, "h": 14336, "act": "silu", "dtype": "bf16"},
        # a training step of the Gemma-like dense block (four slices of 512), ragged batch
        {"name": "ffn_step_small", "op": "ffn_step", "T": 2000, "d": 640, "h": 2048, "act": "gelu_tanh", "dtype": "bf16"},
        # a training step at the Qwen-style width
        {"name": "ffn_step_batch", "op": "ffn_step", "T": 4096, "d": 2048, "h": 5632, "act": "silu", "dtype": "bf16"},
        # a few rows of a serving batch against a large 8-bit weight: its bytes
        {"name": "linear_fp8_decode", "op": "linear_fp8", "M": 9, "N": 14336, "K": 4096, "dtype": "bf16"},
        # prefill in 8 bits: the tensor cores' rate
        {"name": "linear_fp8_prefill", "op": "linear_fp8", "M": 4096, "N": 14336, "K": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "ffn", "ffn_step", "linear_fp8"])
    if op in ("norm", "norm_grad"):
        d = _log(rng, 8, 16384)
        if rng.random() < 0.7:   # mostly widths of whole 16-byte pieces, else any
            d = max(8, d // 8 * 8)
        T = min(_log(rng, 1, 65536), max(1, 8192 * 4096 // d))
        dtype = rng.choice(["bf16", "f16", "f32"])
        kind = rng.choice(["layer", "rms"])
        return {"op": op, "T": T, "d": d, "kind": kind, "dtype": dtype, "w_dtype": rng.choice([dtype, "f32"]),
                "residual": rng.random() < 0.5, "bias": kind == "layer" and rng.random() < 0.7}
    if op == "linear_fp8":
        N, K = 16 * _log(rng, 4, 896), 16 * _log(rng, 4, 896)
        M = min(_log(rng, 1, 8192), max(1, 4096 * 14336 * 4096 // (N * K)))
        return {"op": op, "M": M, "N": N, "K": K, "dtype": rng.choice(["bf16", "f16"])}
    d, h = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 1792)
    most = 4096 * 4096 * 14336 if op == "ffn" else 4096 * 2048 * 5632
    T = min(_log(rng, 1, 8192), max(1, most // (d * h)))
    return {"op": op, "T": T, "d": d, "h": h, "act": rng.choice(["silu", "gelu_tanh"]), "dtype": rng.choice(["bf16", "f16"])}


# ------------------------------------------------------------------ inputs

def _stream_rows(g, T, d):
    """Rows of a residual stream: unit spread, a few channels far larger, a mean of its own per row."""
    x = torch.randn(T, d, generator=g, device="cuda")
    scale = torch.ones(d, device="cuda")
    scale[torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")] = 12.0
    return x * scale + 0.5 * torch.randn(T, 1, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"op": op, "case": case, "dt": dt}

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    if op in ("norm", "norm_grad"):
        T, d, wt = case["T"], case["d"], DTYPES[case["w_dtype"]]
        s["eps"] = 1e-5
        s["x"] = _stream_rows(g, T, d).to(dt)
        s["weight"] = normal(d, std=0.1, mean=1.0, dtype=wt)
        s["bias"] = normal(d, std=0.1, dtype=wt) if case["bias"] else None
        if op == "norm":
            s["residual"] = _stream_rows(g, T, d).to(dt) if case["residual"] else None
        else:
            # what the forward pass kept: the normalised rows' mean and 1 / spread
            s["dy"] = normal(T, d)
            s["dh"] = normal(T, d) if case["residual"] else None
            x = s["x"].float()
            s["mean"] = x.mean(1) if case["kind"] == "layer" else None
            xc = x - s["mean"][:, None] if case["kind"] == "layer" else x
            s["rstd"] = torch.rsqrt(xc.square().mean(1) + s["eps"])
    elif op in ("ffn", "ffn_step"):
        T, d, h = case["T"], case["d"], case["h"]
        s["x"] = normal(T, d)
        s["w_gate"], s["w_up"] = normal(h, d, std=1 / math.sqrt(d)), normal(h, d, std=1 / math.sqrt(d))
        s["w_down"] = normal(d, h, std=1 / math.sqrt(h))
        if op == "ffn_step":
            s["dy"] = normal(T, d)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _stream_rows(g, M, K).to(dt)
        # a weight as a checkpoint in 8 bits holds it: codes, and one scale per 128 x 128 block
        s["w_q"], s["w_s"] = _quantize(torch.randn(N, K, generator=g, device="cuda") * 0.02, BLOCK)
    return s


# ------------------------------------------------------------------ plain forms

def _blocks(v, rows, cols, block_rows):
    """Each element's value of a [rows / block_rows, cols / 128] table of blocks."""
    v = v.repeat_interleave(BLOCK, 1)[:, :cols]
    return v if block_rows == 1 else v.repeat_interleave(block_rows, 0)[:rows]


def _quantize(x, block_rows):
    """e4m3 codes and the scales max|x| / 448 of blocks of block_rows x 128 elements."""
    rows, cols = x.shape
    br, bc = -(-rows // block_rows), -(-cols // BLOCK)
    whole = torch.zeros(br * block_rows, bc * BLOCK, device=x.device)
    whole[:rows, :cols] = x.float().abs()
    scale = whole.view(br, block_rows, bc, BLOCK).amax((1, 3)) / whole.new_full((), FP8_MAX)   # by a tensor: a correctly rounded quotient
    by = _blocks(scale, rows, cols, block_rows)
    q = torch.where(by > 0, x.float() / by, torch.zeros((), device=x.device)).clamp(-FP8_MAX, FP8_MAX)
    return q.to(torch.float8_e4m3fn), scale


def _act(name, u):
    """The activation and its derivative."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-u))
        return u * s, s * (1 + u * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (u + 0.044715 * u * u * u))
    return 0.5 * u * (1 + t), 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * c * (1 + 3 * 0.044715 * u * u)


def _plain_norm(s):
    x = s["x"]
    h = None
    if s["residual"] is not None:
        h = (x.float() + s["residual"].float()).to(x.dtype)   # the rows the residual stream goes on with
        x = h
    x = x.float()
    mean = x.mean(1) if s["case"]["kind"] == "layer" else None
    xc = x - mean[:, None] if mean is not None else x
    rstd = torch.rsqrt(xc.square().mean(1) + s["eps"])
    y = xc * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"y": y.to(s["dt"]), "h": h, "mean": mean, "rstd": rstd}


def _plain_norm_grad(s):
    x, dy = s["x"].float(), s["dy"].float()
    r = s["rstd"][:, None]
    xhat = (x - s["mean"][:, None] if s["mean"] is not None else x) * r
    dxhat = dy * s["weight"].float()
    dx = dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - dxhat.mean(1, keepdim=True)
    dx = dx * r
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["dt"]), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0) if s["bias"] is not None else None}


def _plain_ffn(s):
    x, wg, wu, wd = (s[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    u, v = x @ wg.T, x @ wu.T
    a, da_du = _act(s["case"]["act"], u)
    y = ((a * v) @ wd.T).to(s["dt"])
    if s["op"] == "ffn":
        return y
    dy = s["dy"].float()
    r = dy @ wd
    du, dv = r * v * da_du, r * a
    out = {"y": y, "dx": du @ wg + dv @ wu, "dw_gate": du.T @ x, "dw_up": dv.T @ x, "dw_down": dy.T @ (a * v)}
    return {k: t.to(s["dt"]) for k, t in out.items()}


def _plain_linear_fp8(s):
    x = s["x"]
    q, scale = _quantize(x, 1)
    w = s["w_q"].float() * _blocks(s["w_s"], *s["w_q"].shape, BLOCK)
    y = (q.float() * _blocks(scale, *x.shape, 1)) @ w.T
    return {"y": y.to(s["dt"]), "q": q, "scale": scale}


# ------------------------------------------------------------------ one pass

def run(s):
    op, c = s["op"], s["case"]
    if not own:
        if op == "norm":
            return _plain_norm(s)
        if op == "norm_grad":
            return _plain_norm_grad(s)
        return _plain_linear_fp8(s) if op == "linear_fp8" else _plain_ffn(s)
    from sparse_mixture_experts_sigmoid_b200 import binding as B
    if op == "norm":
        cfg = B.norm_config(c["T"], c["d"], kind=c["kind"], eps=s["eps"], dtype=c["dtype"], w_dtype=c["w_dtype"])
        y, h, mean, rstd = B.norm_forward(cfg, s["x"], s["weight"], bias=s["bias"], residual=s["residual"], want_stats=True)
        return {"y": y, "h": h, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        cfg = B.norm_config(c["T"], c["d"], kind=c["kind"], eps=s["eps"], dtype=c["dtype"], w_dtype=c["w_dtype"])
        dx, dweight, dbias = B.norm_backward(cfg, s["x"], s["weight"], s["mean"], s["rstd"], s["dy"], dh=s["dh"],
                                             want_bias=s["bias"] is not None)
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "linear_fp8":
        q, scale = B.quantize_fp8(s["x"])
        y = B.gemm_fp8(q, scale, s["w_q"], s["w_s"], out_dtype=c["dtype"])
        return {"y": y, "q": q, "scale": scale}
    cfg = B.ffn_config(c["T"], c["d"], c["h"], act=c["act"], dtype=c["dtype"])
    if "ws" not in s:   # a program keeps its workspace from step to step
        s["ws"] = B.alloc_ffn_workspace(cfg, train=op == "ffn_step")
    ws = s["ws"]
    if op == "ffn":
        return B.ffn_forward(cfg, s["x"], s["w_gate"], s["w_up"], s["w_down"], ws=ws)
    y = B.ffn_forward_train(cfg, s["x"], s["w_gate"], s["w_up"], s["w_down"], ws)
    return {"y": y, **B.ffn_backward(cfg, s["x"], s["w_gate"], s["w_up"], s["w_down"], s["dy"], ws)}


def work(case):
    op, e = case["op"], 4 if case["dtype"] == "f32" else 2
    if op in ("norm", "norm_grad"):
        T, d = case["T"], case["d"]
        we = 4 if case["w_dtype"] == "f32" else 2
        stats = 4 * T * (2 if case["kind"] == "layer" else 1)
        if op == "norm":   # x (and the residual) in, y (and their sum) out
            return {"bytes": T * d * e * (4 if case["residual"] else 2) + d * we * (2 if case["bias"] else 1) + stats,
                    "flops": 8 * T * d}
        return {"bytes": T * d * e * (4 if case["residual"] else 3) + d * we + 4 * d * (2 if case["bias"] else 1) + stats,
                "flops": 14 * T * d}
    if op == "linear_fp8":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // BLOCK)
        # x in, its codes and scales out, the weight's in, y out; each product at two operations
        return {"bytes": M * K * 3 + 4 * M * kb + N * K + 4 * kb * -(-N // BLOCK) + M * N * e, "flops": 2 * M * N * K}
    T, d, h = case["T"], case["d"], case["h"]
    if op == "ffn":
        return {"bytes": e * (2 * T * d + 3 * d * h), "flops": 6 * T * d * h}
    return {"bytes": e * (4 * T * d + 6 * d * h), "flops": 18 * T * d * h}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.dtype != torch.float8_e4m3fn else v for k, v in s.items()}
    op = case["op"]
    if op == "norm":
        h = None
        x = f["x"]
        if s["residual"] is not None:
            h = x + f["residual"]
            x = h.to(s["dt"]).double()   # the norm is of the rows as they are stored
        n = x.shape[1]
        mean = x.sum(1) / n if case["kind"] == "layer" else None
        var = ((x - (mean.unsqueeze(1) if mean is not None else 0)) ** 2).sum(1) / n
        rstd = 1 / (var + s["eps"]).sqrt()
        y = (x - (mean.unsqueeze(1) if mean is not None else 0)) * rstd.unsqueeze(1) * f["weight"]
        return {"y": y if s["bias"] is None else y + f["bias"], "h": h, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        # by differentiation of sum(y * dy) + sum(x * dh)
        x = f["x"].requires_grad_()
        w = f["weight"].requires_grad_()
        b = torch.zeros_like(w).requires_grad_()
        z = x - x.mean(1, keepdim=True) if case["kind"] == "layer" else x
        y = z / (z.pow(2).mean(1, keepdim=True) + s["eps"]).sqrt() * w + b
        total = (y * f["dy"]).sum() + ((x * f["dh"]).sum() if s["dh"] is not None else 0)
        dx, dw, db = torch.autograd.grad(total, (x, w, b))
        return {"dx": dx, "dweight": dw, "dbias": db if s["bias"] is not None else None}
    if op in ("ffn", "ffn_step"):
        keys = ("x", "w_gate", "w_up", "w_down")
        x, wg, wu, wd = leaves = [f[k].requires_grad_(op == "ffn_step") for k in keys]
        u = x.mm(wg.t())
        if case["act"] == "silu":
            a = u * torch.sigmoid(u)
        else:
            a = u * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3))   # (1 + tanh z) / 2 = sigmoid(2 z)
        y = (a * x.mm(wu.t())).mm(wd.t())
        if op == "ffn":
            return y
        dx, dg, du, dd = torch.autograd.grad((y * f["dy"]).sum(), leaves)
        return {"y": y.detach(), "dx": dx, "dw_gate": dg, "dw_up": du, "dw_down": dd}
    M, N, K = case["M"], case["N"], case["K"]
    x = f["x"]
    pieces, scales, weights = [], [], []
    w = s["w_q"].double()
    for b, c0 in enumerate(range(0, K, BLOCK)):
        piece = x[:, c0:c0 + BLOCK]
        scale = (piece.abs().max(1).values / FP8_MAX).float().double()   # the scales are 32-bit numbers
        codes = (piece / torch.where(scale > 0, scale, 1.0).unsqueeze(1)).float().clamp(-FP8_MAX, FP8_MAX)
        pieces.append(codes.to(torch.float8_e4m3fn).double())
        scales.append(scale)
        rows = torch.arange(N, device=w.device) // BLOCK
        weights.append(w[:, c0:c0 + BLOCK] * f["w_s"][rows, b].unsqueeze(1))
    y = sum((p * sc.unsqueeze(1)).mm(wb.t()) for p, sc, wb in zip(pieces, scales, weights))
    return {"y": y, "q": torch.cat(pieces, 1), "scale": torch.stack(scales, 1)}
