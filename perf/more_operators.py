"""The operators of a dense feed-forward block, as measured: each in a plain form (elementary torch
operations in 32 bits, rounded once at the end) and through this package's entry points.

The block reads, for hidden states x: a layer norm that also adds the residual (and can give 8-bit
rows with scales), the gated product act(x . gate) * (x . value) with its backward pass, and, where
weights and rows are held in 8 bits, the product with a scale for each block of 128 and what turns
16-bit matrices into such operands. ``own`` selects the side: False is the plain form, True calls
``dense_gemm_tensor_gb300.feedforward``.
"""

import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0
EPS = 1e-5
BLOCK = 128


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token's norm between two layers of a serving step
        dict(name="norm_decode", op="norm", rows=1, cols=4096, dtype="bf16", out="bf16", residual=True, bias=True),
        # a prefill batch, 8-bit rows for the next product
        dict(name="norm_prefill", op="norm", rows=8192, cols=8192, dtype="bf16", out="e4m3", residual=True, bias=True),
        # the norm's backward pass in a training step, an odd number of tokens
        dict(name="norm_train", op="norm_grad", rows=4097, cols=5120, dtype="bf16", residual=True, bias=True),
        # a serving step of 16 tokens: bound by reading the weights
        dict(name="gated_decode", op="gated", M=16, K=4096, F=8192, dtype="bf16", layout=1, act="silu", bias=False,
             keep=False),
        # a prefill batch
        dict(name="gated_prefill", op="gated", M=8192, K=4096, F=8192, dtype="bf16", layout=1, act="silu", bias=False,
             keep=False),
        # odd, ragged sizes: row-major weights with padded rows, a bias, fp16, the sums kept for a backward pass
        dict(name="gated_ragged", op="gated", M=1111, K=1000, F=1500, dtype="f16", layout=0, act="gelu_tanh", bias=True,
             keep=True),
        # a training step's gradients: of the input rows and of both weights
        dict(name="gated_train", op="gated_grad", M=8192, K=4096, F=4096, dtype="bf16", layout=1, act="silu",
             bias=False),
        # a serving step with 8-bit weights in blocks of 128 x 128
        dict(name="blocks_decode", op="blocks", M=16, N=8192, K=8192, b="blocks"),
        # a prefill batch of the same product
        dict(name="blocks_prefill", op="blocks", M=8192, N=8192, K=8192, b="blocks"),
        # a weight's gradient: both operands in runs of 128 tokens, an odd number of them
        dict(name="blocks_train", op="blocks", M=4096, N=5120, K=4099, b="rows"),
        # a prefill batch's rows to 8 bits
        dict(name="quantize_prefill", op="quantize", rows=8192, cols=8192, dtype="bf16", tall=1, transpose=False),
        # a training batch's rows transposed, in runs of 128 tokens, for the weight's gradient
        dict(name="quantize_train", op="quantize", rows=4099, cols=5120, dtype="bf16", tall=1, transpose=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm; odd ones are as likely as even ones."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "gated", "gated", "gated_grad", "blocks", "blocks", "blocks", "quantize",
                     "quantize"])
    if op in ("norm", "norm_grad"):
        c = dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192),
                 dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), residual=rng.random() < 0.7,
                 bias=rng.random() < 0.7)
        if op == "norm":
            c["out"] = rng.choice(["e4m3", c["dtype"]])
        return c
    if op in ("gated", "gated_grad"):
        c = dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 128, 4096), F=_log(rng, 64, 4096),
                 dtype=rng.choice(["bf16", "bf16", "f16"]), layout=rng.choice([0, 1]),
                 act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]), bias=rng.random() < 0.3)
        if op == "gated":
            c["keep"] = rng.random() < 0.5
        return c
    if op == "blocks":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 64, 8192), K=_log(rng, 64, 8192),
                    b=rng.choice(["blocks", "blocks", "rows"]))
    return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                tall=rng.choice([1, 1, BLOCK]), transpose=rng.random() < 0.4)


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    op, c = case["op"], case
    if op in ("norm", "norm_grad"):
        n, es = c["rows"] * c["cols"], BYTES[c["dtype"]]
        if op == "norm":
            reads = 2 * es if c["residual"] else es
            writes = (es if c["residual"] else 0) + BYTES[c["out"]]
            return {"bytes": n * (reads + writes) + c["cols"] * es * (2 if c["bias"] else 1) +
                    4 * c["rows"] * (3 if c["out"] == "e4m3" else 2), "flops": 8 * n}
        return {"bytes": n * es * (4 if c["residual"] else 3) + 3 * c["cols"] * es + 8 * c["rows"], "flops": 11 * n}
    if op in ("gated", "gated_grad"):
        m, k, f, es = c["M"], c["K"], c["F"], BYTES[c["dtype"]]
        if op == "gated":
            return {"bytes": es * (m * k + 2 * f * k + m * f * (3 if c["keep"] else 1) + (2 * f if c["bias"] else 0)),
                    "flops": 4.0 * m * k * f}
        return {"bytes": es * (m * f * 3 + 2 * m * k + 4 * f * k + (2 * f if c["bias"] else 0)), "flops": 8.0 * m * k * f}
    if op == "blocks":
        m, n, k = c["M"], c["N"], c["K"]
        kb = _blocks(k)
        return {"bytes": m * k + n * k + 2 * m * n + 4 * kb * (m + (n if c["b"] == "rows" else _blocks(n))),
                "flops": 2.0 * m * n * k}
    n = c["rows"] * c["cols"]
    along, across = (c["rows"], c["cols"]) if c["transpose"] else (c["cols"], c["rows"])
    scales = _blocks(along) * (across if c["tall"] == 1 else _blocks(across))
    return {"bytes": n * (BYTES[c["dtype"]] + 1) + 4 * scales, "flops": 3 * n}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (int(seed) + 1))
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _pitched(shape, dtype):
    """An empty matrix whose rows start on 16-byte boundaries (the row pitch is padded where it must be)."""
    per = 16 // dtype.itemsize
    return torch.empty((shape[0], -(-shape[1] // per) * per), dtype=dtype, device="cuda")[:, :shape[1]]


def _padded(g, shape, dtype, std=1.0):
    t = _pitched(shape, dtype)
    t.copy_(_normal(g, shape, dtype, std))
    return t


def _spread(g, rows, cols):
    """fp32 rows whose columns differ in size, a few of them by far, as the activations of a model do."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    return x * torch.exp(1.5 * torch.randn((cols,), generator=g, device="cuda"))


def _tiles(x, tall):
    """x as (row blocks, tall, column blocks, 128), padded with zeros."""
    r, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % BLOCK, 0, -r % tall))
    return x.view(-(-r // tall), tall, _blocks(c), BLOCK)


def _to_blocks(x, tall):
    """fp32 rows in 8 bits with a scale for each block: (q, scales with the blocks of a row as the outer dimension)."""
    t = _tiles(x, tall)
    scale = t.abs().amax(dim=(1, 3)).clamp(min=1e-12) / E4M3_MAX
    q = (t * (1.0 / scale)[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.reshape(t.shape[0] * tall, -1)[:x.shape[0], :x.shape[1]], scale


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    if op in ("norm", "norm_grad"):
        dt, shape = DT[c["dtype"]], (c["rows"], c["cols"])
        # rows with a mean of their own, as hidden states have
        x = torch.randn(shape, generator=g, device="cuda") + torch.randn((c["rows"], 1), generator=g, device="cuda")
        s = dict(x=x.to(dt), w=(1 + _normal(g, (c["cols"],), torch.float32, 0.1)).to(dt),
                 b=_normal(g, (c["cols"],), dt, 0.1) if c["bias"] else None)
        if op == "norm":
            s["residual"] = _normal(g, shape, dt, 2.0) if c["residual"] else None
        else:
            s["dy"] = _normal(g, shape, dt)
            s["dh"] = _normal(g, shape, dt) if c["residual"] else None
            h = s["x"].double()
            s["mean"] = h.mean(1).float()
            s["rstd"] = torch.rsqrt((h - s["mean"][:, None]).square().mean(1) + EPS).float()
    elif op in ("gated", "gated_grad"):
        dt = DT[c["dtype"]]
        s = dict(A=_padded(g, (c["M"], c["K"]), dt))
        s["W"] = _padded(g, (2 * c["F"], c["K"]) if c["layout"] == 1 else (c["K"], 2 * c["F"]), dt, c["K"] ** -0.5)
        s["bias"] = _normal(g, (2 * c["F"],), dt, 0.5) if c["bias"] else None
        if op == "gated_grad":
            s["up"] = _normal(g, (c["M"], 2 * c["F"]), dt, 1.1)
            s["dC"] = _normal(g, (c["M"], c["F"]), dt)
    elif op == "blocks":
        s = {}
        for name, n, tall in (("A", c["M"], 1), ("B", c["N"], BLOCK if c["b"] == "blocks" else 1)):
            q, scale = _to_blocks(_spread(g, n, c["K"]) * (1.0 if name == "A" else c["K"] ** -0.5), tall)
            s[name] = _pitched((n, c["K"]), torch.float8_e4m3fn)
            s[name].copy_(q)
            # scales of 1 x 128 blocks lie block column by block column, as `quantize` gives them
            s[name + "_scale"] = scale.t().contiguous().t() if tall == 1 else scale.contiguous()
    else:
        s = dict(x=_spread(g, c["rows"], c["cols"]).to(DT[c["dtype"]]))
    s["case"] = c
    return s


# ---------------------------------------------------------------- plain forms

def _norm_plain(c, s):
    x = s["x"].float()
    h = (x + s["residual"].float()).to(s["x"].dtype) if s["residual"] is not None else s["x"]
    hf = h.float()
    mean = hf.sum(1) / c["cols"]
    d = hf - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / c["cols"] + EPS)
    y = d * rstd[:, None] * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    out = dict(mean=mean, rstd=rstd)
    if c["residual"]:
        out["h"] = h
    if c["out"] == "e4m3":
        scale = y.abs().amax(1).clamp(min=1e-12) / E4M3_MAX
        out["y"], out["scale"] = (y * (1.0 / scale)[:, None]).to(torch.float8_e4m3fn), scale
    else:
        out["y"] = y.to(DT[c["out"]])
    return out


def _norm_grad_plain(c, s):
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - (g.sum(1) / c["cols"])[:, None] - xhat * ((g * xhat).sum(1) / c["cols"])[:, None])
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dt = s["x"].dtype
    return dict(dx=dx.to(dt), dw=(dy * xhat).sum(0).to(dt), db=dy.sum(0).to(dt))


_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def _act(x, act):
    if act == "relu":
        return torch.where(x < 0, 0.0, x)
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(_C0 * (x + _C1 * x * x * x)))
    return x / (1.0 + torch.exp(-x))


def _act_slope(x, act):
    if act == "relu":
        return torch.where(x > 0, 1.0, 0.0)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_C0 * (x + _C1 * x * x * x))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * _C0 * (1.0 + 3.0 * _C1 * x * x)
    sig = 1.0 / (1.0 + torch.exp(-x))
    return sig * (1.0 + x * (1.0 - sig))


def _weights(c, s):
    w = s["W"].float()
    return w.t() if c["layout"] == 1 else w  # K x 2F


def _gated_plain(c, s):
    up = s["A"].float() @ _weights(c, s)
    if s["bias"] is not None:
        up = up + s["bias"].float()
    gate, value = up.chunk(2, dim=1)
    dt = s["A"].dtype
    out = dict(c=(_act(gate, c["act"]) * value).to(dt))
    if c["keep"]:
        out["up"] = up.to(dt)
    return out


def _gated_grad_plain(c, s):
    gate, value = s["up"].float().chunk(2, dim=1)
    d = s["dC"].float()
    dup = torch.cat((d * value * _act_slope(gate, c["act"]), d * _act(gate, c["act"])), dim=1)
    da = dup @ _weights(c, s).t()
    a = s["A"].float()
    dw = dup.t() @ a if c["layout"] == 1 else a.t() @ dup
    dt = s["A"].dtype
    out = dict(da=da.to(dt), dw=dw.to(dt))
    if c["bias"]:
        out["db"] = dup.sum(0).to(dt)
    return out


def _value(q, scale, tall):
    """The fp32 numbers that 8-bit blocks stand for."""
    t = _tiles(q.float(), tall)
    return (t * scale[:, None, :, None]).reshape(t.shape[0] * tall, -1)[:q.shape[0], :q.shape[1]]


def _blocks_plain(c, s):
    a = _value(s["A"], s["A_scale"], 1)
    b = _value(s["B"], s["B_scale"], BLOCK if c["b"] == "blocks" else 1)
    return (a @ b.t()).to(torch.bfloat16)


def _quantize_plain(c, s):
    x = s["x"].float()
    q, scale = _to_blocks(x.t() if c["transpose"] else x, c["tall"])
    return dict(q=q, scale=scale)


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if not own:
        return {"norm": _norm_plain, "norm_grad": _norm_grad_plain, "gated": _gated_plain,
                "gated_grad": _gated_grad_plain, "blocks": _blocks_plain, "quantize": _quantize_plain}[op](c, s)

    from dense_gemm_tensor_gb300 import feedforward

    if op == "norm":
        r = feedforward.layer_norm(s["x"], s["w"], s["b"], s["residual"], eps=EPS, out_dtype=DT[c["out"]])
        out = dict(mean=r.mean, rstd=r.rstd, y=r.y)
        if c["residual"]:
            out["h"] = r.h
        if c["out"] == "e4m3":
            out["scale"] = r.scale
        return out
    if op == "norm_grad":
        dx, dw, db = feedforward.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], dh=s["dh"])
        return dict(dx=dx, dw=dw, db=db)
    if op == "gated":
        r = feedforward.gated_matmul(s["A"], s["W"], layout=c["layout"], activation=c["act"], bias=s["bias"],
                                     keep=c["keep"])
        return dict(c=r.c, up=r.up) if c["keep"] else dict(c=r.c)
    if op == "gated_grad":
        r = feedforward.gated_matmul_backward(s["dC"], s["A"], s["W"], s["up"], layout=c["layout"],
                                              activation=c["act"], bias=c["bias"])
        return dict(da=r.dA, dw=r.dW, db=r.dbias) if c["bias"] else dict(da=r.dA, dw=r.dW)
    if op == "blocks":
        return feedforward.matmul_blocks(s["A"], s["B"], s["A_scale"], s["B_scale"])
    r = feedforward.quantize_blocks(s["x"], rows=c["tall"], transpose=c["transpose"])
    return dict(q=r.q, scale=r.scale)


# ---------------------------------------------------------------- the definitions in 64 bits

def _np(t):
    return t.detach().double().cpu().numpy()


def _exact_gate(x, act):
    """(activation, its slope) in float64."""
    if act == "relu":
        return x.clamp(min=0), (x > 0).double()
    if act == "silu":
        p = torch.sigmoid(x)
        return x * p, p + x * p * (1 - p)
    if act == "gelu":
        p = torch.special.ndtr(x)
        return x * p, p + x * torch.exp(-x.square() / 2) / math.sqrt(2 * math.pi)
    u = 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    p = torch.sigmoid(u)
    return x * p, p + x * p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x ** 2)


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "norm":
        x = _np(s["x"])
        h = x
        if c["residual"]:  # h is held in the input's type: the norm is of the held values
            h = _np((torch.from_numpy(x) + torch.from_numpy(_np(s["residual"]))).to(s["x"].dtype))
        mean = h.mean(1)
        rstd = (h.var(1) + EPS) ** -0.5
        y = rstd[:, None] * (h - mean[:, None]) * _np(s["w"])[None, :]
        if c["bias"]:
            y += _np(s["b"])[None, :]
        out = dict(mean=mean, rstd=rstd, y=y)
        if c["residual"]:
            out["h"] = h
        if c["out"] == "e4m3":
            out["scale"] = np.maximum(np.abs(y).max(1), 1e-12) / E4M3_MAX
            out["y"] = y / out["scale"][:, None]
        return out
    if op == "norm_grad":
        h, dy, w, m, r = _np(s["x"]), _np(s["dy"]), _np(s["w"]), _np(s["mean"]), _np(s["rstd"])
        xh = (h - m[:, None]) * r[:, None]
        n = h.shape[1]
        dx = r[:, None] * (dy * w - (dy @ w / n)[:, None]) - xh * (r * np.einsum("ij,ij,j->i", dy, xh, w) / n)[:, None]
        return dict(dx=dx + _np(s["dh"]) if c["residual"] else dx, dw=np.einsum("ij,ij->j", dy, xh), db=dy.sum(0))
    if op in ("gated", "gated_grad"):
        a, w = s["A"].double(), s["W"].double()
        w = w if c["layout"] == 1 else w.t()  # 2F x K
        f = c["F"]
        if op == "gated":
            g, v = a @ w[:f].t(), a @ w[f:].t()
            if c["bias"]:
                g, v = g + s["bias"][:f].double(), v + s["bias"][f:].double()
            out = dict(c=_exact_gate(g, c["act"])[0] * v)
            if c["keep"]:
                out["up"] = torch.cat((g, v), 1)
            return out
        up, d = s["up"].double(), s["dC"].double()
        y, slope = _exact_gate(up[:, :f], c["act"])
        dg, dv = d * up[:, f:] * slope, d * y
        dw = torch.cat((dg.t() @ a, dv.t() @ a))
        out = dict(da=dg @ w[:f] + dv @ w[f:], dw=dw if c["layout"] == 1 else dw.t().contiguous())
        if c["bias"]:
            out["db"] = torch.cat((dg.sum(0), dv.sum(0)))
        return out
    if op == "blocks":
        a = s["A"].double() * s["A_scale"].double().repeat_interleave(BLOCK, 1)[:, :c["K"]]
        sb = s["B_scale"].double().repeat_interleave(BLOCK, 1)[:, :c["K"]]
        if c["b"] == "blocks":
            sb = sb.repeat_interleave(BLOCK, 0)[:c["N"]]
        return a @ (s["B"].double() * sb).t()
    x = s["x"].double()
    if c["transpose"]:
        x = x.t()
    scale = torch.stack([t.abs().amax(1) for t in x.split(BLOCK, 1)], 1)
    if c["tall"] > 1:
        scale = torch.stack([t.amax(0) for t in scale.split(BLOCK, 0)])
    scale = scale.clamp(min=1e-12) / E4M3_MAX
    full = scale.repeat_interleave(BLOCK, 1)[:, :x.shape[1]]
    if c["tall"] > 1:
        full = full.repeat_interleave(BLOCK, 0)[:x.shape[0]]
    return dict(q=x / full, scale=scale)
