"""The operators of a mixture-of-experts block, as measured: each in a plain form (elementary
torch operations in 32 bits, rounded once at the end) and through this package's entry points.

The block reads, for hidden states x: a root-mean-square norm that also adds the residual (and can
give 8-bit rows with scales), a router that picks experts and orders the rows by expert, the
product of each expert's rows with its weights, and the weighted sum that returns the rows to
their tokens; in training, the backward pass of each. ``own`` selects the side: False is the plain
form, True calls ``dense_gemm_tensor_gb300.experts``.
"""

import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0
EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token's norm between two layers of a serving step; the next product takes 8-bit rows
        dict(name="norm_decode", op="norm", rows=1, cols=4096, dtype="bf16", out="e4m3", residual=True),
        # a prefill batch of the 8192-token projection workload, 8-bit rows for the next product
        dict(name="norm_prefill", op="norm", rows=8192, cols=8192, dtype="bf16", out="e4m3", residual=True),
        # the norm's backward pass in a training step, an odd number of tokens
        dict(name="norm_train", op="norm_grad", rows=4097, cols=5120, dtype="bf16", residual=True),
        # a small serving batch: sigmoid scores, balance bias, four of eight groups, eight of 256 experts
        dict(name="route_decode", op="route", tokens=16, experts=256, k=8, dtype="f32", score="sigmoid", bias=True,
             groups=8, kept=4, masked=0),
        # prefill: 16-bit logits (so exact ties occur), padding tokens masked out
        dict(name="route_prefill", op="route", tokens=16384, experts=128, k=8, dtype="bf16", score="softmax",
             bias=False, groups=1, kept=1, masked=100),
        # the router's gradient in a training step
        dict(name="route_train", op="route_grad", tokens=8192, experts=64, k=6, dtype="f32", score="softmax",
             bias=True, groups=1, kept=1, masked=0),
        # a serving step of 16 tokens: few rows an expert, bound by reading the experts' weights
        dict(name="experts_decode", op="experts", tokens=16, experts=64, k=4, K=2048, N=4096, dtype="bf16", layout=1,
             act="silu_gated", bias=False, gather=True),
        # a prefill batch with 8-bit rows and weights, the first (gate and up) product of the experts
        dict(name="experts_prefill", op="experts", tokens=8192, experts=32, k=4, K=4096, N=4096, dtype="e4m3",
             layout=1, act="silu_gated", bias=False, gather=True),
        # odd, ragged sizes: row-major weights with padded rows, a bias and an activation, fp16
        dict(name="experts_ragged", op="experts", tokens=1111, experts=5, k=2, K=1000, N=1500, dtype="f16", layout=0,
             act="gelu_tanh", bias=True, gather=True),
        # a training step's gradients of one product, of its input rows and of its weights
        dict(name="experts_train", op="experts_grad", tokens=8192, experts=16, k=2, K=4096, N=4096, dtype="bf16",
             layout=1, gather=True),
        # the end of the block over a prefill batch
        dict(name="combine_prefill", op="combine", tokens=8192, cols=4096, k=8, dtype="bf16", residual=True, masked=50),
        # its backward pass, an odd number of tokens
        dict(name="combine_train", op="combine_grad", tokens=4099, cols=2048, k=6, dtype="bf16", masked=0),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm; odd ones are as likely as even ones."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    c = _draw(rng)
    while 3072 in c.values():
        c = _draw(rng)
    return c


def _draw(rng):
    op = rng.choice(["norm", "norm_grad", "route", "route_grad", "experts", "experts", "experts", "experts_grad",
                     "experts_grad", "combine", "combine_grad"])
    if op in ("norm", "norm_grad"):
        c = dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192),
                 dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), residual=rng.random() < 0.7)
        if op == "norm":
            c["out"] = rng.choice(["e4m3", c["dtype"]])
        return c
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * _log(rng, max(2, 8 // groups), 256 // groups)
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(8, kept * (experts // groups)))
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, k=k, dtype=rng.choice(["f32", "bf16", "f16"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, kept=kept,
                    masked=rng.choice([0, 0, 3]))
    if op == "experts":
        dtype = rng.choice(["bf16", "f16", "e4m3"])
        act = rng.choice(["none", "silu_gated", "relu", "gelu"])
        c = dict(op=op, tokens=_log(rng, 1, 8192), experts=_log(rng, 2, 64), dtype=dtype,
                 layout=1 if dtype == "e4m3" else rng.choice([0, 1]), act=act, bias=rng.random() < 0.3,
                 gather=rng.random() < 0.7)
        c["k"] = rng.randint(1, min(4, c["experts"]))
        c["K"] = _log(rng, 128, 4096)
        c["N"] = 2 * _log(rng, 64, 2048) if act == "silu_gated" else _log(rng, 128, 4096)
        return c
    if op == "experts_grad":
        c = dict(op=op, tokens=_log(rng, 16, 8192), experts=_log(rng, 2, 16), K=_log(rng, 128, 4096),
                 N=_log(rng, 128, 4096), dtype=rng.choice(["bf16", "f16"]), layout=rng.choice([0, 1]),
                 gather=rng.random() < 0.7)
        c["k"] = rng.randint(1, 2)
        return c
    return dict(op=op, tokens=_log(rng, 1, 8192), cols=_log(rng, 64, 4096), k=rng.randint(1, 8),
                dtype=rng.choice(["bf16", "f16"]), masked=rng.choice([0, 0, 2]),
                **({"residual": rng.random() < 0.5} if op == "combine" else {}))


def work(case):
    op, c = case["op"], case
    es = BYTES[c["dtype"]]
    if op == "norm":
        n = c["rows"] * c["cols"]
        reads = 2 * es if c["residual"] else es
        writes = (es if c["residual"] else 0) + BYTES[c["out"]]
        return {"bytes": n * (reads + writes) + c["cols"] * es + 4 * c["rows"] * (2 if c["out"] == "e4m3" else 1),
                "flops": 5 * n}
    if op == "norm_grad":
        n = c["rows"] * c["cols"]
        return {"bytes": n * es * (4 if c["residual"] else 3) + 2 * c["cols"] * es + 4 * c["rows"], "flops": 8 * n}
    if op == "route":
        t, e, k = c["tokens"], c["experts"], c["k"]
        return {"bytes": t * e * es + 16 * t * k + 4 * e, "flops": 4 * t * e}
    if op == "route_grad":
        t, e, k = c["tokens"], c["experts"], c["k"]
        return {"bytes": 2 * t * e * es + 12 * t * k, "flops": 6 * t * e}
    if op in ("experts", "experts_grad"):
        t, e, k, K, N = c["tokens"], c["experts"], c["k"], c["K"], c["N"]
        r = t * k
        active = e * (1.0 - (1.0 - k / e) ** t)  # experts with at least one row
        a_rows = t if c["gather"] else r
        if op == "experts":
            out = N // 2 if c["act"] == "silu_gated" else N
            return {"bytes": a_rows * K * es + active * K * N * es + 2 * r * out, "flops": 2.0 * r * K * N}
        # the input gradient reads dC and W and writes r x K; the weight gradient reads A and dC again and writes e x K x N
        return {"bytes": es * (r * N + active * K * N + r * K + a_rows * K + e * K * N), "flops": 4.0 * r * K * N}
    t, h, k = c["tokens"], c["cols"], c["k"]
    if op == "combine":
        return {"bytes": es * (t * k * h + t * h * (2 if c["residual"] else 1)) + 8 * t * k, "flops": 2 * t * k * h}
    return {"bytes": es * (2 * t * k * h + t * h) + 12 * t * k, "flops": 4 * t * k * h}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (int(seed) + 1))
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _order(ids, experts):
    """The expert order of T x k expert numbers (-1: none): slots, rows, offsets."""
    t, k = ids.shape
    flat = torch.where(ids < 0, experts, ids).reshape(-1)
    srt, order = torch.sort(flat, stable=True)
    edges = torch.arange(experts + 1, device=ids.device, dtype=flat.dtype)
    offsets = torch.searchsorted(srt, edges).to(torch.int32)
    place = torch.arange(t * k, device=ids.device, dtype=torch.int32)
    slots = torch.empty_like(place)
    slots[order] = place
    none = srt == experts
    rows = torch.where(none, -1, order // k).to(torch.int32)
    slots = torch.where(ids < 0, -1, slots.view(t, k))
    return slots, rows, offsets


def _pick(g, tokens, experts, k, masked=0):
    """Distinct experts for each token, some experts more popular than others; the last `masked` tokens have none."""
    pop = torch.randn((experts,), generator=g, device="cuda") * 0.5
    noise = torch.rand((tokens, experts), generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    ids = torch.topk(pop - torch.log(-torch.log(noise)), k, dim=1).indices.to(torch.int32)
    if masked:
        ids[-min(masked, tokens):] = -1
    return ids


def _padded(g, shape, dtype, std=1.0):
    """A matrix or a stack of them whose rows start on 16-byte boundaries (the row pitch is padded where it must be)."""
    per = 16 // dtype.itemsize
    ld = -(-shape[-1] // per) * per
    return _normal(g, (*shape[:-1], ld), dtype, std)[..., :shape[-1]]


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    dt = DT[c["dtype"]]
    if op == "norm":
        s = dict(x=_normal(g, (c["rows"], c["cols"]), dt), w=(1 + _normal(g, (c["cols"],), torch.float32, 0.1)).to(dt))
        s["residual"] = _normal(g, (c["rows"], c["cols"]), dt, 2.0) if c["residual"] else None
    elif op == "norm_grad":
        h = _normal(g, (c["rows"], c["cols"]), dt, 2.0)
        s = dict(h=h, dy=_normal(g, h.shape, dt), w=(1 + _normal(g, (c["cols"],), torch.float32, 0.1)).to(dt),
                 rstd=torch.rsqrt(h.float().square().mean(1) + EPS))
        s["dh"] = _normal(g, h.shape, dt) if c["residual"] else None
    elif op in ("route", "route_grad"):
        logits = _normal(g, (c["tokens"], c["experts"]), dt, 1.5)
        if c["masked"]:
            logits[-min(c["masked"], c["tokens"]):] = -math.inf
        s = dict(logits=logits, bias=_normal(g, (c["experts"],), torch.float32, 0.02) if c["bias"] else None)
        if op == "route_grad":
            s["dweights"] = _normal(g, (c["tokens"], c["k"]), torch.float32)
            s["ids"], s["weights"] = _route_plain(c, s)[:2]
    elif op in ("experts", "experts_grad"):
        t, e, k, K, N = c["tokens"], c["experts"], c["k"], c["K"], c["N"]
        ids = _pick(g, t, e, k)
        _, rows, offsets = _order(ids, e)
        s = dict(offsets=offsets, rows=rows if c["gather"] else None,
                 cap=int((offsets[1:] - offsets[:-1]).max()))  # the largest group: the plain form pads to it
        s["A"] = _padded(g, (t if c["gather"] else t * k, K), dt)
        wstd = 1.0 if c["dtype"] == "e4m3" else 1.0 / math.sqrt(K)
        s["W"] = _padded(g, (e, N, K) if c["layout"] == 1 else (e, K, N), dt, wstd)
        if op == "experts":
            s["bias"] = _normal(g, (e, N), torch.bfloat16 if c["dtype"] == "e4m3" else dt) if c["bias"] else None
            s["a_scale"] = s["w_scale"] = None
            if c["dtype"] == "e4m3":
                s["a_scale"] = 0.5 + torch.rand((s["A"].shape[0],), generator=g, device="cuda")
                s["w_scale"] = (0.5 + torch.rand((e, N), generator=g, device="cuda")) / math.sqrt(K)
        else:
            s["dC"] = _padded(g, (t * k, N), dt)
    else:
        t, h, k = c["tokens"], c["cols"], c["k"]
        ids = _pick(g, t, max(16, k), k, c["masked"])
        slots, rows, offsets = _order(ids, max(16, k))
        s = dict(slots=slots, rows=rows, offsets=offsets, z=_normal(g, (t * k, h), dt),
                 weights=torch.softmax(_normal(g, (t, k), torch.float32), 1))
        if op == "combine":
            s["residual"] = _normal(g, (t, h), dt) if c["residual"] else None
        else:
            s["dy"] = _normal(g, (t, h), dt)
    s["case"] = c
    return s


# ---------------------------------------------------------------- plain forms

def _norm_plain(c, s):
    x = s["x"].float()
    h = (x + s["residual"].float()).to(s["x"].dtype) if s["residual"] is not None else s["x"]
    hf = h.float()
    rstd = 1.0 / torch.sqrt((hf * hf).sum(1) / c["cols"] + EPS)
    y = hf * rstd[:, None] * s["w"].float()
    out = dict(rstd=rstd)
    if c["residual"]:
        out["h"] = h
    if c["out"] == "e4m3":
        scale = y.abs().amax(1).clamp(min=1e-12) / E4M3_MAX
        out["y"], out["scale"] = (y * (1.0 / scale)[:, None]).to(torch.float8_e4m3fn), scale
    else:
        out["y"] = y.to(DT[c["out"]])
    return out


def _norm_grad_plain(c, s):
    xhat = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - xhat * ((g * xhat).sum(1) / c["cols"])[:, None])
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dict(dx=dx.to(s["h"].dtype), dw=(dy * xhat).sum(0).to(s["w"].dtype))


def _halves(x):
    """The sum over the last axis by adding halves, the axis padded with zeros to a power of two: the
    order in which the router's softmax denominator is defined, since the choice depends on its last bit."""
    n = 1 << max(0, (x.shape[-1] - 1).bit_length())
    x = torch.nn.functional.pad(x, (0, n - x.shape[-1]))
    return _fold(x)


def _fold(x):
    n = x.shape[-1]
    return x[..., 0] if n == 1 else _fold(x[..., :n // 2] + x[..., n // 2:])


def _scores(c, s):
    l = s["logits"].float()
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    m = l.amax(1, keepdim=True)
    e = torch.where(l > -math.inf, torch.exp(l - torch.where(m > -math.inf, m, 0.0)), 0.0)
    z = _halves(e)[:, None]
    return e / torch.where(z > 0, z, 1.0)


def _top(key, k):
    """The k largest of each row, ties to the lowest index."""
    v, i = torch.sort(key, dim=1, descending=True, stable=True)
    return v[:, :k], i[:, :k]


def _route_plain(c, s):
    e, k = c["experts"], c["k"]
    score = _scores(c, s)
    key = score + s["bias"] if s["bias"] is not None else score
    key = torch.where(s["logits"].float() > -math.inf, key, -math.inf)
    if c["groups"] > 1:
        per = e // c["groups"]
        best = _top(key.reshape(-1, per), min(2, per))[0]
        group = best.sum(1).view(-1, c["groups"]) if per > 1 else best.view(-1, c["groups"])
        keep = torch.zeros_like(group, dtype=torch.bool).scatter_(1, _top(group, c["kept"])[1], True)
        key = torch.where(keep.repeat_interleave(per, 1), key, -math.inf)
    v, ids = _top(key, k)
    none = v == -math.inf
    w = torch.where(none, 0.0, torch.gather(score, 1, ids))
    w = w / (w.sum(1, keepdim=True) + 1e-20)
    ids = torch.where(none, -1, ids).to(torch.int32)
    return (ids, w, *_order(ids, e))


def _route_grad_plain(c, s):
    score = _scores(c, s)
    there = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    dw = torch.where(there, s["dweights"], 0.0)
    sc = torch.where(there, torch.gather(score, 1, ids), 0.0)
    total = sc.sum(1, keepdim=True) + 1e-20
    ds = torch.where(there, (dw - (dw * s["weights"]).sum(1, keepdim=True)) / total, 0.0)
    full = torch.zeros_like(score).scatter_add_(1, ids, ds)
    if c["score"] == "sigmoid":
        d = full * score * (1.0 - score)
    else:
        d = score * (full - (full * score).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _act(x, act):
    if act == "relu":
        return torch.where(x < 0, 0.0, x)
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "silu_gated":
        a, b = x.chunk(2, dim=1)
        return a / (1.0 + torch.exp(-a)) * b
    return x


def _groups(s, n):
    """For each row: its expert, and its place among that expert's rows."""
    at = torch.arange(n, device="cuda")
    e = torch.searchsorted(s["offsets"].long(), at, right=True) - 1
    return e, at - s["offsets"].long()[e]


def _spread(x, e, p, experts, cap):
    full = torch.zeros((experts, cap, x.shape[1]), dtype=torch.float32, device="cuda")
    full[e, p] = x.float()
    return full


def _experts_plain(c, s):
    n = c["tokens"] * c["k"]
    e, p = _groups(s, n)
    rows = s["rows"].long() if s["rows"] is not None else torch.arange(n, device="cuda")
    w = s["W"].float()
    x = torch.bmm(_spread(s["A"][rows], e, p, c["experts"], s["cap"]), w.transpose(1, 2) if c["layout"] == 1 else w)
    x = x[e, p]
    if s["a_scale"] is not None:
        x = x * s["a_scale"][rows][:, None] * s["w_scale"][e]
    if s["bias"] is not None:
        x = x + s["bias"].float()[e]
    return _act(x, c["act"]).to(torch.bfloat16 if c["dtype"] == "e4m3" else DT[c["dtype"]])


def _experts_grad_plain(c, s):
    n = c["tokens"] * c["k"]
    e, p = _groups(s, n)
    rows = s["rows"].long() if s["rows"] is not None else torch.arange(n, device="cuda")
    w = s["W"].float()
    d = _spread(s["dC"], e, p, c["experts"], s["cap"])
    a = _spread(s["A"][rows], e, p, c["experts"], s["cap"])
    da = torch.bmm(d, w if c["layout"] == 1 else w.transpose(1, 2))[e, p]
    dw = torch.bmm(d.transpose(1, 2), a) if c["layout"] == 1 else torch.bmm(a.transpose(1, 2), d)
    return dict(da=da.to(DT[c["dtype"]]), dw=dw.to(DT[c["dtype"]]))


def _combine_plain(c, s):
    there = (s["slots"] >= 0)[:, :, None]
    z = torch.where(there, s["z"][s["slots"].clamp(min=0).long()].float(), 0.0)
    y = (z * s["weights"][:, :, None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["z"].dtype)


def _combine_grad_plain(c, s):
    there = s["slots"] >= 0
    slots = s["slots"].clamp(min=0).long()
    dy = s["dy"].float()
    dw = torch.where(there, (s["z"][slots].float() * dy[:, None, :]).sum(2), 0.0)
    dz = torch.zeros_like(s["z"])
    dz[slots[there]] = (s["weights"][:, :, None] * dy[:, None, :])[there].to(dz.dtype)
    return dict(dz=dz, dweights=dw)


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "route":
            return dict(zip(("ids", "weights", "slots", "rows", "offsets"), _route_plain(c, s)))
        return {"norm": _norm_plain, "norm_grad": _norm_grad_plain, "route_grad": _route_grad_plain,
                "experts": _experts_plain, "experts_grad": _experts_grad_plain, "combine": _combine_plain,
                "combine_grad": _combine_grad_plain}[op](c, s)

    from dense_gemm_tensor_gb300 import experts

    if op == "norm":
        r = experts.rms_norm(s["x"], s["w"], s["residual"], eps=EPS, out_dtype=DT[c["out"]])
        out = dict(rstd=r.rstd, y=r.y)
        if c["residual"]:
            out["h"] = r.h
        if c["out"] == "e4m3":
            out["scale"] = r.scale
        return out
    if op == "norm_grad":
        dx, dw = experts.rms_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], dh=s["dh"])
        return dict(dx=dx, dw=dw)
    if op == "route":
        r = experts.route(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                          kept_groups=c["kept"])
        return dict(ids=r.ids, weights=r.weights, slots=r.slots, rows=r.rows, offsets=r.offsets)
    if op == "route_grad":
        return experts.route_backward(s["dweights"], s["logits"], s["ids"], score=c["score"])
    if op == "experts":
        return experts.expert_matmul(s["A"], s["W"], s["offsets"], s["rows"], layout=c["layout"], bias=s["bias"],
                                     activation=c["act"], a_scale=s["a_scale"], w_scale=s["w_scale"])
    if op == "experts_grad":
        da = experts.expert_matmul(s["dC"], s["W"], s["offsets"], layout=1 - c["layout"])
        dw = experts.expert_weight_grad(s["A"], s["dC"], s["offsets"], s["rows"], layout=c["layout"])
        return dict(da=da, dw=dw)
    if op == "combine":
        return experts.combine(s["z"], s["slots"], s["weights"], residual=s["residual"])
    dz, dw = experts.combine_backward(s["dy"], s["z"], s["slots"], s["weights"], s["offsets"])
    return dict(dz=dz, dweights=dw)


# ---------------------------------------------------------------- the definitions in 64 bits

def _np(t):
    return t.detach().double().cpu().numpy()


def _exact_route(c, s):
    """Scores, choice and weights of each token in float64; the key that chooses is held in 32 bits, as the
    operator defines it (two experts whose keys round to the same value are a tie)."""
    l = _np(s["logits"])
    t, e = l.shape
    with np.errstate(all="ignore"):
        if c["score"] == "sigmoid":
            score = 1.0 / (1.0 + np.exp(-l))
        else:
            top = l.max(1, keepdims=True)
            score = np.exp(l - np.where(np.isfinite(top), top, 0.0))
            score = score / np.maximum(score.sum(1, keepdims=True), 1e-300)
    score[np.isneginf(l)] = 0.0
    return score


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "norm":
        x = _np(s["x"])
        h = x
        if c["residual"]:  # h is held in the input's type: the norm is of the held values
            h = _np((torch.from_numpy(x) + torch.from_numpy(_np(s["residual"]))).to(s["x"].dtype))
        rstd = (np.einsum("ij,ij->i", h, h) / h.shape[1] + EPS) ** -0.5
        y = rstd[:, None] * h * _np(s["w"])[None, :]
        out = dict(rstd=rstd, y=y)
        if c["residual"]:
            out["h"] = h
        if c["out"] == "e4m3":
            out["scale"] = np.maximum(np.abs(y).max(1), 1e-12) / E4M3_MAX
            out["y"] = y / out["scale"][:, None]
        return out
    if op == "norm_grad":
        h, dy, w, r = _np(s["h"]), _np(s["dy"]), _np(s["w"]), _np(s["rstd"])
        xh = h * r[:, None]
        dx = r[:, None] * dy * w - xh * (r * np.einsum("ij,ij,j->i", dy, xh, w) / h.shape[1])[:, None]
        return dict(dx=dx + _np(s["dh"]) if c["residual"] else dx, dw=np.einsum("ij,ij->j", dy, xh))
    if op == "route":
        score = _exact_route(c, s)
        l = _np(s["logits"])
        b = _np(s["bias"]) if c["bias"] else np.zeros(c["experts"])
        key = (score.astype(np.float32) + b.astype(np.float32)).astype(np.float64)
        key[np.isneginf(l)] = -np.inf
        if c["groups"] > 1:
            per = c["experts"] // c["groups"]
            g = np.sort(key.reshape(len(key), c["groups"], per), 2)[:, :, -2:].astype(np.float32)
            g = g.sum(2, dtype=np.float32)
            for row, gi in zip(key, np.argsort(-g, 1, kind="stable")[:, c["kept"]:]):
                row.reshape(c["groups"], per)[gi] = -np.inf
        ids = np.argsort(-key, 1, kind="stable")[:, :c["k"]]
        w = np.take_along_axis(score, ids, 1) * (np.take_along_axis(key, ids, 1) > -np.inf)
        return dict(ids=None, weights=w / (w.sum(1, keepdims=True) + 1e-20), slots=None, rows=None, offsets=None)
    if op == "route_grad":
        score = _exact_route(c, s)
        ids, dw = _np(s["ids"]).astype(int), _np(s["dweights"])
        at = np.where(ids >= 0, ids, 0)
        chosen = np.take_along_axis(score, at, 1) * (ids >= 0)
        total = chosen.sum(1, keepdims=True) + 1e-20
        ds = (ids >= 0) * (dw / total - (dw * chosen).sum(1, keepdims=True) / total ** 2)
        d = np.zeros_like(score)
        for j in range(c["k"]):
            d[np.arange(len(d)), at[:, j]] += ds[:, j]
        if c["score"] == "sigmoid":
            return d * score * (1 - score)
        return score * (d - np.einsum("ij,ij->i", d, score)[:, None])
    if op in ("experts", "experts_grad"):
        off = s["offsets"].tolist()
        n = c["tokens"] * c["k"]
        rows = s["rows"].long() if c["gather"] else torch.arange(n, device="cuda")
        da, dw, ys = [], [], []
        for e in range(c["experts"]):
            at = rows[off[e]:off[e + 1]]
            a, w = s["A"][at].double(), s["W"][e].double()
            w = w if c["layout"] == 1 else w.t()  # N x K
            if op == "experts_grad":
                d = s["dC"][off[e]:off[e + 1]].double()
                da.append(d @ w)
                m = d.t() @ a
                dw.append(m if c["layout"] == 1 else m.t())
                continue
            y = a @ w.t()
            if c["dtype"] == "e4m3":
                y = y * torch.outer(s["a_scale"][at].double(), s["w_scale"][e].double())
            if c["bias"]:
                y = y + s["bias"][e].double()
            if c["act"] == "silu_gated":
                y = y[:, :c["N"] // 2] * torch.sigmoid(y[:, :c["N"] // 2]) * y[:, c["N"] // 2:]
            elif c["act"] == "relu":
                y = y.clamp(min=0)
            elif c["act"] == "gelu":
                y = y * torch.special.ndtr(y)
            elif c["act"] == "gelu_tanh":
                y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
            ys.append(y)
        return dict(da=torch.cat(da), dw=torch.stack(dw)) if op == "experts_grad" else torch.cat(ys)
    slots, z, w = _np(s["slots"]).astype(int), s["z"].double(), s["weights"].double()
    if op == "combine":
        y = s["residual"].double().clone() if c["residual"] else torch.zeros((c["tokens"], c["cols"]), device="cuda",
                                                                             dtype=torch.float64)
        for j in range(c["k"]):
            t = torch.from_numpy(np.flatnonzero(slots[:, j] >= 0)).cuda()
            y[t] += w[t, j, None] * z[s["slots"][t, j].long()]
        return y
    dz, dw, dy = torch.zeros_like(z), torch.zeros_like(w), s["dy"].double()
    for j in range(c["k"]):
        t = torch.from_numpy(np.flatnonzero(slots[:, j] >= 0)).cuda()
        at = s["slots"][t, j].long()
        dz[at] = w[t, j, None] * dy[t]
        dw[t, j] = torch.einsum("ij,ij->i", dy[t], z[at])
    return dict(dz=dz, dweights=dw)
