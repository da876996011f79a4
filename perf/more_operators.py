"""Layer norm, the expert router and the mixture-of-experts layer of a decode step, as they are measured.

Five operators: the layer norm that adds the residual and writes per-token FP8 codes, its backward pass, the router that
picks each token's experts from its logits, the router's backward pass, and the whole expert layer for a few tokens (both
products, the activation between them and the weighted sum) on the FP8 weights that the grouped product reads.

``run`` computes them in plain torch operations in float32 or, where ``own`` is true, through the package's entry points.
"""
import math

import torch

own = False

FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
REAL = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
FLOOR = 2.0 ** -126  # smallest scale
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of a decode step, before a projection of depth 7168
        dict(name="norm 1x7168 bf16", op="norm", rows=1, cols=7168, xt="bf16", fmt="e4m3", residual=True, ckpt=0),
        # a short float32 prompt, nothing added
        dict(name="norm 130x1040 f32", op="norm", rows=130, cols=1040, xt="f32", fmt="e4m3", residual=False, ckpt=0),
        # a large training batch: the stream is updated and kept as an 8-bit checkpoint for the backward pass
        dict(name="norm 16384x4096 ckpt", op="norm", rows=16384, cols=4096, xt="bf16", fmt="e4m3", residual=True, ckpt=128),
        # the gradient of a small, ragged float32 batch
        dict(name="norm_bwd 300x1040 f32", op="norm_bwd", rows=300, cols=1040, xt="f32", residual=True, ckpt=0),
        # the backward pass of a training batch whose stream was kept in 8 bits
        dict(name="norm_bwd 8192x4096 ckpt", op="norm_bwd", rows=8192, cols=4096, xt="bf16", residual=True, ckpt=128),
        # the router of one decoded token
        dict(name="route 1x128 bf16", op="route", tokens=1, experts=128, k=8, xt="bf16", score="softmax", renorm=True),
        # the router of a long prompt or a training batch, float32 logits
        dict(name="route 16384x128 f32", op="route", tokens=16384, experts=128, k=8, xt="f32", score="softmax", renorm=True),
        # that batch's gradient, weights not renormalised: every expert's logit gets one
        dict(name="route_bwd 16384x128", op="route_bwd", tokens=16384, experts=128, k=8, xt="bf16", score="softmax", renorm=False),
        # one token through a small layer of eight experts (the grouped product's weights, 2048 x 1024)
        dict(name="moe 1 of 8x1024x1024", op="moe", tokens=1, experts=8, k=2, hidden=1024, inner=1024, wf="e4m3", gated=True,
             act="silu", bias=False, residual=False),
        # one token through eight of 64 experts
        dict(name="moe 1 of 64x4096x1408", op="moe", tokens=1, experts=64, k=8, hidden=4096, inner=1408, wf="e4m3", gated=True,
             act="silu", bias=False, residual=True),
        # a ragged batch through a layer with biases, not gated
        dict(name="moe 13 of 24x1040x368", op="moe", tokens=13, experts=24, k=3, hidden=1040, inner=368, wf="e4m3", gated=False,
             act="gelu_tanh", bias=True, residual=False),
        # a decode batch that touches nearly every expert
        dict(name="moe 64 of 64x4096x1408", op="moe", tokens=64, experts=64, k=8, hidden=4096, inner=1408, wf="e4m3", gated=True,
             act="silu", bias=False, residual=True),
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, -(-lo // step) * step), hi // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "route", "route_bwd", "moe", "moe"])
    if op in ("norm", "norm_bwd"):
        while True:
            rows, cols = _log(rng, 1, 16384), _log(rng, 128, 16384, 16)
            if rows * cols <= 8192 * 4096:
                break
        c = dict(op=op, rows=rows, cols=cols, xt=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.7,
                 ckpt=rng.choice([0, 32, 64, 128]))
        if op == "norm":
            c["fmt"] = rng.choice(["e4m3", "e4m3", "e5m2"])
        return c
    if op in ("route", "route_bwd"):
        experts = _log(rng, 4, 512)
        # (one renormalised weight is 1 whatever the logits: no gradient)
        return dict(op=op, tokens=_log(rng, 1, 16384 * 128 // max(experts, 128)), experts=experts,
                    k=rng.randint(1 if op == "route" else 2, min(8, experts)), xt=rng.choice(["bf16", "f32"]),
                    score=rng.choice(["softmax", "softmax", "sigmoid"]), renorm=rng.random() < 0.5)
    gated = rng.random() < 0.7
    while True:
        experts = _log(rng, 4, 128)
        hidden, inner = _log(rng, 256, 7168, 16), _log(rng, 128, 4096, 32 if gated else 16)
        if experts * hidden * inner <= 64 * 4096 * 1408 // 2:
            break
    return dict(op=op, tokens=_log(rng, 1, 64), experts=experts, k=rng.randint(1, min(8, experts)), hidden=hidden, inner=inner,
                wf=rng.choice(["e4m3", "e4m3", "e5m2"]), gated=gated, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                bias=rng.random() < 0.3, residual=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _blocks(v, bs):
    """[rows, cols] in blocks of bs along the row, the last one padded with zeros."""
    rows, cols = v.shape
    nb = -(-cols // bs)
    return torch.nn.functional.pad(v, (0, nb * bs - cols)).view(rows, nb, bs)


def _encode(v, s, fmt):
    return (v * (1.0 / s)).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])


def _scale(amax, fmt):
    return (amax / FMAX[fmt]).clamp_min(FLOOR)


def _quantize_rows(v, fmt):
    """Per-token codes and scales of a float32 tensor."""
    s = _scale(v.abs().amax(1), fmt)
    return _encode(v, s[:, None], fmt), s


def _quantize_blocks(v, bs):
    """Block-wise E4M3 codes and scales of a float32 tensor."""
    b = _blocks(v, bs)
    s = _scale(b.abs().amax(2), "e4m3")
    return _encode(b, s[..., None], "e4m3").reshape(v.shape[0], -1)[:, : v.shape[1]].contiguous(), s


def _decode_blocks(q, s, bs):
    return q.float() * s.repeat_interleave(bs, 1)[:, : q.shape[1]]


def _preshuffled(wq):
    """The weight layout that the a8w8 products read: 16-slot x 128-byte fragments, padded with zeros."""
    n, k = wq.shape
    w = torch.nn.functional.pad(wq.view(torch.uint8), (0, -k % 128, 0, -n % 32))
    w = w.view((n + 31) // 32, 4, 2, 4, (k + 127) // 128, 4, 2, 16)
    return w.permute(0, 2, 4, 6, 5, 1, 3, 7).contiguous().view(-1)


def _pick(logits, k):
    """The k largest of each row, equal ones by index."""
    return torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std

    c = dict(case)
    st = {"case": c}
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        rows, cols, xt = c["rows"], c["cols"], REAL[c["xt"]]
        # the stream: rows off centre, a few channels much larger than the others
        wide = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 8.0, 1.0)
        st["weight"] = (1.0 + normal(cols, std=0.1)).to(xt)
        st["bias"] = normal(cols, std=0.1).to(xt)
        x = normal(rows, cols) + normal(rows, 1, std=0.5)
        if op == "norm":
            st["x"] = x.to(xt)
            st["r"] = (normal(rows, cols, std=2.0) * wide).to(xt) if c["residual"] else None
            return st
        h = (2.0 * x * wide).to(xt)
        st["mean"] = h.float().mean(1)
        st["rstd"] = torch.rsqrt((h.float() - st["mean"][:, None]).square().mean(1) + EPS)
        if c["ckpt"]:
            st["hq"], st["hs"] = _quantize_blocks(h.float(), c["ckpt"])
        else:
            st["h"] = h
        st["dy"] = normal(rows, cols, std=1e-2).to(xt)
        st["dr"] = normal(rows, cols, std=1e-2).to(xt) if c["residual"] else None
        return st
    tokens, experts, k = c["tokens"], c["experts"], c["k"]
    # some experts are asked for more often than others
    logits = normal(tokens, experts, std=1.5) + normal(1, experts)
    if op in ("route", "route_bwd"):
        st["logits"] = logits.to(REAL[c["xt"]])
        if op == "route_bwd":
            st["ids"] = _pick(st["logits"], k).to(torch.int32)
            st["dw"] = normal(tokens, k, std=1e-2)
        return st
    ids = _pick(logits, k)
    st["ids"] = ids.to(torch.int32)
    st["w"] = torch.softmax(torch.gather(logits, 1, ids), 1)
    d, f, wide = c["hidden"], c["inner"], (2 if c["gated"] else 1)
    st["xq"], st["xs"] = _quantize_rows(normal(tokens, d), "e4m3")
    st["w1"], st["s1"], st["p1"], st["w2"], st["s2"], st["p2"] = [], [], [], [], [], []
    for _ in range(experts):
        for i, (n, kk, std) in enumerate(((wide * f, d, 1.0 / math.sqrt(d)), (d, f, 1.0 / math.sqrt(f))), 1):
            q, s = _quantize_rows(normal(n, kk, std=std), c["wf"])
            st[f"w{i}"].append(q)
            st[f"s{i}"].append(s)
            st[f"p{i}"].append(_preshuffled(q))
    for key in ("w1", "s1", "w2", "s2"):
        st[key] = torch.stack([t.view(torch.uint8) if t.element_size() == 1 else t for t in st[key]])
    st["p1"], st["p2"] = torch.cat(st["p1"]), torch.cat(st["p2"])
    st["b1"] = normal(experts, wide * f, std=0.1).bfloat16() if c["bias"] else None
    st["b2"] = normal(experts, d, std=0.1).bfloat16() if c["bias"] else None
    st["res"] = normal(tokens, d).bfloat16() if c["residual"] else None
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _act(name, z):
    if name == "relu":
        return z.clamp_min(0.0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _scores(name, l):
    if name == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "norm":
        x = st["x"].float()
        h = x + st["r"].float() if c["residual"] else x
        mean = h.mean(1)
        d = h - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(1) + EPS)
        q, s = _quantize_rows(d * rstd[:, None] * st["weight"].float() + st["bias"].float(), c["fmt"])
        out = {"q": q, "s": s, "mean": mean, "rstd": rstd}
        if c["residual"]:
            out["h"] = h.to(st["x"].dtype)
        if c["ckpt"]:
            out["hq"], out["hs"] = _quantize_blocks(h, c["ckpt"])
        return out
    if op == "norm_bwd":
        h = _decode_blocks(st["hq"], st["hs"], c["ckpt"]) if c["ckpt"] else st["h"].float()
        dy, rstd = st["dy"].float(), st["rstd"][:, None]
        xh = (h - st["mean"][:, None]) * rstd
        t = dy * st["weight"].float()
        dx = rstd * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + st["dr"].float()
        return {"dx": dx.to(st["dy"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}
    if op == "route":
        l = st["logits"].float()
        ids = _pick(l, c["k"])
        w = torch.gather(_scores(c["score"], l), 1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return {"ids": ids.to(torch.int32), "w": w}
    if op == "route_bwd":
        l, ids, dw = st["logits"].float(), st["ids"].long(), st["dw"]
        p = _scores(c["score"], l)
        w = torch.gather(p, 1, ids)
        if c["renorm"]:
            total = w.sum(1, keepdim=True)
            dw = (dw - (dw * w).sum(1, keepdim=True) / total) / total
        dp = torch.zeros_like(p).scatter_add(1, ids, dw)
        dl = dp * p * (1.0 - p) if c["score"] == "sigmoid" else p * (dp - (dp * p).sum(1, keepdim=True))
        return {"dl": dl.to(st["logits"].dtype)}
    f8, f = F8[c["wf"]], c["inner"]
    x = st["xq"].float() * st["xs"][:, None]
    total = st["res"].float() if c["residual"] else torch.zeros(c["tokens"], c["hidden"], device=x.device)
    for e in range(c["experts"]):
        z = x @ (st["w1"][e].view(f8).float() * st["s1"][e][:, None]).t()
        if c["bias"]:
            z = z + st["b1"][e].float()
        a = _act(c["act"], z[:, :f]) * z[:, f:] if c["gated"] else _act(c["act"], z)
        y = a @ (st["w2"][e].view(f8).float() * st["s2"][e][:, None]).t()
        if c["bias"]:
            y = y + st["b2"][e].float()
        total = total + ((st["ids"] == e) * st["w"]).sum(1, keepdim=True) * y
    return {"out": total.bfloat16()}


def _codes(t, fmt):
    return t.view(F8[fmt])


def _own(st):
    import fp8_dynamic_quantization_amd as hq

    c = st["case"]
    op = c["op"]
    fmts = {"e4m3": hq.HQ_E4M3, "e5m2": hq.HQ_E5M2}
    if op == "norm":
        r = hq.hq_layernorm_quantize_fp8(st["x"], st["weight"], st["bias"], EPS, fmts[c["fmt"]], residual=st["r"],
                                         checkpoint=c["ckpt"])
        out = {"q": _codes(r.q, c["fmt"]), "s": r.scale, "mean": r.mean, "rstd": r.rstd}
        if c["residual"]:
            out["h"] = r.h
        if c["ckpt"]:
            out["hq"], out["hs"] = _codes(r.checkpoint.q, "e4m3"), r.checkpoint.scales
        return out
    if op == "norm_bwd":
        h = hq.Checkpoint(st["hq"].view(torch.uint8), st["hs"], c["ckpt"]) if c["ckpt"] else st["h"]
        dx, dw, db = hq.hq_layernorm_backward(st["dy"], h, st["weight"], st["mean"], st["rstd"], dresidual=st["dr"])
        return {"dx": dx, "dw": dw, "db": db}
    if op in ("route", "route_bwd"):
        score = hq.HQ_ROUTE_SOFTMAX if c["score"] == "softmax" else hq.HQ_ROUTE_SIGMOID
        if op == "route":
            ids, w = hq.hq_moe_route(st["logits"], c["k"], score=score, renormalize=c["renorm"])
            return {"ids": ids, "w": w}
        return {"dl": hq.hq_moe_route_backward(st["logits"], st["ids"], st["dw"], score=score, renormalize=c["renorm"])}
    acts = {"relu": hq.HQ_ACT_RELU, "gelu": hq.HQ_ACT_GELU, "gelu_tanh": hq.HQ_ACT_GELU_TANH, "silu": hq.HQ_ACT_SILU}
    out = hq.hq_moe_a8w8(st["xq"].view(torch.uint8), hq.HQ_E4M3, st["xs"], st["ids"], st["w"], st["p1"], st["s1"], st["p2"],
                         st["s2"], fmts[c["wf"]], act=acts[c["act"]], gated=c["gated"], bias1=st["b1"], bias2=st["b2"],
                         residual=st["res"])
    return {"out": out}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        rows, cols, e = c["rows"], c["cols"], SIZE[c["xt"]]
        numel = rows * cols
        copy = numel + 4 * rows * -(-cols // c["ckpt"]) if c["ckpt"] else 0
        if op == "norm":
            return {"bytes": numel * (e + 1) + (2 * e * numel if c["residual"] else 0) + 12 * rows + 2 * e * cols + copy,
                    "flops": 11 * numel}
        return {"bytes": 2 * e * numel + (e * numel if c["residual"] else 0) + 8 * rows + (e + 8) * cols + (copy or e * numel),
                "flops": 14 * numel}
    tokens, experts, k = c["tokens"], c["experts"], c["k"]
    if op == "route":
        return {"bytes": tokens * (experts * SIZE[c["xt"]] + 8 * k), "flops": 4 * tokens * experts}
    if op == "route_bwd":
        return {"bytes": tokens * (2 * experts * SIZE[c["xt"]] + 8 * k), "flops": 8 * tokens * experts}
    # experts that tokens * k independent, even choices reach
    d, f, wide = c["hidden"], c["inner"], (2 if c["gated"] else 1)
    active = experts * (1.0 - (1.0 - k / experts) ** tokens)
    weights = active * ((wide + 1) * d * f + 4 * (wide * f + d) + (2 * (wide * f + d) if c["bias"] else 0))
    return {"bytes": int(weights) + tokens * (d + 4 + 8 * k + 2 * d * (2 if c["residual"] else 1)),
            "flops": 2 * tokens * k * (wide + 1) * d * f}


# ---------------------------------------------------------------------------
# the operators from their definitions in 64 bits
# ---------------------------------------------------------------------------
def _grid64(v, amax, fmt):
    """The values on the code grid before they are rounded to codes, and their scales."""
    s = torch.clamp(amax / FMAX[fmt], min=FLOOR)
    return v / s, s


def _blocks64(v, bs):
    rows, cols = v.shape
    full = torch.zeros(rows, -(-cols // bs) * bs, dtype=torch.float64, device=v.device)
    full[:, :cols] = v
    full = full.view(rows, -1, bs)
    q, s = _grid64(full, full.abs().amax(2, keepdim=True), "e4m3")
    return q.reshape(rows, -1)[:, :cols], s[..., 0]


def _value64(q, s, bs):
    at = torch.arange(q.shape[1], device=q.device) // bs
    return q.double() * s.double()[:, at]


def _act64(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def _weights64(c, l, ids):
    """A row's routing weights, from the logarithms of the scores."""
    log = -torch.log1p(torch.exp(-l)) if c["score"] == "sigmoid" else l - torch.logsumexp(l, 1, keepdim=True)
    at = log[torch.arange(l.shape[0], device=l.device)[:, None], ids]
    return torch.exp(at - torch.logsumexp(at, 1, keepdim=True)) if c["renorm"] else torch.exp(at)


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    op = c["op"]
    if op == "norm":
        h = st["x"].double()
        if c["residual"]:
            h = h + st["r"].double()
        var, mean = torch.var_mean(h, 1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        y = (h - mean[:, None]) * (rstd[:, None] * st["weight"].double()) + st["bias"].double()
        q, s = _grid64(y, y.abs().amax(1, keepdim=True), c["fmt"])
        out = {"q": q, "s": s[:, 0], "mean": mean, "rstd": rstd}
        if c["residual"]:
            out["h"] = h
        if c["ckpt"]:
            out["hq"], out["hs"] = _blocks64(h, c["ckpt"])
        return out
    if op == "norm_bwd":
        h = _value64(st["hq"], st["hs"], c["ckpt"]) if c["ckpt"] else st["h"].double()
        dy, mean, rstd = st["dy"].double(), st["mean"].double(), st["rstd"].double()
        xh = (h - mean[:, None]) * rstd[:, None]
        t = dy * st["weight"].double()
        dx = rstd[:, None] * (t - (t.sum(1, keepdim=True) + xh * (t * xh).sum(1, keepdim=True)) / c["cols"])
        if c["residual"]:
            dx += st["dr"].double()
        return {"dx": dx, "dw": (dy * xh).sum(0), "db": dy.sum(0)}
    if op == "route":
        l = st["logits"].double()
        ids = torch.argsort(-l, dim=1, stable=True)[:, : c["k"]]
        return {"ids": ids.to(torch.int32), "w": _weights64(c, l, ids)}
    if op == "route_bwd":
        # the derivative of sum(dw * weights), by the chain rule through the logarithms
        l = st["logits"].double().requires_grad_()
        (st["dw"].double() * _weights64(c, l, st["ids"].long())).sum().backward()
        return {"dl": l.grad}
    f8, f = F8[c["wf"]], c["inner"]
    x = st["xq"].double() * st["xs"].double()[:, None]
    out = st["res"].double().clone() if c["residual"] else torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device=x.device)
    for e in range(c["experts"]):
        t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        z = torch.mm(x[t], st["w1"][e].view(f8).double().t().contiguous()) * st["s1"][e].double()
        if c["bias"]:
            z += st["b1"][e].double()
        a = _act64(c["act"], z[:, :f])
        if c["gated"]:
            a = a * z[:, f:]
        y = torch.mm(a, st["w2"][e].view(f8).double().t().contiguous()) * st["s2"][e].double()
        if c["bias"]:
            y += st["b2"][e].double()
        out.index_add_(0, t, y * st["w"][t, j].double()[:, None])
    return {"out": out}
