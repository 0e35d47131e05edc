"""The feed-forward operators as they are measured: the product with a fused
epilogue, the routing to experts and the experts' products.

A case is a dict of plain values; prepare() makes its inputs from a seed,
run() makes one pass, exact() gives the same outputs in 64 bits and work()
what a pass cannot do without.  With ``own`` false run() takes the plain form
(elementary torch operations in 32 bits, 64 for the routing keys); with it
true, the library's operators.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GATED = ("swiglu", "geglu")
FAR = 6.0 * 4096 * 4096 * 4096   # most flops of a drawn case


def _lib():
    import dense_tiled_gemm_bf16_amd as tg
    return tg


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _epilogue(name, m, n, k, dtype, layout, act, bias, residual, train=False):
    c = {"op": "epilogue", "m": m, "n": n, "k": k, "dtype": dtype, "layout": layout, "act": act, "bias": bias,
         "residual": residual, "train": train}
    return {"name": name, **c} if name else c


def _route(name, t, e, k, score, dtype, bias, groups, used, renorm, scale, train=False):
    c = {"op": "route", "t": t, "e": e, "k": k, "score": score, "dtype": dtype, "bias": bias, "groups": groups,
         "used": used, "renorm": renorm, "scale": scale, "train": train}
    return {"name": name, **c} if name else c


def _experts(name, t, e, k, d, f, dtype, act, bias, train=False):
    c = {"op": "experts", "t": t, "e": e, "k": k, "d": d, "f": f, "dtype": dtype, "act": act, "bias": bias,
         "train": train}
    return {"name": name, **c} if name else c


def listed():
    return [
        # One new token through a projection: latency and the read of the weight.
        _epilogue("epilogue_token", 1, 4096, 4096, "bf16", "nt", "silu", True, True),
        # A batch of decoded tokens through a gated layer's first product.
        _epilogue("epilogue_batch_gated", 48, 8192, 4096, "bf16", "nt", "swiglu", False, False),
        # The repository's benchmark shape with a whole epilogue.
        _epilogue("epilogue_prompt", 4096, 4096, 8192, "bf16", "nt", "gelu", True, True),
        # Its ragged shape, weights stored K x N, fp16.
        _epilogue("epilogue_ragged", 4000, 3000, 5000, "f16", "nn", "gelu_tanh", True, True),
        # A training step of one layer: forward, then every gradient.
        _epilogue("epilogue_train", 4096, 4096, 2048, "bf16", "nt", "gelu_tanh", True, True, True),
        # Routing of a few decoded tokens: groups, balance bias, sigmoid scores.
        _route("route_tokens", 8, 256, 8, "sigmoid", "f32", True, 8, 4, True, 2.5),
        # Routing of a long packed prompt.
        _route("route_prompt", 32768, 256, 8, "sigmoid", "f32", True, 8, 4, True, 2.5),
        # Routing with its gradient in a training step, an odd number of experts and tokens.
        _route("route_train", 16381, 97, 6, "softmax", "bf16", False, 1, 1, False, 1.0, True),
        # One token through its experts: the weights of the chosen experts are read once.
        _experts("experts_token", 1, 64, 6, 2048, 1024, "bf16", "swiglu", False),
        # A batch of decoded tokens, most experts hit by a few of them.
        _experts("experts_batch", 37, 64, 6, 2048, 1024, "bf16", "swiglu", False),
        # A prompt: every expert has hundreds of rows, unevenly.
        _experts("experts_prompt", 8192, 32, 4, 2048, 2048, "bf16", "swiglu", False),
        # A training step of a whole expert layer, routing and its gradient included.
        _experts("experts_train", 4096, 16, 2, 2048, 1536, "bf16", "gelu", True, True),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    while True:
        op = rng.choice(("epilogue", "route", "experts"))
        train = rng.random() < 0.3
        if op == "epilogue":
            act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu", "swiglu", "geglu"))
            gated = act in GATED
            layout = rng.choice(("nt", "nt", "nn")) if gated else rng.choice(("nt", "nt", "nn", "tn", "tt"))
            m = _log(rng, 1, 8192)
            if layout[0] == "t":
                m = (m + 7) // 8 * 8       # rows of the stored array are whole 16-byte pieces
            n = _log(rng, 128, 8192, 16)
            k = _log(rng, 128, 8192, 8)
            case = _epilogue("", m, n, k, rng.choice(("bf16", "bf16", "f16")), layout, act, rng.random() < 0.6,
                             rng.random() < 0.5, train)
        elif op == "route":
            score = rng.choice(("softmax", "sigmoid"))
            groups = rng.choice((1, 1, 4, 8))
            e = groups * _log(rng, 8, 64) if groups > 1 else _log(rng, 8, 512)
            used = 1 if groups == 1 else rng.randint(1, groups)
            k = rng.randint(1, min(12, used * (e // groups)))
            case = _route("", _log(rng, 1, 32768), e, k, score, rng.choice(("f32", "bf16", "f16")),
                          rng.random() < 0.5, groups, used, rng.random() < 0.6, rng.choice((1.0, 2.5)), train)
        else:
            case = _experts("", _log(rng, 1, 8192), _log(rng, 4, 128), rng.randint(1, 4), _log(rng, 256, 4096, 8),
                            _log(rng, 128, 2048, 8), rng.choice(("bf16", "bf16", "f16")),
                            rng.choice(("swiglu", "geglu", "gelu", "relu")), rng.random() < 0.4, train)
            if case["e"] * case["d"] * case["f"] > 1 << 27:
                continue
        if work(case)["flops"] <= FAR:
            return case


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _stored(x, transposed, dt):
    """x's values in storage of type dt, as the transpose of a row-major array if asked."""
    return x.t().contiguous().to(dt).t() if transposed else x.to(dt)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[case["dtype"]]
    s = {"case": case}
    if case["op"] == "epilogue":
        m, n, k = case["m"], case["n"], case["k"]
        f = n // 2 if case["act"] in GATED else n
        s["a"] = _stored(_randn(g, m, k), case["layout"][0] == "t", dt)
        s["b"] = _stored(_randn(g, k, n) / math.sqrt(k), case["layout"][1] == "t", dt)
        s["bias"] = (0.5 * _randn(g, n)).to(dt) if case["bias"] else None
        s["residual"] = _randn(g, m, f).to(dt) if case["residual"] else None
        s["dy"] = _randn(g, m, f).to(dt) if case["train"] else None
    elif case["op"] == "route":
        t, e = case["t"], case["e"]
        # Some experts are liked by most tokens, as in a trained router.
        s["logits"] = (_randn(g, t, e) + 0.7 * _randn(g, e)).to(dt)
        s["bias"] = 0.1 * _randn(g, e) if case["bias"] else None
        s["dw"] = _randn(g, t, case["k"]) if case["train"] else None
    else:
        t, e, d, f = case["t"], case["e"], case["d"], case["f"]
        n = 2 * f if case["act"] in GATED else f
        s["x"] = _randn(g, t, d).to(dt)
        s["logits"] = (_randn(g, t, e) + 0.5 * _randn(g, e)).to(dt)
        # Weights as linear layers keep them: one row for each output.
        s["w1"] = torch.empty(e, n, d, dtype=dt, device="cuda")
        s["w2"] = torch.empty(e, d, f, dtype=dt, device="cuda")
        for i in range(e):
            s["w1"][i] = _randn(g, n, d) / math.sqrt(d)
            s["w2"][i] = _randn(g, d, f) / math.sqrt(f)
        s["b1"] = (0.5 * _randn(g, e, n)).to(dt) if case["bias"] else None
        s["b2"] = (0.5 * _randn(g, e, d)).to(dt) if case["bias"] else None
        s["dy"] = _randn(g, t, d).to(dt) if case["train"] else None
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _gelu(z):
    return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _gelu_grad(z):
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act in ("gelu", "geglu"):
        return _gelu(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z))          # silu, swiglu


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act in ("gelu", "geglu"):
        return _gelu_grad(z)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _apply(z, act):
    if act in GATED:
        gate, up = z.chunk(2, dim=-1)
        return _act(gate, act) * up
    return _act(z, act)


def _apply_grad(dy, z, act):
    if act in GATED:
        gate, up = z.chunk(2, dim=-1)
        return torch.cat((dy * up * _act_grad(gate, act), dy * _act(gate, act)), dim=-1)
    return dy * _act_grad(z, act)


def _plain_epilogue(s):
    c, dt = s["case"], s["a"].dtype
    a, b = s["a"].float(), s["b"].float()
    z = a @ b
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _apply(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(dt)
    if not c["train"]:
        return y
    dz = _apply_grad(s["dy"].float(), z, c["act"])
    out = {"y": y, "da": (dz @ b.t()).to(dt), "db": (a.t() @ dz).to(dt)}
    if s["bias"] is not None:
        out["dbias"] = dz.sum(0).to(dt)
    return out


def _plain_topk(logits, k, score, bias, groups, used, renorm, scale):
    """(weights, ids, scores); the keys are compared in 64 bits, ties to the lowest index."""
    x = logits.double()
    if score == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    key = p if bias is None else p + bias.double()
    if groups > 1:
        t, e = key.shape
        by = key.view(t, groups, e // groups)
        best = by.sort(dim=2, descending=True).values[:, :, :2].sum(2)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :used]
        keep = torch.zeros(t, groups, dtype=torch.bool, device=key.device).scatter_(1, order, True)
        key = by.masked_fill(~keep[:, :, None], -math.inf).view(t, e)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if renorm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return (w * scale).float(), ids.to(torch.int32), p


def _plain_topk_grad(dw, p, ids, score, renorm, scale, dt):
    at = ids.long()
    p = p.float()
    sel = p.gather(1, at)
    dw = dw.float() * scale
    if renorm:
        total = sel.sum(1, keepdim=True)
        ds = (dw - (dw * (sel / total)).sum(1, keepdim=True)) / total
    else:
        ds = dw
    dp = torch.zeros_like(p).scatter_(1, at, ds)
    if score == "softmax":
        return (p * (dp - (dp * p).sum(1, keepdim=True))).to(dt)
    return (dp * p * (1.0 - p)).to(dt)


def _plain_plan(ids, e):
    """(offsets, token of each row, row of each choice) with the rows sorted by expert, tokens in order."""
    t, k = ids.shape
    flat = ids.reshape(-1).long()
    order = flat.sort(stable=True).indices
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.zeros(e, dtype=torch.int64, device=ids.device).scatter_add_(
        0, flat, torch.ones_like(flat)).cumsum(0)
    slots = torch.empty_like(order).scatter_(0, order, torch.arange(t * k, device=ids.device))
    return offsets, order // k, slots.view(t, k)


def _plain_route(s):
    c = s["case"]
    w, ids, p = _plain_topk(s["logits"], c["k"], c["score"], s["bias"], c["groups"], c["used"], c["renorm"],
                            c["scale"])
    offsets, rows, slots = _plain_plan(ids, c["e"])
    out = {"weights": w, "ids": ids, "offsets": offsets.to(torch.int32), "rows": rows.to(torch.int32),
           "slots": slots.to(torch.int32)}
    if c["train"]:
        out["dlogits"] = _plain_topk_grad(s["dw"], p, ids, c["score"], c["renorm"], c["scale"], s["logits"].dtype)
    return out


class _Padded:
    """The experts' rows side by side in one batch (E, most rows of one expert, columns), or one row each."""

    def __init__(self, ids, e):
        self.offsets, self.rows, self.slots = _plain_plan(ids, e)
        n = self.rows.numel()
        expert = ids.reshape(-1).long().sort(stable=True).values
        self.each = n <= e
        if self.each:
            self.e, self.cap, self.pick = n, 1, expert
            self.at = torch.arange(n, device=ids.device)
        else:
            self.e, self.pick = e, None
            self.cap = int((self.offsets[1:] - self.offsets[:-1]).max())
            self.at = expert * self.cap + torch.arange(n, device=ids.device) - self.offsets[expert]

    def pad(self, x):
        out = torch.zeros(self.e * self.cap, x.shape[1], device=x.device)
        out[self.at] = x
        return out.view(self.e, self.cap, -1)

    def rows_of(self, x):
        return x.reshape(self.e * self.cap, -1)[self.at]

    def weight(self, w):
        return (w if self.pick is None else w[self.pick]).float()

    def grad(self, x, n):
        """The gradient for each of n experts from one for each batch entry."""
        if self.pick is None:
            return x
        return torch.zeros(n, *x.shape[1:], device=x.device).index_add_(0, self.pick, x)


def _plain_experts(s):
    c, dt = s["case"], s["x"].dtype
    e, act = c["e"], c["act"]
    w, ids, p = _plain_topk(s["logits"], c["k"], "softmax", None, 1, 1, True, 1.0)
    m = _Padded(ids, e)
    x = m.pad(s["x"].float()[m.rows])
    w1, w2 = m.weight(s["w1"]), m.weight(s["w2"])
    z = torch.bmm(x, w1.transpose(1, 2).contiguous())
    if s["b1"] is not None:
        z = z + m.weight(s["b1"])[:, None]
    h = _apply(z, act)
    y = torch.bmm(h, w2.transpose(1, 2).contiguous())
    if s["b2"] is not None:
        y = y + m.weight(s["b2"])[:, None]
    rows = m.rows_of(y)
    out = (rows[m.slots] * w[:, :, None]).sum(1).to(dt)
    if not c["train"]:
        return out
    dy = s["dy"].float()
    dw = (rows[m.slots] * dy[:, None]).sum(2)
    drows = torch.empty_like(rows)
    drows[m.slots.reshape(-1)] = (dy[:, None] * w[:, :, None]).reshape(-1, dy.shape[1])
    dout = m.pad(drows)
    dz = _apply_grad(torch.bmm(dout, w2), z, act)
    dx = m.rows_of(torch.bmm(dz, w1))[m.slots].sum(1)
    got = {"y": out, "dx": dx.to(dt),
           "dw1": m.grad(torch.bmm(dz.transpose(1, 2).contiguous(), x), e).to(dt),
           "dw2": m.grad(torch.bmm(dout.transpose(1, 2).contiguous(), h), e).to(dt),
           "dlogits": _plain_topk_grad(dw, p, ids, "softmax", True, 1.0, s["logits"].dtype)}
    if s["b1"] is not None:
        got["db1"] = m.grad(dz.sum(1), e).to(dt)
        got["db2"] = m.grad(dout.sum(1), e).to(dt)
    return got


# --------------------------------------------------------------------------
# The library's operators
# --------------------------------------------------------------------------
def _own_epilogue(s):
    tg, c = _lib(), s["case"]
    a, b = s["a"], s["b"]
    if not c["train"]:
        return tg.gemm_epilogue(a, b, bias=s["bias"], act=c["act"], residual=s["residual"])
    z = torch.empty(c["m"], c["n"], dtype=a.dtype, device=a.device)
    y = tg.gemm_epilogue(a, b, bias=s["bias"], act=c["act"], residual=s["residual"], preact=z)
    dz, dbias = tg.epilogue_backward(s["dy"], z, c["act"], want_dbias=s["bias"] is not None)
    out = {"y": y, "da": tg.gemm(dz, b.t()), "db": tg.gemm(a.t(), dz)}
    if s["bias"] is not None:
        out["dbias"] = dbias
    return out


def _own_route(s):
    tg, c = _lib(), s["case"]
    w, ids = tg.route_topk(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                           groups_used=c["used"], renormalize=c["renorm"], scale=c["scale"])
    offsets, rows, slots = tg.route_plan(ids, c["e"])
    out = {"weights": w, "ids": ids, "offsets": offsets, "rows": rows, "slots": slots}
    if c["train"]:
        out["dlogits"] = tg.route_topk_backward(s["dw"], s["logits"], ids, score=c["score"],
                                                renormalize=c["renorm"], scale=c["scale"])
    return out


def _own_experts(s):
    tg, c = _lib(), s["case"]
    act = c["act"]
    x, w1, w2 = s["x"], s["w1"].transpose(1, 2), s["w2"].transpose(1, 2)     # (E, K, N) views
    w, ids = tg.route_topk(s["logits"], c["k"])
    offsets, rows, slots = tg.route_plan(ids, c["e"])
    if not c["train"]:
        h = tg.gemm_grouped(x, w1, offsets, rows=rows, bias=s["b1"], act=act)
        return tg.expert_combine(tg.gemm_grouped(h, w2, offsets, bias=s["b2"]), slots, w)
    xs = tg.expert_gather(x, rows)
    z = torch.empty(xs.shape[0], w1.shape[2], dtype=x.dtype, device=x.device)
    h = tg.gemm_grouped(xs, w1, offsets, bias=s["b1"], act=act, preact=z)
    rows_out = tg.gemm_grouped(h, w2, offsets, bias=s["b2"])
    y = tg.expert_combine(rows_out, slots, w)
    dout, dw = tg.expert_combine_backward(s["dy"], rows_out, slots, w)
    got = {"y": y, "dw2": tg.gemm_grouped_tn(dout, h, offsets)}
    dh = tg.gemm_grouped(dout, s["w2"], offsets)
    dz, db1 = tg.epilogue_backward(dh, z, act, offsets=offsets, want_dbias=s["b1"] is not None)
    got["dw1"] = tg.gemm_grouped_tn(dz, xs, offsets)
    got["dx"] = tg.expert_combine(tg.gemm_grouped(dz, s["w1"], offsets), slots)
    got["dlogits"] = tg.route_topk_backward(dw, s["logits"], ids)
    if s["b1"] is not None:
        got["db1"] = db1
        got["db2"] = tg.epilogue_backward(dout, None, "none", offsets=offsets)[1]
    return got


def run(state):
    op = state["case"]["op"]
    if own:
        return {"epilogue": _own_epilogue, "route": _own_route, "experts": _own_experts}[op](state)
    return {"epilogue": _plain_epilogue, "route": _plain_route, "experts": _plain_experts}[op](state)


# --------------------------------------------------------------------------
# Work
# --------------------------------------------------------------------------
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "epilogue":
        m, n, k = case["m"], case["n"], case["k"]
        f = n // 2 if case["act"] in GATED else n
        nbytes = m * k + k * n + m * f + (n if case["bias"] else 0) + (m * f if case["residual"] else 0)
        flops = 2.0 * m * n * k
        if case["train"]:
            nbytes += m * f + m * k + k * n + (n if case["bias"] else 0)
            flops *= 3
        return {"bytes": nbytes * 2, "flops": flops}
    t, e, k = case["t"], case["e"], case["k"]
    if case["op"] == "route":
        nbytes = t * e * size + t * k * 16 + 4 * (e + 1) + (4 * e if case["bias"] else 0)
        if case["train"]:
            nbytes += t * k * 4 + t * e * size
        # An exponential and a comparison for each score, the selection aside.
        return {"bytes": nbytes, "flops": 4.0 * t * e}
    d, f = case["d"], case["f"]
    n = 2 * f if case["act"] in GATED else f
    # Experts that uniform choices hit, on average.
    hit = e * (1.0 - (1.0 - k / e) ** t)
    weights = hit * (n * d + d * f)
    bias = hit * (n + d) if case["bias"] else 0
    flops = 2.0 * t * k * (n * d + d * f)
    nbytes = 2 * (2 * t * d + t * e + weights + bias)
    if case["train"]:
        nbytes += 2 * (2 * t * d + t * e + e * (n * d + d * f) + (e * (n + d) if case["bias"] else 0))
        flops *= 3
    return {"bytes": nbytes, "flops": flops}


# --------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------
def _exact_act(z, act):
    """(value, derivative) of an activation."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act in ("gelu", "geglu"):
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        u = c * (z + 0.044715 * z ** 3)
        sig = torch.sigmoid(2 * u)          # (1 + tanh u) / 2
        return z * sig, sig + z * 2 * sig * (1 - sig) * c * (1 + 0.134145 * z ** 2)
    sig = torch.sigmoid(z)
    return z * sig, sig + z * sig * (1 - sig)


def _exact_layer(z, act):
    """Output of the epilogue and a function giving dZ from its gradient."""
    if act in GATED:
        f = z.shape[1] // 2
        g, u = z[:, :f], z[:, f:]
        v, dv = _exact_act(g, act)
        return v * u, lambda dy: torch.cat([dy * u * dv, dy * v], 1)
    v, dv = _exact_act(z, act)
    return v, lambda dy: dy * dv


def _exact_select(x, k, score, bias, groups, used):
    """Scores and chosen experts, from the definition, one comparison table at a time, on the host."""
    x = x.double().cpu().numpy()
    if score == "softmax":
        p = np.exp(x - x.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    else:
        p = 1.0 / (1.0 + np.exp(-x))
    key = p + (0.0 if bias is None else bias.double().cpu().numpy())
    t, e = key.shape
    if groups > 1:
        per = e // groups
        two = np.partition(key.reshape(t, groups, per), per - 2, axis=2)[:, :, -2:].sum(2)
        drop = np.argsort(-two, axis=1, kind="stable")[:, used:]
        mask = np.zeros((t, groups), bool)
        np.put_along_axis(mask, drop, True, 1)
        key = np.where(np.repeat(mask, per, axis=1), -np.inf, key)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    return p, ids


def _exact_plan(ids, e):
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=e))])
    slots = np.empty_like(order)
    slots[order] = np.arange(order.size)
    return offsets, order // ids.shape[1], slots.reshape(ids.shape)


def _exact_weights(p, ids, renorm, scale):
    sel = np.take_along_axis(p, ids, 1)
    return sel, sel / (sel.sum(1, keepdims=True) if renorm else 1.0) * scale


def _exact_dlogits(dw, p, ids, score, renorm, scale):
    """By the chain rule through each chosen score."""
    sel, _ = _exact_weights(p, ids, renorm, scale)
    if renorm:
        total = sel.sum(1, keepdims=True)
        w = sel / total
        dsel = scale * (dw - (dw * w).sum(1, keepdims=True)) / total
    else:
        dsel = dw * scale
    dp = np.zeros_like(p)
    np.put_along_axis(dp, ids, dsel, 1)
    if score == "softmax":
        return p * dp - p * (p * dp).sum(1, keepdims=True)
    return p * (1 - p) * dp


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "epilogue":
        a, b = s["a"].double(), s["b"].double()
        z = torch.mm(a, b)
        if s["bias"] is not None:
            z += s["bias"].double()
        y, back = _exact_layer(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].double()
        if not c["train"]:
            return y
        dz = back(s["dy"].double())
        out = {"y": y, "da": torch.mm(dz, b.t()), "db": torch.mm(a.t(), dz)}
        if s["bias"] is not None:
            out["dbias"] = dz.sum(0)
        return out
    if c["op"] == "route":
        p, ids = _exact_select(s["logits"], c["k"], c["score"], s["bias"], c["groups"], c["used"])
        _, w = _exact_weights(p, ids, c["renorm"], c["scale"])
        offsets, rows, slots = _exact_plan(ids, c["e"])
        out = {"weights": w, "ids": ids, "offsets": offsets, "rows": rows, "slots": slots}
        if c["train"]:
            out["dlogits"] = _exact_dlogits(s["dw"].double().cpu().numpy(), p, ids, c["score"], c["renorm"],
                                            c["scale"])
        return out
    p, ids = _exact_select(s["logits"], c["k"], "softmax", None, 1, 1)
    _, w = _exact_weights(p, ids, True, 1.0)
    offsets, rows, slots = _exact_plan(ids, c["e"])
    dev = s["x"].device
    at, wt = torch.from_numpy(rows).to(dev), torch.from_numpy(w).to(dev)
    put = torch.from_numpy(slots).to(dev)
    x = s["x"].double()
    n, d = len(rows), c["d"]
    y_rows = torch.zeros(n, d, dtype=torch.float64, device=dev)
    keep = []
    for e in range(c["e"]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        z = x[at[lo:hi]] @ s["w1"][e].double().t()
        if s["b1"] is not None:
            z = z + s["b1"][e].double()
        h, back = _exact_layer(z, c["act"])
        y_rows[lo:hi] = h @ s["w2"][e].double().t()
        if s["b2"] is not None:
            y_rows[lo:hi] += s["b2"][e].double()
        if c["train"]:
            keep.append((lo, hi, h, back))
    y = torch.zeros_like(x)
    for j in range(c["k"]):
        y += wt[:, j:j + 1] * y_rows[put[:, j]]
    if not c["train"]:
        return y
    dy = s["dy"].double()
    out = {"y": y, "dx": torch.zeros_like(x), "dw1": torch.zeros(s["w1"].shape, dtype=torch.float64, device=dev),
           "dw2": torch.zeros(s["w2"].shape, dtype=torch.float64, device=dev)}
    if s["b1"] is not None:
        out["db1"] = torch.zeros(s["b1"].shape, dtype=torch.float64, device=dev)
        out["db2"] = torch.zeros(s["b2"].shape, dtype=torch.float64, device=dev)
    dw = torch.zeros_like(wt)
    of_row = torch.zeros(n, dtype=torch.float64, device=dev)
    for j in range(c["k"]):
        dw[:, j] = (dy * y_rows[put[:, j]]).sum(1)
        of_row[put[:, j]] = wt[:, j]
    for e, (lo, hi, h, back) in enumerate(keep):
        tok = at[lo:hi]
        dr = dy[tok] * of_row[lo:hi, None]
        dz = back(dr @ s["w2"][e].double())
        out["dw2"][e] = dr.t() @ h
        out["dw1"][e] = dz.t() @ x[tok]
        out["dx"].index_add_(0, tok, dz @ s["w1"][e].double())
        if s["b1"] is not None:
            out["db1"][e] = dz.sum(0)
            out["db2"][e] = dr.sum(0)
    out["dlogits"] = _exact_dlogits(dw.cpu().numpy(), p, ids, "softmax", True, 1.0)
    return out
