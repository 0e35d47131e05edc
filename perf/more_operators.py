"""The 4-bit feed-forward operators and the layer norm as they are measured:
the norm with its gradients, quantisation to MXFP4, the MXFP4 product with a
fused epilogue and the experts' MXFP4 products.

A case is a dict of plain values; prepare() makes its inputs from a seed,
run() makes one pass, exact() gives the same outputs in 64 bits and work()
what a pass cannot do without.  With ``own`` false run() takes the plain form
(elementary torch operations in 32 bits); with it true, the library's
operators.

MXFP4: blocks of 32 values along a row share a scale 2^e, kept as the byte
e + 127; an element is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign, code
0 .. 7 in the low three bits of a nibble, the first of two in the low one.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GATED = ("swiglu", "geglu")
EPS = 1e-5
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MOST_VALUES = 8192 * 4096                # of a drawn norm or quantisation
MOST_FLOPS = 2.0 * 32768 * 4096 * 2048   # of a drawn product


def _lib():
    import dense_tiled_gemm_bf16_amd as tg
    return tg


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _norm(name, m, n, dtype, wdtype, train=False, residual=False):
    c = {"op": "norm", "m": m, "n": n, "dtype": dtype, "wdtype": wdtype, "train": train, "residual": residual}
    return {"name": name, **c} if name else c


def _quant(name, m, n, dtype, columns):
    c = {"op": "quant", "m": m, "n": n, "dtype": dtype, "columns": columns}
    return {"name": name, **c} if name else c


def _product(name, m, n, k, dtype, act, bias, residual, train=False):
    c = {"op": "product", "m": m, "n": n, "k": k, "dtype": dtype, "act": act, "bias": bias, "residual": residual,
         "train": train}
    return {"name": name, **c} if name else c


def _experts(name, t, e, k, d, f, dtype, act, bias, down=False):
    """down: the second product of the layer (F -> D), its rows in the experts' order, else the first (D -> F)."""
    c = {"op": "experts", "t": t, "e": e, "k": k, "d": d, "f": f, "dtype": dtype, "act": act, "bias": bias,
         "down": down}
    return {"name": name, **c} if name else c


def listed():
    return [
        # The norm of a few decoded tokens: latency.
        _norm("norm_tokens", 8, 4096, "bf16", "bf16"),
        # A training step's norm over a long batch, the residual stream's gradient added.
        _norm("norm_train", 8192, 4096, "bf16", "f32", True, True),
        # Odd rows, a width that is no power of two, fp16.
        _norm("norm_ragged", 4093, 5000, "f16", "f16", True),
        # The rows of a long prompt on their way into a product, and back as a check of the layer would read them.
        _quant("quant_prompt", 8192, 4096, "bf16", False),
        # What a training step quantises: both orientations, binary32 values, odd rows.
        _quant("quant_train", 3999, 4992, "f32", True),
        # One new token through a projection: latency and the read of the 4-bit weight.
        _product("product_token", 1, 4096, 4096, "bf16", "silu", True, True),
        # A batch of decoded tokens through a gated layer's first product.
        _product("product_batch_gated", 48, 8192, 4096, "bf16", "swiglu", False, False),
        # The repository's benchmark shape with a whole epilogue.
        _product("product_prompt", 4096, 4096, 8192, "bf16", "gelu", True, True),
        # A training step of a linear layer in 4 bits: forward, then every gradient; odd rows.
        _product("product_train", 4001, 4096, 2048, "bf16", "none", True, False, True),
        # A batch of decoded tokens through the experts' first product, most of them hit by a few rows.
        _experts("experts_batch", 37, 64, 6, 2048, 1024, "bf16", "swiglu", False),
        # A prompt through the first product: every expert has about a thousand rows, unevenly.
        _experts("experts_prompt", 8192, 32, 4, 2048, 2048, "bf16", "swiglu", False),
        # The second product with its bias, a prompt's rows as the first one left them, fp16.
        _experts("experts_down", 1000, 16, 2, 2048, 1536, "f16", "gelu", True, True),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    while True:
        op = rng.choice(("norm", "quant", "product", "experts"))
        train = rng.random() < 0.4
        if op == "norm":
            dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
            case = _norm("", _log(rng, 1, 16384), _log(rng, 64, 16384, 8), dtype, rng.choice((dtype, "f32")), train,
                         rng.random() < 0.5)
            if case["m"] * case["n"] > MOST_VALUES:
                continue
            return case
        if op == "quant":
            case = _quant("", _log(rng, 1, 16384), _log(rng, 64, 16384, 32), rng.choice(("bf16", "bf16", "f16", "f32")),
                          train)
            if case["m"] * case["n"] > MOST_VALUES // 2:
                continue
            return case
        dtype = rng.choice(("bf16", "bf16", "f16"))
        if op == "product":
            act = "none" if train else rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu", "swiglu", "geglu"))
            # (A training step quantises both ways: whole blocks of the weight's rows, too.)
            case = _product("", _log(rng, 1, 8192), _log(rng, 128, 8192, 32 if train else 16), _log(rng, 128, 8192, 32),
                            dtype, act, rng.random() < 0.6, not train and rng.random() < 0.5, train)
        else:
            case = _experts("", _log(rng, 1, 8192), _log(rng, 4, 128), rng.randint(1, 4), _log(rng, 256, 4096, 32),
                            _log(rng, 128, 2048, 32), dtype, rng.choice(("swiglu", "geglu", "gelu", "relu")),
                            rng.random() < 0.4, rng.random() < 0.4)
            if case["e"] * case["d"] * case["f"] > 1 << 27:
                continue
        if work(case)["flops"] <= MOST_FLOPS:
            return case


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _power(e):
    """2^e in binary32, exactly, for whole e from -127 to 127."""
    return ((e + 1023).long() << 52).view(torch.float64).float()


def _plain_quantize(x):
    """The codes (sign in bit 3) and the scales' exponents of x's rows, padded with zeros to whole blocks."""
    r, c = x.shape
    pad = -c % 32
    if pad:
        x = torch.cat((x, torch.zeros(r, pad, dtype=x.dtype, device=x.device)), 1)
    b = x.float().reshape(r, -1, 32)
    m = b.abs().amax(2)
    f, e = torch.frexp(m)                    # m = f 2^e, f from 0.5 to below 1; 6 = 0.75 2^3
    e = torch.where(f > 0.75, e - 2, e - 3)
    e = torch.where(m > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    a = b * _power(-e)[:, :, None]
    neg = torch.signbit(a)
    a = a.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (code + 8 * neg).view(r, -1), e


def _plain_values(code, e):
    """What codes (R,C) and exponents (R,C/32) stand for, in binary32."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=code.device)
    return (grid[code.long()].view(e.shape[0], -1, 32) * _power(e)[:, :, None]).view(code.shape)


def _pack(code, e):
    """As bytes: two codes each, the scales."""
    c = code.to(torch.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _unpack(q, s):
    code = torch.stack((q & 15, q >> 4), -1).view(q.shape[0], -1)
    return _plain_values(code, s.int() - 127)


def _requantized(x):
    return _plain_values(*_plain_quantize(x))


def _act(z, act):
    if act in GATED:
        gate, up = z.chunk(2, dim=-1)
        return _act(gate, "silu" if act == "swiglu" else "gelu") * up
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z))


def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    n = x.shape[1]
    d = x - x.sum(1, keepdim=True) / n
    r = 1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / n + EPS)
    xh = d * r
    y = (xh * w + b).to(dt)
    if not c["train"]:
        return y
    dy = s["dy"].float()
    g = dy * w
    dx = r * (g - g.sum(1, keepdim=True) / n - xh * ((g * xh).sum(1, keepdim=True) / n))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return {"y": y, "dx": dx.to(dt), "dw": (dy * xh).sum(0).to(s["w"].dtype), "db": dy.sum(0).to(s["b"].dtype)}


def _plain_quant(s):
    x, dt = s["x"], s["out"]
    rows = _requantized(x).to(dt)
    return (rows, _requantized(x.t()).to(dt)) if s["case"]["columns"] else rows


def _plain_product(s):
    c, x = s["case"], s["x"]
    dt = x.dtype
    xq = _requantized(x)
    w = _requantized(s["w"]) if c["train"] else _unpack(s["wq"], s["ws"])
    z = xq @ w.t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(dt)
    if not c["train"]:
        return y
    dy = s["dy"]
    dyt, xt, wt = (_requantized(v.t()) for v in (dy, x, s["w"]))
    out = {"y": y, "dx": (_requantized(dy) @ wt.t()).to(dt), "dw": (dyt @ xt.t()).to(dt)}
    if s["bias"] is not None:
        out["dbias"] = dy.float().sum(0).to(dt)
    return out


def _plain_experts(s):
    c, x, dt = s["case"], s["x"], s["x"].dtype
    xq = _requantized(x)
    out = []
    lo = 0
    for e, hi in enumerate(s["ends"]):
        if hi > lo:
            a = xq[lo:hi] if c["down"] else xq[s["rows"][lo:hi].long()]
            z = a @ _unpack(s["wq"][e], s["ws"][e]).t()
            if s["bias"] is not None:
                z = z + s["bias"][e].float()
            out.append(z if c["down"] else _act(z, c["act"]))
        lo = hi
    return torch.cat(out).to(dt)


# --------------------------------------------------------------------------
# The library's operators
# --------------------------------------------------------------------------
def _own_norm(s):
    tg, c, x = _lib(), s["case"], s["x"]
    if not c["train"]:
        return tg.layer_norm(x, s["w"], s["b"], eps=EPS)
    mean = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    y = tg.layer_norm(x, s["w"], s["b"], eps=EPS, mean=mean, rstd=rstd)
    dx, dw, db = tg.layer_norm_backward(s["dy"], x, s["w"], mean, rstd, residual=s["res"])
    return {"y": y, "dx": dx, "dw": dw, "db": db}


def _own_quant(s):
    tg, c = _lib(), s["case"]
    if not c["columns"]:
        return tg.dequantize_mxfp4(*tg.quantize_mxfp4(s["x"]), dtype=s["out"])
    q, sc, qt, sct = tg.quantize_mxfp4(s["x"], columns=True)
    return tg.dequantize_mxfp4(q, sc, dtype=s["out"]), tg.dequantize_mxfp4(qt, sct, dtype=s["out"])


def _own_product(s):
    tg, c, x = _lib(), s["case"], s["x"]
    if not c["train"]:
        a, sa = tg.quantize_mxfp4(x)
        return tg.gemm_mxfp4_epilogue(a, s["wq"], sa, s["ws"], bias=s["bias"], act=c["act"], residual=s["residual"],
                                      dtype=x.dtype)
    a, sa, at, sat = tg.quantize_mxfp4(x, columns=True)
    w, sw, wt, swt = tg.quantize_mxfp4(s["w"], columns=True)
    d, sd, dtr, sdt = tg.quantize_mxfp4(s["dy"], columns=True)
    out = {"y": tg.gemm_mxfp4_epilogue(a, w, sa, sw, bias=s["bias"], dtype=x.dtype),
           "dx": tg.gemm_mxfp4_epilogue(d, wt, sd, swt, dtype=x.dtype),
           "dw": tg.gemm_mxfp4_epilogue(dtr, at, sdt, sat, dtype=x.dtype)}
    if s["bias"] is not None:
        out["dbias"] = tg.epilogue_backward(s["dy"], None, "none")[1]
    return out


def _own_experts(s):
    tg, c, x = _lib(), s["case"], s["x"]
    a, sa = tg.quantize_mxfp4(x)
    if c["down"]:
        return tg.gemm_mxfp4_grouped(a, s["wq"], sa, s["ws"], s["offsets"], bias=s["bias"], dtype=x.dtype)
    return tg.gemm_mxfp4_grouped(a, s["wq"], sa, s["ws"], s["offsets"], rows=s["rows"], bias=s["bias"], act=c["act"],
                                 dtype=x.dtype)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "quant": _own_quant, "product": _own_product, "experts": _own_experts}[op](state)
    return {"norm": _plain_norm, "quant": _plain_quant, "product": _plain_product, "experts": _plain_experts}[op](state)


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, rows, cols):
    """Values of a residual stream: some columns much larger than the others, rows of their own size."""
    x = _randn(g, rows, cols) * torch.exp(0.5 * _randn(g, rows, 1))
    return x * torch.exp(0.7 * _randn(g, cols))


def _weight(g, n, k):
    return _randn(g, n, k) / math.sqrt(k)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, dt = case, DT[case["dtype"]]
    s = {"case": case}
    if c["op"] == "norm":
        m, n, wt = c["m"], c["n"], DT[c["wdtype"]]
        s["x"] = (_activations(g, m, n) + 0.3 * _randn(g, m, 1)).to(dt)
        s["w"] = (1.0 + 0.2 * _randn(g, n)).to(wt)
        s["b"] = (0.1 * _randn(g, n)).to(wt)
        if c["train"]:
            s["dy"] = _randn(g, m, n).to(dt)
            s["res"] = _randn(g, m, n).to(dt) if c["residual"] else None
    elif c["op"] == "quant":
        s["x"] = _activations(g, c["m"], c["n"]).to(dt)
        s["out"] = torch.float32 if c["dtype"] == "f32" else torch.bfloat16   # either holds every value exactly
    elif c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        f = n // 2 if c["act"] in GATED else n
        # Rows as a norm leaves them, some columns larger.
        s["x"] = (_randn(g, m, k) * torch.exp(0.3 * _randn(g, k))).to(dt)
        s["bias"] = (0.5 * _randn(g, n)).to(dt) if c["bias"] else None
        s["residual"] = _randn(g, m, f).to(dt) if c["residual"] else None
        if c["train"]:
            s["w"] = _weight(g, n, k).to(dt)
            s["dy"] = _randn(g, m, n).to(dt)
        else:
            # A served weight is kept in 4 bits.
            s["wq"], s["ws"] = _pack(*_plain_quantize(_weight(g, n, k)))
    else:
        t, e, k, d, f = c["t"], c["e"], c["k"], c["d"], c["f"]
        rows = t * k
        n, kk = (d, f) if c["down"] else ((2 * f if c["act"] in GATED else f), d)
        s["x"] = _randn(g, rows if c["down"] else t, kk).to(dt)
        # The plan that the routing leaves: some experts are liked by most tokens.
        like = _randn(g, t, e) + 0.5 * _randn(g, e)
        ids = like.sort(dim=1, descending=True, stable=True).indices[:, :k]
        flat = ids.reshape(-1)
        order = flat.sort(stable=True).indices
        ends = torch.zeros(e, dtype=torch.int64, device="cuda").scatter_add_(0, flat, torch.ones_like(flat)).cumsum(0)
        s["offsets"] = torch.cat((ends.new_zeros(1), ends)).to(torch.int32)
        s["rows"] = (order // k).to(torch.int32)
        s["ends"] = ends.tolist()
        s["wq"] = torch.empty(e, n, kk // 2, dtype=torch.uint8, device="cuda")
        s["ws"] = torch.empty(e, n, kk // 32, dtype=torch.uint8, device="cuda")
        for i in range(e):
            s["wq"][i], s["ws"][i] = _pack(*_plain_quantize(_weight(g, n, kk)))
        s["bias"] = (0.5 * _randn(g, e, n)).to(dt) if c["bias"] else None
    return s


# --------------------------------------------------------------------------
# Work
# --------------------------------------------------------------------------
def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "norm":
        m, n, ws = c["m"], c["n"], 4 if c["wdtype"] == "f32" else 2
        nbytes = 2 * m * n * size + 2 * n * ws
        if c["train"]:
            # dy in, dx out, x once (a second read of it is none that has to be).
            nbytes += (3 if c["residual"] else 2) * m * n * size + 2 * n * ws
        return {"bytes": nbytes, "flops": (24.0 if c["train"] else 8.0) * m * n}
    if c["op"] == "quant":
        m, n = c["m"], c["n"]
        ways = 2 if c["columns"] else 1
        return {"bytes": m * n * (size + ways * (4 if c["dtype"] == "f32" else 2)), "flops": 4.0 * ways * m * n}
    bits = 17 / 32            # bytes of a value in MXFP4, its share of the scale with it
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        f = n // 2 if c["act"] in GATED else n
        nbytes = 2 * (m * k + m * f + (n if c["bias"] else 0) + (m * f if c["residual"] else 0))
        nbytes += 2 * n * k if c["train"] else int(bits * n * k)
        flops = 2.0 * m * n * k
        if c["train"]:
            nbytes += 2 * (m * n + m * k + n * k + (n if c["bias"] else 0))
            flops *= 3
        return {"bytes": nbytes, "flops": flops}
    t, e, k, d, f = c["t"], c["e"], c["k"], c["d"], c["f"]
    gated = c["act"] in GATED
    n, kk = (d, f) if c["down"] else ((2 * f if gated else f), d)
    hit = e * (1.0 - (1.0 - k / e) ** t)       # experts that uniform choices hit, on average
    nbytes = bits * hit * n * kk + (2 * hit * n if c["bias"] else 0)
    # Rows in and out: of the first product a token's row is read once, whoever takes it.
    nbytes += 2 * t * k * (f + d) if c["down"] else 2 * (t * d + t * k * f) + 4 * t * k
    return {"bytes": int(nbytes), "flops": 2.0 * t * k * n * kk}


# --------------------------------------------------------------------------
# The definition in 64 bits
# --------------------------------------------------------------------------
def _exact_blocks(x):
    """Nearest MXFP4 values of x's rows: steps of a half below 2, of 1 below 4, of 2 up to 6, halves to even."""
    r, c = x.shape
    b = torch.zeros(r, -(-c // 32) * 32, dtype=torch.float64, device=x.device)
    b[:, :c] = x.double()
    b = b.view(r, -1, 32)
    m = b.abs().amax(2, keepdim=True)
    scale = torch.full_like(m, 2.0 ** -127)
    # The least power of two whose sixfold reaches the largest value, found by steps of halved size.
    for p in (128, 64, 32, 16, 8, 4, 2, 1):
        far = 6.0 * scale * 2.0 ** (p - 1) < m
        scale = torch.where(far, scale * 2.0 ** p, scale)
    v = b / scale
    a = v.abs()
    near = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2)))
    return (torch.copysign(near, v) * scale).view(r, -1)


def _exact_stored(q, s):
    """Values of bytes, element by element from the format's definition: exponent bits 1-2, mantissa bit 0."""
    code = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.int64, device=q.device)
    code[:, 0::2] = q.long() % 16
    code[:, 1::2] = q.long() // 16
    man, ex, sign = code % 2, code // 2 % 4, code // 8
    mag = torch.where(ex == 0, 0.5 * man, (1 + 0.5 * man) * 2.0 ** (ex - 1).double())
    val = (1 - 2 * sign) * mag
    return val * (2.0 ** (s.double() - 127)).repeat_interleave(32, dim=1)


def _exact_act(z, act):
    if act in GATED:
        f = z.shape[1] // 2
        g = z[:, :f]
        return z[:, f:] * (g * torch.sigmoid(g) if act == "swiglu" else 0.5 * g * torch.erfc(-g / math.sqrt(2.0)))
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if act == "silu" else z


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        x, w = s["x"].double(), s["w"].double()
        var, mu = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        r = (var + EPS).rsqrt()
        xh = (x - mu) * r
        y = xh * w + s["b"].double()
        if not c["train"]:
            return y
        dy = s["dy"].double()
        g = dy * w
        dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if s["res"] is not None:
            dx = dx + s["res"].double()
        return {"y": y, "dx": dx, "dw": (dy * xh).sum(0), "db": dy.sum(0)}
    if c["op"] == "quant":
        rows = _exact_blocks(s["x"])
        return (rows, _exact_blocks(s["x"].t())) if c["columns"] else rows
    if c["op"] == "product":
        x = _exact_blocks(s["x"])
        w = _exact_blocks(s["w"]) if c["train"] else _exact_stored(s["wq"], s["ws"])
        z = torch.mm(x, w.t())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].double()
        if not c["train"]:
            return y
        dy = s["dy"]
        out = {"y": y, "dx": torch.mm(_exact_blocks(dy), _exact_blocks(s["w"].t()).t()),
               "dw": torch.mm(_exact_blocks(dy.t()), _exact_blocks(s["x"].t()).t())}
        if s["bias"] is not None:
            out["dbias"] = dy.double().sum(0)
        return out
    x = _exact_blocks(s["x"])
    off = s["offsets"].tolist()
    n = s["wq"].shape[1]
    z = torch.empty(off[-1], n, dtype=torch.float64, device=x.device)
    for e in range(c["e"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        a = x[lo:hi] if c["down"] else x.index_select(0, s["rows"][lo:hi].long())
        z[lo:hi] = torch.mm(a, _exact_stored(s["wq"][e], s["ws"][e]).t())
        if s["bias"] is not None:
            z[lo:hi] += s["bias"][e].double()
    return z if c["down"] else _exact_act(z, c["act"])
