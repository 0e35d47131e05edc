"""Plain 64-bit forms of the feed-forward operators, for the tests (CPU
tensors), with what their arithmetic in the kernels may be off by."""
import math

import torch

GATED = ("swiglu", "geglu")
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step
#: Smallest normal value: below it half a step stops shrinking.
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -14, torch.float32: 2.0 ** -126}


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name in ("gelu", "geglu"):
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        # (1 + tanh u) / 2 = sigmoid(2 u), which keeps its digits where tanh is near -1.
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


def layer(z, name):
    if name in GATED:
        g, u = z.chunk(2, dim=-1)
        return act(g, name) * u
    return act(z, name)


def rounding(ref, dtype):
    """Half a step of dtype at ref."""
    return EPS[dtype] * ref.abs().clamp(min=TINY[dtype])


# Slopes of the activations are at most 1.13 (gelu's largest); their kernels'
# values are within 2^-17 of |z|, relatively: the exponential's argument is
# rounded to 24 bits at up to 128 octaves (2^-17), the fits are within 2^-19.
SLOPE, VALUE = 1.13, 2.0 ** -17


def product_error(a, b, bias=None):
    """Of a @ b + bias summed in 32 bits in any order: K + 1 roundings of
    partial sums no larger than the sum of magnitudes; twice that for
    instructions that keep fewer guard bits."""
    s = a.abs() @ b.abs()
    if bias is not None:
        s = s + bias.abs()
    return 2 * (a.shape[1] + 2) * 2.0 ** -24 * s


def layer_error(z, dz, name):
    """Of act(z) (times the other half) where z is off by dz."""
    if name in GATED:
        g, u = z.chunk(2, dim=-1)
        dg, du = dz.chunk(2, dim=-1)
        v = act(g, name).abs()
        dv = SLOPE * dg + VALUE * g.abs()
        return dv * (u.abs() + du) + v * du + 2.0 ** -23 * v * u.abs()
    if name in ("none", "relu"):
        return dz
    return SLOPE * dz + VALUE * z.abs()


def epilogue(a, b, bias, name, residual, dtype):
    """(out, its tolerance, z, its tolerance) of act(a b + bias) + residual."""
    a, b = a.double(), b.double()
    bias = None if bias is None else bias.double()
    z = a @ b if bias is None else a @ b + bias
    dz = product_error(a, b, bias)
    y = layer(z, name)
    dy = layer_error(z, dz, name)
    if residual is not None:
        y = y + residual.double()
        dy = dy + 2.0 ** -23 * (y.abs() + residual.double().abs())
    return y, dy + rounding(y, dtype) * 1.001, z, dz + rounding(z, dtype) * 1.001


def assert_near(got, ref, tol, what=""):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}, not {tuple(ref.shape)}"
    off = (got - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off by more than may be; worst "
                           f"{float((off / tol.clamp(min=1e-300))[bad].max()):.3g} times")


def topk(logits, k, score="softmax", bias=None, groups=1, used=1, renorm=True, scale=1.0):
    """(weights, ids) by the definition, row by row."""
    x = logits.double()
    T, E = x.shape
    w = torch.zeros(T, k, dtype=torch.float64)
    ids = torch.full((T, k), -1, dtype=torch.int64)
    for t in range(T):
        ok = ~(torch.isnan(x[t]) | (x[t] == -math.inf))
        if not ok.any():
            continue
        row = torch.where(ok, x[t], torch.full_like(x[t], -math.inf))
        # Value by value: an array's exponential may round the same number
        # differently in its last, partial vector, and equal logits would not tie.
        if score == "softmax":
            top = float(row.max())
            s = torch.tensor([1.0 if v == top else math.exp(v - top) for v in row.tolist()], dtype=torch.float64)
            s = s / s.sum()
        else:
            s = torch.tensor([1.0 / (1.0 + math.exp(-v)) if v > -700 else math.exp(max(v, -800.0)) for v in row.tolist()],
                             dtype=torch.float64)
        key = s if bias is None else s + bias.double()
        key = torch.where(ok & ~torch.isnan(key), key, torch.full_like(key, -math.inf))
        if groups > 1:
            per = E // groups
            sums = []
            for g in range(groups):
                two = sorted((v for v in key[g * per:(g + 1) * per].tolist() if v > -math.inf), reverse=True)[:2]
                sums.append(sum(two) if two else -math.inf)
            keep = sorted(range(groups), key=lambda g: (-sums[g], g))[:used]
            dropped = [g for g in range(groups) if g not in keep]
        else:
            per, dropped = E, []
        if bias is None:
            key = row.clone()          # the order of the scores, without their ties
        for g in dropped:
            key[g * per:(g + 1) * per] = -math.inf
        best = [e for e in sorted(range(E), key=lambda e: (-key[e].item(), e)) if key[e] > -math.inf][:k]
        at = torch.tensor(best, dtype=torch.int64)
        if not len(best):
            continue
        sel = s[at]
        if renorm and score == "softmax":
            c = row[at]
            sel = torch.where(c == c.max(), torch.ones_like(c), torch.exp(c - c.max()))
        v = sel / (sel.sum() + 1e-20) if renorm else sel
        ids[t, :len(best)] = at
        w[t, :len(best)] = v * scale
    return w, ids


def plan(ids, experts):
    """(offsets, rows, slots) by the definition."""
    T, k = ids.shape
    lists = [[] for _ in range(experts)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < experts:
            lists[e].append(i)
    offsets, rows = [0], []
    slots = torch.full((T * k,), -1, dtype=torch.int32)
    for l in lists:
        for i in l:
            slots[i] = len(rows)
            rows.append(i // k)
        offsets.append(len(rows))
    rows += [-1] * (T * k - len(rows))
    return (torch.tensor(offsets, dtype=torch.int32), torch.tensor(rows, dtype=torch.int32), slots.view(T, k))
