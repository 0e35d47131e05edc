"""Plain 64-bit forms of the layer norm and of the MXFP4 operators, for the
tests (CPU tensors), with what their arithmetic in the kernels may be off by."""
import torch

import _ffn_ref as ref

U = 2.0 ** -24   # half a step of binary32, relatively

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantize(x):
    """(q (M,P/2), scales (M,P/32)) of the rows of x, zeros up to whole blocks of 32, by the definition."""
    M, n = x.shape
    P = (n + 31) // 32 * 32
    b = torch.zeros(M, P, dtype=torch.float64)
    b[:, :n] = x.double()
    neg = torch.zeros(M, P, dtype=torch.bool)
    neg[:, :n] = torch.signbit(x)
    b = b.view(M, -1, 32)
    odd = ~torch.isfinite(b).all(2)
    top = torch.where(odd, torch.zeros_like(b[:, :, 0]), b.abs().amax(2))
    e = torch.full(top.shape, -127, dtype=torch.int64)
    for k in range(127 + 127):        # the least e with top <= 6 2^e
        e = torch.where((e < 127) & (top > 6.0 * 2.0 ** e.double()), e + 1, e)
    a = (b.abs() * 2.0 ** -e.double()[:, :, None]).view(M, P)
    # Nearest of the grid; halfway the one with an even code.
    d = (a[:, :, None] - GRID).abs()
    best = d.amin(2, keepdim=True)
    even = torch.arange(8) % 2 == 0
    hit = d == best
    code = torch.where((hit & even).any(2), (hit & even).int().argmax(2), hit.int().argmax(2))
    code = code + 8 * neg
    code = torch.where(odd.repeat_interleave(32, 1), torch.zeros_like(code), code)
    s = torch.where(odd, torch.full_like(e, 255), e + 127)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8), s.to(torch.uint8)


def values(q, s):
    """What they stand for (float64; NaN in blocks with scale 255)."""
    q = q.long()
    code = torch.stack((q & 15, q >> 4), -1).view(q.shape[0], 2 * q.shape[1])
    v = torch.cat((GRID, -GRID))[code]
    scale = torch.where(s == 255, torch.full_like(s, 0, dtype=torch.float64) / 0, 2.0 ** (s.double() - 127))
    return v * scale.repeat_interleave(32, 1)


def layer_norm(x, w, b, eps, dtype):
    """(y, its tolerance, mean, rstd, their tolerances).

    A sum of N values goes through at most D = 64 + N / 512 additions one after
    the other (a thread's own, 6 between lanes, 16 between waves), so it is off
    by D U of the sum of magnitudes; 1 / N's rounding adds one U, and so on."""
    x = x.double()
    M, N = x.shape
    D = 64 + N / 512
    w = torch.ones(N, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(N, dtype=torch.float64) if b is None else b.double()
    mu = x.mean(1, keepdim=True)
    dmu = (D + 2) * U * x.abs().mean(1, keepdim=True)
    c = x - mu
    dc = dmu + U * c.abs()
    var = (c * c).mean(1, keepdim=True)
    dvar = (2 * c.abs() * dc + dc * dc).mean(1, keepdim=True) + (D + 4) * U * var
    r = 1 / torch.sqrt(var + eps)
    dr = r * (dvar / (var + eps) + 6 * U)     # twice the half of dvar / var: room for its second order
    h, dh = c * r, dc * r + c.abs() * dr + U * (c * r).abs()
    y = h * w + b
    dy = dh * w.abs() + 2 * U * ((h * w).abs() + y.abs())
    return y, dy + ref.rounding(y, dtype) * 1.001, mu[:, 0], r[:, 0], dmu[:, 0] + U * mu[:, 0].abs(), dr[:, 0], h, dh


def layer_norm_backward(dout, x, w, eps, residual, dtype, wdtype):
    """{name: (value, tolerance)} of dx, dweight, dbias."""
    N = x.shape[1]
    M = x.shape[0]
    D = 64 + N / 512
    _, _, _, r, _, dr, h, dh = layer_norm(x, None, None, eps, dtype)
    r, dr = r[:, None], dr[:, None]
    d = dout.double()
    ww = torch.ones(N, dtype=torch.float64) if w is None else w.double()
    g = d * ww
    c0, c1 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dc0 = (D + 3) * U * g.abs().mean(1, keepdim=True)
    dc1 = (D + 4) * U * (g * h).abs().mean(1, keepdim=True) + (g.abs() * dh).mean(1, keepdim=True)
    i = g - c0 - h * c1
    di = dc0 + h.abs() * dc1 + dh * (c1.abs() + dc1) + 3 * U * (g.abs() + c0.abs() + (h * c1).abs())
    dx = r * i
    ddx = (r + dr) * di + dr * i.abs() + U * dx.abs()
    if residual is not None:
        dx = dx + residual.double()
        ddx = ddx + 2 * U * dx.abs()
    out = {"dx": (dx, ddx + ref.rounding(dx, dtype) * 1.001)}
    for name, v, dv in (("dweight", d * h, d.abs() * dh + U * (d * h).abs()), ("dbias", d, 0 * d)):
        s = v.sum(0)
        ds = dv.sum(0) + (M + 4) * U * v.abs().sum(0)
        out[name] = (s, ds + ref.rounding(s, wdtype) * 1.001)
    return out


def product(a, sa, b, sb, bias, name, residual, dtype):
    """As _ffn_ref.epilogue, of MXFP4 operands a, b (N,K/2)."""
    return ref.epilogue(values(a, sa), values(b, sb).t(), bias, name, residual, dtype)
