"""Plain 64-bit restatements of the dense operators, with bounds on how far a correct 32-bit / bf16
computation can be from them. Roundings are counted as in rows_reference: bf16 2^-8 of the value, a
sum of n products in fp32 n 2^-23 of the sum of their magnitudes."""

import torch

from tests.rows_reference import BF16, FP32, _gate_up, mlp


def codes(x):
    """(int8, fp32): the nearest whole number of 127 x / max |x|, halves to the even one. The products and
    halves are exact in 64 bits, the quotient's rounding does not reach a half's neighbour."""
    x = x.double()
    top = x.abs().amax(1, keepdim=True)
    bad = ~torch.isfinite(x).all(1, keepdim=True)
    one = torch.ones_like(top)
    q = torch.round(torch.where(bad, 0.0, x) * 127 / torch.where((top > 0) & ~bad, top, one))
    # one rounding of the quotient. (No quotient of a 24-bit number by 127 is a half of an fp32 step -- 127 times an
    # odd 25-bit number is odd and longer -- nor within 2^-33 of one, so that rounding to 64 bits first changes nothing.
    # torch divides fp32 tensors by a number through its reciprocal, which does.)
    scale = (top[:, 0] / 127).float()
    return q.to(torch.int8), torch.where(bad[:, 0], torch.nan, scale)


def int8(q, s, w, c, addend=None, swiglu=False, bf16=True):
    """(out, bound) of a product of codes."""
    q, w = q.double(), w.double()
    scale = s.double()[:, None] * c.double()
    size = scale.abs()
    y, mag = (q @ w.t()) * scale, (q.abs() @ w.abs().t()) * size
    # whole sums below 2^24 are exact; above, a rounding at each of K additions. Two products with scales, their product
    bound = torch.where(mag <= 2.0 ** 24 * size, 0.0, q.shape[1] * FP32 * mag) + 4 * FP32 * y.abs()
    if swiglu:
        o = y.shape[1] // 2
        g, u, dg, du = y[:, :o], y[:, o:], bound[:, :o], bound[:, o:]
        h = g * torch.sigmoid(g) * u
        # |silu'| <= 1.1; fp32 exp (the argument's rounding counts by its size), two divisions, products
        y, bound = h, 1.1 * dg * (u.abs() + du) + (g * torch.sigmoid(g)).abs() * du + 16 * FP32 * (1 + g.abs()) * h.abs()
    if addend is not None:
        y = y + addend.double()
        bound = bound + FP32 * (y.abs() + bound)
    return y, bound + (BF16 if bf16 else FP32) * (y.abs() + bound)


def block(x, w13, w2, residual=None):
    """(out, bound, gate_up, its bound) of the bf16 block."""
    x, w13, w2 = x.double(), w13.double(), w2.double()
    both, mag = x @ w13.t(), x.abs() @ w13.abs().t()
    d = x.shape[1] * FP32 * mag
    y, bound = mlp(x, w13, w2, False)
    if residual is not None:
        y = y + residual.double()
        bound = bound + FP32 * (y.abs() + bound)
    return y, bound + BF16 * (y.abs() + bound), both, d + BF16 * (both.abs() + d)


def block_int8(x, w13, s13, w2, s2, residual=None):
    """The int8 block's out by the definition, and how far a code of h that falls the other way of a half
    (h is fp32) moves it: the codes' steps times the down weights, for values next to a half."""
    i = w13.shape[0] // 2
    h, dh = int8(*codes(x), w13, s13, swiglu=True, bf16=False)
    top = h.abs().amax(1, keepdim=True)
    v = torch.where(top > 0, h * 127 / torch.where(top > 0, top, 1.0), 0.0)
    off = torch.where(top > 0, 127 * (dh / torch.where(top > 0, top, 1.0) + v.abs() / 127 * (dh.amax(1, keepdim=True) / torch.where(top > 0, top, 1.0))), 0.0)
    near = ((v - torch.floor(v) - 0.5).abs() <= off + 1e-9).double()  # may be one step off
    q = torch.round(v)
    scale = top / 127 * s2.double()
    dscale = dh.amax(1, keepdim=True) / 127 * s2.double() + 2 * FP32 * scale
    y = (q @ w2.double().t()) * scale
    bound = (near @ w2.double().abs().t()) * scale + (q.abs() @ w2.double().abs().t()) * (dscale + i * FP32 * scale)
    if residual is not None:
        y = y + residual.double()
        bound = bound + FP32 * (y.abs() + bound)
    return y, bound + BF16 * (y.abs() + bound)


def gradients(grad, x, w13, w2, gate_up, bf16_weights=True, operand=BF16):
    """((dx, bound), (dw13, bound), (dw2, bound)); the bounds count dg, du and h rounded by `operand` (two bf16
    numbers: BF16 of what BF16 leaves)."""
    grad, x, w13, w2 = grad.double(), x.double(), w13.double(), w2.double()
    g, u = gate_up.double().chunk(2, 1)
    dh, e = grad @ w2, grad.shape[1] * FP32 * (grad.abs() @ w2.abs())
    sig = torch.sigmoid(g)
    r = 16 * FP32 * (1 + g.abs())  # sigmoid by fp32 exp and division, relative
    s, d = g * sig, sig + g * sig * (1 - sig)
    # of d: sig's error by (1 + |g|), and a rounding of each of its four operations on values of at most that
    ed = (r + 4 * FP32) * sig * (1 + g.abs())
    dg, du, h = dh * u * d, dh * s, s * u
    eg = u.abs() * (dh.abs() * ed + e * (d.abs() + ed)) + 4 * FP32 * dg.abs()
    eu = (dh.abs() * (r + 2 * FP32) + e * (1 + r)) * s.abs()
    eh = (r + 2 * FP32) * h.abs()
    both, eb = torch.cat((dg, du), 1), torch.cat((eg, eu), 1)
    eb, eh = eb + operand * (both.abs() + eb), eh + operand * (h.abs() + eh)
    last = BF16 if bf16_weights else FP32

    def product(a, ea, b, n, rounding):
        y = a @ b
        bound = ea @ b.abs() + n * FP32 * ((a.abs() + ea) @ b.abs())
        return y, bound + rounding * (y.abs() + bound)

    t = x.shape[0]
    dw2 = grad.t() @ h
    bound2 = grad.abs().t() @ eh + t * FP32 * (grad.abs().t() @ (h.abs() + eh))
    return (product(both, eb, w13, both.shape[1], BF16), product(both.t(), eb.t(), x, t, last),
            (dw2, bound2 + last * (dw2.abs() + bound2)))


def within(out, want, bound, floor=0.0):
    """Whether every value is; NaN where the definition has NaN."""
    out = out.double()
    nan = torch.isnan(want)
    return bool((torch.isnan(out) == nan).all()) and bool(((out - want).abs() <= bound + floor)[~nan].all())
