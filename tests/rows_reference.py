"""Plain 64-bit restatements of the many-row operators, with bounds on how far a
correct 32-bit / bf16 computation can be from them.

Roundings counted: bf16 is off by at most 2^-8 of the value (half a step), a sum of
n products in fp32 by n 2^-23 of the sum of their magnitudes (one step for each
addition), CUDA's exp and division by a few steps of fp32.
"""

import math

import torch

BF16, FP32 = 2.0 ** -8, 2.0 ** -23


def route(logits, k, score, bias=None, groups=1, kept=1, best=1, renormalise=True, scale=1.0):
    """(idx, w) as lists, row by row and by the definition; python floats are 64-bit."""
    idx, w = [], []
    size = logits.shape[1] // groups
    for row in logits.double().cpu().tolist():
        row = [min(v, 3e38) if v > -1e38 else -math.inf for v in row]  # NaN compares false
        live = [e for e, v in enumerate(row) if v > -math.inf]
        if score == "softmax":
            top = max((row[e] for e in live), default=0.0)
            total = math.fsum(math.exp(row[e] - top) for e in live)
            s = {e: math.exp(row[e] - top) / total for e in live}
        else:
            s = {e: 1 / (1 + math.exp(-row[e])) if row[e] > -700 else 0.0 for e in live}
        b = [0.0] * len(row) if bias is None else bias.double().cpu().tolist()
        key = {e: s[e] + b[e] for e in live}
        value = []
        for g in range(groups):
            of = sorted((key[e] for e in live if e // size == g), reverse=True)[:best]
            value.append(sum(of) if of else -math.inf)
        keep = sorted(range(groups), key=lambda g: (-value[g], g))[:kept]
        # without a bias the keys are ordered as the logits (also where 64 bits cannot tell the scores apart)
        order = sorted((e for e in live if e // size in keep),
                       key=lambda e: (-(row[e] if bias is None else key[e]), e))[:k]
        weights = [s[e] for e in order]
        if renormalise and order:
            if score == "sigmoid" and max(weights) < 1e-13:
                weights = [math.exp(row[e] - max(row[i] for i in order)) for e in order]
            total = math.fsum(weights)
            weights = [v / total for v in weights]
        idx.append(order + [-1] * (k - len(order)))
        w.append([scale * v for v in weights] + [0.0] * (k - len(order)))
    return torch.tensor(idx, dtype=torch.int32), torch.tensor(w, dtype=torch.float64)


def route_tolerance(logits, score, renormalise):
    """Relative: exp of a difference rounded to fp32 (its size times half a step), two steps each for exp and
    division, and one for each addition of the longest sum (a lane's share of E and 5 exchanges, or top_k)."""
    live = logits.float()[logits > -1e38]
    span = float(live.max() - live.min()) if live.numel() else 0.0
    span = min(span, 104.0)  # beyond it fp32 holds nothing of exp
    return (span + 16 + logits.shape[1] / 32 + 16) * FP32 / 2


def fp8(q, s):
    r, k = q.shape
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 0)[:r].repeat_interleave(128, 1)[:, :k]


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def nvfp4(q, s, ts):
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device=q.device)
    v = torch.stack((table[(q & 15).long()], table[(q >> 4).long()]), -1).flatten(1)
    v = v * s.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    ts = ts.double().reshape(-1)
    return v * ts.repeat_interleave(v.shape[0] // ts.numel())[:, None]


def matrix(layer, name, wdtype, e):
    if wdtype == "bf16":
        return layer[name][e].double()
    if wdtype == "fp8":
        return fp8(layer[name + "_q"][e], layer[name + "_s"][e])
    return nvfp4(layer[name + "_q"][e], layer[name + "_s"][e], layer[name + "_gs"][e])


def _gate_up(g, u, dg, du):
    """(silu(g) u, its bound) for sums off by dg and du: |silu'| <= 1.1; fp32 exp and divisions, bf16 result."""
    s = g * torch.sigmoid(g)
    h = s * u
    dh = 1.1 * dg * (u.abs() + du) + s.abs() * du + 16 * FP32 * (1 + g.abs()) * h.abs()
    return h, dh + BF16 * (h.abs() + dh)


def mlp(x, w13, w2, widened):
    """(y, bound): the kernels' bf16 intermediate, and where ``widened`` weights that were rounded to bf16."""
    i = w13.shape[0] // 2
    off = (BF16 if widened else 0.0) + w13.shape[1] * FP32
    both, mag = x @ w13.t(), x.abs() @ w13.abs().t()
    h, dh = _gate_up(both[:, :i], both[:, i:], off * mag[:, :i], off * mag[:, i:])
    off2 = (BF16 if widened else 0.0) + w2.shape[1] * FP32
    return h @ w2.t(), dh @ w2.abs().t() + off2 * ((h.abs() + dh) @ w2.abs().t())


def experts(shape, layer, x, idx, w, residual=None):
    """(out, bound) in 64 bits; bound covers the final rounding to bf16."""
    x = x.double()
    out = torch.zeros(x.shape[0], shape.hidden, dtype=torch.float64, device=x.device) if residual is None \
        else residual.double().clone()
    bound, mag = torch.zeros_like(out), out.abs()
    widened = shape.wdtype == "fp8"
    for t in range(idx.shape[1]):
        for e in range(shape.num_experts):
            rows = torch.nonzero(idx[:, t] == e).flatten()
            if rows.numel():
                y, d = mlp(x[rows], matrix(layer, "w13", shape.wdtype, e), matrix(layer, "w2", shape.wdtype, e), widened)
                f = w[rows, t].double()[:, None]
                out[rows] += f * y
                bound[rows] += f.abs() * d
                mag[rows] += (f * y).abs()
    for e in range(shape.num_shared):
        y, d = mlp(x, matrix(layer, "sh_w13", shape.wdtype, e), matrix(layer, "sh_w2", shape.wdtype, e), widened)
        out, bound, mag = out + y, bound + d, mag + y.abs()
    bound = bound + (2 * idx.shape[1] + 8) * FP32 * (mag + bound)
    return out, bound + BF16 * (out.abs() + bound)


def project(x, weight, adapters=None, ids=None, addend=None, swiglu=False, widened=False, bf16=True):
    """(out, bound) in 64 bits; ``weight`` holds 64-bit values."""
    x = x.double()
    k = x.shape[1]
    y, bound = x @ weight.t(), ((BF16 if widened else 0.0) + k * FP32) * (x.abs() @ weight.abs().t())
    if adapters is not None:
        for a in range(adapters.a.shape[0]):
            rows = torch.nonzero(ids == a).flatten()
            if not rows.numel():
                continue
            s = 1.0 if adapters.scale is None else float(adapters.scale[a])
            a_, b_ = adapters.a[a].double(), adapters.b[a].double()
            u = s * (x[rows] @ a_.t())
            du = (k + 2) * FP32 * abs(s) * (x[rows].abs() @ a_.abs().t())
            du = du + BF16 * (u.abs() + du)
            y[rows] += u @ b_.t()
            bound[rows] += (du + (b_.shape[1] + k) * FP32 * (u.abs() + du)) @ b_.abs().t()
    if addend is not None:
        y = y + addend.double()
    bound = bound + 4 * FP32 * (y.abs() + bound)
    if swiglu:
        o = y.shape[1] // 2
        return _gate_up(y[:, :o], y[:, o:], bound[:, :o], bound[:, o:])
    return y, bound + (BF16 if bf16 else 0.0) * (y.abs() + bound)
