"""The dense gated feed-forward block and the 8-bit integer products, as cases that can be timed.

A mixture-of-experts model has dense layers beside its expert layers, and linear maps around both. These
operators are what such a layer runs on its rows, and what trains it:

quantise         rows in bf16 or fp32 -> 8-bit integers, and one scale a row (a token): codes
                 round(127 x / max |x|) to the nearest, halves to even, scale max |x| / 127
project_int8     y = s_t c_o sum_k q_tk W_ok (+ addend), integers with a scale for each token and each output
                 channel; x comes quantised (several projections share it), or as rows that the call
                 quantises; plain, or with the gate/up product silu(g) * u
feed_forward     y = W2 (silu(Wg x) * (Wu x)) (+ residual); bf16 weights, for training with the gate and up
                 sums kept; or 8-bit integer weights, with x and the intermediate row quantised by the token
feed_forward_backward
                 the gradients of x, of [Wg; Wu] and of W2 from that of y and the kept sums

``own`` selects what run() computes them with: plain torch operations in 32 bits (64 where a rounding
to an integer decides), or the calls of this repository's package.
"""

from __future__ import annotations

import math

import torch

own = False


def listed() -> list[dict]:
    return [
        # one token before a decode projection: latency alone
        dict(name="quantise-token", op="quantise", rows=1, inner=4096, dtype="bfloat16"),
        # a long prompt batch of intermediate rows that were kept in fp32
        dict(name="quantise-long", op="quantise", rows=16384, inner=8192, dtype="float32"),
        # one token: the weights' bytes are the time
        dict(name="int8-token", op="project_int8", rows=1, inner=4096, outer=8192, swiglu=True, given="codes",
             addend=False, out="bfloat16"),
        # requests of an odd decode batch, quantised in the call, output fp32 (logits of a head)
        dict(name="int8-requests", op="project_int8", rows=27, inner=2560, outer=16000, swiglu=False, given="bfloat16",
             addend=False, out="float32"),
        # a prompt chunk, added to the residual
        dict(name="int8-chunk", op="project_int8", rows=777, inner=8192, outer=4096, swiglu=False, given="codes",
             addend=True, out="bfloat16"),
        # one token through the whole block
        dict(name="ff-token", op="feed_forward", rows=1, hidden=4096, inter=8192, wdtype="bf16", residual=True, keep=False),
        # a prompt chunk of an odd number of rows
        dict(name="ff-chunk", op="feed_forward", rows=1001, hidden=2560, inter=6912, wdtype="bf16", residual=True,
             keep=False),
        # decode requests over 8-bit weights
        dict(name="ff-int8-requests", op="feed_forward", rows=32, hidden=4096, inter=8192, wdtype="int8", residual=True,
             keep=False),
        # a training batch's forward pass, the gate and up sums kept
        dict(name="ff-train", op="feed_forward", rows=8192, hidden=4096, inter=8192, wdtype="bf16", residual=False,
             keep=True),
        # the backward pass of a short, odd batch: the weights' gradients are most of the bytes
        dict(name="ffb-short", op="feed_forward_backward", rows=203, hidden=2560, inter=6912),
        # the training batch's backward pass: all four products are large
        dict(name="ffb-train", op="feed_forward_backward", rows=8192, hidden=4096, inter=8192),
    ]


def draw(rng) -> dict:
    """One more case of the listed ranges; sizes over their logarithm, odd ones among them."""
    log = lambda a, b: max(a, min(b, round(math.exp(rng.uniform(math.log(a), math.log(b + 1))))))  # noqa: E731
    of = lambda step, a, b: step * max(1, round(log(a, b) / step))  # noqa: E731
    op = rng.choice(["quantise", "project_int8", "project_int8", "feed_forward", "feed_forward", "feed_forward_backward"])
    if op == "quantise":
        inner = of(8, 64, 16384)
        return dict(op=op, rows=min(log(1, 65536), 16384 * 8192 // inner), inner=inner,
                    dtype=rng.choice(["bfloat16", "float32"]))
    if op == "project_int8":
        swiglu = rng.random() < 0.4
        inner, outer = of(16, 128, 8192), of(8, 128, 8192 if swiglu else 16384)
        most = 8192 * 4096 * 8192 // (inner * outer)
        return dict(op=op, rows=min(log(1, 8192), max(1, most)), inner=inner, outer=outer, swiglu=swiglu,
                    given=rng.choice(["codes", "codes", "bfloat16"]), addend=not swiglu and rng.random() < 0.4,
                    out=rng.choice(["bfloat16", "bfloat16", "float32"]))
    wdtype = "int8" if op == "feed_forward" and rng.random() < 0.35 else "bf16"
    step = 16 if wdtype == "int8" else 8
    hidden, inter = of(step, 128, 8192), of(step, 128, 16384)
    rows = min(log(1, 8192), max(1, 8192 * 4096 * 8192 // (hidden * inter)))
    if op == "feed_forward":
        return dict(op=op, rows=rows, hidden=hidden, inter=inter, wdtype=wdtype, residual=rng.random() < 0.5,
                    keep=wdtype == "bf16" and rng.random() < 0.4)
    return dict(op=op, rows=rows, hidden=hidden, inter=inter)


# --------------------------------------------------------------------------- inputs


def _channels(w):
    """8-bit integers of a weight matrix and one scale for each of its rows (output channels)."""
    scale = w.abs().amax(1) / 127
    return torch.round(w / scale.clamp(min=1e-30)[:, None]).clamp(-127, 127).to(torch.int8), scale


def prepare(case: dict, seed: int) -> dict:
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    s, t = dict(case), case["rows"]
    if case["op"] in ("quantise", "project_int8"):
        # a few channels of activations are far larger than the others
        x = normal(t, case["inner"]) * torch.exp(0.7 * normal(case["inner"]))
        if case["op"] == "quantise":
            s["x"] = x.to(getattr(torch, case["dtype"]))
            return s
        s["x"] = x.bfloat16()
        if case["given"] == "codes":
            s["codes"], s["scale"] = _channels(s["x"].float())
        o = case["outer"] * (2 if case["swiglu"] else 1)
        s["w"], s["w_scale"] = _channels(normal(o, case["inner"]) / math.sqrt(case["inner"]))
        s["addend_values"] = normal(t, o).bfloat16() if case["addend"] else None
        return s
    h, i = case["hidden"], case["inter"]
    s["x"] = normal(t, h).bfloat16()
    w13, w2 = normal(2 * i, h) / math.sqrt(h), normal(h, i) / math.sqrt(i)
    if case["op"] == "feed_forward" and case["wdtype"] == "int8":
        s["w13"], s["s13"] = _channels(w13)
        s["w2"], s["s2"] = _channels(w2)
    else:
        s["w13"], s["w2"] = w13.bfloat16(), w2.bfloat16()
    if case["op"] == "feed_forward":
        s["residual_values"] = normal(t, h).bfloat16() if case["residual"] else None
    else:
        s["grad"] = (0.1 * normal(t, h)).bfloat16()
        s["gate_up"] = s["x"] @ s["w13"].t()  # what the forward pass kept
    return s


# --------------------------------------------------------------------------- the plain forms


def _plain_codes(x):
    """Codes, as the whole numbers that they are, and scales. The rounding decides: in 64 bits."""
    x = x.double()
    top = x.abs().amax(1, keepdim=True)
    q = torch.round(x * 127 / torch.where(top > 0, top, 1.0))
    return q.float(), (top[:, 0] / 127).float()


def _plain_silu(g):
    return g / (1 + torch.exp(-g))


def _plain_quantise(s):
    q, scale = _plain_codes(s["x"])
    return q * scale[:, None], scale


def _plain_product(q, scale, w, w_scale):
    return (q @ w.float().t()) * (scale[:, None] * w_scale)


def _plain_project_int8(s):
    q, scale = (s["codes"].float(), s["scale"]) if s["given"] == "codes" else _plain_codes(s["x"])
    y = _plain_product(q, scale, s["w"], s["w_scale"])
    if s["swiglu"]:
        g, u = y.chunk(2, dim=1)
        y = _plain_silu(g) * u
    if s["addend_values"] is not None:
        y = y + s["addend_values"].float()
    return y.to(getattr(torch, s["out"]))


def _plain_feed_forward(s):
    if s["wdtype"] == "int8":
        both = _plain_product(*_plain_codes(s["x"]), s["w13"], s["s13"])
    else:
        both = s["x"].float() @ s["w13"].float().t()
    g, u = both.chunk(2, dim=1)
    h = _plain_silu(g) * u
    y = _plain_product(*_plain_codes(h), s["w2"], s["s2"]) if s["wdtype"] == "int8" else h @ s["w2"].float().t()
    if s["residual_values"] is not None:
        y = y + s["residual_values"].float()
    return (y.bfloat16(), both.bfloat16()) if s["keep"] else y.bfloat16()


def _plain_feed_forward_backward(s):
    x, grad = s["x"].float(), s["grad"].float()
    g, u = s["gate_up"].float().chunk(2, dim=1)
    sig = 1 / (1 + torch.exp(-g))
    dh = grad @ s["w2"].float()
    both = torch.cat((dh * u * (sig + g * sig * (1 - sig)), dh * (g * sig)), 1)
    return (both @ s["w13"].float()).bfloat16(), (both.t() @ x).bfloat16(), (grad.t() @ (g * sig * u)).bfloat16()


# --------------------------------------------------------------------------- this repository's calls


def _own_quantise(s):
    from moe_decode_layer_gb300 import batch
    codes, scale = batch.quantise(s["x"])
    return codes * scale[:, None], scale


def _own_project_int8(s):
    from moe_decode_layer_gb300 import batch
    x = (s["codes"], s["scale"]) if s["given"] == "codes" else s["x"]
    return batch.project_int8(x, (s["w"], s["w_scale"]), addend=s["addend_values"], swiglu=s["swiglu"],
                              out_dtype=getattr(torch, s["out"]))


def _own_feed_forward(s):
    from moe_decode_layer_gb300 import batch
    if s["wdtype"] == "int8":
        return batch.feed_forward(s["x"], (s["w13"], s["s13"]), (s["w2"], s["s2"]), wdtype="int8",
                                  residual=s["residual_values"])
    if not s["keep"]:
        return batch.feed_forward(s["x"], s["w13"], s["w2"], residual=s["residual_values"])
    kept = torch.empty((s["rows"], 2 * s["inter"]), dtype=torch.bfloat16, device="cuda")
    return batch.feed_forward(s["x"], s["w13"], s["w2"], residual=s["residual_values"], gate_up=kept), kept


def _own_feed_forward_backward(s):
    from moe_decode_layer_gb300 import batch
    return batch.feed_forward_backward(s["grad"], s["x"], s["w13"], s["w2"], s["gate_up"])


def run(state: dict):
    if own:
        return {"quantise": _own_quantise, "project_int8": _own_project_int8, "feed_forward": _own_feed_forward,
                "feed_forward_backward": _own_feed_forward_backward}[state["op"]](state)
    return {"quantise": _plain_quantise, "project_int8": _plain_project_int8, "feed_forward": _plain_feed_forward,
            "feed_forward_backward": _plain_feed_forward_backward}[state["op"]](state)


# --------------------------------------------------------------------------- floors


def work(case: dict) -> dict:
    t = case["rows"]
    if case["op"] == "quantise":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": t * case["inner"] * (size + 1) + 4 * t, "flops": 3 * t * case["inner"]}
    if case["op"] == "project_int8":
        k, o = case["inner"], case["outer"]
        rows = o * (2 if case["swiglu"] else 1)
        x = t * (k + 4) if case["given"] == "codes" else 2 * t * k
        out = t * o * ((4 if case["out"] == "float32" else 2) + (2 if case["addend"] else 0))
        return {"bytes": rows * (k + 4) + x + out, "flops": 2 * t * k * rows}
    h, i = case["hidden"], case["inter"]
    if case["op"] == "feed_forward":
        weights = 3 * h * i + 4 * (2 * i + h) if case["wdtype"] == "int8" else 6 * h * i
        return {"bytes": weights + 2 * t * h * (3 if case["residual"] else 2) + (4 * t * i if case["keep"] else 0),
                "flops": 6 * t * h * i}
    # x, grad, dx; the kept sums; both weights and their gradients
    return {"bytes": 6 * t * h + 4 * t * i + 12 * h * i, "flops": 12 * t * h * i}


# --------------------------------------------------------------------------- the definitions in 64 bits


def _exact_codes(x):
    x = x.to(torch.float64)
    top = x.abs().max(dim=1, keepdim=True).values
    scale = top / 127
    # nearest whole number of steps, halves to the even one
    steps = torch.where(top > 0, 127 * x / torch.where(top > 0, top, torch.ones_like(top)), torch.zeros_like(x))
    low = torch.floor(steps)
    part = steps - low
    up = (part > 0.5) | ((part == 0.5) & (torch.remainder(low, 2) == 1))
    return low + up, scale


def _exact_swiglu(both, i):
    gate, up = both[:, :i], both[:, i:]
    return gate * torch.sigmoid(gate) * up


def _exact_int8(codes, scale, w, w_scale):
    return torch.matmul(codes, w.to(torch.float64).transpose(0, 1)) * scale * w_scale.to(torch.float64)


def exact(case: dict, seed: int):
    if work(case)["flops"] > 1e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "quantise":
        codes, scale = _exact_codes(s["x"])
        return codes * scale, scale[:, 0]
    if case["op"] == "project_int8":
        codes, scale = (s["codes"].double(), s["scale"].double()[:, None]) if case["given"] == "codes" else _exact_codes(s["x"])
        y = _exact_int8(codes, scale, s["w"], s["w_scale"])
        if case["swiglu"]:
            y = _exact_swiglu(y, case["outer"])
        return y + s["addend_values"].double() if case["addend"] else y
    i, x = case["inter"], s["x"].double()
    if case["op"] == "feed_forward":
        if case["wdtype"] == "int8":
            h = _exact_swiglu(_exact_int8(*_exact_codes(s["x"]), s["w13"], s["s13"]), i)
            y = _exact_int8(*_exact_codes(h), s["w2"], s["s2"])
        else:
            both = torch.matmul(x, s["w13"].double().transpose(0, 1))
            y = torch.matmul(_exact_swiglu(both, i), s["w2"].double().transpose(0, 1))
        if case["residual"]:
            y = y + s["residual_values"].double()
        return (y, both) if case["keep"] else y
    grad, gate, up = s["grad"].double(), s["gate_up"][:, :i].double(), s["gate_up"][:, i:].double()
    dh = torch.matmul(grad, s["w2"].double())
    sg = torch.sigmoid(gate)
    dgate, dup = dh * up * sg * (1 + gate * (1 - sg)), dh * gate * sg
    w13 = s["w13"].double()
    dx = torch.matmul(dgate, w13[:i]) + torch.matmul(dup, w13[i:])
    d13 = torch.cat((torch.matmul(dgate.transpose(0, 1), x), torch.matmul(dup.transpose(0, 1), x)))
    return dx, d13, torch.matmul(grad.transpose(0, 1), gate * sg * up)
