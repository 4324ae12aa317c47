"""The many-row operators of a mixture-of-experts layer, as cases that can be timed.

Three operators that one layer runs one after another on a batch of any number of rows (a chunk of a
prompt, the rows of many requests, a wide verify batch):

route    router logits [T, E] -> the k chosen experts of each row and their weights: softmax or sigmoid
         scores, a selection bias, groups of experts of which the best are kept, masked experts
experts  out = residual + sum_j w_j W2_e (silu(Wg_e x) * (Wu_e x)) over the chosen experts e, plus shared
         experts that every row takes; bf16, FP8 (128 x 128 blocks) or NVFP4 (blocks of 16) weights
project  y = W x + s_a B_a (A_a x) (+ addend): one projection shared by all rows and, beside it, the
         low-rank adapter a of each row's request; plain, or with the gate/up product silu(g) * u

``own`` selects what run() computes them with: plain torch operations in 32 bits (64 where a comparison
decides), or the calls of this repository's package.
"""

from __future__ import annotations

import math

import torch
import torch.nn.functional as F

own = False

# Logits at or below this value stand for "this expert is not to be had" (masks of -inf or of a
# type's lowest value); so does NaN.
MASKED = -1e38

# Sizes: LING, MUSE and TINY are the layers of this repository's own workloads, the rest is generic.
LING = dict(hidden=2560, inter=768, num_experts=512, top_k=8)
MUSE = dict(hidden=4096, inter=1024, num_experts=256, top_k=8)
TINY = dict(hidden=256, inter=128, num_experts=16, top_k=2)


def listed() -> list[dict]:
    return [
        # one decoded token of a 512-expert layer: nothing but latency
        dict(name="route-token", op="route", rows=1, experts=512, top_k=8, score="softmax", dtype="float32",
             groups=1, top_groups=1, group_best=1, bias=False, renormalise=True, scale=1.0, masked=0),
        # a prompt chunk under the bias-corrected sigmoid rule, half of eight groups kept
        dict(name="route-chunk-groups", op="route", rows=4096, experts=256, top_k=8, score="sigmoid", dtype="float32",
             groups=8, top_groups=4, group_best=2, bias=True, renormalise=True, scale=2.5, masked=0),
        # an odd batch in bf16 (logits of bf16 tie often), some experts not to be had
        dict(name="route-odd-bf16", op="route", rows=777, experts=160, top_k=6, score="softmax", dtype="bfloat16",
             groups=8, top_groups=3, group_best=1, bias=False, renormalise=False, scale=16.0, masked=5),
        # the longest prompt batch: logits far larger than the caches' reach of one launch
        dict(name="route-long", op="route", rows=65536, experts=512, top_k=8, score="softmax", dtype="float32",
             groups=1, top_groups=1, group_best=1, bias=False, renormalise=True, scale=1.0, masked=0),
        # a few rows of a small layer: latency of the whole chain
        dict(name="experts-tiny", op="experts", rows=5, **TINY, shared=1, wdtype="bf16", padded=0),
        # just more rows than one decode step takes
        dict(name="experts-verify", op="experts", rows=24, **LING, shared=1, wdtype="bf16", padded=0),
        # a prompt chunk that touches all 512 experts: all weights are read for 16 rows each; padded tail
        dict(name="experts-chunk", op="experts", rows=1001, **LING, shared=1, wdtype="bf16", padded=9),
        # quantised weights
        dict(name="experts-chunk-fp8", op="experts", rows=300, **LING, shared=1, wdtype="fp8", padded=0),
        dict(name="experts-chunk-nvfp4", op="experts", rows=512, **MUSE, shared=0, wdtype="nvfp4", padded=0),
        # many rows for each expert: bound by the matrix products
        dict(name="experts-long", op="experts", rows=8192, hidden=2048, inter=1024, num_experts=64, top_k=8, shared=1,
             wdtype="bf16", padded=0),
        # decode: 32 requests with 24 adapters at the shared expert's gate/up projection
        dict(name="project-requests", op="project", rows=32, inner=2560, outer=768, swiglu=True, rank=16, adapters=64,
             requests=24, addend=False),
        # prompt chunks of seven requests at a down projection, ragged, added to the residual
        dict(name="project-chunk", op="project", rows=5003, inner=2048, outer=4096, swiglu=False, rank=64, adapters=16,
             requests=7, addend=True),
    ]


def draw(rng) -> dict:
    """One more case of the listed ranges; sizes over their logarithm, odd ones among them."""
    log = lambda a, b: max(a, min(b, round(math.exp(rng.uniform(math.log(a), math.log(b + 1))))))  # noqa: E731
    op = rng.choice(["route", "experts", "project"])
    if op == "route":
        e = rng.choice([8, 16, 60, 64, 96, 128, 160, 256, 384, 512, 1024])
        g = rng.choice([n for n in (1, 1, 2, 4, 8, 16) if e % n == 0 and e // n >= 2])
        tg = rng.randint(1, g)
        k = rng.randint(1, min(16, tg * (e // g)))
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op="route", rows=min(log(1, 65536), 65536 * 512 // e), experts=e, top_k=k, score=score,
                    dtype=rng.choice(["float32", "bfloat16"]), groups=g, top_groups=tg, group_best=rng.choice([1, 2]),
                    bias=rng.random() < 0.5, renormalise=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    masked=rng.choice([0, 0, e // 8]))
    if op == "experts":
        wdtype = rng.choice(["bf16", "bf16", "fp8", "nvfp4"])
        step = {"bf16": 8, "fp8": 128, "nvfp4": 256}[wdtype]
        hidden = step * round(log(256, 4096) / step)
        inter = step * max(1, round(log(128, 1024) / step))
        e = rng.choice([8, 16, 40, 64, 128, 256])
        k = rng.randint(1, min(8, e))
        most = int(8192 * 8 * 2048 * 1024 / (hidden * inter * k))
        return dict(op="experts", rows=min(log(1, 6000), max(1, most)), hidden=hidden, inter=inter, num_experts=e, top_k=k,
                    shared=rng.choice([0, 1, 2]) if k < 8 else 0, wdtype=wdtype, padded=rng.choice([0, 0, 1]))
    inner, outer = 8 * round(log(128, 4096) / 8), 8 * round(log(128, 4096) / 8)
    swiglu = rng.random() < 0.4
    rows = log(1, 6000)
    adapters = rng.choice([1, 4, 16, 64])
    return dict(op="project", rows=rows, inner=inner, outer=outer // 2 // 8 * 8 if swiglu else outer, swiglu=swiglu,
                rank=rng.choice([8, 16, 24, 32, 64, 128]) if adapters <= 16 else rng.choice([8, 16, 32]), adapters=adapters,
                requests=rng.randint(1, max(1, min(adapters, rows))), addend=not swiglu and rng.random() < 0.5)


# --------------------------------------------------------------------------- inputs


def _codes_fp4(w):
    """[..., K] -> e2m1 codes (two a byte, the even one low), e4m3 scales of 16, one fp32 scale for the last two dims."""
    ts = (w.abs().amax(dim=(-2, -1)) / (6 * 448)).clamp(min=1e-30)
    b = w.unflatten(-1, (-1, 16)) / ts[..., None, None, None]
    sc = (b.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    q = b / sc.float().clamp(min=2.0 ** -9)[..., None]
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    c = (torch.bucketize(q.abs(), mid) + 8 * (q < 0)).to(torch.uint8).flatten(-2)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), sc.view(torch.uint8), ts


def _codes_fp8(w):
    """[..., R, K] -> e4m3 codes and one fp32 scale for each 128 x 128 block."""
    b = w.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    sc = (b.abs().amax(dim=(-3, -1)) / 448).clamp(min=1e-30)
    q = (b / sc[..., :, None, :, None]).to(torch.float8_e4m3fn)
    return q.flatten(-2).flatten(-3, -2).view(torch.uint8).contiguous(), sc


def _weights(out, prefix, n, h, i, wdtype, g):
    """n experts' gate/up [2I, H] and down [H, I] matrices into ``out``, a few at a time."""
    per = max(1, (1 << 28) // (2 * h * i))
    parts: dict[str, list] = {}
    for s in range(0, n, per):
        m = min(per, n - s)
        for name, shape in (("w13", (m, 2 * i, h)), ("w2", (m, h, i))):
            w = torch.randn(shape, generator=g, device="cuda").mul_(0.02)
            if wdtype == "bf16":
                parts.setdefault(name, []).append(w.bfloat16())
            elif wdtype == "fp8":
                for key, t in zip(("_q", "_s"), _codes_fp8(w)):
                    parts.setdefault(name + key, []).append(t)
            else:
                halves = w.unflatten(1, (2, i)) if name == "w13" else w  # gate and up rows: a scale each
                q, sc, ts = _codes_fp4(halves)
                flat = (lambda t: t.flatten(1, 2)) if name == "w13" else (lambda t: t)
                for key, t in zip(("_q", "_s", "_gs"), (flat(q), flat(sc), ts)):
                    parts.setdefault(name + key, []).append(t)
    for name, t in parts.items():
        out[prefix + name] = torch.cat(t).contiguous() if len(t) > 1 else t[0].contiguous()


def prepare(case: dict, seed: int) -> dict:
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    t = case["rows"]
    if case["op"] == "route":
        e = case["experts"]
        l = normal(t, e) + 0.5 * normal(e)
        if case["masked"]:
            l[:, torch.randperm(e, generator=g, device="cuda")[:case["masked"]]] = -math.inf
        s["logits"] = l.to(getattr(torch, case["dtype"]))
        s["bias_values"] = 0.05 * normal(e) if case["bias"] else None
    elif case["op"] == "experts":
        h, i, e, k = case["hidden"], case["inter"], case["num_experts"], case["top_k"]
        w = s["weights"] = {}
        _weights(w, "", e, h, i, case["wdtype"], g)
        if case["shared"]:
            _weights(w, "sh_", case["shared"], h, i, case["wdtype"], g)
        s["x"] = normal(t, h).bfloat16()
        s["residual"] = normal(t, h).bfloat16()
        top = torch.topk(normal(t, e) + 0.5 * normal(e), k, dim=1)
        s["idx"] = top.indices.int()
        s["w"] = torch.softmax(top.values, 1)
        if case["padded"] and t > case["padded"]:  # rows of a padded batch have no expert
            s["idx"][t - case["padded"]:] = -1
    else:
        k, o, r, n = case["inner"], case["outer"] * (2 if case["swiglu"] else 1), case["rank"], case["adapters"]
        s["x"] = normal(t, k).bfloat16()
        s["weight"] = (0.02 * normal(o, k)).bfloat16()
        s["a"] = (normal(n, r, k) / math.sqrt(k)).bfloat16()
        s["b"] = (0.05 * normal(n, o, r)).bfloat16()
        s["scales"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        # rows of one request are adjacent and have one adapter; one request in eight has none
        q = case["requests"]
        request = torch.sort(torch.randint(q, (t,), generator=g, device="cuda")).values
        chosen = torch.randperm(n, generator=g, device="cuda")[torch.arange(q, device="cuda") % n]
        chosen[7::8] = -1
        s["ids"] = chosen[request].int()
        s["addend_values"] = normal(t, o).bfloat16() if case["addend"] else None
    return s


# --------------------------------------------------------------------------- the plain forms


def _plain_route(s):
    # comparisons decide here, so the scores are taken in 64 bits
    l = s["logits"].double()
    gone = ~(l > MASKED)
    l = l.masked_fill(gone, -math.inf)
    if s["score"] == "softmax":
        top = l.amax(1, keepdim=True).clamp(min=MASKED)
        p = torch.exp(l - top)
        score = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = torch.sigmoid(l)
    key = score if s["bias_values"] is None else score + s["bias_values"].double()
    key = key.masked_fill(gone, -math.inf)
    t, e = key.shape
    if s["top_groups"] < s["groups"]:
        of = torch.sort(key.view(t, s["groups"], -1), dim=2, descending=True).values[:, :, :s["group_best"]]
        value = of.masked_fill(of == -math.inf, 0).sum(2).masked_fill(of[:, :, 0] == -math.inf, -math.inf)
        best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, best, True)
        key = key.masked_fill(~kept.repeat_interleave(e // s["groups"], 1), -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    idx, there = order.indices[:, :s["top_k"]], order.values[:, :s["top_k"]] > -math.inf
    w = score.gather(1, idx) * there
    if s["renormalise"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return idx.masked_fill(~there, -1).int(), (w * s["scale"]).float()


def _values(w, name, wdtype, rows=None):
    """The 32-bit values of stored weights (those of the experts ``rows``)."""
    pick = (lambda t: t) if rows is None else (lambda t: t[rows])
    if wdtype == "bf16":
        return pick(w[name]).float()
    if wdtype == "fp8":
        q = pick(w[name + "_q"]).view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
        return (q * pick(w[name + "_s"])[..., :, None, :, None]).flatten(-2).flatten(-3, -2)
    c = pick(w[name + "_q"])
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=c.device)
    q = table[torch.stack((c & 15, c >> 4), -1).flatten(-2).int()]
    q = q.unflatten(-1, (-1, 16)) * pick(w[name + "_s"]).view(torch.float8_e4m3fn).float()[..., None]
    q, ts = q.flatten(-2), pick(w[name + "_gs"])
    if ts.dim() == 2:
        return (q.unflatten(1, (2, -1)) * ts[:, :, None, None]).flatten(1, 2)
    return q * ts[:, None, None]


def _mlp(x, w13, w2):
    g, u = torch.bmm(x, w13.transpose(1, 2)).chunk(2, dim=2)
    return torch.bmm(F.silu(g) * u, w2.transpose(1, 2))


def _plain_experts(s):
    x, idx, w, wdtype = s["x"].float(), s["idx"], s["w"], s["wdtype"]
    t, k = idx.shape
    # the pairs sorted by expert, each used expert's rows in a batch padded to the longest
    flat = idx.flatten().long()
    pair = torch.nonzero(flat >= 0).flatten()
    used, slot, count = torch.unique(flat[pair], return_inverse=True, return_counts=True)
    out = s["residual"].float()
    if pair.numel():
        order = torch.argsort(slot, stable=True)
        at = torch.arange(pair.numel(), device=x.device) - (count.cumsum(0) - count)[slot[order]]
        rows, slot = pair[order] // k, slot[order]
        xs = x.new_zeros(used.numel(), int(count.max()), x.shape[1])
        xs[slot, at] = x[rows]
        y = _mlp(xs, _values(s["weights"], "w13", wdtype, used), _values(s["weights"], "w2", wdtype, used))
        each = x.new_zeros(t * k, x.shape[1])
        each[pair[order]] = y[slot, at]
        out = out + (each.view(t, k, -1) * w[:, :, None]).sum(1)
    if s["shared"]:
        n = s["shared"]
        out = out + _mlp(x.expand(n, -1, -1), _values(s["weights"], "sh_w13", wdtype),
                         _values(s["weights"], "sh_w2", wdtype)).sum(0)
    return out.bfloat16()


def _plain_project(s):
    x, ids = s["x"].float(), s["ids"].long()
    n, r, k = s["a"].shape
    y = x @ s["weight"].float().t()
    # all adapters' first halves at once, each row keeping its own
    u = (x @ s["a"].float().view(n * r, k).t()).view(-1, n, r)
    mine = (ids[:, None] == torch.arange(n, device=x.device)).float() * s["scales"]
    y = y + (u * mine[:, :, None]).flatten(1) @ s["b"].float().transpose(1, 2).reshape(n * r, -1)
    if s["addend_values"] is not None:
        y = y + s["addend_values"].float()
    if s["swiglu"]:
        g, u = y.chunk(2, dim=1)
        y = F.silu(g) * u
    return y.bfloat16()


# --------------------------------------------------------------------------- this repository's calls


def _own_route(s):
    from moe_decode_layer_gb300 import batch
    return batch.route(s["logits"], s["top_k"], score=s["score"], bias=s["bias_values"], num_groups=s["groups"],
                       top_groups=s["top_groups"], group_best=s["group_best"], renormalise=s["renormalise"],
                       scale=s["scale"])


def _own_experts(s):
    from moe_decode_layer_gb300 import LayerShape, batch
    shape = LayerShape(s["hidden"], s["inter"], s["num_experts"], s["top_k"], s["shared"], s["wdtype"])
    return batch.experts(shape, s["weights"], s["x"], s["idx"], s["w"], residual=s["residual"])


def _own_project(s):
    from moe_decode_layer_gb300 import batch
    return batch.project(s["x"], s["weight"], adapters=batch.Adapters(s["a"], s["b"], s["scales"]),
                         adapter_ids=s["ids"], addend=s["addend_values"], swiglu=s["swiglu"])


def run(state: dict):
    if own:
        return {"route": _own_route, "experts": _own_experts, "project": _own_project}[state["op"]](state)
    return {"route": _plain_route, "experts": _plain_experts, "project": _plain_project}[state["op"]](state)


# --------------------------------------------------------------------------- floors


def work(case: dict) -> dict:
    t = case["rows"]
    if case["op"] == "route":
        e, k = case["experts"], case["top_k"]
        size = 4 if case["dtype"] == "float32" else 2
        # a score, a key and one comparison for each logit
        return {"bytes": t * e * size + 8 * t * k + (4 * e if case["bias"] else 0), "flops": 8 * t * e}
    if case["op"] == "experts":
        h, i, e, k, n = case["hidden"], case["inter"], case["num_experts"], case["top_k"], case["shared"]
        real = t - (case["padded"] if t > case["padded"] else 0)
        each = {"bf16": 6 * h * i, "fp8": 3 * h * i + 3 * h * i // 128 // 128 * 4, "nvfp4": 3 * h * i // 2 + 3 * h * i // 16}
        touched = e * (1 - (1 - k / e) ** real) + n
        return {"bytes": touched * each[case["wdtype"]] + 6 * t * h + 8 * t * k, "flops": 6 * h * i * (real * k + t * n)}
    k, o, r = case["inner"], case["outer"] * (2 if case["swiglu"] else 1), case["rank"]
    used = min(case["requests"] - case["requests"] // 8, case["adapters"], t)
    return {"bytes": 2 * (o * k + used * r * (k + o) + t * (k + case["outer"] + (o if case["addend"] else 0))) + 4 * t,
            "flops": 2 * t * (o * k + r * (k + o))}


# --------------------------------------------------------------------------- the definitions in 64 bits


def _exact_route(case, s):
    l = s["logits"].to(torch.float64)
    t, e = l.shape
    ok = l > MASKED
    if case["score"] == "softmax":
        score = torch.exp(torch.where(ok, l, l.new_tensor(-1e300)) - torch.logsumexp(torch.where(ok, l, l.new_tensor(-1e300)), 1, True))
    else:
        score = 1 / (1 + torch.exp(-torch.where(ok, l, l.new_tensor(0.0))))
    key = score + (s["bias_values"].to(torch.float64) if case["bias"] else 0.0)
    key = torch.where(ok, key, key.new_tensor(-math.inf))
    at = torch.arange(e, device=l.device).expand(t, e)

    def first_of_largest(v, pos):
        return torch.where(v == v.amax(1, True), pos, pos.shape[1]).amin(1)

    if case["top_groups"] < case["groups"]:
        size = e // case["groups"]
        rest, value = key.reshape(t * case["groups"], size).clone(), 0.0
        none = torch.isinf(rest.amax(1))
        for _ in range(min(case["group_best"], size)):
            best = rest.amax(1)
            value = value + torch.where(torch.isinf(best), best.new_zeros(()), best)
            rest.scatter_(1, first_of_largest(rest, at[:1, :size].expand_as(rest))[:, None], -math.inf)
        value = torch.where(none, value.new_tensor(-math.inf), value).view(t, -1).clone()
        keep = torch.zeros_like(value)
        for _ in range(case["top_groups"]):
            # a group that is taken is passed over from then on, also among groups of nothing
            left = torch.where(keep > 0, value.new_tensor(math.nan), value)
            top = torch.nan_to_num(left, nan=-math.inf, neginf=-1e300).masked_fill(keep > 0, -math.inf)
            keep.scatter_(1, first_of_largest(top, at[:, :case["groups"]])[:, None], 1.0)
        key = torch.where(keep.repeat_interleave(size, 1) > 0, key, key.new_tensor(-math.inf))
    idx, w = [], []
    for _ in range(case["top_k"]):
        there = ~torch.isinf(key.amax(1))
        i = first_of_largest(key, at)
        idx.append(torch.where(there, i, -1))
        w.append(torch.where(there, score.gather(1, i[:, None])[:, 0], 0.0))
        key = key.scatter(1, i[:, None], -math.inf)
    w = torch.stack(w, 1)
    if case["renormalise"]:
        total = w.sum(1, True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.stack(idx, 1).int(), case["scale"] * w


def _exact_matrix(w, name, wdtype, e):
    if wdtype == "bf16":
        return w[name][e].double()
    q = w[name + "_q"][e]
    if wdtype == "fp8":
        r, k = q.shape
        scale = w[name + "_s"][e].double()
        return q.view(torch.float8_e4m3fn).double() * scale.repeat_interleave(128, 0)[:r].repeat_interleave(128, 1)[:, :k]
    bits = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.int64, device=q.device)
    bits[:, 0::2], bits[:, 1::2] = (q & 15).long(), (q >> 4).long()
    ex, man = (bits >> 1) & 3, (bits & 1).double()
    v = torch.where(ex > 0, (1 + man / 2) * torch.exp2((ex - 1).double()), man / 2) * (1 - 2 * (bits >> 3)).double()
    v = v * w[name + "_s"][e].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    ts = w[name + "_gs"][e].double()
    if ts.dim():
        return v * ts.repeat_interleave(v.shape[0] // 2)[:, None]
    return v * ts


def _exact_mlp(x, w, prefix, wdtype, e):
    w13 = _exact_matrix(w, prefix + "w13", wdtype, e)
    i = w13.shape[0] // 2
    g, u = x @ w13[:i].t(), x @ w13[i:].t()
    return (g / (1 + torch.exp(-g)) * u) @ _exact_matrix(w, prefix + "w2", wdtype, e).t()


def _exact_experts(case, s):
    x, out, w = s["x"].double(), s["residual"].double(), s["weights"]
    for e in range(case["num_experts"]):
        row, j = torch.nonzero(s["idx"] == e, as_tuple=True)
        if row.numel():
            out.index_add_(0, row, s["w"][row, j].double()[:, None] * _exact_mlp(x[row], w, "", case["wdtype"], e))
    for e in range(case["shared"]):
        out += _exact_mlp(x, w, "sh_", case["wdtype"], e)
    return out


def _exact_project(case, s):
    x = s["x"].double()
    y = x @ s["weight"].double().t()
    for a in range(case["adapters"]):
        row = torch.nonzero(s["ids"] == a).flatten()
        if row.numel():
            y[row] += s["scales"][a].double() * ((x[row] @ s["a"][a].double().t()) @ s["b"][a].double().t())
    if case["addend"]:
        y += s["addend_values"].double()
    if case["swiglu"]:
        g, u = y[:, :case["outer"]], y[:, case["outer"]:]
        y = g / (1 + torch.exp(-g)) * u
    return y


def exact(case: dict, seed: int):
    if 100 * work(case)["flops"] > 1e14:
        return None
    s = prepare(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "project": _exact_project}[case["op"]](case, s)
