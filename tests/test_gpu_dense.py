"""The dense operators against 64-bit restatements: 8-bit rows and products, the gated block and its gradients."""

import pytest
import torch

from moe_decode_layer_gb300 import _lib, batch
from tests import dense_reference as ref

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *size, scale=1.0):
    return torch.randn(size, generator=g, device="cuda") * scale


def _bf16(g, *size, scale=1.0):
    return _normal(g, *size, scale=scale).bfloat16()


def _int8(g, rows, cols):
    """Codes of the whole range (-128 too) and scales, some of them zero or negative."""
    q = torch.randint(-128, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)
    s = _normal(g, rows, scale=0.01)
    s[::7] = 0
    return q, s


# --------------------------------------------------------------------------- rows to integers


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,inner", [(1, 8), (2, 16), (7, 1016), (9, 1024), (8, 1032), (33, 2048), (5, 2056), (3, 8200), (2, 65536),
                                        (512, 8), (600, 264), (513, 1032), (515, 2048), (520, 4096), (512, 4104)])
def test_quantise(dtype, rows, inner):
    x = (_normal(_gen(rows + inner), rows, inner) * torch.exp(_normal(_gen(1), inner))).to(dtype)
    q, s = batch.quantise(x)
    want, scale = ref.codes(x)
    assert torch.equal(q, want) and torch.equal(s, scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantise_values(dtype):
    """Halves, rows of zeros, single values, the ends of the type's range, values that are not finite."""
    big = torch.finfo(dtype).max
    tiny = torch.tensor([1], dtype=torch.int16 if dtype is torch.bfloat16 else torch.int32).view(dtype).item()  # the least subnormal
    rows = [[0.0] * 8, [-0.0] * 8, [1.0, 0.5, -0.5, 1 / 128, -1 / 128, 0.25, 0.75, -1.0], [127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5],
            [254, 1, 3, 5, -1, -3, -5, 253], [big, -big, big / 2, -big / 2, big / 256, 1.0, tiny, 0.0], [tiny, -tiny, 0, 0, 0, 0, 0, 0],
            [5 * tiny, tiny, 2 * tiny, 3 * tiny, 4 * tiny, -tiny, -2 * tiny, 0], [1e-30, 5e-31, -5e-31, 1e-32, 0, 0, 0, 0], [1e-38, 5e-39, -2.5e-39, 1e-40, 0, 0, 0, 0],
            [1e30, 5e29, 1e-30, -1e30, 0, 0, 0, 0], [3.0] * 8, [float("inf"), 1, 2, 3, 4, 5, 6, 7], [1, 2, 3, float("nan"), 5, 6, 7, 8],
            [float("-inf"), float("nan"), 0, 0, 0, 0, 0, 0]]
    x = torch.tensor(rows, dtype=torch.float64).to(dtype).cuda()
    q, s = batch.quantise(x)
    want, scale = ref.codes(x)
    assert torch.equal(q, want)
    assert torch.equal(s.nan_to_num(nan=-1.0), scale.nan_to_num(nan=-1.0))
    # every multiple of a half of a step, near and at it
    k = torch.arange(-254, 255, device="cuda").double() / 2
    x = torch.cat((k, torch.tensor([127.0] * 3, device="cuda")))[None].to(dtype)
    x = torch.cat((x, torch.nextafter(x.float(), x.float() * 2).to(dtype), torch.nextafter(x.float(), x.float() * 0).to(dtype)))
    x[:, -3:] = 127
    assert torch.equal(batch.quantise(x)[0], ref.codes(x)[0])


def test_quantise_strides_places_and_rows_behind():
    wide = _bf16(_gen(3), 21, 640)
    x = wide[:, 64:64 + 256]
    codes = torch.full((24, 256), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((24,), 99.0, device="cuda")
    q, s = batch.quantise(x, codes=codes[:21], scale=scale[:21])
    want, ws = ref.codes(x)
    assert q.data_ptr() == codes.data_ptr() and torch.equal(codes[:21], want) and torch.equal(scale[:21], ws)
    assert bool((codes[21:] == 99).all()) and bool((scale[21:] == 99).all())
    assert batch.quantise(x[:0])[0].shape == (0, 256)


# --------------------------------------------------------------------------- integer products

INT8 = [(1, 16, 8), (2, 128, 72), (5, 4096, 264), (8, 48, 4104), (9, 144, 200), (16, 1040, 136), (17, 16, 8), (31, 2048, 96),
        (64, 640, 1000), (100, 4096, 512), (128, 272, 264), (129, 1024, 72), (300, 208, 776), (512, 512, 256), (513, 16, 8),
        (700, 1008, 520), (1100, 256, 264),
        # rows on the weights' other side: one CTA a tile, and clusters of 2, 4 and 8
        (12, 400, 10008), (40, 1040, 6000), (33, 2064, 4008), (63, 3088, 1000), (96, 2064, 984), (127, 1168, 4504), (160, 784, 9736),
        (192, 2064, 3000), (250, 2320, 1032), (256, 16, 9800)]


@pytest.mark.parametrize("rows,inner,outer", INT8)
@pytest.mark.parametrize("swiglu", [False, True])
def test_project_int8(rows, inner, outer, swiglu):
    g = _gen(rows * 7 + inner)
    q, s = _int8(g, rows, inner)
    w, c = _int8(g, outer * (2 if swiglu else 1), inner)
    for out_dtype in (torch.bfloat16, torch.float32):
        addend = None if swiglu else _bf16(g, rows, outer)
        for a in {None, addend}:
            out = batch.project_int8((q, s), (w, c), addend=a, swiglu=swiglu, out_dtype=out_dtype)
            assert out.dtype is out_dtype
            assert ref.within(out, *ref.int8(q, s, w, c, a, swiglu, out_dtype is torch.bfloat16))


@pytest.mark.parametrize("rows", [3, 40, 600])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_project_int8_quantises_rows(rows, dtype):
    """Rows that the call quantises give the bits of rows that came quantised."""
    g = _gen(rows)
    x = _normal(g, rows, 528)[:, :512].to(dtype) if dtype is torch.float32 else _bf16(g, rows, 528)[:, :512]
    w = _int8(g, 264, 512)
    assert torch.equal(batch.project_int8(x, w), batch.project_int8(batch.quantise(x), w))


@pytest.mark.parametrize("rows", [8, 16, 100, 600])
def test_project_int8_long_sums(rows):
    """Sums of one sign far above 2^24, and the same weights with alternating signs: nothing is lost beyond fp32."""
    q = torch.full((rows, 16384), 127, dtype=torch.int8, device="cuda")
    w = torch.full((16, 16384), -128, dtype=torch.int8, device="cuda")
    w[8:, ::2] = 127
    s, c = torch.ones(rows, device="cuda"), torch.ones(16, device="cuda")
    out = batch.project_int8((q, s), (w, c), out_dtype=torch.float32)
    assert ref.within(out, *ref.int8(q, s, w, c, bf16=False))


@pytest.mark.parametrize("rows", [4, 12, 50, 520])
def test_project_int8_rows_are_their_own(rows):
    """A row with a NaN scale gives NaN, and no other row changes; rows behind the last stay as they were."""
    g = _gen(rows)
    q, s = _int8(g, rows, 272)
    w, c = _int8(g, 136, 272)
    want = batch.project_int8((q, s), (w, c))
    s2 = s.clone()
    s2[rows // 2] = float("nan")
    place = torch.full((rows + 40, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    out = batch.project_int8((q, s2), (w, c), out=place[:rows])
    keep = torch.arange(rows, device="cuda") != rows // 2
    assert bool(torch.isnan(out[rows // 2]).all()) and torch.equal(out[keep], want[keep])
    assert bool((place[rows:] == 7.0).all())


# --------------------------------------------------------------------------- the block

BLOCKS = [(1, 64, 8), (2, 8, 8), (7, 264, 136), (8, 1000, 520), (9, 128, 64), (15, 64, 2056), (16, 520, 1032), (17, 8, 8), (33, 72, 200),
          (64, 512, 264), (127, 256, 384), (128, 1032, 136), (129, 64, 64), (200, 328, 776), (256, 512, 512), (257, 128, 1000),
          (400, 2560, 768), (700, 200, 264), (1100, 136, 328),
          # a CTA a tile, and clusters of 2, 4 and 8; a second wave of CTAs
          (33, 9800, 40), (40, 1032, 5000), (70, 2056, 1040), (96, 4104, 520), (120, 72, 10008)]


def _block(g, hidden, inter):
    return _bf16(g, 2 * inter, hidden, scale=hidden ** -0.5), _bf16(g, hidden, inter, scale=inter ** -0.5)


@pytest.mark.parametrize("rows,hidden,inter", BLOCKS)
def test_feed_forward(rows, hidden, inter):
    g = _gen(rows + hidden)
    w13, w2 = _block(g, hidden, inter)
    x, residual = _bf16(g, rows, hidden), _bf16(g, rows, hidden)
    ws = torch.full((batch.feed_forward_workspace(hidden, inter, rows),), 255, dtype=torch.uint8, device="cuda")
    kept = torch.empty(rows, 2 * inter, dtype=torch.bfloat16, device="cuda")
    y, bound, both, near = ref.block(x, w13, w2, residual)
    out = batch.feed_forward(x, w13, w2, residual=residual, gate_up=kept, workspace=ws)
    assert batch.status(ws) == _lib.MOE_OK
    assert ref.within(out, y, bound) and ref.within(kept, both, near)
    y, bound, _, _ = ref.block(x, w13, w2)
    assert ref.within(batch.feed_forward(x, w13, w2, workspace=ws), y, bound)
    assert batch.status(ws) == _lib.MOE_OK


@pytest.mark.parametrize("rows,hidden,inter", [(1, 64, 16), (5, 512, 256), (12, 272, 128), (40, 256, 528), (300, 128, 144), (530, 512, 256)])
def test_feed_forward_int8(rows, hidden, inter):
    g = _gen(rows + inter)
    w13, w2 = batch.quantise(_normal(g, 2 * inter, hidden, scale=hidden ** -0.5)), batch.quantise(_normal(g, hidden, inter, scale=inter ** -0.5))
    x, residual = _bf16(g, rows, hidden), _bf16(g, rows, hidden)
    ws = torch.full((batch.feed_forward_workspace(hidden, inter, rows, wdtype="int8"),), 255, dtype=torch.uint8, device="cuda")
    for r in (None, residual):
        out = batch.feed_forward(x, w13, w2, wdtype="int8", residual=r, workspace=ws)
        assert batch.status(ws) == _lib.MOE_OK
        assert ref.within(out, *ref.block_int8(x, *w13, *w2, r))


@pytest.mark.parametrize("rows", [3, 12, 60, 300])
@pytest.mark.parametrize("wdtype", ["bf16", "int8"])
def test_feed_forward_strides_and_places(rows, wdtype):
    """A row stride, results in the residual's and in x's place, rows behind the last untouched."""
    g = _gen(rows)
    w13, w2 = _block(g, 256, 128)
    if wdtype == "int8":
        w13, w2 = batch.quantise(w13), batch.quantise(w2)
    wide = _bf16(g, rows, 264 + 256)
    x, residual = wide[:, 264:], _bf16(g, rows, 256)
    want = batch.feed_forward(x, w13, w2, wdtype=wdtype, residual=residual)
    place = torch.full((rows + 300, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    place[:rows] = residual
    assert torch.equal(batch.feed_forward(x, w13, w2, wdtype=wdtype, residual=place[:rows], out=place[:rows]), want)
    assert bool((place[rows:] == 7.0).all())
    same = x.contiguous()
    want = batch.feed_forward(same.clone(), w13, w2, wdtype=wdtype, residual=same.clone())
    assert torch.equal(batch.feed_forward(same, w13, w2, wdtype=wdtype, residual=same, out=same), want)
    if wdtype == "bf16":
        kept = torch.full((rows + 300, 256), 7.0, dtype=torch.bfloat16, device="cuda")
        batch.feed_forward(x, w13, w2, gate_up=kept[:rows])
        assert bool((kept[rows:] == 7.0).all())
    assert batch.feed_forward(x[:0], w13, w2, wdtype=wdtype).shape == (0, 256)


@pytest.mark.parametrize("rows", [4, 12, 50, 300])
def test_feed_forward_rows_are_their_own(rows):
    """What one row holds (an infinity, a NaN) reaches no other."""
    g = _gen(rows)
    w13, w2 = _block(g, 136, 72)
    x = _bf16(g, rows, 136)
    want = batch.feed_forward(x, w13, w2)
    bad = x.clone()
    bad[0, 3], bad[rows // 2, 100] = float("inf"), float("nan")
    out = batch.feed_forward(bad, w13, w2)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[0] = keep[rows // 2] = False
    assert torch.equal(out[keep], want[keep]) and not bool(torch.isfinite(out[~keep]).any())


# --------------------------------------------------------------------------- gradients


@pytest.mark.parametrize("rows,hidden,inter", BLOCKS)
def test_backward(rows, hidden, inter):
    g = _gen(rows + inter)
    w13, w2 = _block(g, hidden, inter)
    x, grad = _bf16(g, rows, hidden), _bf16(g, rows, hidden, scale=0.3)
    kept = torch.empty(rows, 2 * inter, dtype=torch.bfloat16, device="cuda")
    batch.feed_forward(x, w13, w2, gate_up=kept)
    ws = torch.full((batch.feed_forward_backward_workspace(hidden, inter, rows),), 255, dtype=torch.uint8, device="cuda")
    found = batch.feed_forward_backward(grad, x, w13, w2, kept, workspace=ws)
    assert batch.status(ws) == _lib.MOE_OK
    for out, (want, bound) in zip(found, ref.gradients(grad, x, w13, w2, kept)):
        assert out.dtype is torch.bfloat16 and ref.within(out, want, bound)
    # fp32 weight gradients, and added to what was there
    d13, d2 = _normal(g, 2 * inter, hidden), _normal(g, hidden, inter)
    b13, b2 = d13.clone(), d2.clone()
    batch.feed_forward_backward(grad, x, w13, w2, kept, dw13=d13, dw2=d2, input_grad=False, workspace=ws)
    want = ref.gradients(grad, x, w13, w2, kept, bf16_weights=False)[1:]
    assert all(ref.within(d, *w) for d, w in zip((d13, d2), want))
    once = d13.clone(), d2.clone()
    d13.copy_(b13), d2.copy_(b2)
    batch.feed_forward_backward(grad, x, w13, w2, kept, dw13=d13, dw2=d2, accumulate=True, workspace=ws)
    assert torch.equal(d13, b13 + once[0]) and torch.equal(d2, b2 + once[1])  # one rounding of the same sum
    assert batch.status(ws) == _lib.MOE_OK


@pytest.mark.parametrize("rows,hidden,inter", [(1, 64, 8), (3, 1032, 136), (7, 264, 136), (15, 64, 2056), (17, 8, 72), (200, 8, 264), (512, 8, 8)])
def test_backward_of_few_rows_keeps_two_numbers(rows, hidden, inter):
    """dg, du and h as two bf16 numbers each: the gradients' errors are those of rounding by 2^-16 and of fp32 sums
    of twice the products."""
    g = _gen(rows)
    w13, w2 = _block(g, hidden, inter)
    x, grad, kept = _bf16(g, rows, hidden), _bf16(g, rows, hidden), _bf16(g, rows, 2 * inter)
    d13, d2 = torch.empty(2 * inter, hidden, device="cuda"), torch.empty(hidden, inter, device="cuda")
    dx, _, _ = batch.feed_forward_backward(grad, x, w13, w2, kept, dw13=d13, dw2=d2)
    want = ref.gradients(grad, x, w13, w2, kept, bf16_weights=False, operand=ref.BF16 ** 2 + 2 * max(rows, 2 * inter) * ref.FP32)
    assert all(ref.within(d, *w) for d, w in zip((dx, d13, d2), want))
    # an infinite dh stays one (no inf - inf in its second number); an infinite grad meets h's second number, of either sign
    grad[0], grad[0, 0] = 0, float("inf")
    w2[0], kept[0], x[0] = w2[0].abs() + 0.125, kept[0].abs() + 0.125, x[0].abs() + 0.125
    batch.feed_forward_backward(grad, x, w13, w2, kept, dw13=d13, dw2=d2)
    assert bool((d13 == float("inf")).all()) and bool(torch.isfinite(d2[1:]).all()) and not bool(torch.isfinite(d2[0]).any())


def test_gradients_against_differences():
    """The loss along random directions of x, W13 and W2, in 64 bits, against the gradients' products with them."""
    g = _gen(5)
    rows, hidden, inter = 40, 72, 136
    w13, w2 = _block(g, hidden, inter)
    x, grad = _bf16(g, rows, hidden), _bf16(g, rows, hidden)
    kept = (x.double() @ w13.double().t()).bfloat16()
    # the kept sums are rounded: differences are taken of the block whose first product gives just them
    g0, u0 = kept.double().chunk(2, 1)

    def loss(dx, d13, d2):
        both = kept.double() + dx @ w13.double().t() + x.double() @ d13.t()
        a, b = both.chunk(2, 1)
        return float(((a * torch.sigmoid(a) * b) @ (w2.double() + d2).t() * grad.double()).sum())

    found = batch.feed_forward_backward(grad, x, w13, w2, kept)
    bounds = [b for _, b in ref.gradients(grad, x, w13, w2, kept)]
    zero = [torch.zeros_like(t.double()) for t in (x, w13, w2)]
    for k in range(3):
        for seed in range(4):
            v = torch.randn(zero[k].shape, generator=_gen(100 + seed), device="cuda", dtype=torch.float64)
            step = 1e-6
            plus, minus = list(zero), list(zero)
            plus[k], minus[k] = step * v, -step * v
            slope = (loss(*plus) - loss(*minus)) / (2 * step)
            got = float((found[k].double() * v).sum())
            # what each value may be off by, and the difference's own error: third derivatives times step^2 and 2^-52 / step
            assert abs(got - slope) <= float((bounds[k] * v.abs()).sum()) + 1e-5 * (1 + abs(slope))


@pytest.mark.parametrize("rows", [6, 60, 300])
def test_backward_strides_places_and_parts(rows):
    g = _gen(rows)
    w13, w2 = _block(g, 136, 72)
    wide, wide2 = _bf16(g, rows, 400), _bf16(g, rows, 400)
    x, grad = wide[:, 8:144], wide2[:, 200:336]
    kept = _bf16(g, rows, 144)
    want = batch.feed_forward_backward(grad.contiguous(), x.contiguous(), w13, w2, kept)
    place = torch.full((rows + 300, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    found = batch.feed_forward_backward(grad, x, w13, w2, kept, dx=place[:rows])
    assert all(torch.equal(a, b) for a, b in zip(found, want)) and bool((place[rows:] == 7.0).all())
    dx, none13, none2 = batch.feed_forward_backward(grad, x, w13, w2, kept, weight_grad=False)
    assert torch.equal(dx, want[0]) and none13 is None and none2 is None
    none, d13, d2 = batch.feed_forward_backward(grad, x, w13, w2, kept, input_grad=False)
    assert none is None and torch.equal(d13, want[1]) and torch.equal(d2, want[2])


@pytest.mark.parametrize("rows", [5, 300])
def test_one_weight_gradient(rows):
    """A call that asks for one matrix's gradient alone gives the bits of the whole one."""
    g = _gen(rows)
    w13, w2 = _block(g, 136, 72)
    x, grad, kept = _bf16(g, rows, 136), _bf16(g, rows, 136), _bf16(g, rows, 144)
    _, want13, want2 = batch.feed_forward_backward(grad, x, w13, w2, kept)
    ws = torch.empty(batch.feed_forward_backward_workspace(136, 72, rows), dtype=torch.uint8, device="cuda")
    weights = _lib.FfWeights(w13.data_ptr(), w2.data_ptr(), None, None)
    for want, places in ((want13, lambda d: (None, d.data_ptr(), None)), (want2, lambda d: (None, None, d.data_ptr()))):
        d = torch.full_like(want, 7.0)
        assert _lib.load().moe_decode_ff_backward(
            _lib.FfConfig(136, 72, 0), weights, grad.data_ptr(), 136, x.data_ptr(), 136, kept.data_ptr(), *places(d), 0, 0, rows,
            ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == _lib.MOE_OK
        assert torch.equal(d, want)


def test_backward_without_rows():
    w13, w2 = _block(_gen(1), 64, 72)
    x, kept = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 144, dtype=torch.bfloat16, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        d13, d2 = torch.ones(144, 64, dtype=dtype, device="cuda"), torch.ones(64, 72, dtype=dtype, device="cuda")
        dx, _, _ = batch.feed_forward_backward(x, x, w13, w2, kept, dw13=d13, dw2=d2)
        assert dx.shape == (0, 64) and not bool(d13.any()) and not bool(d2.any())
    d13, d2 = torch.ones(144, 64, device="cuda"), torch.ones(64, 72, device="cuda")
    batch.feed_forward_backward(x, x, w13, w2, kept, dw13=d13, dw2=d2, accumulate=True)
    assert bool((d13 == 1).all()) and bool((d2 == 1).all())


def test_saturated_gates():
    """Gates far out on both sides: the gradient ends at 0 or at dh u, and nothing overflows."""
    g = _gen(2)
    w13, w2 = _block(g, 64, 64)
    x, grad = _bf16(g, 32, 64), _bf16(g, 32, 64)
    kept = _bf16(g, 32, 128)
    kept[:, :8], kept[:, 8:16], kept[:, 16:24], kept[:, 24:32] = -1e4, 1e4, -95.0, 95.0
    for out, (want, bound) in zip(batch.feed_forward_backward(grad, x, w13, w2, kept), ref.gradients(grad, x, w13, w2, kept)):
        # fp32's sigmoid is 0 from exp(-g) = 2^126 on (g = -87.3): silu and its slope lose at most 89 * 2^-126 there
        assert ref.within(out, want, bound, floor=1e-30)


# --------------------------------------------------------------------------- streams, graphs, long offsets


def _calls(rows):
    """A training step over the block, and an int8 block, as callables over buffers of their own."""
    g = _gen(rows)
    w13, w2 = _block(g, 264, 136)
    q13, q2 = batch.quantise(_normal(g, 544, 272)), batch.quantise(_normal(g, 272, 272))
    x, grad, x8 = _bf16(g, rows, 264), _bf16(g, rows, 264), _bf16(g, rows, 272)
    kept = torch.empty(rows, 272, dtype=torch.bfloat16, device="cuda")
    bufs = dict(out=torch.empty_like(x), dx=torch.empty_like(x), dw13=torch.empty_like(w13), dw2=torch.empty_like(w2), out8=torch.empty_like(x8))
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
        batch.feed_forward_workspace(264, 136, rows), batch.feed_forward_backward_workspace(264, 136, rows),
        batch.feed_forward_workspace(272, 272, rows, wdtype="int8"))]

    def step(stream=None):
        batch.feed_forward(x, w13, w2, residual=x, gate_up=kept, out=bufs["out"], workspace=ws[0], stream=stream)
        batch.feed_forward_backward(grad, x, w13, w2, kept, dx=bufs["dx"], dw13=bufs["dw13"], dw2=bufs["dw2"], workspace=ws[1], stream=stream)
        batch.feed_forward(x8, q13, q2, wdtype="int8", residual=x8, out=bufs["out8"], workspace=ws[2], stream=stream)
    return step, (x, grad, x8), bufs, ws


@pytest.mark.parametrize("rows", [5, 40, 300, 700])
def test_calls_are_repeatable_and_captured(rows):
    """The same bits again, on another stream, and from a graph with new inputs; two graphs side by side."""
    one, two = _calls(rows), _calls(rows + 1)
    for step, _, bufs, _ in (one, two):
        step()
    torch.cuda.synchronize()
    want = [{n: t.clone() for n, t in c[2].items()} for c in (one, two)]
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for c in (one, two):
        for t in c[2].values():
            t.fill_(5)
    torch.cuda.synchronize()
    for _ in range(3):
        one[0](s), two[0](s2)
    torch.cuda.synchronize()
    for c, w in zip((one, two), want):
        assert all(torch.equal(t, w[n]) for n, t in c[2].items())
    graphs = []
    for c in (one, two):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c[0]()
        graphs.append(graph)
    # new inputs: each graph has the other's size, so compare with an eager run on the same
    for c in (one, two):
        for t in c[1]:
            t.mul_(-0.5)
    with torch.cuda.stream(s):
        graphs[0].replay()
    with torch.cuda.stream(s2):
        graphs[1].replay()
    torch.cuda.synchronize()
    found = [{n: t.clone() for n, t in c[2].items()} for c in (one, two)]
    for c, f in zip((one, two), found):
        c[0]()
        torch.cuda.synchronize()
        assert all(torch.equal(t, f[n]) for n, t in c[2].items())
        assert all(batch.status(w) == _lib.MOE_OK for w in c[3])


def test_offsets_past_32_bits():
    """More than 2^31 kept sums and gradients; rows from the start, the middle and the end."""
    rows, hidden, inter = 70001, 64, 16384
    g = _gen(9)
    w13, w2 = _block(g, hidden, inter)
    x, grad = _bf16(g, rows, hidden), _bf16(g, rows, hidden)
    kept = torch.empty(rows, 2 * inter, dtype=torch.bfloat16, device="cuda")
    out = batch.feed_forward(x, w13, w2, gate_up=kept)
    dx, d13, d2 = batch.feed_forward_backward(grad, x, w13, w2, kept)
    for part in (slice(0, 40), slice(34990, 35010), slice(rows - 41, rows)):
        y, bound, both, near = ref.block(x[part], w13, w2)
        assert ref.within(out[part], y, bound) and ref.within(kept[part], both, near)
        assert ref.within(dx[part], *ref.gradients(grad[part], x[part], w13, w2, kept[part])[0])
    # weight gradients as a sum over parts of the rows
    total = [0, 0, 0, 0]
    for r in range(0, rows, 8192):
        p = slice(r, r + 8192)
        for k, (v, b) in enumerate(ref.gradients(grad[p], x[p], w13, w2, kept[p])[1:]):
            total[2 * k], total[2 * k + 1] = total[2 * k] + v, total[2 * k + 1] + b
    assert ref.within(d13, total[0], total[1]) and ref.within(d2, total[2], total[3])


def test_int8_offsets_past_32_bits():
    rows, inner = 140000, 16384
    g = _gen(4)
    q = torch.randint(-128, 128, (rows, inner), generator=g, device="cuda", dtype=torch.int8)
    s, (w, c) = _normal(g, rows), _int8(g, 64, inner)
    out = batch.project_int8((q, s), (w, c))
    for part in (slice(0, 30), slice(131060, 131090), slice(rows - 30, rows)):
        assert ref.within(out[part], *ref.int8(q[part], s[part], w, c))
