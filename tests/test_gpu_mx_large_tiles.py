"""4-bit projections by tiles of 256 outputs by 256 rows, which calls of 1,024 tiles of 128 or more take (rows and outputs in
128s, rounded up, by each other), against the 64-bit definition.

The reduction goes through two buffers in turn, in steps of 256 values: one step, whole steps and a short last one behind
whole ones, with rows and outputs that end inside a tile, next to its end, and at it."""
import math

import pytest
import torch

import more_operators_ref as ref
import test_gpu_mx as mx

pytestmark = pytest.mark.gpu

SIZES = [(4100, 1100, 4100), (2049, 2112, 8200), (4096, 768, 4096), (8193, 250, 2047), (4351, 513, 4097)]


def want_of(x, codes, scales, bias):
    """As test_gpu_mx has it, with the 64-bit product on the GPU."""
    K = x.shape[1]
    xv = ref.mx_values(*ref.mx_quantize(x), K).cuda()
    w = ref.mx_values(codes, scales, K).cuda().t().contiguous()
    y, size = xv @ w, xv.abs() @ w.abs()
    return (y, size) if bias is None else (y + bias.double().cuda(), size + bias.double().abs().cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows, K, O", SIZES)
def test_project(rows, K, O, dtype):
    assert -(-rows // 128) * -(-O // 128) >= 1024
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, K + 1, generator=g).to(ref.TYPES[dtype])[:, :K]
    codes, scales = mx.weights(g, O, K)
    bias = torch.randn(O, generator=g).to(x.dtype) if O % 2 == 0 else None
    y = mx.project(x, codes, scales, bias, O, dtype, stride=3)
    want, size = want_of(x, codes, scales, bias)
    err, tol = (y.double() - want).abs(), mx.tol_of(want, size, dtype, K)
    assert (err <= tol).all(), float((err / tol).max())
    if dtype == "f32":  # a random sum is far below its magnitudes: as in test_gpu_mx
        assert (y.double() - want).norm() <= 3 * K ** 0.5 * 2 ** -24 * want.norm()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_do_not_depend_on_others(dtype):
    """A row's bits depend on the row alone, wherever it lies in a tile, and rows that are not finite spoil no other."""
    g = torch.Generator().manual_seed(1)
    rows, K, O = 4100, 1100, 4100
    x = torch.randn(rows, K, generator=g).to(ref.TYPES[dtype])
    codes, scales = mx.weights(g, O, K)
    y = mx.project(x, codes, scales, None, O, dtype)
    order = torch.randperm(rows, generator=g)
    assert torch.equal(mx.project(x[order], codes, scales, None, O, dtype), y[order.cuda()])
    bad = x.clone()
    bad[7, K - 1], bad[300, 0], bad[rows - 1, 515] = math.nan, math.inf, -math.inf
    scales[O - 1, 2] = 255  # a weight row's block that stands for NaN
    spoilt = mx.project(bad, codes, scales, None, O, dtype)
    few = torch.tensor([7, 300, rows - 1], device="cuda")
    assert torch.isnan(spoilt[few]).all() and torch.isnan(spoilt[:, O - 1]).all()
    spoilt[few] = y[few]
    assert torch.equal(spoilt[:, :O - 1], y[:, :O - 1])


def test_scales_of_any_size():
    g = torch.Generator().manual_seed(2)
    rows, K, O = 4100, 160, 4100
    x = torch.randn(rows, K, generator=g)
    codes, scales = mx.weights(g, O, K)
    for ex, ew in ((-120, 120), (100, -100), (0, -126), (120, -127)):
        xs = torch.ldexp(x, torch.tensor(ex))
        ws = (127 + ew + torch.randint(0, 3, scales.shape, generator=g)).clamp(0, 254).to(torch.uint8)
        want, size = want_of(xs, codes, ws, None)
        y = mx.project(xs, codes, ws, None, O, "f32")
        assert ((y.double() - want).abs() <= mx.tol_of(want, size, "f32", K)).all(), (ex, ew)


def test_streams_and_graphs():
    from zero_order_recurrent_amd import binding as b
    g = torch.Generator().manual_seed(3)
    rows, K, O = 4100, 700, 4100
    codes, scales = mx.weights(g, O, K)
    layer = b.MxProjection(b.make_mx_config(K, O, "bf16"), codes.cuda(), scales.cuda())
    x, other = (torch.randn(rows, K, generator=g).bfloat16().cuda() for _ in range(2))
    y = torch.empty(rows, O, dtype=torch.bfloat16, device="cuda")
    want = layer.project(x, y).clone()
    want_other = layer.project(other, y).clone()
    side = torch.cuda.Stream()
    y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    layer.project(x, y, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    graph, held = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        layer.project(held, y)
    for values, expect in ((x, want), (other, want_other), (x, want)):
        held.copy_(values)
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert torch.equal(y, expect)
