"""Microscaled 4-bit floating point: quantisation, the values back, and the product, against 64-bit definitions."""
import math

import pytest
import torch

import more_operators_ref as ref
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu


def quantize(x, dtype):
    f = b.MxFormat(b.make_mx_config(x.shape[1], 1, dtype))
    codes, scales = f.empty(x.shape[0])
    codes.fill_(0x55)
    scales.fill_(0x55)
    f.quantize(x.cuda() if x._base is None else x._base.cuda()[:, :x.shape[1]], codes, scales)
    return f, codes, scales


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows, K", [(1, 1), (3, 31), (2, 32), (5, 33), (7, 100), (2, 1000), (3, 4099), (1, 70000), (300, 40)])
def test_quantize_and_back(rows, K, dtype):
    g = torch.Generator().manual_seed(K)
    x = (torch.randn(rows, K + 3, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))).to(ref.TYPES[dtype])[:, :K]
    f, codes, scales = quantize(x, dtype)
    want_codes, want_scales = ref.mx_quantize(x)
    assert torch.equal(scales.cpu(), want_scales)
    # a zero may have either sign
    values = ref.mx_values(want_codes, want_scales, K)
    assert torch.equal(ref.mx_values(codes.cpu(), scales.cpu(), K), values)
    back = torch.full((rows, K + 2), 7.0, dtype=x.dtype, device="cuda")
    f.dequantize(codes, scales, back[:, :K])
    assert torch.equal(back[:, :K].double().cpu(), values) and (back[:, K:] == 7.0).all()
    pad = ref.mx_values(codes.cpu(), scales.cpu(), 32 * scales.shape[1])[:, K:]
    assert (pad == 0).all()
    # quantising the values again changes nothing
    again, twice = f.empty(rows)
    f.quantize(back[:, :K], again, twice)
    assert torch.equal(ref.mx_values(again.cpu(), twice.cpu(), K), values)


def test_borders_and_extremes():
    """Every border between two codes, its neighbours, at every magnitude that a block may have, and what has no scale."""
    grid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.99]
    base = torch.tensor([4.0] + grid + [-v for v in grid] + [0.0, -0.0, 6.0, -6.0], dtype=torch.float64)
    rows = []
    for e in (-149, -140, -127, -126, -125, -124, -60, -1, 0, 1, 60, 100, 124):
        v = torch.ldexp(base, torch.tensor(e)).float()
        rows += [v, torch.nextafter(v, torch.tensor(math.inf)), torch.nextafter(v, torch.tensor(-math.inf))]
    x = torch.stack(rows)
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    _, codes, scales = quantize(x, "f32")
    want_codes, want_scales = ref.mx_quantize(x)
    assert torch.equal(scales.cpu(), want_scales)
    assert torch.equal(ref.mx_values(codes.cpu(), scales.cpu(), x.shape[1]), ref.mx_values(want_codes, want_scales, x.shape[1]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_is_not_finite(dtype):
    x = torch.randn(4, 100, generator=torch.Generator().manual_seed(0)).to(ref.TYPES[dtype])
    x[0, 40], x[1, 99], x[2, 0], x[3, 64:96] = math.nan, math.inf, -math.inf, 0.0
    f, codes, scales = quantize(x, dtype)
    back = torch.empty_like(x, device="cuda")
    f.dequantize(codes, scales, back)
    assert torch.isnan(back[0, 32:64]).all() and torch.isnan(back[1, 96:]).all() and torch.isnan(back[2, :32]).all()
    assert int(torch.isnan(back).sum()) == 32 + 4 + 32 and (back[3, 64:96] == 0).all() and int(scales[3, 2]) == 0


def project(x, w_codes, w_scales, bias, O, dtype, stride=0):
    K = x.shape[1]
    layer = b.MxProjection(b.make_mx_config(K, O, dtype), w_codes.cuda(), w_scales.cuda(), None if bias is None else bias.cuda())
    y = torch.full((x.shape[0], O + stride), 7.0, dtype=x.dtype, device="cuda")
    layer.project(x.cuda() if x._base is None else x._base.cuda()[:, :K], y[:, :O])
    assert (y[:, O:] == 7.0).all()
    return y[:, :O]


def weights(g, O, K):
    blocks = -(-K // 32)
    codes = torch.randint(0, 256, (O, 16 * blocks), generator=g, dtype=torch.uint8)
    scales = torch.randint(120, 130, (O, blocks), generator=g, dtype=torch.uint8)
    return codes, scales


def want_of(x, codes, scales, bias):
    """y and the sums of its terms' magnitudes. Codes past the end of a row count for nothing: Q(x) is zero there."""
    K = x.shape[1]
    xv = ref.mx_values(*ref.mx_quantize(x), K)
    w = ref.mx_values(codes, scales, K)
    y, size = xv @ w.t(), xv.abs() @ w.t().abs()
    return (y, size) if bias is None else (y + bias.double(), size + bias.double().abs())


# Products of codes are exact; a float32 sum of K of them is off by 2^-24 of their magnitudes an addition, and by as much
# again where the matrix core cuts off instead of rounding.
def tol_of(y, size, dtype, K):
    return ref.HALF_STEP[dtype] * y.abs() + (2 * K + 64) * 2 ** -24 * size + 1e-38


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows, K, O", [(1, 1, 1), (1, 1024, 100), (2, 64, 33), (4, 3333, 70), (5, 3333, 70), (16, 130, 16), (17, 100, 50), (48, 1000, 129), (64, 32, 64),
                                        (65, 256, 70), (100, 5000, 20), (130, 515, 260), (257, 96, 300), (300, 1024, 512)])
def test_project(rows, K, O, dtype):
    g = torch.Generator().manual_seed(rows + K)
    x = (torch.randn(rows, K + 1, generator=g)).to(ref.TYPES[dtype])[:, :K]
    codes, scales = weights(g, O, K)
    bias = torch.randn(O, generator=g).to(x.dtype) if K % 2 else None
    y = project(x, codes, scales, bias, O, dtype, stride=3)
    want, size = want_of(x, codes, scales, bias)
    err, tol = (y.double().cpu() - want).abs(), tol_of(want, size, dtype, K)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("rows", [3, 100, 300])
def test_precision_in_the_2_norm(rows):
    """Float32 sums of exact products: a random sum is far below its magnitudes, and K^(1/2) roundings of 2^-24 of the sum
    so far, three times that allowed for sums that are cut off."""
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, 2048, generator=g)
    codes, scales = weights(g, 256, 2048)
    want, _ = want_of(x, codes, scales, None)
    y = project(x, codes, scales, None, 256, "f32").double().cpu()
    assert (y - want).norm() <= 3 * 2048 ** 0.5 * 2 ** -24 * want.norm()


@pytest.mark.parametrize("rows", [2, 70, 300])
def test_project_scales_of_any_size(rows):
    """Scales from the smallest to the largest, of weights and of rows, whose product is a float32."""
    g = torch.Generator().manual_seed(rows)
    K, O = 160, 40
    x = torch.randn(rows, K, generator=g)
    codes, scales = weights(g, O, K)
    for ex, ew in ((-120, 120), (100, -100), (-60, -50), (0, -126), (120, -127)):
        xs = torch.ldexp(x, torch.tensor(ex))
        ws = (127 + ew + torch.randint(0, 3, scales.shape, generator=g)).clamp(0, 254).to(torch.uint8)
        want, size = want_of(xs, codes, ws, None)
        y = project(xs, codes, ws, None, O, "f32")
        assert ((y.double().cpu() - want).abs() <= tol_of(want, size, "f32", K)).all(), (ex, ew)


@pytest.mark.parametrize("rows", [1, 5, 70, 300])
def test_project_what_is_not_finite(rows):
    g = torch.Generator().manual_seed(rows)
    K, O = 300, 90
    x = torch.randn(rows, K, generator=g)
    codes, scales = weights(g, O, K)
    good = project(x, codes, scales, None, O, "f32")
    bad = x.clone()
    bad[rows // 2, 299] = math.nan
    y = project(bad, codes, scales, None, O, "f32")
    others = [r for r in range(rows) if r != rows // 2]
    assert torch.isnan(y[rows // 2]).all() and torch.equal(y[others], good[others])
    scales[3, 1] = 255  # a weight row's block that stands for NaN
    y = project(x, codes, scales, None, O, "f32")
    rest = [o for o in range(O) if o != 3]
    assert torch.isnan(y[:, 3]).all() and torch.equal(y[:, rest], good[:, rest])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_do_not_depend_on_others(dtype):
    """Among rows of one call, and of calls that take the same kernel, a row's bits depend on the row alone."""
    g = torch.Generator().manual_seed(5)
    K, O = 700, 200
    x = torch.randn(300, K, generator=g).to(ref.TYPES[dtype])
    codes, scales = weights(g, O, K)
    y = project(x, codes, scales, None, O, dtype)
    order = torch.randperm(300, generator=g)
    assert torch.equal(project(x[order], codes, scales, None, O, dtype), y[order.cuda()])


def test_streams_and_graphs():
    g = torch.Generator().manual_seed(6)
    K, O = 500, 130
    codes, scales = weights(g, O, K)
    layer = b.MxProjection(b.make_mx_config(K, O, "bf16"), codes.cuda(), scales.cuda())
    f = b.MxFormat(b.make_mx_config(K, O, "bf16"))
    for rows in (1, 40, 300):
        x = torch.randn(rows, K, generator=g).bfloat16().cuda()
        y, back = torch.empty(rows, O, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
        c, s = f.empty(rows)

        def call(stream=None):
            layer.project(x, y, stream=stream)
            f.quantize(x, c, s, stream=stream)
            f.dequantize(c, s, back, stream=stream)

        call()
        want = y.clone(), back.clone()
        y.zero_(), back.zero_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        call(side)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(back, want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for _ in range(3):
            y.zero_(), back.zero_()
            torch.cuda.synchronize()
            graph.replay()
            assert torch.equal(y, want[0]) and torch.equal(back, want[1])


def test_classes_refuse():
    u8 = torch.uint8
    f = b.MxFormat(b.make_mx_config(70, 10, "f32"))
    codes, scales = f.empty(4)
    assert codes.shape == (4, 48) and scales.shape == (4, 3)
    x = torch.zeros(4, 70, device="cuda")
    for args in ((x[:3], codes, scales), (x.bfloat16(), codes, scales), (x, codes[:, :32], scales), (x, codes, scales[:, :2]),
                 (x.cpu(), codes, scales), (x, codes.int(), scales)):
        with pytest.raises(ValueError):
            f.quantize(*args)
        with pytest.raises(ValueError):
            f.dequantize(args[1], args[2], args[0])
    with pytest.raises(ValueError):
        b.MxProjection(b.make_mx_config(70, 4, "f32"), codes, scales, torch.zeros(5, device="cuda"))
    layer = b.MxProjection(b.make_mx_config(70, 4, "f32"), codes.zero_(), scales.zero_())
    with pytest.raises(ValueError):
        layer.project(x, torch.zeros(4, 5, device="cuda"))
    with pytest.raises(ValueError):
        layer.project(x[:, :64], torch.zeros(4, 4, device="cuda"))
    assert layer.project(x[:0], torch.zeros(0, 4, device="cuda")).shape == (0, 4)
    assert u8 is codes.dtype


@pytest.mark.parametrize("rows, K, O", [(1100, 300, 4100), (2049, 2112, 2050), (4097, 64, 1000)])
def test_project_large_tiles(rows, K, O):
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, K, generator=g).bfloat16()
    codes, scales = weights(g, O, K)
    bias = torch.randn(O, generator=g).bfloat16()
    y = project(x, codes, scales, bias, O, "bf16", stride=1)
    want, size = want_of(x, codes, scales, bias)
    err, tol = (y.double().cpu() - want).abs(), tol_of(want, size, "bf16", K)
    assert (err <= tol).all(), float((err / tol).max())
