"""Low-rank adapters beside a shared projection against the formula in 64 bits, row by row."""
import pytest
import torch

import operators_ref as ref
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    def __init__(self, dtype, rows, K, O, A, R, bias=True, ranks=None, scale=True, order="mixed", seed=0, xpad=3, wpad=0, ypad=2):
        g = torch.Generator().manual_seed(seed)
        t = T[dtype]
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.dtype, self.K, self.O, self.R, self.A, self.n = dtype, K, O, R, A, rows
        self.x = rand(rows, K + xpad).to(t)[:, :K]
        self.w = (rand(O, K + wpad) * K ** -0.5).to(t)[:, :K]
        self.bias = rand(O).to(t) if bias else None
        self.down, self.up = (rand(A, R, K) * K ** -0.5).to(t), (rand(A, O, R) * R ** -0.5).to(t)
        self.ranks = ranks
        self.scale = (rand(rows) if scale else None)
        who = torch.randint(-1, max(A, 1), (rows,), generator=g)
        self.who = (torch.sort(who)[0] if order == "runs" else who).to(torch.int32)
        self.ypad = ypad

    def operator(self):
        dev = lambda v: None if v is None else v.cuda()  # noqa: E731
        cfg = b.make_adapter_config(self.K, self.O, self.A, self.R, self.dtype)
        ranks = None if self.ranks is None else torch.tensor(self.ranks, dtype=torch.int32).cuda()
        wide = torch.zeros(self.O, self.w.stride(0), dtype=T[self.dtype], device="cuda")
        wide[:, :self.K] = self.w.cuda()
        return b.AdapterProjection(cfg, wide[:, :self.K], dev(self.bias), dev(self.down), dev(self.up), ranks)

    def inputs(self):
        wide = torch.zeros(self.n, self.x.stride(0), dtype=T[self.dtype], device="cuda")
        wide[:, :self.K] = self.x.cuda()
        y = torch.full((self.n, self.O + self.ypad), 7.0, dtype=T[self.dtype], device="cuda")
        return wide[:, :self.K], self.who.cuda(), y, None if self.scale is None else self.scale.cuda()

    def check(self, y, rows=None):
        want, shared, low = ref.adapters(self.x, self.w, self.bias, self.down, self.up, self.ranks, self.who, self.scale)
        tol = ref.adapters_tol(want, shared, low, self.dtype, self.K, self.R) + 1e-30
        err = (y.double().cpu() - want).abs() / tol
        err = err if rows is None else err[rows]
        assert torch.isfinite(err).all()
        assert err.max() <= 1, f"{float(err.max()):.2f} of the tolerance"


CASES = [
    # dtype, rows, K, O, A, R
    ("bf16", 1, 64, 64, 1, 16), ("bf16", 1, 1000, 515, 3, 8), ("bf16", 5, 33, 7, 4, 1), ("bf16", 16, 256, 192, 16, 16),
    ("bf16", 17, 512, 130, 5, 13), ("bf16", 40, 1024, 256, 40, 16), ("bf16", 64, 96, 64, 2, 64), ("bf16", 129, 320, 257, 9, 32),
    ("bf16", 300, 640, 512, 3, 8), ("bf16", 513, 192, 384, 7, 128), ("bf16", 260, 70, 66, 4, 40),
    ("f32", 1, 64, 64, 1, 16), ("f32", 3, 129, 515, 2, 12), ("f32", 33, 130, 65, 5, 5), ("f32", 150, 256, 256, 6, 64), ("f32", 90, 17, 300, 30, 128),
]


@pytest.mark.parametrize("order", ["mixed", "runs"])
@pytest.mark.parametrize("case", CASES)
def test_project(case, order):
    c = Case(*case, order=order, seed=case[1])
    x, who, y, scale = c.inputs()
    c.operator().project(x, who, y[:, :c.O], row_scale=scale)
    c.check(y[:, :c.O])
    assert (y[:, c.O:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows, K, O, A, R", [(1, 8, 5, 1, 1), (1, 2047, 33, 3, 30), (4, 1000, 100, 3, 16), (2, 513, 17, 2, 23), (3, 96, 160, 5, 9),
                                              (4, 1, 1, 2, 7), (16, 300, 70, 0, 1), (1, 4096, 48, 2, 16), (1, 33, 20, 2, 64), (5, 64, 40, 9, 4),
                                              (2, 4100, 40, 2, 16)])
def test_a_row_or_a_few(dtype, rows, K, O, A, R):
    """Either side of the one-launch form's limits, the same adapter twice, ranks of zero, rows without one or with a bad one."""
    c = Case(dtype, rows, K, O, A, R, seed=rows * K, ranks=[(R + 1) // 2 * (i % 3) for i in range(A)] if A else None)
    op, (x, who, y, scale) = c.operator(), c.inputs()
    op.project(x, who, y[:, :c.O], row_scale=scale)
    if not A:  # every adapter is out of range
        bad, c.who = c.who >= 0, torch.full_like(c.who, -1)
        assert bad.any() and y[bad.cuda(), :c.O].isnan().all()
    c.check(y[:, :c.O], rows=slice(None) if A else ~bad)
    assert (y[:, c.O:] == 7).all()
    if A:
        c.who[:] = A - 1
        op.project(x, c.who.cuda(), y[:, :c.O], row_scale=scale)
        c.check(y[:, :c.O])
        who = c.who.clone()
        who[0] = A
        c.down[0] = float("nan")  # an adapter that no row names
        bad = b.AdapterProjection(op.cfg, op._held[0], op._held[1], c.down.cuda(), op._held[3], op._held[4])
        bad.project(x, who.cuda(), y[:, :c.O], row_scale=scale)
        assert y[0, :c.O].isnan().all()
        if rows > 1 and A > 1:
            c.check(y[:, :c.O], rows=slice(1, None))


@pytest.mark.parametrize("counts", [[64], [40, 24], [33, 17, 14], [1] * 64, [0, 50, 3], [16, 16, 31, 1], [48, 150, 2]])
@pytest.mark.parametrize("dtype, K, R", [("bf16", 1000, 16), ("bf16", 130, 40), ("f32", 515, 20)])
def test_rows_of_an_adapter_lie_anywhere(dtype, K, R, counts):
    """Adapters that few, some and most of a tile's rows name, in any order."""
    n = sum(counts)
    c = Case(dtype, n, K, 96, len(counts), R, seed=n)
    who = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    c.who = who[torch.randperm(n, generator=torch.Generator().manual_seed(n))].to(torch.int32)
    x, who, y, scale = c.inputs()
    c.operator().project(x, who, y[:, :c.O], row_scale=scale)
    c.check(y[:, :c.O])


@pytest.mark.parametrize("dtype, rows, K, O, R, pad", [("bf16", 3333, 192, 3880, 8, 0), ("bf16", 3333, 70, 3880, 40, 3), ("f32", 3100, 64, 4070, 24, 0)])
def test_many_rows(dtype, rows, K, O, R, pad):
    """The largest tiles, with rows and outputs that end inside one, aligned and not."""
    c = Case(dtype, rows, K, O, 5, R, order="runs", seed=rows, xpad=pad, ranks=[R, R - 1, 0, 3, R])
    x, who, y, scale = c.inputs()
    c.operator().project(x, who, y[:, :c.O], row_scale=scale)
    c.check(y[:, :c.O])
    assert (y[:, c.O:] == 7).all()


@pytest.mark.parametrize("dtype, rows", [("bf16", 4), ("bf16", 200), ("f32", 70)])
def test_ranks_and_no_scale(dtype, rows):
    c = Case(dtype, rows, 128, 96, 6, 24, bias=False, ranks=[0, 24, 1, 17, -4, 99], scale=False, xpad=0, ypad=0, wpad=8)
    x, who, y, _ = c.inputs()
    # what lies past a rank is not used, whatever it holds
    for a, r in enumerate(c.ranks):
        r = min(max(r, 0), 24)
        c.down[a, r:] = float("nan")
        c.up[a, :, r:] = float("inf")
    c.operator().project(x, who, y)
    c.check(y)


@pytest.mark.parametrize("dtype, rows, O", [("bf16", 6, 80), ("bf16", 150, 320), ("f32", 40, 80)])
def test_rows_do_not_meet(dtype, rows, O):
    """Another row's NaN input, another request's NaN or infinite adapter, an adapter out of range."""
    c = Case(dtype, rows, 96, O, 4, 8)
    c.who = torch.arange(rows).remainder(6).to(torch.int32) - 1  # -1 .. 4; 4 is out of range
    c.x[1::12] = float("nan")
    c.down[1] = float("nan")
    c.up[2] = float("inf")
    x, who, y, scale = c.inputs()
    c.operator().project(x, who, y[:, :c.O], row_scale=scale)
    y = y[:, :c.O]
    nan = torch.zeros(rows, dtype=torch.bool)
    nan[1::12] = True
    wild = (c.who == 1) | (c.who == 2) | (c.who == 4) | nan
    assert torch.isnan(y.cpu()[(c.who == 4) | (c.who == 1) | nan]).all()
    assert not torch.isfinite(y.cpu()[c.who == 2]).any()
    c.who = torch.where(wild, torch.full_like(c.who, -1), c.who)
    c.x = torch.where(nan[:, None], torch.zeros_like(c.x), c.x)
    c.check(y, ~wild)


@pytest.mark.parametrize("dtype, rows", [("bf16", 3), ("bf16", 140), ("f32", 20)])
def test_without_adapters(dtype, rows):
    c = Case(dtype, rows, 64, 72, 2, 8)
    x, _, y, scale = c.inputs()
    c.who = torch.full_like(c.who, -1)
    a = c.operator().project(x, None, y[:, :c.O], row_scale=scale).clone()
    c.check(a)
    assert torch.equal(a, c.operator().project(x, c.who.cuda(), y[:, :c.O], row_scale=scale))
    none = b.AdapterProjection(b.make_adapter_config(64, 72, 0, 8, dtype), c.w.cuda(), c.bias.cuda())
    assert torch.equal(a, none.project(x, None, y[:, :c.O]))
    none.project(x[:0], None, y[:0, :c.O])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_antithetic_pair_shares_its_probe(dtype):
    """Rows at +s and -s of one adapter: their mean is the shared product, their difference the low-rank one."""
    c = Case(dtype, 2 * 48, 128, 64, 1, 4, bias=False)
    c.x[48:] = c.x[:48]
    c.who[:] = 0
    c.scale = torch.cat([torch.full((48,), 0.25), torch.full((48,), -0.25)])
    x, who, y, scale = c.inputs()
    c.operator().project(x, who, y[:, :64], row_scale=scale)
    c.check(y[:, :64])


@pytest.mark.parametrize("rows", [3, 100, 400])
def test_row_order_does_not_matter(rows):
    c = Case("bf16", rows, 256, 128, 5, 8)
    x, who, y, scale = c.inputs()
    op = c.operator()
    a = op.project(x, who, y[:, :128], row_scale=scale).clone()
    p = torch.randperm(rows, generator=torch.Generator().manual_seed(1)).cuda()
    again = op.project(x[p], who[p], y[:, :128], row_scale=scale[p])
    assert torch.equal(a[p], again)


@pytest.mark.parametrize("rows", [2, 300])
def test_graph_replays_and_other_stream(rows):
    c = Case("bf16", rows, 256, 320, 5, 16)
    x, who, y, scale = c.inputs()
    op, out = c.operator(), torch.zeros(rows, 320, dtype=torch.bfloat16, device="cuda")
    eager = op.project(x, who, out, row_scale=scale).clone()
    out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    op.project(x, who, out, row_scale=scale, stream=side)
    side.synchronize()
    assert torch.equal(out, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.project(x, who, out, row_scale=scale)
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert torch.equal(out, eager)
        torch.ones(1000, device="cuda").sum().item()


def test_operator_checks_its_tensors():
    c = Case("bf16", 8, 64, 72, 2, 8)
    x, who, y, scale = c.inputs()
    op = c.operator()
    for call in (lambda: op.project(x.float(), who, y[:, :72]), lambda: op.project(x[:, :-1], who, y[:, :72]),
                 lambda: op.project(x, who.long(), y[:, :72]), lambda: op.project(x, who[:-1], y[:, :72]),
                 lambda: op.project(x, who, y), lambda: op.project(x, who, y[:, :72], row_scale=scale.double()),
                 lambda: op.project(x, who.cpu(), y[:, :72]),
                 lambda: b.AdapterProjection(op.cfg, c.w.cuda(), None, c.down.cuda()[:, :4], c.up.cuda())):
        with pytest.raises(ValueError):
            call()
