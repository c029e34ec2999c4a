"""Log probabilities, entropy, alternatives and their gradients against the 64-bit definition."""
import math

import pytest
import torch

import more_operators_ref as ref
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu


def draw(g, rows, V, dtype, spread=2.5, stride=None):
    wide = V if stride is None else stride
    x = (torch.randn(rows, wide, generator=g) * spread).to(ref.TYPES[dtype])[:, :V]
    tokens = torch.randint(0, V, (rows,), generator=g).to(torch.int32)
    return x, tokens


def device(x):
    base = x._base
    return x.cuda() if base is None else base.cuda()[:, :x.shape[1]]


def run(x, tokens, k, tau, dtype):
    op = b.TokenScores(b.make_score_config(x.shape[1], k, tau, dtype))
    n = x.shape[0]
    lp, h = torch.full((n,), 9.0, device="cuda"), torch.full((n,), 9.0, device="cuda")
    ids = torch.full((n, k), -7, dtype=torch.int32, device="cuda")
    lps = torch.full((n, k), 9.0, device="cuda")
    op.scores(device(x), tokens.cuda(), lp, h, ids if k else None, lps if k else None)
    return lp.cpu().double(), h.cpu().double(), ids.cpu(), lps.cpu().double()


def bounds(x, tau):
    """Half steps that a row's logprob and entropy may be off by. A scaled distance from the largest is off by three
    roundings (the difference, the factor's and the product), the sum by as much relative to itself and by its additions,
    V / 64 in a thread's share at most and 16 across; its logarithm and the last subtraction by a few more."""
    z = x.double() / tau
    z = torch.where(torch.isfinite(z), z, z.max(1, keepdim=True)[0])
    return 2 ** -24 * (x.shape[1] / 64 + 64 + 8 * (1 + z.amax(1) - z.amin(1)))


SIZES = [(1, 1, 1), (3, 2, 2), (37, 50, 5), (5, 50, 50), (16, 64, 64), (9, 257, 3), (4, 511, 100), (3, 1000, 1000), (2, 4097, 64),
         (3, 8191, 20), (2, 30011, 300), (2, 32768, 64), (1, 70001, 1024), (1, 300007, 20)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows, V, k", SIZES)
def test_scores(rows, V, k, dtype):
    g = torch.Generator().manual_seed(V)
    tau = 0.7
    x, tokens = draw(g, rows, V, dtype, stride=V + 5)
    tokens[rows // 2] = -3 if rows > 2 else tokens[rows // 2]
    lp, h, ids, lps = run(x, tokens, k, tau, dtype)
    want, entropy, _, _ = ref.scores(x, tokens, tau)
    tol = bounds(x, tau)
    assert ((lp - want).abs() <= tol).all()
    assert ((h - entropy).abs() <= tol * (1 + entropy)).all()
    expect = ref.top(x, k)
    assert torch.equal(ids, expect)
    for j in range(0, k, max(1, k // 5)):
        at, _, _, _ = ref.scores(x, expect[:, j], tau)
        assert ((lps[:, j] - at).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V, k", [(50, 20), (900, 5), (900, 300), (8000, 64), (30011, 1024), (40000, 1), (300007, 40)])
@pytest.mark.parametrize("kind", ["equal", "few values", "falling", "rising", "zeros of both signs", "one thread's"])
def test_alternatives_of_awkward_rows(V, k, kind, dtype):
    """Rows of ties (the lowest ids), sorted rows, and the largest all in one thread's pieces."""
    g = torch.Generator().manual_seed(V + k)
    t = ref.TYPES[dtype]
    x = {"equal": torch.full((2, V), 1.25), "few values": torch.randint(0, 3, (2, V), generator=g).float(),
         "falling": -torch.arange(V).float()[None].expand(2, V) / 7, "rising": torch.arange(V).float()[None].expand(2, V) / 7,
         "zeros of both signs": torch.where(torch.rand(2, V, generator=g) < 0.5, -0.0, 0.0),
         "one thread's": torch.randn(2, V, generator=g)}[kind].to(t).contiguous()
    if kind == "one thread's":
        per = 8 if dtype == "bf16" else 4
        x[:, :per] += 20
    _, _, ids, lps = run(x, torch.zeros(2, dtype=torch.int32), k, 1.0, dtype)
    assert torch.equal(ids, ref.top(x, k))
    assert (lps[:, :-1] >= lps[:, 1:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 100, 3000, 33333])
def test_masked_and_spoilt_rows(V, dtype):
    g = torch.Generator().manual_seed(V)
    x, tokens = draw(g, 9, V, dtype)
    inf, k = math.inf, 4
    x[1, 1:] = -inf  # a sure row
    x[2] = -inf
    x[3, V // 2] = math.nan
    x[4, V - 1] = inf
    x[5, ::2] = -inf
    x[6] = torch.finfo(x.dtype).min  # the type's lowest value everywhere
    x[7, 1:] = torch.finfo(x.dtype).min
    tokens[:] = torch.tensor([0, 0, 1, 2, 3, 0, 1, 0, V], dtype=torch.int32)
    lp, h, ids, lps = run(x, tokens, k, 1.0, dtype)
    nan = [2, 3, 4]
    assert torch.isnan(lp[nan + [8]]).all() and torch.isnan(h[nan]).all() and torch.isnan(lps[nan]).all() and (ids[nan] == -1).all()
    ok = [0, 1, 5, 6, 7]
    want, entropy, _, _ = ref.scores(x[ok], tokens[ok], 1.0)
    assert lp[5] == -inf and want[2] == -inf
    tol = 2 ** -24 * (V / 64 + 64 + 8 * 40)
    rest = [0, 1, 3, 4]
    assert ((lp[[0, 1, 6, 7]] - want[rest]).abs() <= tol).all()
    assert ((h[ok] - entropy).abs() <= tol * (1 + entropy)).all()
    assert torch.isfinite(h[8]) and (ids[8] >= 0).all()
    assert torch.equal(ids[ok], ref.top(x[ok], k))
    assert lps[1, 0] == 0 and (lps[1, 1:] == -inf).all() and h[1] == 0
    # padding's logprob is zero whatever its row holds
    lp, _, _, _ = run(x, torch.full((9,), -1, dtype=torch.int32), 0, 1.0, dtype)
    assert (lp == 0).all()


@pytest.mark.parametrize("V", [50, 5000])
def test_sure_rows_keep_their_bits(V):
    """What a row leaves for all but its largest logit is far below float32's step at one; its logarithm and entropy are
    held relative to themselves: each term by 2^-23 of its exponent's size, and the sums."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, V, generator=g)
    x[:, 3] = torch.tensor([20.0, 25.0, 30.0, 50.0, 70.0, 80.0])
    tokens = torch.full((6,), 3, dtype=torch.int32)
    lp, h, _, _ = run(x, tokens, 0, 1.0, "f32")
    rest = torch.exp(x.double() - x.double()[:, 3:4])
    rest[:, 3] = 0
    want = -torch.log1p(rest.sum(1))
    entropy = torch.log1p(rest.sum(1)) + (rest * (x.double()[:, 3:4] - x.double())).sum(1) / (1 + rest.sum(1))
    tol = 2 ** -24 * (V / 64 + 64 + 8 * 90)
    assert ((lp - want).abs() <= tol * want.abs()).all()
    assert ((h - entropy).abs() <= tol * entropy).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows, V", [(1, 1), (33, 50), (3, 513), (2, 8191), (2, 33000), (1, 150001)])
def test_gradient(rows, V, dtype):
    g = torch.Generator().manual_seed(V)
    tau = 1.3
    x, tokens = draw(g, rows, V, dtype, stride=V + 3)
    up, uh = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    if rows > 2:
        tokens[0] = -1
        x[1, V // 2:] = -math.inf
        tokens[1] = 0
    op = b.TokenScores(b.make_score_config(V, 0, tau, dtype))
    _, entropy, d_lp, d_h = ref.scores(x, tokens, tau)
    p = torch.softmax(x.double() / tau, 1)
    size = p * (up.abs()[:, None] + uh.abs()[:, None] * (torch.log(p.clamp(min=1e-300)).abs() + entropy[:, None])) / tau
    for a, c in ((up, uh), (up, None), (None, uh)):
        want = (0 if a is None else a.double()[:, None] * d_lp) + (0 if c is None else c.double()[:, None] * d_h)
        out = torch.full((rows, V + 3), 7.0, dtype=x.dtype, device="cuda")
        args = (tokens.cuda(), None if a is None else a.cuda(), None if c is None else c.cuda())
        op.grad(device(x), *args, out[:, :V])
        # p's relative error is that of its exponent and of the sum, as in `bounds`; a term's rounding comes on top
        tol = ref.HALF_STEP[dtype] * want.abs() + bounds(x, tau)[:, None] * (size + want.abs()) + 1e-37
        if dtype == "bf16":
            tol = tol + 2.0 ** -133
        assert ((out[:, :V].double().cpu() - want).abs() <= tol).all()
        assert (out[:, V:] == 7.0).all()
        inplace = device(x.clone()) if x._base is None else device(x).clone()
        op.grad(inplace, *args, inplace)
        assert torch.equal(inplace, out[:, :V])


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(2)
    V, tau, e = 11, 0.8, 1e-6
    x, tokens = draw(g, 4, V, "f32")
    up, uh = torch.randn(4, generator=g), torch.randn(4, generator=g)
    out = torch.empty(4, V, device="cuda")
    b.TokenScores(b.make_score_config(V, 0, tau, "f32")).grad(x.cuda(), tokens.cuda(), up.cuda(), uh.cuda(), out)
    for v in range(V):
        ends = []
        for s in (e, -e):
            z = x.double().clone()
            z[:, v] += s
            lp, h, _, _ = ref.scores(z, tokens, tau)
            ends.append(up * lp + uh * h)
        # the difference's own error: e^2 of the third derivative and 2^-52 / e
        assert ((out[:, v].double().cpu() - (ends[0] - ends[1]) / (2 * e)).abs() <= 1e-6).all()


def test_gradient_of_spoilt_and_idle_rows():
    V = 600
    x = torch.randn(6, V)
    x[0, 5] = math.nan
    x[1] = -math.inf
    x[2, 3] = math.inf
    x[3, 7] = math.nan
    tokens = torch.tensor([1, 1, 1, -1, V, V], dtype=torch.int32)
    up = torch.tensor([1.0, 1.0, 1.0, 1.0, 1.0, 0.0])
    out = torch.empty(6, V, device="cuda")
    op = b.TokenScores(b.make_score_config(V, 0, 1.0, "f32"))
    op.grad(x.cuda(), tokens.cuda(), up.cuda(), None, out)
    assert torch.isnan(out[[0, 1, 2, 4]]).all() and (out[[3, 5]] == 0).all()
    op.grad(x.cuda(), tokens.cuda(), None, torch.tensor([1.0, 1.0, 1.0, 0.0, 1.0, 1.0]).cuda(), out)
    assert torch.isnan(out[:3]).all() and (out[3] == 0).all() and torch.isfinite(out[4:]).all()


@pytest.mark.parametrize("tau", [2.0 ** -60, 2.0 ** -20, 2.0 ** 60])
def test_far_temperatures(tau):
    g = torch.Generator().manual_seed(3)
    x, tokens = draw(g, 4, 300, "f32", spread=min(tau, 2.0 ** 20))
    lp, h, ids, _ = run(x, tokens, 5, tau, "f32")
    want, entropy, _, _ = ref.scores(x, tokens, tau)
    assert ((lp - want).abs() <= bounds(x, tau) * (1 + want.abs())).all()
    assert ((h - entropy).abs() <= bounds(x, tau) * (1 + entropy)).all()
    assert torch.equal(ids, ref.top(x, 5))


def test_optional_outputs_streams_and_graphs():
    g = torch.Generator().manual_seed(4)
    x, tokens = draw(g, 40, 3000, "bf16")
    op = b.TokenScores(b.make_score_config(3000, 7, 1.0, "bf16"))
    xs, ts = x.cuda(), tokens.cuda()
    lp, h, ids, lps = torch.empty(40, device="cuda"), torch.empty(40, device="cuda"), torch.empty(40, 7, dtype=torch.int32, device="cuda"), torch.empty(40, 7, device="cuda")
    d, up = torch.empty_like(xs), torch.randn(40, generator=g).cuda()
    op.scores(xs, ts, lp, h, ids, lps)
    op.grad(xs, ts, up, up, d)
    want = [t.clone() for t in (lp, h, ids, lps, d)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (lp, h, lps, d):
        t.zero_()
    torch.cuda.synchronize()
    op.scores(xs, ts, lp, h, ids, lps, stream=side)
    op.grad(xs, ts, up, up, d, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip((lp, h, ids, lps, d), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.scores(xs, ts, lp, h, ids, lps)
        op.grad(xs, ts, up, up, d)
    for _ in range(3):
        for t in (lp, h, ids, lps, d):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip((lp, h, ids, lps, d), want))
    h.zero_()
    op.scores(xs, None, None, h, ids, lps)
    assert torch.equal(h, want[1])
    op.scores(xs, ts, lp, None, ids, lps)
    with pytest.raises(b.CdrgeError):
        op.scores(xs, None, lp, h, ids, lps)
    with pytest.raises(b.CdrgeError):
        op.scores(xs, ts, lp, h)
    with pytest.raises(ValueError):
        op.scores(xs, ts, lp, h, ids.long(), lps)
    with pytest.raises(ValueError):
        op.scores(xs[:, :2999], ts, lp, h, ids, lps)


def test_many_rows():
    """More rows than a grid's first dimension of workgroups would be tried with: 1.1 million of 3 logits."""
    n = 1100003
    x = torch.randn(n, 3, generator=torch.Generator().manual_seed(5))
    tokens = (torch.arange(n) % 3).to(torch.int32)
    lp, h, ids, _ = run(x, tokens, 2, 1.0, "f32")
    want, entropy, _, _ = ref.scores(x, tokens, 1.0)
    assert ((lp - want).abs() <= bounds(x, 1.0)).all() and ((h - entropy).abs() <= bounds(x, 1.0) * 3).all()
    assert torch.equal(ids.long(), torch.sort(x, dim=1, descending=True, stable=True)[1][:, :2])
