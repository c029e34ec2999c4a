"""Distillation loss and gradient against the definition in 64 bits, and against differences of it."""
import pytest
import torch

import operators_ref as ref
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}
NINF = -float("inf")


def make(dtype, rows, V, k, seed=0, pad=3, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(rows, V + pad, generator=g) * spread).to(T[dtype])[:, :V]
    ids = torch.stack([torch.randperm(V, generator=g)[:k] if k <= V else torch.randint(0, V, (k,), generator=g) for _ in range(rows)])
    return logits, ids.to(torch.int32), torch.randn(rows, k, generator=g) * 3


def put(t, pad):
    wide = torch.full((t.shape[0], t.shape[1] + pad), 7.0, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


def check(dtype, logits, ids, teacher, tau, models, row_grad=None, pad=3, in_place=False, finite=True):
    n, V = logits.shape
    op = b.DistillLoss(b.make_distill_config(V, ids.shape[1], models, tau, dtype))
    row, losses = torch.empty(n, device="cuda"), torch.empty(models, device="cuda")
    x = put(logits, pad)
    ids, teacher = ids.contiguous(), teacher.contiguous()
    op.losses(x, ids.cuda(), teacher.cuda(), row, losses)
    want, each, grad, width = ref.distill(logits, ids, teacher, tau, models, row_grad)
    tol = tau * tau * width * 2 ** -24 + 2 ** -24 * want.abs() + 1e-30
    err = (row.double().cpu() - want).abs() / tol
    assert err.max() <= 1, f"row losses: {float(err.max()):.2f} of the tolerance"
    scored = (ids >= 0).any(1)
    mean_tol = (tol * scored).view(models, -1).sum(1) / scored.view(models, -1).sum(1) + 2 ** -24 * each.abs()
    both = torch.isnan(losses.cpu()) & torch.isnan(each)
    assert (both | ((losses.double().cpu() - each).abs() <= mean_tol)).all()
    d = x if in_place else put(torch.zeros_like(logits), pad)
    row_again, losses_again = torch.empty_like(row), torch.empty_like(losses)
    up = None if row_grad is None else row_grad.cuda()
    op.grad(x, ids.cuda(), teacher.cuda(), up, row_again, losses_again, d)
    assert torch.equal(row_again, row) and torch.equal(losses_again.nan_to_num(), losses.nan_to_num())
    q = torch.softmax(logits.double() / tau, 1)
    scale = (torch.ones(n) if row_grad is None else row_grad).double().abs()[:, None] * tau
    # the difference of two numbers that each are off by width 2^-24 of themselves, then its rounding
    gtol = ref.HALF_STEP[dtype] * grad.abs() + 2 ** -24 * width[:, None] * (grad.abs() + 2 * scale * q) + 1e-38
    gerr = (d.double().cpu() - grad).abs() / gtol
    assert gerr.max() <= 1, f"gradient: {float(gerr.max()):.2f} of the tolerance"
    if not in_place and pad:
        assert (d.as_strided((n, pad), (V + pad, 1), V) == 7).all()
    return row, d


SHAPES = [
    # dtype, rows, V, k, models
    ("f32", 64, 50, 8, 8), ("bf16", 33, 50, 8, 1), ("f32", 1, 1, 1, 1), ("bf16", 7, 2, 5, 7), ("f32", 10, 63, 63, 2), ("bf16", 6, 1000, 100, 3),
    ("f32", 5, 2047, 20, 1), ("bf16", 4, 2049, 64, 2), ("f32", 3, 10007, 33, 3), ("bf16", 2, 30011, 1024, 1), ("f32", 2, 50001, 257, 2),
    ("bf16", 3, 8192, 64, 1), ("bf16", 2, 140000, 20, 1), ("f32", 1, 140001, 5, 1),
]


@pytest.mark.parametrize("tau", [1.0, 2.5, 0.5])
@pytest.mark.parametrize("dtype, rows, V, k, models", SHAPES)
def test_losses_and_gradient(dtype, rows, V, k, models, tau):
    logits, ids, teacher = make(dtype, rows, V, k, seed=V)
    check(dtype, logits, ids, teacher, tau, models, row_grad=torch.randn(rows, generator=torch.Generator().manual_seed(1)))


@pytest.mark.parametrize("V", [64, 4096])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_aligned_rows_and_in_place(dtype, V):
    logits, ids, teacher = make(dtype, 9, V, 16)
    _, apart = check(dtype, logits, ids, teacher, 1.5, 3, pad=0)
    _, same = check(dtype, logits, ids, teacher, 1.5, 3, pad=0, in_place=True)
    assert torch.equal(apart, same)


def test_in_place_odd_rows():
    logits, ids, teacher = make("bf16", 5, 5001, 40)
    check("bf16", logits, ids, teacher, 1.0, 1, pad=2, in_place=True)


@pytest.mark.parametrize("V", [50, 3000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_absent_entries(dtype, V):
    """Fewer than k entries, none, teacher logits of minus infinity, an id twice; a model without a scored row."""
    logits, ids, teacher = make(dtype, 8, V, 6)
    ids[0, 3:] = -1
    ids[1] = -1
    teacher[2] = NINF
    teacher[3, 1:4] = NINF
    ids[4, 1] = ids[4, 0]
    ids[4, 5] = ids[4, 0]
    ids[5, 0] = -7
    ids[6], ids[7] = -1, -2
    teacher[7] = float("nan")  # absent, whatever it holds
    row, d = check(dtype, logits, ids, teacher, 1.0, 4)
    for r in (1, 2, 6, 7):
        assert row[r] == 0 and (d[r] == 0).all()


@pytest.mark.parametrize("V", [50, 3000])
def test_masked_vocabulary(V):
    """Student logits of minus infinity and of the type's lowest value: no NaN where the teacher puts no mass."""
    for dtype in ("f32", "bf16"):
        logits, ids, teacher = make(dtype, 4, V, 5)
        ids = torch.stack([torch.arange(5)] * 4).to(torch.int32)
        logits[0, 20:] = NINF
        logits[1, 5:] = torch.finfo(T[dtype]).min
        logits[2, 7] = NINF
        op = b.DistillLoss(b.make_distill_config(V, 5, 1, 1.0, dtype))
        x, row, d = logits.cuda(), torch.empty(4, device="cuda"), torch.empty_like(logits, device="cuda")
        op.grad(x.contiguous(), ids.cuda(), teacher.cuda(), None, row, None, d)
        want, _, grad, _ = ref.distill(logits, ids, teacher, 1.0, 1)
        assert torch.isfinite(row).all() and torch.isfinite(d).all()
        assert (row.double().cpu() - want).abs().max() <= 2 ** -24 * (V / 64 + 64 + 32 * 40)
        assert (d[0, 20:] == 0).all() and d[2, 7] == 0 and (d[1, 5:] == 0).all()
        # the teacher wants what the student rules out: an infinite loss
        logits[3, 2] = NINF
        op.losses(logits.cuda().contiguous(), ids.cuda(), teacher.cuda(), row)
        assert row[3] == float("inf")


def test_bad_rows_are_nan_and_alone():
    for V in (50, 3000):
        logits, ids, teacher = make("f32", 6, V, 5)
        clean = check("f32", logits, ids, teacher, 1.0, 1)
        ids[1, 2] = V
        ids[3, 4] = 2 ** 31 - 1
        logits[4, 17] = float("nan")
        op = b.DistillLoss(b.make_distill_config(V, 5, 6, 1.0, "f32"))
        row, losses, d = torch.empty(6, device="cuda"), torch.empty(6, device="cuda"), torch.empty(6, V, device="cuda")
        op.grad(logits.cuda().contiguous(), ids.cuda(), teacher.cuda(), None, row, losses, d)
        bad = [1, 3, 4]
        assert torch.isnan(row[bad]).all() and torch.isnan(losses[bad]).all() and torch.isnan(d[bad]).all()
        good = [0, 2, 5]
        assert torch.equal(row[good], clean[0][good]) and torch.equal(d[good], clean[1][good])


@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_gradient_against_differences(tau):
    logits, ids, teacher = make("f32", 3, 12, 4, pad=0)
    _, d = check("f32", logits, ids, teacher, tau, 1, pad=0)
    h, x = 1e-4, logits.double()
    for v in range(12):
        e = torch.zeros(12, dtype=torch.float64)
        e[v] = h
        up, down = (ref.distill(x + s * e, ids, teacher, tau, 1)[0] for s in (1, -1))
        # differences are off by h^2 / 6 times a third derivative of at most 1 / tau; the kernel by its own bound
        assert ((up - down) / (2 * h) - d[:, v].double().cpu()).abs().max() <= h * h + 1e-10 / h + 2 ** -24 * 2000 * tau


def test_means_read_like_update_losses():
    """2K models' means in the order that the update takes; rows of a model lie together."""
    logits, ids, teacher = make("f32", 6 * 300, 20, 4)
    check("f32", logits, ids, teacher, 1.0, 6)


def test_no_rows():
    op = b.DistillLoss(b.make_distill_config(20, 4, 2, 1.0, "f32"))
    losses = torch.zeros(2, device="cuda")
    op.losses(torch.empty(0, 20, device="cuda"), torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda"),
              torch.empty(0, device="cuda"), losses)
    assert torch.isnan(losses).all()


@pytest.mark.parametrize("V", [50, 5000])
def test_graph_replays_and_other_stream(V):
    logits, ids, teacher = make("bf16", 12, V, 8)
    op = b.DistillLoss(b.make_distill_config(V, 8, 2, 1.0, "bf16"))
    x, i, t = logits.cuda().contiguous(), ids.cuda(), teacher.cuda()
    outs = torch.empty(12, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(x)

    def call(stream=None):
        op.grad(x, i, t, None, outs[0], outs[1], outs[2], stream=stream)

    call()
    eager = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert all(torch.equal(a, e) for a, e in zip(outs, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert all(torch.equal(a, e) for a, e in zip(outs, eager))
        torch.ones(1000, device="cuda").sum().item()


def test_loss_checks_its_tensors():
    logits, ids, teacher = make("f32", 4, 20, 3)
    op = b.DistillLoss(b.make_distill_config(20, 3, 2, 1.0, "f32"))
    x, i, t, row = logits.cuda(), ids.cuda(), teacher.cuda(), torch.empty(4, device="cuda")
    for call in (lambda: op.losses(x.bfloat16(), i, t, row), lambda: op.losses(x, i.long(), t, row), lambda: op.losses(x, i, t[:, :2], row),
                 lambda: op.losses(x, i, t, row[:2]), lambda: op.losses(x, i, t, row, torch.empty(3, device="cuda")),
                 lambda: op.losses(x, i.cpu(), t, row), lambda: op.losses(x[:, :-1], i, t, row),
                 lambda: op.grad(x, i, t, None, row, None, x.double())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(b.CdrgeError):
        b.DistillLoss(b.make_distill_config(20, 3, 3, 1.0, "f32")).losses(x, i, t, row)
