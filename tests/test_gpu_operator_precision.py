"""How exact the population operators are as a whole, in the 2-norm over many outputs.

A bound of each element by the magnitudes of its sum's terms holds for any inputs, but over random terms of either sign
those magnitudes are many times the sum: precision that is lost in every operand can hide below it. Over thousands of
outputs of random terms the roundings are independent and add as squares, relative to the outputs themselves, so the
norm of the error shows what each operand was rounded to.
"""
import pytest
import torch

import operators_ref as ref
from test_gpu_adapters import Case as Adapters
from test_gpu_scan import Case, ints
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu

# A prompt's outputs. Entries enter products in two halves of 11 bits, rounded by at most 2^-22 (in the 2-norm that over
# sqrt 3); a product leaves out the two low halves' (2^-22 again). Two such products in a row with two roundings each make
# sqrt(6 / 3) 2^-22 = 2^-21.5. Up to 3 x 256 + 3 x 64 additions in float32, each rounded by 2^-24 / sqrt 3 of a partial sum
# whose square grows evenly to the whole's: sqrt(960 / 6) 2^-24 = 2^-20.3. Convolution, exponentials and gates: a few
# 2^-23. As squares: 2^-19.9, held to 2^-19.
SCAN = 2 ** -19


def off(got, want):
    """The norm of the difference over the norm of `want`; bf16 against `want` rounded to bf16."""
    if got.dtype == torch.bfloat16:
        want = want.to(torch.bfloat16).double()
    return float((got.double().cpu() - want).norm() / want.norm())


def bound(dtype, e):
    # A value that is off by e of itself before it is rounded to bf16 ends a step (at most 2^-7 of it, 2^-7.5 in the mean)
    # from the nearest with the probability |e| / step: the mean square is step |e|, at most 2^-7 e.
    return (2 ** -7 * e) ** 0.5 if dtype == "bf16" else e


@pytest.mark.parametrize("shape, lengths", [
    (("bf16", 2, 64, 1, 128, 4), [600, 70]), (("f32", 2, 64, 1, 128, 4), [600, 70]), (("bf16", 2, 32, 2, 16, 3), [150, 33]),
    (("bf16", 2, 80, 1, 64, 4), [400]), (("f32", 3, 40, 1, 100, 2), [300, 5]), (("bf16", 1, 128, 1, 256, 4), [330]),
    (("f32", 1, 64, 1, 256, 4), [130])])
def test_prompts(shape, lengths):
    n = len(lengths)
    c = Case(*shape, tokens=sum(lengths), seqs=n, slots=n, seed=11)
    bounds = [(sum(lengths[:i]), sum(lengths[:i + 1])) for i in range(n)]
    xbc, dt, z = c.rows()
    conv, ssm = c.conv.cuda(), c.ssm.cuda()
    y = c.layer().prompt(xbc, dt, c.y(), n, z=z, offsets=ints([0] + [e for _, e in bounds]), positions=ints([7] * n), conv_state=conv,
                         ssm_state=ssm)
    want, _, carried = c.expect(bounds, list(range(n)), [7] * n)
    assert off(y, want) <= bound(c.dtype, SCAN)
    for i in range(n):
        assert off(ssm[i], carried[i][0]) <= SCAN


def steps_and_decays(c, steps, decay):
    """Makes the case's tokens take these steps ([tokens], every head) with one decay; the definition's y in 64 bits, for
    equal sequences that start at zero. (A softplus that holds for any step, which exp does not from 709 on.)"""
    H, P, G, N = c.dims
    raw = torch.as_tensor(steps, dtype=torch.float32).expm1().log().where(torch.as_tensor(steps) < 30, torch.as_tensor(steps, dtype=torch.float32))
    c.dt.copy_(raw[:, None].expand(-1, H))
    c.dt_bias, c.decay = None, torch.full((H,), float(decay))
    dt = c.dt.double()
    step = dt.clamp(min=0) + torch.log1p(torch.exp(-dt.abs()))
    y, each = torch.zeros(c.tokens, H, P, dtype=torch.float64), c.tokens // c.n
    for i in range(c.n):
        x = torch.cat([torch.zeros(c.width - 1, c.ch, dtype=torch.float64), c.xbc[i * each:i * each + each].double()])
        u = c.cb.double() + sum(x[j:j + each] * c.cw[:, j].double() for j in range(c.width))
        u = u * torch.sigmoid(u)
        S = torch.zeros(H, P, N, dtype=torch.float64)
        for t in range(each):
            at = i * each + t
            X, B, C = u[t, :c.d].view(H, P), *(u[t, o:o + G * N].view(G, N).repeat_interleave(H // G, 0) for o in (c.d, c.d + G * N))
            S = S * torch.exp(step[at] * c.decay.double())[:, None, None] + (step[at][:, None] * X)[:, :, None] * B[:, None, :]
            y[at] = (S * C[:, None]).sum(2) + c.skip.double()[:, None] * X
    gate = c.z.double()
    return y.view(c.tokens, -1) * gate * torch.sigmoid(gate)


@pytest.mark.parametrize("step, decay", [(50, -16), (200, -16), (1000, -16), (5000, -16), (20, -64), (10, -1000), (100, -1000), (1e-3, -0.01)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seqs, each", [(1, 200), (5, 12)])  # in blocks, and in the kernel for short ones
def test_prompts_with_long_steps(dtype, step, decay, seqs, each):
    """Long steps leave nothing of what was before: a token's own weight, its step, has to come out as exact as ever. Token
    by token the same."""
    c = Case(dtype, 2, 64, 1, 32, 4, tokens=seqs * each, seqs=seqs, slots=seqs, seed=4)
    want = steps_and_decays(c, [float(step)] * c.tokens, decay)
    xbc, dt, z = c.rows()
    layer = c.layer()
    y = layer.prompt(xbc, dt, c.y(), seqs, z=z)
    assert off(y, want) <= bound(dtype, SCAN)
    conv, ssm, alone = c.conv.cuda(), c.ssm.cuda(), c.y()
    for t in range(each):
        at = slice(t, None, each)
        layer.step(xbc[at], dt[at], alone[at], ints([t] * seqs), conv, ssm, z=z[at])
    assert off(alone, want) <= bound(dtype, SCAN)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("each, far", [(60, 20), (15, 4)])
def test_prompt_with_one_far_step(dtype, each, far):
    """One token of a step beyond all others: the decays behind it are as exact as before it."""
    c = Case(dtype, 2, 64, 1, 32, 4, tokens=each, seqs=1, seed=5)
    steps = [1.0] * each
    steps[far] = 1e20
    want = steps_and_decays(c, steps, -0.1)
    xbc, dt, z = c.rows()
    y = c.layer().prompt(xbc, dt, c.y(), 1, z=z)
    # What a token's row holds of the far one is e^-4 of it at the least: far above the 2^-38 of the largest weight that
    # operands are rounded to.
    for t in range(far, each):
        err = (y[t].double().cpu() - want[t]).norm() / want[t].norm()
        assert err <= ref.HALF_STEP[dtype] + 2 * SCAN, t  # 128 outputs scatter more than thousands


def distill(logits, ids, teacher, tau):
    n, V = logits.shape
    op = b.DistillLoss(b.make_distill_config(V, ids.shape[1], 1, tau, "bf16" if logits.dtype == torch.bfloat16 else "f32"))
    row, d = torch.empty(n, device="cuda"), torch.empty(logits.shape, dtype=logits.dtype, device="cuda")
    op.grad(logits.cuda(), ids.cuda(), teacher.cuda(), None, row, None, d)
    z, t = logits.double() / tau, teacher.double() / tau
    logq, logp = torch.log_softmax(z, 1), torch.log_softmax(t, 1)
    q, p = torch.exp(logq), torch.exp(logp)
    at = torch.gather(logq, 1, ids.long())
    want = tau * tau * torch.where(p > 0, p * (logp - at), torch.zeros_like(p)).sum(1)
    grad = tau * q.scatter_add(1, ids.long(), -p)
    # A logit's distance from the largest is rounded once, scaled by a factor that is off by two roundings and rounded
    # again: four of 2^-24 of the exponent, four of the teacher's. Sums of V and k terms, their logarithms, products:
    # V / 64 + 64 more. An exponential is off by its exponent's error times itself.
    near = lambda v: torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v))  # noqa: E731
    each = 4 * (near(at) + near(logp)) + V / 64 + 64 + near(at) + near(logp)
    tol = tau * tau * 2 ** -24 * torch.where(p > 0, p * (4 * near(logp) + 1) * each, torch.zeros_like(p)).sum(1) + 1e-38
    assert ((row.double().cpu() - want).abs() <= tol).all()
    mass = torch.zeros_like(q).scatter_add(1, ids.long(), p * (4 * near(logp) + V / 64 + 64))
    gtol = ref.HALF_STEP["bf16" if logits.dtype == torch.bfloat16 else "f32"] * grad.abs() + tau * 2 ** -24 * (
        q * (4 * near(logq) + V / 64 + 64) + mass) + 1e-38
    assert ((d.double().cpu() - grad).abs() <= gtol).all()


@pytest.mark.parametrize("tau", [2.0 ** e for e in (-60, -40, -30, -28, -20, -10, 10, 20, 40, 60)])
@pytest.mark.parametrize("V", [50, 3000, 140000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_distill_at_every_temperature(dtype, V, tau):
    g = torch.Generator().manual_seed(V)
    logits = (torch.randn(4, V, generator=g) * 2).to(dtype)
    ids = torch.stack([torch.randperm(V, generator=g)[:7] for _ in range(4)]).to(torch.int32)
    ids[0, 0] = logits[0].float().argmax()
    ids[0, 1:] = (ids[0, 0] + torch.arange(1, 7)) % V
    teacher = torch.randn(4, 7, generator=g) * 3
    teacher[0, 0] = 20.0  # the teacher is as sure as the student, and of the same
    distill(logits, ids, teacher, tau)


@pytest.mark.parametrize("offset", [3e4, -3e4, 1.1e10, -3.3e10, 1.7e18])
def test_distill_far_from_zero(offset):
    """What all logits have in common does not count."""
    g = torch.Generator().manual_seed(1)
    logits = torch.randn(5, 700, generator=g) * 2 + offset
    ids = torch.stack([torch.randperm(700, generator=g)[:9] for _ in range(5)]).to(torch.int32)
    ids[:, 0] = logits.argmax(1)
    ids[:, 1:] = (ids[:, :1] + torch.arange(1, 9)) % 700
    distill(logits, ids, torch.randn(5, 9, generator=g), 1.0)


@pytest.mark.parametrize("shape", [("bf16", 2, 64, 1, 32, 4), ("f32", 1, 40, 1, 100, 3), ("bf16", 1, 5, 1, 7, 2)])
def test_rows_before_a_sequence_are_zeros_in_every_form(shape):
    """One token at the start of a sequence, weights of the rows before it that are not finite: the same in the kernel for
    short prompts, in blocks and token by token."""
    n = 4
    c = Case(*shape, tokens=n, seqs=n, slots=n, seed=2)
    c.cw[3, 0], c.cw[c.d + 1, 0], c.cw[-1, -2] = float("inf"), float("nan"), -float("inf")  # in x, in B and in C
    xbc, dt, z = c.rows()
    layer, fresh = c.layer(), ints([0] * n)
    got = [layer.prompt(xbc, dt, c.y(), n, z=z)]
    for form in ("blocks", "step"):
        conv, ssm, y = c.conv.cuda(), c.ssm.cuda(), c.y()
        if form == "blocks":
            layer.prompt(xbc, dt, y, n, z=z, positions=fresh, conv_state=conv, ssm_state=ssm)
        else:
            layer.step(xbc, dt, y, fresh, conv, ssm, z=z)
        got.append(y)
    assert torch.isnan(got[0]).any()
    for y in got[1:]:
        assert torch.equal(torch.isnan(y), torch.isnan(got[0]))


@pytest.mark.parametrize("channel", [3, -1])
def test_a_channel_that_is_not_finite_stays_alone(channel):
    """Of x, one channel's weight spoils that channel's outputs alone; of C every output of the group."""
    c = Case("f32", 2, 20, 2, 24, 4, tokens=2, seqs=2, slots=2, seed=3)
    c.cw[channel, 0] = float("inf")
    xbc, dt, z = c.rows()
    conv, ssm = c.conv.cuda(), c.ssm.cuda()
    y = c.layer().step(xbc, dt, c.y(), ints([0, 0]), conv, ssm, z=z)
    bad = torch.zeros(2, 40, dtype=torch.bool)
    if channel == 3:
        bad[:, 3] = True
    else:
        bad[:, 20:] = True
    assert torch.equal(torch.isnan(y).cpu(), bad)


@pytest.mark.parametrize("dtype, rows, K, O, A, R", [
    ("bf16", 1, 1024, 4096, 1, 16), ("bf16", 48, 512, 640, 40, 16), ("bf16", 48, 512, 640, 7, 40), ("bf16", 300, 640, 512, 3, 8),
    ("bf16", 3333, 192, 3880, 5, 8), ("bf16", 300, 70, 515, 9, 33), ("f32", 1, 1024, 4096, 1, 16), ("f32", 40, 515, 640, 6, 12),
    ("f32", 300, 256, 320, 6, 64), ("f32", 1279, 129, 515, 23, 12), ("f32", 3100, 64, 4070, 5, 24)])
def test_adapters(dtype, rows, K, O, A, R):
    """float32: nothing is rounded but sums of K and of R terms, whose partial sums' squares grow evenly, 2^-24 / sqrt 3 each.
    bf16: the low-rank value enters its product in two halves, rounded by at most 2^-16."""
    c = Adapters(dtype, rows, K, O, A, R, seed=K)
    x, who, y, scale = c.inputs()
    c.operator().project(x, who, y[:, :O], row_scale=scale)
    want, _, _ = ref.adapters(c.x, c.w, c.bias, c.down, c.up, c.ranks, c.who, c.scale)
    shared, _, _ = ref.adapters(c.x, c.w, c.bias, c.down, c.up, c.ranks, None, c.scale)
    low = float((want - shared).norm() / want.norm())
    assert rows == 1 or low > 0.1
    sums = ((K + R) / 6) ** 0.5 * 2 ** -24 + 2 ** -24
    e = 2 * sums if dtype == "f32" else 2 * sums + 2 ** -16 / 3 ** 0.5 * low
    assert off(y[:, :O], want) <= bound(dtype, e)
