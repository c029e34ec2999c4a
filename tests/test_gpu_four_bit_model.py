"""Projections by 4-bit weights, the delta rule, token scores and the distillation loss together, as a program evaluates a
model: a prompt and its scores, a second model's loss against the alternatives, then token by token from the state that
the prompt left. Quantisation is not continuous, so each stage is held against its definition on what the stage before it
gave."""
import pytest
import torch

import more_operators_ref as ref
import operators_ref
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu

B, L, E, H, G, KD, VD, V, TOP = 3, 70, 96, 4, 2, 64, 32, 45, 6
WIDTHS = [G * KD, G * KD, H * VD, H, H]
WIDE = sum(WIDTHS)


def parts_of(wide):
    at = [sum(WIDTHS[:i]) for i in range(6)]
    return [wide[:, a:c] for a, c in zip(at, at[1:])]


def check_projection(x, weights, y, bias=None):
    codes, scales = (w.cpu() for w in weights)
    xv = ref.mx_values(*ref.mx_quantize(x.cpu()), x.shape[1])
    w = ref.mx_values(codes, scales, x.shape[1])
    want, size = xv @ w.t(), xv.abs() @ w.abs().t()
    # exact products, float32 sums, one rounding to bf16
    tol = ref.HALF_STEP["bf16"] * want.abs() + (2 * x.shape[1] + 64) * 2 ** -24 * size
    assert ((y.double().cpu() - want).abs() <= tol).all()


def check_delta(wide, y, decay, bias, bounds, state_in=None, positions=None):
    want, part, carried = ref.delta(*(p.cpu() for p in parts_of(wide)), decay, bias, H, G, KD, VD, bounds, KD ** -0.5,
                                    state_in=state_in, positions=positions)
    assert ((y.double().cpu() - want).abs() <= ref.delta_tol(want, part, "bf16", KD)).all()
    return carried


def test_a_model_of_four_bits():
    g = torch.Generator().manual_seed(0)
    w_in, w_out = torch.randn(WIDE, E, generator=g) * E ** -0.5, torch.randn(V, H * VD, generator=g) * 3 * (H * VD) ** -0.5
    decay, bias = -0.5 - 4 * torch.rand(H, generator=g), torch.randn(H, generator=g) - 3
    emb = torch.randn(V, E, generator=g).bfloat16()
    f_in, f_out = (b.MxFormat(b.make_mx_config(k, 1, "f32")) for k in (E, H * VD))
    in_, out_ = f_in.quantize(w_in.cuda(), *f_in.empty(WIDE)), f_out.quantize(w_out.cuda(), *f_out.empty(V))
    proj = b.MxProjection(b.make_mx_config(E, WIDE, "bf16"), *in_)
    layer = b.DeltaLayer(b.make_delta_config(H, G, KD, VD, "bf16"), decay.cuda(), bias.cuda())
    head = b.MxProjection(b.make_mx_config(H * VD, V, "bf16"), *out_)
    scores = b.TokenScores(b.make_score_config(V, TOP, 1.0, "bf16"))
    loss = b.DistillLoss(b.make_distill_config(V, TOP, 1, 1.0, "bf16"))

    tokens = torch.randint(0, V, (B, L + 1), generator=g)
    n = B * L
    x = emb[tokens[:, :-1]].reshape(n, E).cuda()
    given = tokens[:, 1:].reshape(n).to(torch.int32).cuda()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    wide, y, logits = torch.empty(n, WIDE, **bf), torch.empty(n, H * VD, **bf), torch.empty(n, V, **bf)
    lp, h, top_lp = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, TOP, device="cuda")
    top = torch.empty(n, TOP, dtype=torch.int32, device="cuda")
    state = torch.full((B, H, VD, KD), float("nan"), device="cuda")
    fresh = torch.zeros(B, dtype=torch.int32, device="cuda")
    student = (torch.randn(n, V, generator=g) * 2).bfloat16().cuda()
    row, mean, grad = torch.empty(n, device="cuda"), torch.empty(1, device="cuda"), torch.empty(n, V, **bf)
    d_lp, d_h, d_logits = torch.full((n,), -1.0 / n, device="cuda"), torch.full((n,), -0.01 / n, device="cuda"), torch.empty(n, V, **bf)

    def forward():
        proj.project(x, wide)
        layer.prompt(*parts_of(wide), y, B, positions=fresh, state=state)
        head.project(y, logits)
        scores.scores(logits, given, lp, h, top, top_lp)
        loss.grad(student, top, top_lp, None, row, mean, grad)
        scores.grad(logits, given, d_lp, d_h, d_logits)

    forward()
    check_projection(x, in_, wide)
    carried = check_delta(wide, y, decay, bias, [(i * L, i * L + L) for i in range(B)])
    check_projection(y, out_, logits)
    want, entropy, g_lp, g_h = ref.scores(logits.cpu(), given.cpu(), 1.0)
    tol = 2 ** -24 * (V / 64 + 64 + 8 * 60)
    assert ((lp.double().cpu() - want).abs() <= tol).all() and ((h.double().cpu() - entropy).abs() <= tol * (1 + entropy)).all()
    assert torch.equal(top.cpu(), ref.top(logits.cpu(), TOP))
    g_want = d_lp.double().cpu()[:, None] * g_lp + d_h.double().cpu()[:, None] * g_h
    assert ((d_logits.double().cpu() - g_want).abs() <= 2 ** -8 * g_want.abs() + 2 * tol / n).all()
    # the alternatives are a teacher's entries: their log probabilities are its logits up to a constant
    r_row, r_mean, r_grad, width = operators_ref.distill(student.cpu(), top.cpu(), top_lp.cpu(), 1.0, 1)
    assert ((row.double().cpu() - r_row).abs() <= 2 ** -24 * width * (1 + r_row.abs())).all()
    assert abs(float(mean) - float(r_mean)) <= 2 ** -24 * float(width.max()) * (1 + float(r_row.max()))
    assert ((grad.double().cpu() - r_grad).abs() <= 2 ** -8 * r_grad.abs() + 2 ** -24 * width[:, None]).all()

    # captured, replayed: the same bits, with other work in between
    outs = (wide, y, logits, lp, h, top, top_lp, row, mean, grad, d_logits, state)
    eager = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward()
    for _ in range(3):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(outs, eager))

    # a token more of each sequence, twice
    before = [c[0] for c in carried]
    for t in range(L, L + 2):
        one = emb[torch.randint(0, V, (B,), generator=g)].cuda()
        w1, y1, l1 = torch.empty(B, WIDE, **bf), torch.empty(B, H * VD, **bf), torch.empty(B, V, **bf)
        start = [s.double() for s in state.cpu()]
        # the state is within its bound of the definition's before the first of them
        if t == L:
            for s, c in zip(start, carried):
                assert ((s - c[0]).abs() <= ref.delta_eps(KD) * (c[1] + c[0].flatten(1).norm(dim=1))[:, None, None]).all()
        proj.project(one, w1)
        layer.step(*parts_of(w1), y1, torch.full((B,), t, dtype=torch.int32, device="cuda"), state)
        head.project(y1, l1)
        check_projection(one, in_, w1)
        before = check_delta(w1, y1, decay, bias, [(i, i + 1) for i in range(B)], state_in=start, positions=[t] * B)
        check_projection(y1, out_, l1)
    assert len(before) == B
