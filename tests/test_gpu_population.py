"""The population operators together, as a zero-order step runs them: K antithetic pairs of low-rank probes
share a projection, recur through a state space layer, are read out, and scored against a teacher; the means by
model are the losses of a central-difference update. Then one of the models generates token by token."""
import pytest
import torch

import operators_ref as ref
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu

K, B, L, E, H, P, G, N, W, V, R, TOP = 3, 4, 21, 48, 4, 16, 1, 32, 4, 29, 2, 5
M = 2 * K  # models
CH, D = H * P + 2 * G * N, H * P
WIDE = D + CH + H  # z | x B C | dt


def weights(g):
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(emb=rand(V, E), w_in=rand(WIDE, E) * E ** -0.5, in_d=rand(K, R, E) * E ** -0.5, in_u=rand(K, WIDE, R),
                w_out=rand(V, D) * D ** -0.5, out_d=rand(K, R, D) * D ** -0.5, out_u=rand(K, V, R),
                cw=torch.rand(CH, W, generator=g) - 0.5, cb=rand(CH) * 0.2, decay=-1 - 8 * torch.rand(H, generator=g), skip=rand(H),
                dt_bias=rand(H) - 3)


def operators(w):
    c = {k: v.cuda() for k, v in w.items()}
    return (b.AdapterProjection(b.make_adapter_config(E, WIDE, K, R, "f32"), c["w_in"], None, c["in_d"], c["in_u"]),
            b.ScanLayer(b.make_scan_config(H, P, G, N, W, "f32"), c["cw"], c["cb"], c["decay"], c["skip"], c["dt_bias"]),
            b.AdapterProjection(b.make_adapter_config(D, V, K, R, "f32"), c["w_out"], None, c["out_d"], c["out_u"]))


def test_population_step_and_generation():
    g = torch.Generator().manual_seed(0)
    w, eps = weights(g), 0.05
    tokens = torch.randint(0, V, (B, L), generator=g)
    ids = torch.stack([torch.randperm(V, generator=g)[:TOP] for _ in range(B * L)]).to(torch.int32).repeat(M, 1)
    teacher = torch.randn(B * L, TOP, generator=g).repeat(M, 1).contiguous()
    rows = M * B * L
    model = torch.arange(rows) // (B * L)
    pair, sign = (model // 2).to(torch.int32), (1.0 - 2.0 * (model % 2)) * eps
    x = w["emb"][tokens].reshape(B * L, E).repeat(M, 1)

    proj, layer, out = operators(w)
    wide, y = torch.empty(rows, WIDE, device="cuda"), torch.empty(rows, D, device="cuda")
    logits, row, losses = torch.empty(rows, V, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(M, device="cuda")
    conv, ssm = torch.empty(M * B, W, CH, device="cuda").fill_(float("nan")), torch.empty(M * B, H, P, N, device="cuda").fill_(float("nan"))
    fresh = torch.zeros(M * B, dtype=torch.int32, device="cuda")
    loss = b.DistillLoss(b.make_distill_config(V, TOP, M, 1.0, "f32"))
    who, scale = pair.cuda(), sign.cuda()

    def forward():
        proj.project(x.cuda(), who, wide, row_scale=scale)
        layer.prompt(wide[:, D:D + CH], wide[:, D + CH:], y, M * B, z=wide[:, :D], positions=fresh, conv_state=conv, ssm_state=ssm)
        out.project(y, who, logits, row_scale=scale)
        loss.losses(logits, ids.cuda(), teacher.cuda(), row, losses)

    forward()

    # each model with its own dense weights, in 64 bits
    each, last = [], []
    for m in range(M):
        s = eps * (1 if m % 2 == 0 else -1)
        w_in = w["w_in"].double() + s * w["in_u"][m // 2].double() @ w["in_d"][m // 2].double()
        w_out = w["w_out"].double() + s * w["out_u"][m // 2].double() @ w["out_d"][m // 2].double()
        h = x[:B * L].double() @ w_in.t()
        yy, _, carried = ref.scan(h[:, D:D + CH], h[:, D + CH:], w["cw"], w["cb"], w["decay"], w["skip"], w["dt_bias"], H, P, G, N,
                                  [(i * L, i * L + L) for i in range(B)], z=h[:, :D])
        lg = yy @ w_out.t()
        each.append(ref.distill(lg, ids[:B * L], teacher[:B * L], 1.0, 1)[1][0])
        last.append((w_in, w_out, carried))
    want = torch.stack(each)
    # every stage is within 2^-13 of its magnitudes (split products 8 * 2^-16, float32 sums); the loss moves by at most
    # twice the logits' error, whose magnitudes stay below 2^5 here: 2^-13 * 2^5 * 2 = 2^-7 would be the bound, held to a tenth
    assert (losses.double().cpu() - want).abs().max() <= 2 ** -7 / 10
    diff, ref_diff = (losses[0::2] - losses[1::2]).double().cpu(), want[0::2] - want[1::2]
    assert (diff - ref_diff).abs().max() <= 2 ** -6 / 10

    # one captured step gives the same losses on every replay
    eager = losses.clone()
    graph = torch.cuda.CUDAGraph()
    xs, idc, tc = x.cuda(), ids.cuda(), teacher.cuda()
    with torch.cuda.graph(graph):
        proj.project(xs, who, wide, row_scale=scale)
        layer.prompt(wide[:, D:D + CH], wide[:, D + CH:], y, M * B, z=wide[:, :D], positions=fresh, conv_state=conv, ssm_state=ssm)
        out.project(y, who, logits, row_scale=scale)
        loss.losses(logits, idc, tc, row, losses)
    for _ in range(3):
        losses.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert torch.equal(losses, eager)

    # every model goes on by one token of each of its sequences, from the states that the prompt left
    nxt = torch.randint(0, V, (B,), generator=g)
    one = w["emb"][nxt].repeat(M, 1)
    m1 = torch.arange(M * B) // B
    who1, scale1 = (m1 // 2).to(torch.int32).cuda(), ((1.0 - 2.0 * (m1 % 2)) * eps).cuda()
    wide1, y1, lg1 = torch.empty(M * B, WIDE, device="cuda"), torch.empty(M * B, D, device="cuda"), torch.empty(M * B, V, device="cuda")
    proj.project(one.cuda(), who1, wide1, row_scale=scale1)
    layer.step(wide1[:, D:D + CH], wide1[:, D + CH:], y1, torch.full((M * B,), L, dtype=torch.int32, device="cuda"), conv, ssm, z=wide1[:, :D])
    out.project(y1, who1, lg1, row_scale=scale1)
    for m in range(M):
        w_in, w_out, carried = last[m]
        h = one[:B].double() @ w_in.t()
        yy, mag, _ = ref.scan(h[:, D:D + CH], h[:, D + CH:], w["cw"], w["cb"], w["decay"], w["skip"], w["dt_bias"], H, P, G, N,
                              [(i, i + 1) for i in range(B)], z=h[:, :D], ring=[c[2] for c in carried],
                              state_in=[c[0] for c in carried], positions=[L] * B)
        lg = yy @ w_out.t()
        tol = 2 ** -12 * (mag @ w_out.abs().t() + 1)
        assert ((lg1[m * B:(m + 1) * B].double().cpu() - lg).abs() <= tol).all()
