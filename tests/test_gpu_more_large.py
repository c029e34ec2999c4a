"""The delta rule, token scores and 4-bit rows where counts are large: many sequences with slots named twice, and rows that lie
past 2^32 bytes or elements, against smaller calls, bit by bit, and the definitions."""
import pytest
import torch

import more_operators_ref as ref
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu

BF = dict(dtype=torch.bfloat16, device="cuda")


def delta(g, heads, kd, vd, n, stride=0):
    """Layer, and q, k, v, dt, beta of n rows, all views of one tensor if a stride is given."""
    decay, bias = (-0.5 - 4 * torch.rand(heads, generator=g)).cuda(), (torch.randn(heads, generator=g) - 3).cuda()
    layer = b.DeltaLayer(b.make_delta_config(heads, 1, kd, vd, "bf16"), decay, bias)
    widths = [kd, kd, heads * vd, heads, heads]
    at = [sum(widths[:i]) for i in range(6)]
    wide = torch.empty(n, max(stride, at[-1]), **BF)
    some = torch.randn(997, at[-1], generator=g).bfloat16().cuda()
    for r in range(0, n, 997):  # the same rows again: what matters is where they lie
        wide[r:r + 997, :at[-1]] = some[:min(997, n - r)]
    return layer, [wide[:, a:c] for a, c in zip(at, at[1:])]


@pytest.mark.parametrize("heads, kd, vd, each", [(4, 4, 4, 0), (2, 16, 70, 0), (4, 64, 16, 0), (4, 4, 4, 1), (4, 4, 4, 40)])
def test_many_sequences_and_slots_named_twice(heads, kd, vd, each):
    g = torch.Generator().manual_seed(kd + each)
    seqs, part = 8192, 1024
    layer, rows = delta(g, heads, kd, vd, seqs * max(each, 1))
    slots = torch.randperm(seqs + 5, generator=g)[:seqs].to(torch.int32)
    free = sorted(set(range(seqs + 5)) - set(slots.tolist()))
    twice = [7, 64, 1000, 4097, 8191]
    for i in twice:
        free.append(int(slots[i]))
        slots[i] = slots[i // 2]
    slots[5], slots[5000] = -1, seqs + 5
    positions = torch.randint(0, 3, (seqs,), generator=g, dtype=torch.int32)
    state = (torch.randn(seqs + 5, heads, vd, kd, generator=g) * 0.3).cuda()
    first = state.clone()
    y = torch.full((seqs * max(each, 1), heads * vd), 5.0, **BF)

    def call(rows, y, slots, positions, state):
        s, p = slots.cuda(), positions.cuda()
        if each:
            layer.prompt(*rows, y, len(slots), slots=s, positions=p, state=state)
        else:
            layer.step(*rows, y, p, state, slots=s)

    call(rows, y, slots, positions, state)
    bad = torch.zeros(seqs, dtype=torch.bool)
    bad[twice + [5000]] = True
    want, want_state = torch.full_like(y, 5.0), first.clone()
    alone = torch.where(bad, torch.full_like(slots, -1), slots)
    for i in range(0, seqs, part):
        at = slice(i * max(each, 1), (i + part) * max(each, 1))
        call([r[at] for r in rows], want[at], alone[i:i + part], positions[i:i + part], want_state)
    got, want = y.view(seqs, -1), want.view(seqs, -1)
    assert got[bad.cuda()].isnan().all()
    assert torch.equal(got[~bad.cuda()], want[~bad.cuda()])
    assert torch.equal(state, want_state)
    assert torch.equal(state[free], first[free]) or not free
    assert each or (got[5] == 5.0).all()


def test_delta_rows_far_apart():
    g = torch.Generator().manual_seed(1)
    lengths = [2000, 30, 2500, 70]
    n, stride = sum(lengths), 1 << 20  # 4,600 rows of 2 MB
    layer, rows = delta(g, 2, 128, 48, n, stride)
    y = torch.empty(n, stride, **BF)[:, :96]
    offsets = [0, 2000, 2030, 4530, 4600]
    layer.prompt(*rows, y, 4, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    for a, c in zip(offsets, offsets[1:]):
        near = torch.empty(c - a, 96, **BF)
        layer.prompt(*[r[a:c].contiguous() for r in rows], near, 1, offsets=torch.tensor([0, c - a], dtype=torch.int32, device="cuda"))
        if c - a <= 100:
            want, part, _ = ref.delta(*[r[a:c].cpu() for r in rows], *(w.cpu() for w in layer._held), 2, 1, 128, 48, [(0, c - a)], 128 ** -0.5)
            for got in (near, y[a:c]):
                assert ((got.double().cpu() - want).abs() <= ref.delta_tol(want, part, "bf16", 128)).all()
        # 30 tokens alone are taken token by token, beside long sequences as a block: other sums
        assert c - a == 30 or torch.equal(y[a:c], near)
    whole = torch.empty(n, 96, **BF)
    layer.prompt(*[r.contiguous() for r in rows], whole, 4, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, whole)


def test_scores_rows_far_apart():
    g = torch.Generator().manual_seed(2)
    n, V, k = 2200, 300, 5
    x = torch.empty(n, 1 << 21, **BF)[:, :V]
    x.copy_(torch.randn(n, V, generator=g))
    tokens = torch.randint(0, V, (n,), generator=g, dtype=torch.int32).cuda()
    s = b.TokenScores(b.make_score_config(V, k, 1.0, "bf16"))

    def run(x, dx):
        out = [torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, k, dtype=torch.int32, device="cuda"),
               torch.empty(n, k, device="cuda")]
        s.scores(x, tokens, *out)
        s.grad(x, tokens, out[1], out[0], dx)
        return out + [dx]

    near = run(x.contiguous(), torch.empty(n, V, **BF))
    far = run(x, x)  # in place
    assert all(torch.equal(a, c) for a, c in zip(near, far))


def test_four_bit_rows_far_apart():
    g = torch.Generator().manual_seed(3)
    n, K, O = 1100, 200, 130
    x = torch.empty(n, 1 << 22, **BF)[:, :K]
    x.copy_(torch.randn(n, K, generator=g))
    f = b.MxFormat(b.make_mx_config(K, 1, "bf16"))
    near, far, back = f.quantize(x.contiguous(), *f.empty(n)), f.quantize(x, *f.empty(n)), torch.empty(n, K, **BF)
    assert all(torch.equal(a, c) for a, c in zip(near, far))
    f.dequantize(*near, back)
    w = f.quantize(torch.randn(O, K, generator=g).bfloat16().cuda(), *f.empty(O))
    proj = b.MxProjection(b.make_mx_config(K, O, "bf16"), *w)
    y = torch.empty(n, O, **BF)
    proj.project(x.contiguous(), y)
    for rows in (n, 60):  # tiles, and some rows
        wide = torch.empty(rows, 1 << 22, **BF)[:, :O]
        proj.project(x[n - rows:], wide)
        small = torch.empty(rows, O, **BF)
        proj.project(x[n - rows:].contiguous(), small)
        assert torch.equal(wide, small) and (rows < n or torch.equal(small, y))
    f.dequantize(*near, x)
    assert torch.equal(x, back)


@pytest.mark.parametrize("rows, O, K", [(550_000, 4100, 40), (60, 1 << 20, 40), (16, 1 << 20, 40), (17, 32_650, 1000), (33, 32_640, 700),
                                        (17, 32_641, 1)])
def test_project_many_outputs(rows, O, K):
    g = torch.Generator().manual_seed(4)
    f = b.MxFormat(b.make_mx_config(K, 1, "bf16"))
    w = f.quantize(torch.randn(O, K, generator=g).bfloat16().cuda(), *f.empty(O))
    x = torch.randn(rows, K, generator=g).bfloat16().cuda()
    bias = torch.randn(O, generator=g).bfloat16().cuda()
    y = torch.empty(rows, O, **BF)
    b.MxProjection(b.make_mx_config(K, O, "bf16"), *w, bias).project(x, y)
    at, to = [0, rows // 2, rows - 2, rows - 1], [0, 1, O // 2, O - 70, O - 2, O - 1]
    xv = ref.mx_values(*ref.mx_quantize(x[at].cpu()), K)
    wv = ref.mx_values(w[0][to].cpu(), w[1][to].cpu(), K)
    bv = bias[to].double().cpu()
    want, size = xv @ wv.t() + bv, xv.abs() @ wv.abs().t() + bv.abs()
    tol = ref.HALF_STEP["bf16"] * want.abs() + (2 * K + 64) * 2 ** -24 * size
    assert ((y[at][:, to].double().cpu() - want).abs() <= tol).all()
