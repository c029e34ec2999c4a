"""The gated delta rule against its 64-bit definition, token by token."""
import math

import pytest
import torch

import more_operators_ref as ref
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu

NAN = float("nan")


def inputs(g, n, heads, groups, kd, vd, dtype, wide=True):
    t = ref.TYPES[dtype]
    widths = [groups * kd, groups * kd, heads * vd, heads, heads]
    if wide:  # side by side in one projection's output, a few columns apart from its ends
        x = torch.randn(n, sum(widths) + 3, generator=g).to(t)
        at = [3 + sum(widths[:i]) for i in range(6)]
        parts = [x[:, a:c] for a, c in zip(at, at[1:])]
    else:
        parts = [torch.randn(n, w, generator=g).to(t) for w in widths]
    decay = -0.2 - 8 * torch.rand(heads, generator=g)
    bias = torch.randn(heads, generator=g) - 3
    return parts, decay, bias


def on_gpu(parts):
    base = parts[0]._base
    if base is None:
        return [p.cuda() for p in parts]
    whole = base.cuda()
    return [whole[:, p.storage_offset():p.storage_offset() + p.shape[1]] for p in parts]


def layer_of(heads, groups, kd, vd, dtype, decay, bias, **kw):
    return b.DeltaLayer(b.make_delta_config(heads, groups, kd, vd, dtype, **kw), decay.cuda(), None if bias is None else bias.cuda())


SHAPES = [(1, 1, 1, 1), (4, 2, 16, 16), (6, 2, 100, 40), (8, 4, 128, 128), (2, 1, 256, 256), (3, 3, 33, 5), (2, 2, 64, 192), (4, 1, 24, 129)]
LENGTHS = [0, 1, 63, 64, 65, 130, 2, 200, 17]


def check(y, want, part, dtype, kd, what):
    err = (y.double().cpu() - want).abs()
    tol = ref.delta_tol(want, part, dtype, kd) + 1e-30
    assert (err <= tol).all(), f"{what}: error {float((err / tol).max()):.2f} of what it may be"


LONG = [700, 0, 1, 129, 350, 64, 15, 16, 17]  # more than 128 tokens a sequence on average: no mixed launches


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads, groups, kd, vd, lengths", [(*s, LENGTHS) for s in SHAPES] + [(4, 2, 100, 40, LONG), (2, 1, 128, 32, LONG)])
def test_ragged_prompts(heads, groups, kd, vd, lengths, dtype):
    g = torch.Generator().manual_seed(heads * 1000 + kd)
    n, seqs = sum(lengths) + 4, len(lengths)  # four rows behind the last sequence
    parts, decay, bias = inputs(g, n, heads, groups, kd, vd, dtype)
    offsets = [0]
    for x in lengths:
        offsets.append(offsets[-1] + x)
    bounds = list(zip(offsets, offsets[1:]))
    slots = torch.tensor([4, 0, 7, 2, -1, 9, 1, 3, 10], dtype=torch.int32)  # of 11; one keeps nothing
    positions = torch.tensor([5, 0, 3, 8, 9, -2, 1, 0, 70], dtype=torch.int32)
    state = torch.randn(11, heads, vd, kd, generator=g) * 0.3
    out = torch.full((11, heads, vd, kd), 7.0, device="cuda")
    y = torch.full((n, heads * vd + 3), 5.0, dtype=ref.TYPES[dtype], device="cuda")[:, :heads * vd]
    layer = layer_of(heads, groups, kd, vd, dtype, decay, bias)
    before = state.cuda()
    layer.prompt(*on_gpu(parts), y, seqs, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), slots=slots.cuda(),
                 positions=positions.cuda(), state=before, state_out=out)
    start = [state[s] if s >= 0 else None for s in slots.tolist()]
    pos = [p if s >= 0 else 0 for p, s in zip(positions.tolist(), slots.tolist())]
    want, part, carried = ref.delta(*parts, decay, bias, heads, groups, kd, vd, bounds, kd ** -0.5, state_in=start, positions=pos)
    end = offsets[-1]
    check(y[:end], want[:end], part[:end], dtype, kd, "y")
    assert (y[end:] == 5.0).all()
    assert torch.equal(before.cpu(), state)
    got = out.double().cpu()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            S, E = carried[i]
            tol = ref.delta_eps(kd) * (E[:, None, None] + S.flatten(1).norm(dim=1)[:, None, None]) + 1e-30
            assert ((got[s] - S).abs() <= tol).all(), (i, float(((got[s] - S).abs() / tol).max()))
    assert (got[[5, 6, 8]] == 7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs, each, heads, groups, kd, vd", [(1, 1, 2, 1, 128, 128), (37, 10, 4, 2, 64, 64), (3, 129, 2, 2, 128, 64),
                                                               (2, 500, 1, 1, 32, 16), (5, 32, 2, 1, 128, 32), (5, 33, 2, 1, 128, 32), (5, 16, 2, 1, 200, 32),
                                                               (5, 17, 2, 1, 200, 32)])
def test_equal_prompts_without_a_state(seqs, each, heads, groups, kd, vd, dtype):
    g = torch.Generator().manual_seed(seqs * each)
    parts, decay, _ = inputs(g, seqs * each, heads, groups, kd, vd, dtype, wide=False)
    y = torch.empty(seqs * each, heads * vd, dtype=ref.TYPES[dtype], device="cuda")
    layer = layer_of(heads, groups, kd, vd, dtype, decay, None, q_scale=-1.5, norm_eps=0.25)
    layer.prompt(*on_gpu(parts), y, seqs)
    want, part, _ = ref.delta(*parts, decay, None, heads, groups, kd, vd, [(i * each, i * each + each) for i in range(seqs)], -1.5, 0.25)
    check(y, want, part, dtype, kd, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows, heads, groups, kd, vd", [(1, 8, 4, 128, 128), (5, 4, 4, 16, 16), (7, 6, 2, 100, 40), (3, 2, 1, 256, 256),
                                                         (4, 3, 3, 33, 5), (130, 2, 1, 64, 64), (2, 1, 1, 1, 1), (9, 4, 2, 30, 70)])
def test_steps(rows, heads, groups, kd, vd, dtype):
    g = torch.Generator().manual_seed(rows + kd)
    parts, decay, bias = inputs(g, rows, heads, groups, kd, vd, dtype)
    slots = torch.randperm(rows + 3, generator=g)[:rows].to(torch.int32)
    positions = torch.randint(0, 9, (rows,), generator=g, dtype=torch.int32)
    if rows > 2:
        slots[1] = -1
        positions[2] = 0
    state = torch.randn(rows + 3, heads, vd, kd, generator=g) * 0.3
    y = torch.full((rows, heads * vd), 5.0, dtype=ref.TYPES[dtype], device="cuda")
    layer = layer_of(heads, groups, kd, vd, dtype, decay, bias)
    cache = state.cuda()
    layer.step(*on_gpu(parts), y, positions.cuda(), cache, slots=slots.cuda())
    want, part, carried = ref.delta(*parts, decay, bias, heads, groups, kd, vd, [(i, i + 1) for i in range(rows)], kd ** -0.5,
                                    state_in=[state[max(s, 0)] for s in slots.tolist()], positions=positions.tolist())
    real = slots >= 0
    check(y[real.cuda()], want[real], part[real], dtype, kd, "y")
    assert (y[~real.cuda()] == 5.0).all()
    expect = state.double()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            expect[s] = carried[i][0]
    tol = ref.delta_eps(kd) * (expect.flatten(2).norm(dim=2)[:, :, None, None] * 2 + 2 * vd ** 0.5 * 4)
    assert ((cache.double().cpu() - expect).abs() <= tol).all()
    untouched = [s for s in range(rows + 3) if s not in slots.tolist()]
    assert torch.equal(cache.cpu()[untouched], state[untouched])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_steps_go_on_from_a_prompt(dtype):
    """A prompt, then single tokens, and the whole as one prompt, agree with the definition."""
    g = torch.Generator().manual_seed(3)
    heads, groups, kd, vd, L, more = 4, 2, 64, 48, 70, 5
    parts, decay, bias = inputs(g, 2 * (L + more), heads, groups, kd, vd, dtype, wide=False)
    layer = layer_of(heads, groups, kd, vd, dtype, decay, bias)
    want, part, _ = ref.delta(*parts, decay, bias, heads, groups, kd, vd, [(0, L + more), (L + more, 2 * (L + more))], kd ** -0.5)
    by_seq = [p.view(2, L + more, -1).cuda() for p in parts]
    state = torch.full((2, heads, vd, kd), NAN, device="cuda")
    y = torch.empty(2, L + more, heads * vd, dtype=ref.TYPES[dtype], device="cuda")
    front = [p[:, :L].reshape(2 * L, -1).contiguous() for p in by_seq]
    yf = torch.empty(2 * L, heads * vd, dtype=ref.TYPES[dtype], device="cuda")
    layer.prompt(*front, yf, 2, positions=torch.zeros(2, dtype=torch.int32, device="cuda"), state=state)
    y[:, :L] = yf.view(2, L, -1)
    for t in range(L, L + more):
        one = [p[:, t].contiguous() for p in by_seq]
        yt = torch.empty(2, heads * vd, dtype=ref.TYPES[dtype], device="cuda")
        layer.step(*one, yt, torch.full((2,), t, dtype=torch.int32, device="cuda"), state)
        y[:, t] = yt
    check(y.view(2 * (L + more), -1), want, part, dtype, kd, "y")


@pytest.mark.parametrize("step", [True, False])
def test_bad_slots(step):
    """A slot out of range, and one that an earlier sequence has: NaN rows, no state touched."""
    g = torch.Generator().manual_seed(4)
    rows, heads, groups, kd, vd = 6, 2, 1, 32, 24
    parts, decay, bias = inputs(g, rows, heads, groups, kd, vd, "f32")
    slots = torch.tensor([2, 5, 2, 0, 9, -1], dtype=torch.int32)
    state = torch.randn(6, heads, vd, kd, generator=g)
    cache, y = state.cuda(), torch.full((rows, heads * vd), 5.0, device="cuda")
    pos = torch.ones(rows, dtype=torch.int32, device="cuda")
    layer = layer_of(heads, groups, kd, vd, "f32", decay, bias)
    if step:
        layer.step(*on_gpu(parts), y, pos, cache, slots=slots.cuda())
    else:
        layer.prompt(*on_gpu(parts), y, rows, slots=slots.cuda(), positions=pos, state=cache)
    bad = [2, 4]
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[[0, 1, 3, 5]]).all()
    assert torch.equal(cache.cpu()[[1, 3, 4]], state[[1, 3, 4]]) and torch.isfinite(cache).all()
    assert (y[5] == 5.0).all() == step


def test_offsets_are_clamped():
    g = torch.Generator().manual_seed(5)
    heads, groups, kd, vd, n = 2, 1, 16, 16, 30
    parts, decay, bias = inputs(g, n, heads, groups, kd, vd, "f32")
    layer = layer_of(heads, groups, kd, vd, "f32", decay, bias)
    y = torch.full((n, heads * vd), 5.0, device="cuda")
    layer.prompt(*on_gpu(parts), y, 4, offsets=torch.tensor([-7, 10, 4, 20, 99], dtype=torch.int32, device="cuda"))
    want, part, _ = ref.delta(*parts, decay, bias, heads, groups, kd, vd, [(0, 10), (10, 20), (20, 30)], kd ** -0.5)
    check(y, want, part, "f32", kd, "y")


def test_no_tokens():
    g = torch.Generator().manual_seed(6)
    parts, decay, bias = inputs(g, 0, 2, 1, 16, 16, "f32", wide=False)
    layer = layer_of(2, 1, 16, 16, "f32", decay, bias)
    state = torch.randn(3, 2, 16, 16, generator=g)
    out = torch.full((3, 2, 16, 16), 7.0, device="cuda")
    y = torch.empty(0, 32, device="cuda")
    pos = torch.tensor([4, 0, 1], dtype=torch.int32, device="cuda")
    layer.prompt(*on_gpu(parts), y, 3, positions=pos, state=state.cuda(), state_out=out)
    assert torch.equal(out[[0, 2]].cpu(), state[[0, 2]]) and (out[1] == 0).all()
    layer.prompt(*on_gpu(parts), y, 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 16, 100])
def test_what_is_not_finite_stays_in_its_sequence(L, dtype):
    g = torch.Generator().manual_seed(7)
    heads, groups, kd, vd = 2, 1, 64, 32
    parts, decay, bias = inputs(g, 3 * L, heads, groups, kd, vd, dtype, wide=False)
    layer = layer_of(heads, groups, kd, vd, dtype, decay, bias)
    y0, y1 = (torch.empty(3 * L, heads * vd, dtype=ref.TYPES[dtype], device="cuda") for _ in range(2))
    s0, s1 = (torch.full((3, heads, vd, kd), NAN, device="cuda") for _ in range(2))  # what lies in a fresh slot is not read
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    layer.prompt(*on_gpu(parts), y0, 3, positions=pos, state=s0)
    for which, value in ((0, NAN), (1, math.inf), (2, -math.inf), (3, NAN), (4, NAN), (1, 1.5e38)):
        spoilt = [p.clone() for p in parts]
        spoilt[which][L + L // 2, 0] = value
        s1.fill_(NAN)
        layer.prompt(*on_gpu(spoilt), y1, 3, positions=pos, state=s1)
        mine = slice(L, 2 * L)
        assert torch.equal(y1[:L], y0[:L]) and torch.equal(y1[2 * L:], y0[2 * L:])
        assert torch.equal(s1[[0, 2]], s0[[0, 2]])
        later = y1[mine][L // 2:, 0] if which > 0 else y1[mine][L // 2, 0]  # a query enters no state
        assert not torch.isfinite(later).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_far_gates_and_small_rows(dtype):
    """Steps that forget everything, steps of zero, strengths of zero and one, rows of zeros and tiny rows."""
    g = torch.Generator().manual_seed(8)
    heads, groups, kd, vd, L = 2, 1, 64, 32, 150
    parts, decay, bias = inputs(g, L, heads, groups, kd, vd, dtype, wide=False)
    q, k, v, dt, beta = parts
    dt[5], dt[40], dt[70:80] = 3000.0, -200.0, 30.0
    beta[7], beta[8], beta[9] = -200.0, 200.0, 0.0
    k[20], q[21] = 0.0, 0.0
    k[30] *= 2.0 ** -30
    q[31] *= 2.0 ** -30
    k[33] *= 2.0 ** 50
    q[34] *= 2.0 ** 50
    layer = layer_of(heads, groups, kd, vd, dtype, decay, bias)
    y = torch.empty(L, heads * vd, dtype=ref.TYPES[dtype], device="cuda")
    layer.prompt(*on_gpu(parts), y, 1)
    want, part, _ = ref.delta(*parts, decay, bias, heads, groups, kd, vd, [(0, L)], kd ** -0.5)
    check(y, want, part, dtype, kd, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_precision_in_the_2_norm(dtype):
    """A sum of random terms is far below its magnitudes: y and the state by the 2-norm of their errors. float32: 2^-20
    of them (operands of 24 bits, sums of 128 and 64 terms); bf16's y against the nearest bf16 of the exact one, which an
    operand of 16 bits moves by 2^-15 at most."""
    g = torch.Generator().manual_seed(9)
    heads, groups, kd, vd, L = 4, 2, 128, 64, 700
    parts, decay, bias = inputs(g, L, heads, groups, kd, vd, dtype)
    layer = layer_of(heads, groups, kd, vd, dtype, decay * 0.2, bias)
    y = torch.empty(L, heads * vd, dtype=ref.TYPES[dtype], device="cuda")
    state = torch.zeros(1, heads, vd, kd, device="cuda")
    layer.prompt(*on_gpu(parts), y, 1, state=state)
    want, _, carried = ref.delta(*parts, decay * 0.2, bias, heads, groups, kd, vd, [(0, L)], kd ** -0.5)
    assert (state[0].double().cpu() - carried[0][0]).norm() <= 2 ** -20 * carried[0][0].norm()
    if dtype == "f32":
        assert (y.double().cpu() - want).norm() <= 2 ** -20 * want.norm()
    else:
        # an element next to a border between two bf16 values may fall on the other side: steps of 2^-8, in the share of
        # elements that the error, 2^-15 of them, is of a step's width
        near = want.to(torch.bfloat16).double()
        assert (y.double().cpu() - near).norm() <= (2 ** -15 * 2 ** -7) ** 0.5 * want.norm()


def test_streams_and_graphs():
    g = torch.Generator().manual_seed(10)
    heads, groups, kd, vd, L = 4, 2, 128, 64, 130
    parts, decay, bias = inputs(g, 2 * L, heads, groups, kd, vd, "bf16")
    layer = layer_of(heads, groups, kd, vd, "bf16", decay, bias)
    dev = on_gpu(parts)
    offsets = torch.tensor([0, 100, 2 * L], dtype=torch.int32, device="cuda")
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    state = torch.zeros(2, heads, vd, kd, device="cuda")
    y = torch.zeros(2 * L, heads * vd, dtype=torch.bfloat16, device="cuda")

    def call(stream=None):
        layer.prompt(*dev, y, 2, offsets=offsets, slots=slots, positions=pos, state=state, stream=stream)
        layer.step(*[d[:2] for d in dev], y[:2], pos + 5, state, slots=slots, stream=stream)

    call()
    want_y, want_s = y.clone(), state.clone()
    side = torch.cuda.Stream()
    y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    assert torch.equal(y, want_y) and torch.equal(state, want_s)
    graph = torch.cuda.CUDAGraph()
    later = pos + 5
    with torch.cuda.graph(graph):
        layer.prompt(*dev, y, 2, offsets=offsets, slots=slots, positions=pos, state=state)
        layer.step(*[d[:2] for d in dev], y[:2], later, state, slots=slots)
    for _ in range(3):
        y.zero_()
        state.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert torch.equal(y, want_y) and torch.equal(state, want_s)
    # other slots and lengths in the same buffers
    offsets.copy_(torch.tensor([0, 64, 2 * L - 3]))
    slots.copy_(torch.tensor([0, 1]))
    call()
    want_y, want_s = y.clone(), state.clone()
    y.zero_()
    torch.cuda.synchronize()
    graph.replay()
    assert torch.equal(y[:2 * L - 3], want_y[:2 * L - 3]) and torch.equal(state, want_s)


def test_class_refuses():
    g = torch.Generator().manual_seed(11)
    parts, decay, bias = inputs(g, 4, 2, 1, 16, 16, "f32", wide=False)
    layer = layer_of(2, 1, 16, 16, "f32", decay, bias)
    q, k, v, dt, beta = on_gpu(parts)
    y, state = torch.empty(4, 32, device="cuda"), torch.zeros(4, 2, 16, 16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (dict(q=q[:, :8]), dict(k=k.bfloat16()), dict(v=v[:3]), dict(dt=dt.cpu()), dict(beta=beta.t().contiguous().t()),
                dict(y=y[:, :31]), dict(state=state[:, :, :, :8]), dict(state=None, state_out=state), dict(positions=pos.long()),
                dict(slots=pos[:3])):
        kw = dict(q=q, k=k, v=v, dt=dt, beta=beta, y=y, positions=pos, state=state) | bad
        with pytest.raises((ValueError, b.CdrgeError)):
            layer.step(**kw)
        with pytest.raises((ValueError, b.CdrgeError)):
            layer.prompt(n_seqs=4, **kw)
    with pytest.raises(b.CdrgeError):
        layer.prompt(q, k, v, dt, beta, y, 3)
