"""Calls of more workgroups than one dimension of a launch holds (2^32 threads): many short rows. Their rows repeat
those of a smaller call of the same kernels, whose results they must have, to the bit."""
import pytest
import torch

from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu


def repeats(big, base):
    """Whether big's rows are base's over and over, the last time in part."""
    n, m = big.shape[0], base.shape[0]
    whole = n // m * m
    return bool((big[:whole].view(-1, *base.shape) == base).all()) and torch.equal(big[whole:], base[:n - whole])


def spread(base, n):
    return base.repeat(-(-n // base.shape[0]), *[1] * (base.dim() - 1))[:n].contiguous()


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def test_distill_rows():
    g = torch.Generator(device="cuda").manual_seed(1)
    m, n = 1 << 20, (1 << 28) + 33
    logits = torch.randn(m, 2, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, 2, (m, 1), device="cuda", generator=g, dtype=torch.int32)
    teacher = torch.randn(m, 1, device="cuda", generator=g)
    op = b.DistillLoss(b.make_distill_config(2, 1, 1, 1.5, "bf16"))
    want, d_want = torch.empty(m, device="cuda"), torch.empty_like(logits)
    op.grad(logits, ids, teacher, None, want, None, d_want)
    assert want.min() > 0  # -log q of one of two
    row = torch.zeros(n, device="cuda")
    x = spread(logits, n)
    op.grad(x, spread(ids, n), spread(teacher, n), None, row, None, x)
    assert repeats(row, want) and repeats(x, d_want)


def test_adapter_rows():
    g = torch.Generator(device="cuda").manual_seed(2)
    m, n = 1 << 20, (1 << 28) + 70
    op = b.AdapterProjection(b.make_adapter_config(8, 8, 1, 1, "bf16"), *[
        torch.randn(*s, device="cuda", generator=g).bfloat16() for s in ((8, 8), (8,), (1, 1, 8), (1, 8, 1))])
    x = torch.randn(m, 8, device="cuda", generator=g).bfloat16()
    who = torch.randint(-1, 1, (m,), device="cuda", generator=g, dtype=torch.int32)
    want = op.project(x, who, torch.empty_like(x))
    assert want.isfinite().all()
    y = torch.zeros(n, 8, device="cuda", dtype=torch.bfloat16)
    op.project(spread(x, n), spread(who, n), y)
    assert repeats(y, want)


def scan_layer(heads, groups, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    channels = heads + 2 * groups
    layer = b.ScanLayer(b.make_scan_config(heads, 1, groups, 1, 2, "bf16"), rand(channels, 2).bfloat16(), None, -rand(heads).exp())
    return layer, channels, rand


@pytest.mark.parametrize("form", ["step", "prompt"])
def test_scan_sequences_with_states(form):
    heads, m, n = 32, 1 << 10, 1 << (20 if form == "step" else 19)
    layer, channels, rand = scan_layer(heads, 1, 3)
    xbc, dt = rand(m, channels).bfloat16(), rand(m, heads).bfloat16()
    conv, ssm = rand(m, 2, channels).bfloat16(), rand(m, heads, 1, 1)
    positions = torch.arange(m, device="cuda", dtype=torch.int32) % 5

    def run(k):
        x, y, c, s = spread(xbc, k), torch.zeros(k, heads, device="cuda", dtype=torch.bfloat16), spread(conv, k), spread(ssm, k)
        if form == "step":
            layer.step(x, spread(dt, k), y, spread(positions, k), c, s)
        else:
            layer.prompt(x, spread(dt, k), y, k, positions=spread(positions, k), conv_state=c, ssm_state=s)
        return y, c, s

    base, big = run(m), run(n)
    assert not torch.equal(base[2], ssm) and base[0].isfinite().all()
    for whole, part in zip(big, base):
        assert repeats(whole, part)


def test_scan_short_sequences():
    heads, m, n = 16, 1 << 10, 1 << 20
    layer, channels, rand = scan_layer(heads, heads, 4)
    xbc, dt = rand(m, channels).bfloat16(), rand(m, heads).bfloat16()
    base, big = torch.zeros(m, heads, device="cuda", dtype=torch.bfloat16), torch.zeros(n, heads, device="cuda", dtype=torch.bfloat16)
    layer.prompt(xbc, dt, base, m)
    layer.prompt(spread(xbc, n), spread(dt, n), big, n)
    assert base.isfinite().all() and base.any() and repeats(big, base)


@pytest.mark.parametrize("form", ["step", "prompt"])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_scan_far_positions(form, width):
    """The last positions that 32 bits hold: only their place in the ring counts (12 is a multiple of every width)."""
    heads, slots = 3, 4
    g = torch.Generator(device="cuda").manual_seed(width)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    layer = b.ScanLayer(b.make_scan_config(heads, 5, 1, 6, width, "f32"), rand(27, width), None, -rand(heads).exp())
    n = slots * (1 if form == "step" else 70)
    xbc, dt, conv, ssm = rand(n, 27), rand(n, heads), rand(slots, width, 27), rand(slots, heads, 5, 6)
    far = torch.tensor([2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 8, 2 ** 30], dtype=torch.int64)

    def run(positions):
        y, c, s = torch.zeros(n, 15, device="cuda"), conv.clone(), ssm.clone()
        at = positions.to(torch.int32).cuda()
        if form == "step":
            layer.step(xbc, dt, y, at, c, s)
        else:
            layer.prompt(xbc, dt, y, slots, positions=at, conv_state=c, ssm_state=s)
        return y, c, s

    near = run(far % 12 + 12)
    assert near[0].isfinite().all() and not torch.equal(near[2], ssm)
    for a, c in zip(run(far), near):
        assert torch.equal(a, c)


def test_two_calls_at_once():
    """The same operators on two streams: each call has a workspace of its own."""
    g = torch.Generator(device="cuda").manual_seed(9)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    layer, channels, _ = scan_layer(16, 1, 5)
    adapters = b.AdapterProjection(b.make_adapter_config(256, 320, 3, 8, "f32"), rand(320, 256), None, rand(3, 8, 256), rand(3, 320, 8))
    loss = b.DistillLoss(b.make_distill_config(999, 4, 1, 2.0, "f32"))
    inputs = []
    for _ in range(2):
        ids = torch.randint(0, 999, (300, 4), device="cuda", generator=g, dtype=torch.int32)
        inputs.append((rand(3000, channels).bfloat16(), rand(3000, 16).bfloat16(), rand(300, 256),
                       torch.randint(-1, 3, (300,), device="cuda", generator=g, dtype=torch.int32), rand(300, 999), ids, rand(300, 4)))

    def run(xbc, dt, x, who, logits, ids, teacher):
        y, z = torch.empty(3000, 16, device="cuda", dtype=torch.bfloat16), torch.empty(300, 320, device="cuda")
        few = torch.empty(40, 320, device="cuda")
        row, d = torch.empty(300, device="cuda"), torch.empty_like(logits)
        layer.prompt(xbc, dt, y, 3)
        adapters.project(x, who, z)
        adapters.project(x[:40], who[:40], few)
        loss.grad(logits, ids, teacher, None, row, None, d)
        return y, z, few, row, d

    want = [run(*i) for i in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, i in zip(streams, inputs):
            with torch.cuda.stream(s):
                got.append(run(*i))
        torch.cuda.synchronize()
        for a, c in zip(got, want):
            for u, v in zip(a, c):
                assert torch.equal(u, v)
