"""Selective scan against the token-by-token definition in 64 bits: prompts (equal and ragged, fresh and
continued) and single tokens, odd widths, padding, bad slots, states in place and apart, graphs and streams."""
import pytest
import torch

import operators_ref as ref
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    """A layer and its inputs, made on the CPU from a seed."""

    def __init__(self, dtype, heads, head_dim, groups, state, width, tokens, seqs, slots=0, gate=True, bias=True, extra=0, seed=0,
                 fast=16.0):
        g = torch.Generator().manual_seed(seed)
        t, self.dtype = T[dtype], dtype
        self.dims = (heads, head_dim, groups, state)
        self.d, self.ch, self.n = heads * head_dim, heads * head_dim + 2 * groups * state, seqs
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        # rows further apart than they are long, and starting anywhere (`extra` elements in)
        wide = rand(tokens, extra + self.d + self.ch + heads + 3).to(t)
        self.z = wide[:, extra:extra + self.d] if gate else None
        self.xbc = wide[:, extra + self.d:extra + self.d + self.ch]
        self.dt = wide[:, extra + self.d + self.ch:extra + self.d + self.ch + heads]
        self.wide, self.extra = wide, extra
        self.cw = (torch.rand(self.ch, width, generator=g) - 0.5).to(t)
        self.cb = (rand(self.ch) * 0.2).to(t) if bias else None
        self.decay = -(1 + (fast - 1) * torch.rand(heads, generator=g))
        self.skip = rand(heads) if bias else None
        self.dt_bias = -4 + 2 * rand(heads) if bias else None
        self.width, self.tokens = width, tokens
        if slots:
            self.conv, self.ssm = rand(slots, width, self.ch).to(t), rand(slots, heads, head_dim, state) * 0.3

    def layer(self):
        self.cfg = b.make_scan_config(*self.dims, self.width, self.dtype)
        dev = lambda v: None if v is None else v.cuda()  # noqa: E731
        return b.ScanLayer(self.cfg, dev(self.cw), dev(self.cb), dev(self.decay), dev(self.skip), dev(self.dt_bias))

    def rows(self):
        w, e = self.wide.cuda(), self.extra
        at = e + self.d
        return w[:, at:at + self.ch], w[:, at + self.ch:at + self.ch + self.dims[0]], (w[:, e:at] if self.z is not None else None)

    def y(self, fill=7.0):
        return torch.full((self.tokens, self.d + 5), fill, dtype=T[self.dtype], device="cuda")[:, :self.d]

    def expect(self, bounds, slots=None, positions=None):
        ring = state = None
        if slots is not None:
            ring, state = [self.conv[s] for s in slots], [self.ssm[s] for s in slots]
        return ref.scan(self.xbc, self.dt, self.cw, self.cb, self.decay, self.skip, self.dt_bias, *self.dims, bounds, self.z, ring,
                        state, positions)


def close(c, got, want, mag, what="y"):
    tol = ref.HALF_STEP[c.dtype] * want.abs() + ref.SCAN_Y[c.dtype] * mag + 1e-30
    err = (got.double().cpu() - want).abs()
    assert torch.isfinite(got).all(), what
    worst = (err / tol).max() if err.numel() else 0
    assert worst <= 1, f"{what}: {float(worst):.2f} of the tolerance"


def close_state(got, want, mag):
    err, tol = (got.double().cpu() - want).abs(), ref.SCAN_STATE * mag + 2 ** -24 * want.abs() + 1e-30
    assert (err <= tol).all(), f"state: {float((err / tol).max()):.2f} of the tolerance"


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


SHAPES = [
    # dtype, heads, head_dim, groups, state, width
    ("bf16", 4, 64, 1, 128, 4), ("f32", 4, 64, 2, 64, 4), ("bf16", 2, 32, 2, 16, 3), ("f32", 3, 40, 1, 100, 2),
    ("bf16", 2, 128, 1, 256, 4), ("bf16", 1, 5, 1, 7, 2), ("f32", 6, 17, 3, 33, 4), ("bf16", 2, 72, 1, 31, 4), ("f32", 1, 256, 1, 200, 3),
]


@pytest.mark.parametrize("lengths", [[1], [10], [63, 1], [64], [65, 130], [200]])
@pytest.mark.parametrize("shape", SHAPES)
def test_prompt_fresh(shape, lengths):
    n = len(lengths)
    c = Case(*shape, tokens=sum(lengths), seqs=n, seed=sum(lengths), extra=3)
    off = [0]
    for v in lengths:
        off.append(off[-1] + v)
    xbc, dt, z = c.rows()
    y = c.layer().prompt(xbc, dt, c.y(), n, z=z, offsets=ints(off))
    want, mag, _ = c.expect(list(zip(off, off[1:])))
    close(c, y, want, mag)


@pytest.mark.parametrize("place", ["in place", "apart"])
@pytest.mark.parametrize("shape", SHAPES)
def test_prompt_ragged_with_states(shape, place):
    """Fresh, continued and empty sequences, one without a slot, rows before, between and behind."""
    lengths, positions = [5, 0, 70, 1, 0, 131, 2, 66], [0, 9, 3, 700, 0, 1, 0, 2]
    slots = [4, 2, 0, 6, 1, 8, -1, 3]
    off = [2]
    for v in lengths:
        off.append(off[-1] + v)
    c = Case(*shape, tokens=off[-1] + 4, seqs=8, slots=10, seed=1, gate=shape[0] == "f32")
    xbc, dt, z = c.rows()
    conv, ssm = c.conv.cuda(), c.ssm.cuda()
    co, so = (conv, ssm) if place == "in place" else (torch.full_like(conv, 3.0), torch.full_like(ssm, 3.0))
    y = c.layer().prompt(xbc, dt, c.y(), 8, z=z, offsets=ints(off), slots=ints(slots), positions=ints(positions), conv_state=conv,
                         ssm_state=ssm, conv_out=co, ssm_out=so)
    bounds = list(zip(off, off[1:]))
    want, mag, carried = c.expect(bounds, slots, [p if s >= 0 else 0 for p, s in zip(positions, slots)])
    assert (y[:2] == 7).all() and (y[off[-1]:] == 7).all()
    close(c, y[2:off[-1]], want[2:off[-1]], mag[2:off[-1]])
    for s in (5, 7, 9):  # slots that nobody named
        assert torch.equal(so[s].cpu(), c.ssm[s] if place == "in place" else torch.full_like(c.ssm[s], 3.0))
    for s, (S, Sm, ring), p, n in zip(slots, carried, positions, lengths):
        if s < 0:
            continue
        close_state(so[s], S, Sm)
        assert torch.equal(co[s].double().cpu(), ring), s
    if place == "apart":
        assert torch.equal(conv.cpu(), c.conv) and torch.equal(ssm.cpu(), c.ssm)


def test_prompt_equal_lengths_match_offsets():
    c = Case("bf16", 4, 64, 1, 64, 4, tokens=60, seqs=6)
    xbc, dt, z = c.rows()
    layer = c.layer()
    want, mag, _ = c.expect([(i, i + 10) for i in range(0, 60, 10)])
    close(c, layer.prompt(xbc, dt, c.y(), 6, z=z), want, mag)
    # the two forms take different kernels, each within its bound of the definition: equal bits are not promised
    close(c, layer.prompt(xbc, dt, c.y(), 6, z=z, offsets=ints(list(range(0, 61, 10)))), want, mag)


@pytest.mark.parametrize("length", [1, 2, 10, 15, 16, 17])
@pytest.mark.parametrize("shape", SHAPES + [("bf16", 40, 64, 2, 64, 4)])
def test_prompt_equal_and_short(shape, length):
    """Short equal sequences without a state, the forward pass of a population."""
    c = Case(*shape, tokens=5 * length, seqs=5, seed=length, extra=1, gate=length % 2 == 0)
    xbc, dt, z = c.rows()
    y = c.layer().prompt(xbc, dt, c.y(), 5, z=z)
    want, mag, _ = c.expect([(i * length, i * length + length) for i in range(5)])
    close(c, y, want, mag)


@pytest.mark.parametrize("dtype, heads, head_dim, state, tokens", [("bf16", 2, 64, 128, 1500), ("f32", 1, 48, 64, 1025), ("bf16", 1, 16, 16, 4100)])
def test_prompt_long(dtype, heads, head_dim, state, tokens):
    """The time axis split over many workgroups; slow decays, so that far states matter."""
    c = Case(dtype, heads, head_dim, 1, state, 4, tokens=tokens, seqs=1, slots=1, fast=1.0)
    c.decay *= 0.01
    xbc, dt, z = c.rows()
    conv, ssm = c.conv.cuda(), c.ssm.cuda()
    y = c.layer().prompt(xbc, dt, c.y(), 1, z=z, positions=ints([5]), conv_state=conv, ssm_state=ssm)
    want, mag, carried = c.expect([(0, tokens)], [0], [5])
    close(c, y, want, mag)
    close_state(ssm[0], carried[0][0], carried[0][1])


@pytest.mark.parametrize("shape", SHAPES)
def test_step(shape):
    """A batch of single tokens with padding rows, fresh and continued, in place and apart."""
    slots, positions = [3, -1, 0, 6, -5, 2, 5], [0, 4, 1, 2, 0, 3, 900]
    c = Case(*shape, tokens=7, seqs=7, slots=8, extra=1)
    xbc, dt, z = c.rows()
    layer = c.layer()
    live = [i for i in range(7) if slots[i] >= 0]
    want, mag, carried = c.expect([(i, i + 1) for i in range(7)], [max(s, 0) for s in slots], positions)
    for apart in (True, False):
        conv, ssm = c.conv.cuda(), c.ssm.cuda()
        co, so = (torch.full_like(conv, 3.0), torch.full_like(ssm, 3.0)) if apart else (conv, ssm)
        y = layer.step(xbc, dt, c.y(), ints(positions), conv, ssm, z=z, slots=ints(slots), conv_out=co, ssm_out=so)
        close(c, y[live], want[live], mag[live])
        assert (y[[1, 4]] == 7).all()
        for i in live:
            close_state(so[slots[i]], carried[i][0], carried[i][1])
            assert torch.equal(co[slots[i]].double().cpu(), carried[i][2])
        for s in (1, 4, 7):
            assert torch.equal(so[s].cpu(), torch.full_like(c.ssm[s], 3.0) if apart else c.ssm[s])
            assert torch.equal(co[s].cpu(), torch.full_like(c.conv[s], 3.0) if apart else c.conv[s])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_steps_is_one_prompt(dtype):
    c = Case(dtype, 4, 32, 2, 64, 4, tokens=90, seqs=1, slots=1, seed=3)
    xbc, dt, z = c.rows()
    layer = c.layer()
    conv, ssm, y = c.conv.cuda(), c.ssm.cuda(), c.y()
    cut = 0
    for n in (2, 1, 70):  # pieces of a prompt, then token by token
        layer.prompt(xbc[cut:cut + n], dt[cut:cut + n], y[cut:cut + n], 1, z=z[cut:cut + n], positions=ints([cut]), conv_state=conv,
                     ssm_state=ssm)
        cut += n
    for t in range(cut, 90):
        layer.step(xbc[t:t + 1], dt[t:t + 1], y[t:t + 1], ints([t]), conv, ssm, z=z[t:t + 1])
    want, mag, carried = c.expect([(0, 90)], [0], [0])
    close(c, y, want, mag)
    close_state(ssm[0], carried[0][0], 2 * carried[0][1])
    assert torch.equal(conv[0].double().cpu(), carried[0][2])


def test_step_stale_state_is_not_read_when_fresh():
    """Position 0 starts at zero whatever the slot holds, NaN included; likewise a fresh prompt."""
    c = Case("bf16", 2, 64, 1, 128, 4, tokens=3, seqs=3, slots=3)
    xbc, dt, z = c.rows()
    want, mag, _ = c.expect([(i, i + 1) for i in range(3)])
    layer = c.layer()
    for form in ("step", "prompt"):
        conv, ssm = torch.full_like(c.conv, float("nan")).cuda(), torch.full_like(c.ssm, float("nan")).cuda()
        if form == "step":
            y = layer.step(xbc, dt, c.y(), ints([0, 0, -3]), conv, ssm, z=z)
        else:
            y = layer.prompt(xbc, dt, c.y(), 3, z=z, positions=ints([0, 0, -3]), conv_state=conv, ssm_state=ssm)
        close(c, y, want, mag)
        assert torch.isfinite(ssm).all()


@pytest.mark.parametrize("form", ["step", "prompt"])
def test_bad_slots(form):
    """A slot out of range, and one named twice: NaN rows, states untouched; the others as ever."""
    slots, positions = [1, 9, 1, 0, 1], [2, 2, 2, 2, 0]
    c = Case("f32", 2, 20, 1, 24, 4, tokens=5, seqs=5, slots=3)
    xbc, dt, z = c.rows()
    conv, ssm = c.conv.cuda(), c.ssm.cuda()
    want, mag, carried = c.expect([(i, i + 1) for i in range(5)], [1, 0, 0, 0, 0], positions)
    layer = c.layer()
    if form == "step":
        y = layer.step(xbc, dt, c.y(), ints(positions), conv, ssm, z=z, slots=ints(slots))
    else:
        y = layer.prompt(xbc, dt, c.y(), 5, z=z, slots=ints(slots), positions=ints(positions), conv_state=conv, ssm_state=ssm)
    close(c, y[[0, 3]], want[[0, 3]], mag[[0, 3]])
    assert torch.isnan(y[[1, 2, 4]]).all()
    close_state(ssm[1], carried[0][0], carried[0][1])
    close_state(ssm[0], carried[3][0], carried[3][1])
    assert torch.equal(ssm[2].cpu(), c.ssm[2]) and torch.equal(conv[2].cpu(), c.conv[2])


def test_wild_offsets_stay_inside():
    """Offsets that fall or leave the rows are clamped; nothing outside y's rows is written."""
    c = Case("bf16", 2, 32, 1, 32, 4, tokens=40, seqs=4)
    xbc, dt, z = c.rows()
    buf = torch.full((48, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    c.layer().prompt(xbc, dt, buf[4:44], 4, z=z, offsets=ints([-9, 10, 5, 30, 1000]))
    assert (buf[:4] == 7).all() and (buf[44:] == 7).all()
    want, mag, _ = c.expect([(0, 10), (10, 10), (5, 30), (30, 40)])
    close(c, buf[4 + 30:44], want[30:], mag[30:])


def test_nan_in_one_sequence_stays_there():
    c = Case("bf16", 2, 32, 1, 32, 4, tokens=60, seqs=3)
    c.wide[25] = float("nan")
    xbc, dt, z = c.rows()
    y = c.layer().prompt(xbc, dt, c.y(), 3, z=z)
    want, mag, _ = c.expect([(0, 20), (20, 40), (40, 60)])
    for first, end in ((0, 20), (40, 60)):
        close(c, y[first:end], want[first:end], mag[first:end])
    assert torch.isnan(y[25:40]).all()


@pytest.mark.parametrize("form", ["step", "prompt"])
def test_graph_replays_and_other_stream(form):
    c = Case("bf16", 4, 64, 1, 128, 4, tokens=150 if form == "prompt" else 6, seqs=1 if form == "prompt" else 6, slots=6)
    xbc, dt, z = c.rows()
    layer, pos = c.layer(), ints([3] * c.n)
    conv, ssm = c.conv.cuda(), c.ssm.cuda()
    co, so, y = torch.zeros_like(conv), torch.zeros_like(ssm), c.y()

    def call(stream=None):
        if form == "step":
            layer.step(xbc, dt, y, pos, conv, ssm, z=z, conv_out=co, ssm_out=so, stream=stream)
        else:
            layer.prompt(xbc, dt, y, c.n, z=z, positions=pos, conv_state=conv, ssm_state=ssm, conv_out=co, ssm_out=so, stream=stream)

    call()
    eager = y.clone(), so.clone(), co.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (y, so, co):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert all(torch.equal(a, e) for a, e in zip((y, so, co), eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for t in (y, so, co):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert all(torch.equal(a, e) for a, e in zip((y, so, co), eager))
        torch.ones(1000, device="cuda").sum().item()


def test_layer_checks_its_tensors():
    c = Case("bf16", 2, 32, 1, 32, 4, tokens=4, seqs=4, slots=4)
    layer = c.layer()
    xbc, dt, z = c.rows()
    conv, ssm, pos = c.conv.cuda(), c.ssm.cuda(), ints([0] * 4)
    bad = [
        lambda: layer.step(xbc.float(), dt, c.y(), pos, conv, ssm),
        lambda: layer.step(xbc[:, :-1], dt, c.y(), pos, conv, ssm),
        lambda: layer.step(xbc.t().contiguous().t(), dt, c.y(), pos, conv, ssm),
        lambda: layer.step(xbc, dt, c.y()[:3], pos, conv, ssm),
        lambda: layer.step(xbc, dt, c.y(), pos.long(), conv, ssm),
        lambda: layer.step(xbc, dt, c.y(), pos, conv, ssm.double()),
        lambda: layer.step(xbc, dt, c.y(), pos, conv[:3], ssm),
        lambda: layer.step(xbc, dt, c.y(), pos, conv, ssm, ssm_out=ssm.cpu()),
        lambda: layer.prompt(xbc, dt, c.y(), 2, conv_state=conv),
        lambda: layer.prompt(xbc, dt, c.y(), 4, slots=ints([0, 1, 2])),
        lambda: layer.prompt(xbc, dt, c.y()[:1].expand(4, -1), 4),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(b.CdrgeError):
        layer.prompt(xbc, dt, c.y(), 3)  # 4 rows are no equal shares of 3 sequences
    with pytest.raises(b.CdrgeError):
        layer.prompt(xbc, dt, c.y(), 4, slots=ints([0, 1, 2, 3]))  # slots, but no state


def test_no_tokens():
    c = Case("bf16", 2, 32, 1, 32, 4, tokens=0, seqs=2, slots=2)
    xbc, dt, z = c.rows()
    conv, ssm = c.conv.cuda(), c.ssm.cuda()
    c.layer().prompt(xbc, dt, c.y(), 2, z=z, positions=ints([0, 4]), conv_state=conv, ssm_state=ssm)
    assert (ssm[0] == 0).all() and torch.equal(ssm[1].cpu(), c.ssm[1]) and torch.equal(conv.cpu(), c.conv)
