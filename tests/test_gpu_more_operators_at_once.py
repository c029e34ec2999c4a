"""Calls of the delta rule, the scores and the 4-bit projection that run at once, on two streams and as two graphs."""
import torch

import pytest

import test_gpu_delta as delta
import test_gpu_mx as mx
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu

HEADS, GROUPS, KEYS, VALUES, L, SEQS = 8, 4, 128, 64, 260, 3


def work(seed):
    """A call of each operator on tensors of its own, and what it writes."""
    g = torch.Generator().manual_seed(seed)
    parts, decay, bias = delta.inputs(g, SEQS * L, HEADS, GROUPS, KEYS, VALUES, "bf16")
    layer = delta.layer_of(HEADS, GROUPS, KEYS, VALUES, "bf16", decay, bias)
    rows = delta.on_gpu(parts)
    offsets = torch.tensor([0, L - 7 * seed, 2 * L, SEQS * L], dtype=torch.int32, device="cuda")
    positions = torch.ones(SEQS, dtype=torch.int32, device="cuda")
    state = torch.randn(SEQS, HEADS, VALUES, KEYS, generator=g).cuda()
    out, y = torch.empty_like(state), torch.empty(SEQS * L, HEADS * VALUES, dtype=torch.bfloat16, device="cuda")
    codes, scales = mx.weights(g, 2000, HEADS * VALUES)
    head = b.MxProjection(b.make_mx_config(HEADS * VALUES, 2000, "bf16"), codes.cuda(), scales.cuda())
    logits = torch.empty(SEQS * L, 2000, dtype=torch.bfloat16, device="cuda")
    op = b.TokenScores(b.make_score_config(2000, 20, 1.0, "bf16"))
    tokens = torch.randint(0, 2000, (SEQS * L,), generator=g, dtype=torch.int32).cuda()
    lp, h = (torch.empty(SEQS * L, device="cuda") for _ in range(2))
    ids, lps = torch.empty(SEQS * L, 20, dtype=torch.int32, device="cuda"), torch.empty(SEQS * L, 20, device="cuda")

    def call():
        layer.prompt(*rows, y, SEQS, offsets=offsets, positions=positions, state=state, state_out=out)
        head.project(y, logits)
        op.scores(logits, tokens, lp, h, ids, lps)

    return call, (y, out, logits, lp, h, ids, lps)


def test_on_two_streams_and_as_two_graphs():
    both = [work(1), work(2)]
    want = []
    for call, outputs in both:
        call()
        want.append([t.clone() for t in outputs])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    for call, _ in both:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)

    def check(run):
        for _, outputs in both:
            for t in outputs:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    run(i)
        torch.cuda.synchronize()
        for (_, outputs), expect in zip(both, want):
            assert all(torch.equal(a, c) for a, c in zip(outputs, expect))

    for _ in range(3):
        check(lambda i: both[i][0]())
        check(lambda i: graphs[i].replay())
