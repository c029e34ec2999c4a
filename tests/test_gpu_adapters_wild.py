"""Adapters whose up matrices hold infinities and NaN in places: what follows from them, and nothing else, and in a time
beside the call's own."""
import time

import pytest
import torch

import operators_ref as ref
from test_gpu_adapters import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype, rows, K, O, R", [
    ("bf16", 3, 64, 70, 8), ("bf16", 200, 96, 320, 8), ("bf16", 3333, 192, 3880, 8), ("bf16", 3333, 70, 3880, 40), ("f32", 150, 64, 300, 24),
    ("f32", 3100, 64, 4070, 8), ("f32", 30, 64, 300, 24),
    # after a product in slices, by a launch that joins them: ranks of one product and of several, whole pieces and not
    ("bf16", 60, 200, 130, 12), ("bf16", 60, 200, 130, 16), ("bf16", 30, 300, 70, 40), ("bf16", 150, 2048, 200, 33)])
def test_entries_that_are_not_finite(dtype, rows, K, O, R):
    """Outputs that meet such an entry become what the formula gives; every other one keeps its value to the bit."""
    c = Case(dtype, rows, K, O, 5, R, seed=rows, ranks=[R, R, max(R - 3, 1), 0, R])
    c.x[0], c.x[-1] = 0.0, torch.eye(1, K)  # a value of zero meets infinity as NaN, one that bf16 holds exactly as infinity
    x, who, y, scale = c.inputs()
    clean = c.operator().project(x, who, y[:, :O], row_scale=scale).clone()
    g = torch.Generator().manual_seed(1)
    at = torch.randint(0, 40, c.up.shape, generator=g)
    at[4] = 9  # one adapter stays finite
    inf = float("inf")
    for value, which in ((inf, at == 0), (-inf, at == 1), (float("nan"), at == 2)):
        c.up[which] = value
    got = c.operator().project(x, who, y[:, :O], row_scale=scale)
    want, _, _ = ref.adapters(c.x, c.w, c.bias, c.down, c.up, c.ranks, c.who, c.scale)
    live = torch.isfinite(want)
    assert live.any() and (rows < 4 or not live.all())
    assert torch.equal(got.cpu()[live], clean.cpu()[live])
    assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
    assert torch.equal((got.cpu() == inf), (want == inf)) and torch.equal((got.cpu() == -inf), (want == -inf))
    assert (y[:, O:] == 7).all()


def test_a_diverged_adapter_costs_little():
    """One infinity in every row of an up matrix: the call stays within a few times its own time (rows computed one by one
    took 60 times it)."""
    c = Case("bf16", 4096, 2048, 4096, 2, 8, order="runs", xpad=0, ypad=0)
    x, who, y, scale = c.inputs()

    def seconds(op):
        best = 1e9
        for _ in range(4):
            torch.cuda.synchronize()
            began = time.perf_counter()
            op.project(x, who, y, row_scale=scale)
            torch.cuda.synchronize()
            best = min(best, time.perf_counter() - began)
        return best

    clean = seconds(c.operator())
    c.up[:, :, 3] = float("inf")
    assert seconds(c.operator()) <= 8 * clean + 1e-3
