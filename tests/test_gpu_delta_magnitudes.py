"""The delta rule with rows of q, k and v far from one, as far as the header allows: what a row of k writes is v over its
length, and the state's product with a row of k as it comes is up to 2^100."""
import pytest
import torch

import more_operators_ref as ref
import test_gpu_delta as delta

pytestmark = pytest.mark.gpu

# powers of two of q, k, v and the state
FAR = [(0, 59, -35, -35), (59, 59, 30, 30), (-59, 59, 0, 0), (59, -59, 30, 30), (-30, -30, 95, 95), (0, 0, -90, -90), (0, 20, -60, -60)]
FORMS = [(3, 13), (1, 200), (17, 70)]
IDS = ["token by token", "few blocks", "many workgroups"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs, L", FORMS, ids=IDS)
@pytest.mark.parametrize("eq, ek, ev, es", FAR)
def test_prompts(eq, ek, ev, es, seqs, L, dtype):
    y, state, want, part, carried, kd = run(eq, ek, ev, es, seqs, L, dtype)
    delta.check(y, want, part, dtype, kd, "y")
    check_state(state, carried, kd)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs, L", FORMS, ids=IDS)
def test_queries_too_far_for_the_state(seqs, L, dtype):
    """The state's product with a row of q passes float32: y counts as not finite, and the state is as ever."""
    y, state, _, _, carried, kd = run(59, 0, 90, 90, seqs, L, dtype)
    assert not torch.isfinite(y).any()
    check_state(state, carried, kd)


def check_state(state, carried, kd):
    got = state.double().cpu()
    for i, (S, E) in enumerate(carried):
        tol = ref.delta_eps(kd) * (E + S.flatten(1).norm(dim=1))[:, None, None] + 1e-37
        assert ((got[i] - S).abs() <= tol).all(), (i, float(((got[i] - S).abs() / tol).max()))


def run(eq, ek, ev, es, seqs, L, dtype):
    g = torch.Generator().manual_seed(100 + ek)
    heads, groups, kd, vd, eps = 4, 2, 128, 64, 2.0 ** -60
    parts, decay, bias = delta.inputs(g, seqs * L, heads, groups, kd, vd, dtype, wide=False)
    for part, e in zip(parts, (eq, ek, ev)):
        part.mul_(2.0 ** e)
    start = torch.randn(seqs, heads, vd, kd, generator=g) * 0.3 * 2.0 ** es
    layer = delta.layer_of(heads, groups, kd, vd, dtype, decay, bias, norm_eps=eps)
    y = torch.empty(seqs * L, heads * vd, dtype=ref.TYPES[dtype], device="cuda")
    state = start.cuda()
    layer.prompt(*delta.on_gpu(parts), y, seqs, positions=torch.ones(seqs, dtype=torch.int32, device="cuda"), state=state)
    want, part, carried = ref.delta(*parts, decay, bias, heads, groups, kd, vd, [(i * L, i * L + L) for i in range(seqs)], kd ** -0.5,
                                    eps, state_in=start, positions=[1] * seqs)
    return y, state, want, part, carried, kd
