"""The scores' gradient with factors far from one, as far as the header allows: up to 2^100 times the temperature."""
import math

import pytest
import torch

import more_operators_ref as ref
import test_gpu_scores as scores
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [50, 5000, 70001])
@pytest.mark.parametrize("tau, up", [(2.0 ** -30, 2.0 ** 69), (1.0, 2.0 ** 99), (2.0 ** 40, 2.0 ** -30)])
def test_gradient(tau, up, V):
    """Masked logits have no gradient whatever the factors; the others' scales with these."""
    g = torch.Generator().manual_seed(V)
    x, tokens = scores.draw(g, 4, V, "f32", spread=2.0 * tau)
    x[1, ::3], tokens[1] = -math.inf, 1
    x[2, 1:], tokens[2] = -math.inf, 0
    a, c = torch.full((4,), up), torch.tensor([up, -up, up, 0.0])
    out = torch.empty(4, V, device="cuda")
    b.TokenScores(b.make_score_config(V, 0, tau, "f32")).grad(x.cuda(), tokens.cuda(), a.cuda(), c.cuda(), out)
    _, entropy, d_lp, d_h = ref.scores(x, tokens, tau)
    want = a.double()[:, None] * d_lp + c.double()[:, None] * d_h
    p = torch.softmax(x.double() / tau, 1)
    size = p * (a.abs()[:, None] + c.abs()[:, None] * (torch.log(p.clamp(min=1e-300)).abs() + entropy[:, None])) / tau
    tol = ref.HALF_STEP["f32"] * want.abs() + scores.bounds(x, tau)[:, None] * (size + want.abs()) + 1e-37
    assert ((out.double().cpu() - want).abs() <= tol).all()
    assert (out.cpu()[1, ::3] == 0).all() and (out.cpu()[2] == 0).all()
