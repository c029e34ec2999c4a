"""The gradient of the entropy where a row's logits are nearly equal: it is what is left of two logarithms of the vocabulary's
size, and has to be formed without them."""
import pytest
import torch

import more_operators_ref as ref
import test_gpu_scores as scores
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spread", [1e-2, 1e-4])
@pytest.mark.parametrize("V", [50, 1000, 30011, 70001])
def test_gradient_of_flat_rows(V, spread):
    """log p_v + entropy is d_v - sum p d, with d the scaled distances from the largest, in [-R, 0]. Differences of logits
    this near are exact; d and p d have 8 roundings, the sum of terms of one sign V / 64 + 16 additions, twice (its own and that
    of p), and 8 for what follows: R (V / 32 + 64) 2^-24 of p / tau. p is off as in test_gpu_scores."""
    g = torch.Generator().manual_seed(V)
    rows, tau = 5, 1.3
    x = 5 + torch.randn(rows, V, generator=g) * spread
    tokens = torch.randint(0, V, (rows,), generator=g).to(torch.int32)
    op = b.TokenScores(b.make_score_config(V, 0, tau, "f32"))
    _, _, d_lp, d_h = ref.scores(x, tokens, tau)
    p = torch.softmax(x.double() / tau, 1)
    R = (x.amax(1) - x.amin(1)).double()[:, None] / tau
    uh = torch.tensor([1.0, -2.0, 0.3, 1.7, -0.9])
    for up in (None, torch.full((rows,), 2.0 ** -40)):  # without and with the given token's own formula
        want = d_h * uh.double()[:, None] + (0 if up is None else d_lp * 2.0 ** -40)
        out = torch.empty(rows, V, device="cuda")
        op.grad(x.cuda(), tokens.cuda(), None if up is None else up.cuda(), uh.cuda(), out)
        tol = (2 ** -24 + scores.bounds(x, tau)[:, None]) * (want.abs() + 2.0 ** -40) + uh.abs()[:, None] * p / tau * R * (V / 32 + 64) * 2 ** -24
        err = (out.double().cpu() - want).abs()
        assert (err <= tol).all(), float((err / tol).max())


def test_equal_logits_have_no_gradient():
    x = torch.full((3, 777), 2.5)
    out = torch.empty(3, 777, device="cuda")
    op = b.TokenScores(b.make_score_config(777, 0, 0.7, "f32"))
    op.grad(x.cuda(), None, None, torch.ones(3, device="cuda"), out)
    assert (out == 0).all()
