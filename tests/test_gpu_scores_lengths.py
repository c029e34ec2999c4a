"""Scores without alternatives, and gradients, at vocabularies of every form that a row is held in: 16 to 1,024 threads with one
to 16 pieces each, and rows that are read again."""
import pytest
import torch

import more_operators_ref as ref
import test_gpu_scores as scores

pytestmark = pytest.mark.gpu

# in float32 and bf16 one of each side of 16, 64, 128, 512, 1024, 2048, 4096, 8192 and 16384 pieces of 16 bytes
LENGTHS = [per * pieces + more for pieces in (16, 64, 128, 512, 1024, 2048, 4096, 8192, 16384) for per in (4, 8) for more in (0, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", sorted(set(LENGTHS)))
def test_scores_without_alternatives(V, dtype):
    g = torch.Generator().manual_seed(V)
    x, tokens = scores.draw(g, 3, V, dtype, stride=V + 1)
    tokens[0] = V - 1
    lp, h, _, _ = scores.run(x, tokens, 0, 0.7, dtype)
    want, entropy, _, _ = ref.scores(x, tokens, 0.7)
    tol = scores.bounds(x, 0.7)
    assert ((lp - want).abs() <= tol).all()
    assert ((h - entropy).abs() <= tol * (1 + entropy)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", sorted(set(LENGTHS)))
def test_gradient(V, dtype):
    scores.test_gradient(3, V, dtype)
