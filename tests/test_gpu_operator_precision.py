"""How exact the population operators are as a whole, in the 2-norm over many outputs.

A bound of each element by the magnitudes of its sum's terms holds for any inputs, but over random terms of either sign
those magnitudes are many times the sum: precision that is lost in every operand can hide below it. Over thousands of
outputs of random terms the roundings are independent and add as squares, relative to the outputs themselves, so the
norm of the error shows what each operand was rounded to.
"""
import pytest
import torch

import operators_ref as ref
from test_gpu_scan import Case, ints

pytestmark = pytest.mark.gpu

# A prompt's outputs. Entries enter products in two halves of 11 bits, rounded by at most 2^-22 (in the 2-norm that over
# sqrt 3); a product leaves out the two low halves' (2^-22 again). Two such products in a row with two roundings each make
# sqrt(6 / 3) 2^-22 = 2^-21.5. Up to 3 x 256 + 3 x 64 additions in float32, each rounded by 2^-24 / sqrt 3 of a partial sum
# whose square grows evenly to the whole's: sqrt(960 / 6) 2^-24 = 2^-20.3. Convolution, exponentials and gates: a few
# 2^-23. As squares: 2^-19.9, held to 2^-19.
SCAN = 2 ** -19


def off(got, want):
    """The norm of the difference over the norm of `want`; bf16 against `want` rounded to bf16."""
    if got.dtype == torch.bfloat16:
        want = want.to(torch.bfloat16).double()
    return float((got.double().cpu() - want).norm() / want.norm())


def bound(dtype, e):
    # A value that is off by e of itself before it is rounded to bf16 ends a step (at most 2^-7 of it, 2^-7.5 in the mean)
    # from the nearest with the probability |e| / step: the mean square is step |e|, at most 2^-7 e.
    return (2 ** -7 * e) ** 0.5 if dtype == "bf16" else e


@pytest.mark.parametrize("shape, lengths", [
    (("bf16", 2, 64, 1, 128, 4), [600, 70]), (("f32", 2, 64, 1, 128, 4), [600, 70]), (("bf16", 2, 32, 2, 16, 3), [150, 33]),
    (("bf16", 2, 80, 1, 64, 4), [400]), (("f32", 3, 40, 1, 100, 2), [300, 5]), (("bf16", 1, 128, 1, 256, 4), [330]),
    (("f32", 1, 64, 1, 256, 4), [130])])
def test_prompts(shape, lengths):
    n = len(lengths)
    c = Case(*shape, tokens=sum(lengths), seqs=n, slots=n, seed=11)
    bounds = [(sum(lengths[:i]), sum(lengths[:i + 1])) for i in range(n)]
    xbc, dt, z = c.rows()
    conv, ssm = c.conv.cuda(), c.ssm.cuda()
    y = c.layer().prompt(xbc, dt, c.y(), n, z=z, offsets=ints([0] + [e for _, e in bounds]), positions=ints([7] * n), conv_state=conv,
                         ssm_state=ssm)
    want, _, carried = c.expect(bounds, list(range(n)), [7] * n)
    assert off(y, want) <= bound(c.dtype, SCAN)
    for i in range(n):
        assert off(ssm[i], carried[i][0]) <= SCAN
