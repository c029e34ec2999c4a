"""The gated delta rule's prompts by the 2-norm of their errors, by each of their kernels.

Which kernels a call takes goes by its type, its keys (up to 128, or more; exactly 128 in bf16 read where they lie),
and its workgroups, one for each sequence, head and 16 values: up to 256 of them or more.
"""
import pytest
import torch

import more_operators_ref as ref
import test_gpu_delta as delta

pytestmark = pytest.mark.gpu

HEADS, GROUPS, VALUES = 4, 2, 64  # 16 workgroups a sequence
FORMS = {"few workgroups": (1, 700), "many workgroups": (17, 130), "token by token": (9, 16)}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kd", [100, 128, 200, 256])
@pytest.mark.parametrize("form", list(FORMS))
def test_prompts_in_the_2_norm(form, kd, dtype):
    """y and the state are off by 2^-20 of their norms: operands of 24 bits, a block's sums of up to 128 terms and a few
    blocks' worth of state, whose roundings add up as random ones do; with more keys by the root of their number.

    In bf16 y is the nearest bf16 to a value that is off by that: an element falls to the other side of a border where it is
    no further from it than its error e, in a share |e| / step of them, and is off by a step then: the sum of squares is
    step |e|, with steps of at most 2^-7 of an element, and so at most 2^-7 |y| |e| of the norms."""
    seqs, L = FORMS[form]
    g = torch.Generator().manual_seed(kd + seqs)
    parts, decay, bias = delta.inputs(g, seqs * L, HEADS, GROUPS, kd, VALUES, dtype)
    decay = decay * 0.2
    layer = delta.layer_of(HEADS, GROUPS, kd, VALUES, dtype, decay, bias)
    y = torch.empty(seqs * L, HEADS * VALUES, dtype=ref.TYPES[dtype], device="cuda")
    start = torch.randn(seqs, HEADS, VALUES, kd, generator=g) * 0.3
    state = start.cuda()
    layer.prompt(*delta.on_gpu(parts), y, seqs, positions=torch.ones(seqs, dtype=torch.int32, device="cuda"), state=state)
    want, _, carried = ref.delta(*parts, decay, bias, HEADS, GROUPS, kd, VALUES, [(i * L, i * L + L) for i in range(seqs)],
                                 kd ** -0.5, state_in=start, positions=[1] * seqs)
    off = 2 ** -20 * max(1.0, kd / 128) ** 0.5
    S = torch.stack([c[0] for c in carried])
    err = float((state.double().cpu() - S).norm() / S.norm())
    assert err <= off, f"state: {err:.3g} of {off:.3g}"
    near = want.to(ref.TYPES[dtype]).double() if dtype == "bf16" else want
    tol = (off * 2 ** -7) ** 0.5 if dtype == "bf16" else off
    err = float((y.double().cpu() - near).norm() / want.norm())
    assert err <= tol, f"y: {err:.3g} of {tol:.3g}"
