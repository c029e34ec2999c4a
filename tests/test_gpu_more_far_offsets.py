"""The delta rule with a cache of states, and 4-bit weights, that pass 2^32 elements and bytes, against the same in small ones."""
import pytest
import torch

import more_operators_ref as ref
import test_gpu_delta as delta
from zero_order_recurrent_amd import binding as b

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kd, vd, heads", [(128, 128, 32), (127, 129, 32)])
def test_states_far_in_a_cache(kd, vd, heads):
    g = torch.Generator().manual_seed(kd)
    n_slots = (1 << 32) // (heads * kd * vd) + 6
    far = torch.tensor([n_slots - 1, 3, n_slots - 4, n_slots - 2], dtype=torch.int32)
    cache = torch.empty(n_slots, heads, vd, kd, device="cuda")
    start = torch.randn(4, heads, vd, kd, generator=g).cuda()
    positions = torch.ones(4, dtype=torch.int32, device="cuda")
    lengths = {"step": [1] * 4, "tokens": [5, 30, 8, 2], "blocks": [100, 130, 64, 500]}
    for name, L in lengths.items():
        n = sum(L)
        parts, decay, bias = delta.inputs(g, n, heads, heads, kd, vd, "bf16", wide=False)
        layer = delta.layer_of(heads, heads, kd, vd, "bf16", decay, bias)
        rows = delta.on_gpu(parts)
        offsets = torch.tensor([0] + L).cumsum(0).to(torch.int32).cuda()
        got = []
        for state, slots in ((start.clone(), torch.arange(4, dtype=torch.int32)), (cache, far)):
            if state is cache:
                cache[far.long().cuda()] = start
                cache[n_slots - 3] = 7.0
            y = torch.empty(n, heads * vd, dtype=torch.bfloat16, device="cuda")
            if name == "step":
                layer.step(*rows, y, positions, state, slots=slots.cuda())
            else:
                layer.prompt(*rows, y, 4, offsets=offsets, slots=slots.cuda(), positions=positions, state=state)
            got.append((y, state[slots.long().cuda()]))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]), name
        assert not torch.equal(got[1][1], start) and (cache[n_slots - 3] == 7.0).all()


def test_weights_of_more_than_4_gb():
    g = torch.Generator().manual_seed(1)
    O, K = 1 << 20, 8209  # 257 blocks of 16 bytes a row
    w = torch.randn(4096, K, generator=g).bfloat16().cuda()
    f = b.MxFormat(b.make_mx_config(K, 1, "bf16"))
    some = f.quantize(w, *f.empty(4096))
    x = torch.empty(O, K, dtype=torch.bfloat16, device="cuda")
    for r in range(0, O, 4096):  # the same rows again and again, turned by one each time
        x[r:r + 4096] = w.roll(r // 4096, 0)
    codes, scales = f.quantize(x, *f.empty(O))
    for r in (0, O // 2, O - 4096):
        assert torch.equal(codes[r:r + 4096], some[0].roll(r // 4096, 0)) and torch.equal(scales[r:r + 4096], some[1].roll(r // 4096, 0))
    back = f.dequantize(codes, scales, x)
    near = f.dequantize(*some, torch.empty_like(w))
    assert torch.equal(back[O - 4096:], near.roll((O - 4096) // 4096, 0)) and torch.equal(back[:4096], near)
    to = torch.tensor([0, 1, O // 2, O - 300, O - 2, O - 1])
    wv = ref.mx_values(codes[to.cuda()].cpu(), scales[to.cuda()].cpu(), K)
    for rows in (3, 10, 20):  # quantised by the product's workgroups, before it, and by tiles
        a = torch.randn(rows, K, generator=g).bfloat16()
        y = torch.empty(rows, O, dtype=torch.bfloat16, device="cuda")
        b.MxProjection(b.make_mx_config(K, O, "bf16"), codes, scales).project(a.cuda(), y)
        xv = ref.mx_values(*ref.mx_quantize(a), K)
        want, size = xv @ wv.t(), xv.abs() @ wv.abs().t()
        tol = ref.HALF_STEP["bf16"] * want.abs() + (2 * K + 64) * 2 ** -24 * size
        assert ((y[:, to.cuda()].double().cpu() - want).abs() <= tol).all()
