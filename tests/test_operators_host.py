"""The population operators' refusals, which come before any device work: no GPU is needed, and the
pointers handed over are never followed."""
import ctypes
import os

import pytest

from zero_order_recurrent_amd import binding as b

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(b.LIB_PATH):
        from zero_order_recurrent_amd.build import build
        build()
    return b.lib()


def _set(struct, changes):
    for k, v in changes.items():
        setattr(struct, k, v)
    return struct


def _scan(io=None, weights=None, **cfg):
    c = _set(b.make_scan_config(4, 32, 2, 64, 4, "bf16"), cfg)
    ch = 4 * 32 + 2 * 2 * 64
    w = _set(b.cdrge_scan_weights(FAKE, FAKE, FAKE, FAKE, FAKE), weights or {})
    i = b.cdrge_scan_io(FAKE, ch, FAKE, 4, FAKE, 128, FAKE, 128, 6, 3, 3, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    return c, w, _set(i, io or {})


def _prompt(lib, c, w, i, ws=FAKE, nbytes=1 << 40):
    return lib.cdrge_scan_prompt(ctypes.byref(c), ctypes.byref(w), ctypes.byref(i), ws, nbytes, None)


BAD_SCAN = [
    (dict(abi_version=0), {}, {}, 1), (dict(dtype=2), {}, {}, 1), (dict(n_heads=0), {}, {}, 1),
    (dict(n_heads=3), {}, {}, 1), (dict(state_dim=0), {}, {}, 1), (dict(conv_width=0), {}, {}, 1),
    (dict(conv_width=1), {}, {}, 2), (dict(conv_width=5), {}, {}, 2), (dict(state_dim=257), {}, {}, 2),
    (dict(head_dim=257), {}, {}, 2),
    ({}, dict(n_tokens=-1), {}, 1), ({}, dict(n_seqs=0), {}, 1), ({}, dict(n_tokens=7), {}, 1),
    ({}, dict(xbc_stride=383), {}, 1), ({}, dict(dt_stride=3), {}, 1), ({}, dict(z_stride=127), {}, 1),
    ({}, dict(y_stride=127), {}, 1), ({}, dict(y=None), {}, 1), ({}, dict(xbc=None), {}, 1),
    ({}, dict(ssm_out=None), {}, 1), ({}, dict(conv_in=None, conv_out=None), {}, 1),
    ({}, dict(conv_in=None, conv_out=None, ssm_in=None, ssm_out=None), {}, 1),  # slots without states
    ({}, dict(slots=None, n_slots=2), {}, 1), ({}, dict(n_slots=0), {}, 1), ({}, dict(ssm_in=FAKE + 8), {}, 1),
    ({}, dict(n_tokens=(1 << 30) + 2, n_seqs=2), {}, 2),
    ({}, {}, dict(conv_weight=None), 1), ({}, {}, dict(decay=None), 1),
]


@pytest.mark.parametrize("cfg, io, weights, status", BAD_SCAN)
def test_scan_refuses(lib, cfg, io, weights, status):
    c, w, i = _scan(io, weights, **cfg)
    assert _prompt(lib, c, w, i) == status
    i.n_tokens = i.n_seqs if not io.get("n_tokens") else i.n_tokens
    if "n_tokens" not in io:
        assert lib.cdrge_scan_step(ctypes.byref(c), ctypes.byref(w), ctypes.byref(i), None) == status


def test_scan_prompt_refuses_its_workspace(lib):
    c, w, i = _scan()
    need = b.cdrge_scan_workspace_bytes(c, 6, 3)
    for ws, nbytes in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
        assert _prompt(lib, c, w, i, ws, nbytes) == 3
        assert "cdrge_scan_prompt" in b.cdrge_last_error_detail()


def test_scan_step_refuses(lib):
    for io in (dict(offsets=FAKE), dict(positions=None), dict(n_tokens=6), dict(n_tokens=0),
               dict(conv_in=None, conv_out=None, ssm_in=None, ssm_out=None, slots=None, positions=None)):
        c, w, i = _scan(dict(n_tokens=3) | io)
        assert lib.cdrge_scan_step(ctypes.byref(c), ctypes.byref(w), ctypes.byref(i), None) == 1, io


def _project(lib, rows=5, x=FAKE, y=FAKE, x_stride=64, y_stride=96, adapter=FAKE, ws=FAKE, nbytes=1 << 40, weights=None, **cfg):
    c = _set(b.make_adapter_config(64, 96, 3, 8, "f32"), cfg)
    w = _set(b.cdrge_adapter_weights(FAKE, 64, FAKE, FAKE, FAKE, FAKE), weights or {})
    return lib.cdrge_adapter_project(ctypes.byref(c), ctypes.byref(w), rows, x, x_stride, adapter, None, y, y_stride, ws, nbytes, None)


@pytest.mark.parametrize("kw, status", [
    (dict(abi_version=3), 1), (dict(dtype=2), 1), (dict(in_features=0), 1), (dict(n_adapters=-1), 1), (dict(max_rank=0), 1),
    (dict(max_rank=129), 2), (dict(out_features=(1 << 20) + 1, y_stride=1 << 21), 2), (dict(rows=-1), 1),
    (dict(rows=(1 << 30) + 1), 2), (dict(x=None), 1), (dict(y=None), 1), (dict(x_stride=63), 1), (dict(y_stride=95), 1),
    (dict(weights=dict(weight=None)), 1), (dict(weights=dict(weight_stride=63)), 1), (dict(weights=dict(down=None)), 1),
    (dict(weights=dict(up=None)), 1), (dict(ws=None), 3), (dict(nbytes=4), 3), (dict(ws=FAKE + 4), 3)])
def test_adapters_refuse(lib, kw, status):
    assert _project(lib, **kw) == status


def test_adapters_without_rows(lib):
    assert _project(lib, rows=0, x=None, y=None, ws=None, nbytes=0) == 0


def _distill(lib, rows=6, logits=FAKE, stride=50, ids=FAKE, teacher=FAKE, row=FAKE, **cfg):
    c = _set(b.make_distill_config(50, 4, 2, 1.5, "f32"), cfg)
    return lib.cdrge_distill_losses(ctypes.byref(c), rows, logits, stride, ids, teacher, row, FAKE, None)


@pytest.mark.parametrize("kw, status", [
    (dict(abi_version=9), 1), (dict(dtype=2), 1), (dict(vocab=0), 1), (dict(top_k=0), 1), (dict(n_models=0), 1),
    (dict(n_models=4), 1), (dict(temperature=0.0), 1), (dict(temperature=float("nan")), 1), (dict(temperature=float("inf")), 1),
    (dict(temperature=-1.0), 1), (dict(top_k=1025), 2), (dict(vocab=(1 << 24) + 1, stride=1 << 25), 2), (dict(rows=-2), 1),
    (dict(rows=(1 << 30) + 2), 2), (dict(stride=49), 1), (dict(logits=None), 1), (dict(ids=None), 1),
    (dict(teacher=None), 1), (dict(row=None), 1)])
def test_distill_refuses(lib, kw, status):
    assert _distill(lib, **kw) == status


@pytest.mark.parametrize("tau", [2.0 ** -61, 2.0 ** 61, 1e-40])
def test_distill_refuses_far_temperatures(lib, tau):
    assert _distill(lib, temperature=tau) == 2


def test_distill_grad_refuses(lib):
    c = b.make_distill_config(50, 4, 2, 1.5, "f32")

    def grad(logits, stride, d, d_stride):
        return lib.cdrge_distill_grad(ctypes.byref(c), 6, logits, stride, FAKE, FAKE, None, FAKE, None, d, d_stride, None)

    assert grad(FAKE, 50, None, 50) == 1
    assert grad(FAKE, 50, FAKE + (1 << 30), 49) == 1
    assert grad(FAKE, 50, FAKE, 60) == 1  # in place, but with other strides


def test_layers_refuse_cpu_tensors(lib):
    import torch
    cw = torch.zeros(4 * 32 + 2 * 2 * 64, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        b.ScanLayer(b.make_scan_config(4, 32, 2, 64, 4, "bf16"), cw, None, torch.zeros(4))
    with pytest.raises(ValueError):
        b.AdapterProjection(b.make_adapter_config(64, 96, 0, 8, "f32"), torch.zeros(96, 64))
    with pytest.raises(ValueError):
        b.DistillLoss(b.make_distill_config(50, 4, 2, 1.5, "f32"), device="cpu")
