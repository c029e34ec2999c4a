"""Refusals of the delta rule, the token scores and the 4-bit projections, which come before any device work: no GPU is
needed, and the pointers handed over are never followed."""
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


def _delta(io=None, weights=None, **cfg):
    c = _set(b.make_delta_config(4, 2, 64, 32, "bf16"), cfg)
    w = _set(b.cdrge_delta_weights(FAKE, FAKE), weights or {})
    i = b.cdrge_delta_io(FAKE, 128, FAKE, 128, FAKE, 128, FAKE, 4, FAKE, 4, FAKE, 128, 6, 3, 3, None, FAKE, FAKE, FAKE, FAKE)
    return c, w, _set(i, io or {})


def _prompt(lib, c, w, i, ws=FAKE, nbytes=1 << 40):
    return lib.cdrge_delta_prompt(ctypes.byref(c), ctypes.byref(w), ctypes.byref(i), ws, nbytes, None)


BAD_DELTA = [
    (dict(abi_version=0), {}, {}, 1), (dict(dtype=2), {}, {}, 1), (dict(n_heads=0), {}, {}, 1), (dict(n_heads=3), {}, {}, 1),
    (dict(key_dim=0), {}, {}, 1), (dict(value_dim=0), {}, {}, 1), (dict(n_groups=0), {}, {}, 1), (dict(key_dim=257), {}, {}, 2),
    (dict(value_dim=257), {}, {}, 2), (dict(norm_eps=0.0), {}, {}, 1), (dict(norm_eps=-1.0), {}, {}, 1),
    (dict(norm_eps=float("nan")), {}, {}, 1), (dict(norm_eps=2.0), {}, {}, 2), (dict(norm_eps=2.0 ** -61), {}, {}, 2),
    (dict(q_scale=float("inf")), {}, {}, 1), (dict(q_scale=2.0 ** 61), {}, {}, 2),
    ({}, dict(n_tokens=-1), {}, 1), ({}, dict(n_seqs=0), {}, 1), ({}, dict(n_tokens=7), {}, 1),
    ({}, dict(q_stride=127), {}, 1), ({}, dict(k_stride=127), {}, 1), ({}, dict(v_stride=127), {}, 1),
    ({}, dict(y_stride=127), {}, 1), ({}, dict(dt_stride=3), {}, 1), ({}, dict(beta_stride=3), {}, 1),
    ({}, dict(q=None), {}, 1), ({}, dict(k=None), {}, 1), ({}, dict(v=None), {}, 1), ({}, dict(dt=None), {}, 1),
    ({}, dict(beta=None), {}, 1), ({}, dict(y=None), {}, 1), ({}, dict(state_out=None), {}, 1), ({}, dict(state_in=None), {}, 1),
    ({}, dict(state_in=None, state_out=None), {}, 1),  # slots without states
    ({}, dict(slots=None, n_slots=2), {}, 1), ({}, dict(n_slots=0), {}, 1), ({}, dict(state_in=FAKE + 8), {}, 1),
    ({}, dict(n_tokens=(1 << 30) + 2, n_seqs=2), {}, 2), ({}, {}, dict(decay=None), 1),
]


@pytest.mark.parametrize("cfg, io, weights, status", BAD_DELTA)
def test_delta_refuses(lib, cfg, io, weights, status):
    c, w, i = _delta(io, weights, **cfg)
    assert _prompt(lib, c, w, i) == status
    if "n_tokens" not in io:
        i.n_tokens = i.n_seqs
        assert lib.cdrge_delta_step(ctypes.byref(c), ctypes.byref(w), ctypes.byref(i), None) == status


def test_delta_prompt_refuses_its_workspace(lib):
    c, w, i = _delta()
    need = b.cdrge_delta_workspace_bytes(c, 6, 3)
    for ws, nbytes in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
        assert _prompt(lib, c, w, i, ws, nbytes) == 3
        assert "cdrge_delta_prompt" in b.cdrge_last_error_detail()


def test_delta_step_refuses(lib):
    for io in (dict(offsets=FAKE), dict(positions=None), dict(n_tokens=6), dict(n_tokens=0),
               dict(state_in=None, state_out=None, slots=None, positions=None)):
        c, w, i = _delta(dict(n_tokens=3) | io)
        assert lib.cdrge_delta_step(ctypes.byref(c), ctypes.byref(w), ctypes.byref(i), None) == 1, io


def test_delta_workspace_refuses(lib):
    c = b.make_delta_config(4, 2, 64, 32, "bf16")
    out = ctypes.c_size_t()
    size = lib.cdrge_delta_workspace_bytes
    assert size(ctypes.byref(c), 6, 3, None) == 1
    assert size(ctypes.byref(c), -1, 3, ctypes.byref(out)) == 1
    assert size(ctypes.byref(c), 6, 0, ctypes.byref(out)) == 1
    assert size(ctypes.byref(c), (1 << 30) + 1, 3, ctypes.byref(out)) == 2
    assert size(ctypes.byref(c), 6, (1 << 20) + 1, ctypes.byref(out)) == 2


def _scores(lib, rows=6, logits=FAKE, stride=50, tokens=FAKE, logprobs=FAKE, ids=FAKE, lps=FAKE, **cfg):
    c = _set(b.make_score_config(50, 4, 1.5, "f32"), cfg)
    return lib.cdrge_token_scores(ctypes.byref(c), rows, logits, stride, tokens, logprobs, FAKE, ids, lps, None)


SCORES = [(dict(abi_version=9), 1), (dict(dtype=2), 1), (dict(vocab=0), 1), (dict(top_k=-1), 1), (dict(top_k=51), 1),
          (dict(temperature=0.0), 1), (dict(temperature=float("nan")), 1), (dict(temperature=float("inf")), 1),
          (dict(temperature=-1.0), 1), (dict(temperature=2.0 ** -61), 2), (dict(temperature=2.0 ** 61), 2),
          (dict(vocab=(1 << 24) + 1, stride=1 << 25), 2), (dict(vocab=2000, stride=2000, top_k=1025), 2), (dict(rows=-2), 1),
          (dict(rows=(1 << 30) + 2), 2), (dict(stride=49), 1), (dict(logits=None), 1)]


@pytest.mark.parametrize("kw, status", SCORES + [(dict(tokens=None), 1), (dict(ids=None), 1), (dict(lps=None), 1)])
def test_scores_refuse(lib, kw, status):
    assert _scores(lib, **kw) == status


def _scores_grad(lib, rows=6, logits=FAKE, stride=50, tokens=FAKE, up=FAKE, d=FAKE + (1 << 30), d_stride=1 << 25, **cfg):
    c = _set(b.make_score_config(50, 4, 1.5, "f32"), cfg)
    return lib.cdrge_token_scores_grad(ctypes.byref(c), rows, logits, stride, tokens, up, FAKE, d, d_stride, None)


@pytest.mark.parametrize("kw, status", SCORES + [(dict(tokens=None), 1), (dict(d=None), 1), (dict(d_stride=49), 1),
                                                 (dict(d=FAKE, d_stride=60), 1)])
def test_scores_grad_refuses(lib, kw, status):
    assert _scores_grad(lib, **kw) == status


def test_scores_without_rows(lib):
    assert _scores(lib, rows=0, logits=None, tokens=None, ids=None, lps=None) == 0
    assert _scores_grad(lib, rows=0, logits=None, tokens=None, d=None) == 0


def _project(lib, rows=5, codes=FAKE, scales=FAKE, x=FAKE, y=FAKE, x_stride=1 << 21, y_stride=1 << 21, ws=FAKE, nbytes=1 << 40,
             **cfg):
    c = _set(b.make_mx_config(70, 96, "f32"), cfg)
    return lib.cdrge_mx_project(ctypes.byref(c), codes, scales, FAKE, rows, x, x_stride, y, y_stride, ws, nbytes, None)


MX = [(dict(abi_version=3), 1), (dict(dtype=2), 1), (dict(in_features=0), 1), (dict(out_features=0), 1), (dict(rows=-1), 1),
      (dict(rows=(1 << 30) + 1), 2), (dict(in_features=(1 << 20) + 1), 2), (dict(out_features=(1 << 20) + 1), 2), (dict(codes=None), 1),
      (dict(codes=FAKE + 8), 1), (dict(scales=None), 1), (dict(x=None), 1), (dict(x_stride=69), 1)]


@pytest.mark.parametrize("kw, status", MX + [(dict(y=None), 1), (dict(y_stride=95), 1), (dict(ws=None), 3), (dict(nbytes=4), 3),
                                             (dict(ws=FAKE + 4), 3)])
def test_mx_project_refuses(lib, kw, status):
    assert _project(lib, **kw) == status


@pytest.mark.parametrize("kw, status", MX)
def test_mx_quantize_and_dequantize_refuse(lib, kw, status):
    kw = dict(rows=5, codes=FAKE, scales=FAKE, x=FAKE, x_stride=1 << 21) | kw
    if "codes" in kw and kw["codes"] is None:
        kw["codes"] = 0
    c = b.make_mx_config(70, 96, "f32")
    for name in list(kw):
        if hasattr(c, name):
            setattr(c, name, kw.pop(name))
    c = ctypes.byref(c)
    assert lib.cdrge_mx_quantize(c, kw["rows"], kw["x"], kw["x_stride"], kw["codes"], kw["scales"], None) == status
    assert lib.cdrge_mx_dequantize(c, kw["rows"], kw["codes"], kw["scales"], kw["x"], kw["x_stride"], None) == status


def test_mx_without_rows(lib):
    assert _project(lib, rows=0, x=None, y=None, ws=None, nbytes=0) == 0
    c = ctypes.byref(b.make_mx_config(70, 96, "f32"))
    assert lib.cdrge_mx_quantize(c, 0, None, 70, None, None, None) == 0
    assert lib.cdrge_mx_dequantize(c, 0, None, None, None, 70, None) == 0


def test_classes_refuse_cpu_tensors(lib):
    import torch
    with pytest.raises(ValueError):
        b.DeltaLayer(b.make_delta_config(4, 2, 64, 32, "bf16"), torch.zeros(4))
    with pytest.raises(ValueError):
        b.TokenScores(b.make_score_config(50, 4, 1.5, "f32"), device="cpu")
    with pytest.raises(ValueError):
        b.MxFormat(b.make_mx_config(64, 64, "f32"), device="cpu")
    with pytest.raises(ValueError):
        b.MxProjection(b.make_mx_config(64, 64, "f32"), torch.zeros(64, 32, dtype=torch.uint8), torch.zeros(64, 2, dtype=torch.uint8))
