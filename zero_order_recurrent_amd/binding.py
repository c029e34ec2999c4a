"""ctypes binding of libcdrge.so (include/cdrge.h), argument marshalling only.

Every function mirrors the C entry point of the same name. Device buffers are torch tensors on
the GPU (only their data pointers cross the boundary); the stream is torch's current stream
unless one is given. There is no fallback: if libcdrge.so is missing or does not load, every call
raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libcdrge.so")

CDRGE_ABI_VERSION = 1
CDRGE_F32, CDRGE_BF16, CDRGE_BF16_EXACT = 0, 1, 2
STATUS = {0: "CDRGE_OK", 1: "CDRGE_ERR_INVALID_ARG", 2: "CDRGE_ERR_UNSUPPORTED", 3: "CDRGE_ERR_WORKSPACE",
          4: "CDRGE_ERR_DEVICE", 5: "CDRGE_ERR_NONFINITE"}
KIND_GATES, KIND_CE, KIND_UPDATE, KIND_PREP = 0, 1, 2, 3


class CdrgeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}")
        self.status = status


class cdrge_config(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("n_layers", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("embed", ctypes.c_int32), ("hidden", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("seq_len", ctypes.c_int32), ("n_probes", ctypes.c_int32), ("probes_per_chunk", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("lr", ctypes.c_float),
                ("base_seed", ctypes.c_uint64)]


def make_config(n_layers, vocab, embed, hidden, batch, seq_len, n_probes, dtype, eps, lr, base_seed,
                probes_per_chunk=0) -> cdrge_config:
    dt = {"f32": CDRGE_F32, "bf16": CDRGE_BF16, "bf16x": CDRGE_BF16_EXACT}.get(dtype, dtype)
    return cdrge_config(CDRGE_ABI_VERSION, n_layers, vocab, embed, hidden, batch, seq_len, n_probes,
                        probes_per_chunk, dt, eps, lr, base_seed)


class cdrge_scan_config(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("dtype", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("state_dim", ctypes.c_int32),
                ("conv_width", ctypes.c_int32)]


class cdrge_scan_weights(ctypes.Structure):
    _fields_ = [("conv_weight", ctypes.c_void_p), ("conv_bias", ctypes.c_void_p), ("decay", ctypes.c_void_p),
                ("skip", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p)]


class cdrge_scan_io(ctypes.Structure):
    _fields_ = [("xbc", ctypes.c_void_p), ("xbc_stride", ctypes.c_int64), ("dt", ctypes.c_void_p),
                ("dt_stride", ctypes.c_int64), ("z", ctypes.c_void_p), ("z_stride", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64), ("n_tokens", ctypes.c_int64),
                ("n_seqs", ctypes.c_int32), ("n_slots", ctypes.c_int32), ("offsets", ctypes.c_void_p),
                ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("conv_in", ctypes.c_void_p),
                ("conv_out", ctypes.c_void_p), ("ssm_in", ctypes.c_void_p), ("ssm_out", ctypes.c_void_p)]


class cdrge_adapter_config(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("dtype", ctypes.c_int32), ("in_features", ctypes.c_int32),
                ("out_features", ctypes.c_int32), ("n_adapters", ctypes.c_int32), ("max_rank", ctypes.c_int32)]


class cdrge_adapter_weights(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("weight_stride", ctypes.c_int64), ("bias", ctypes.c_void_p),
                ("down", ctypes.c_void_p), ("up", ctypes.c_void_p), ("ranks", ctypes.c_void_p)]


class cdrge_distill_config(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("dtype", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("n_models", ctypes.c_int32), ("temperature", ctypes.c_float)]


class cdrge_delta_config(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("dtype", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("value_dim", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("key_dim", ctypes.c_int32),
                ("q_scale", ctypes.c_float), ("norm_eps", ctypes.c_float)]


class cdrge_delta_weights(ctypes.Structure):
    _fields_ = [("decay", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p)]


class cdrge_delta_io(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("k_stride", ctypes.c_int64), ("v", ctypes.c_void_p), ("v_stride", ctypes.c_int64),
                ("dt", ctypes.c_void_p), ("dt_stride", ctypes.c_int64), ("beta", ctypes.c_void_p),
                ("beta_stride", ctypes.c_int64), ("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64),
                ("n_tokens", ctypes.c_int64), ("n_seqs", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("offsets", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("state_in", ctypes.c_void_p), ("state_out", ctypes.c_void_p)]


class cdrge_score_config(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("dtype", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("temperature", ctypes.c_float)]


class cdrge_mx_config(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_uint32), ("dtype", ctypes.c_int32), ("in_features", ctypes.c_int32),
                ("out_features", ctypes.c_int32)]


_OPERATOR_DTYPES = {"f32": CDRGE_F32, "bf16": CDRGE_BF16}


def make_scan_config(n_heads, head_dim, n_groups, state_dim, conv_width, dtype) -> cdrge_scan_config:
    return cdrge_scan_config(CDRGE_ABI_VERSION, _OPERATOR_DTYPES.get(dtype, dtype), n_heads, head_dim, n_groups,
                             state_dim, conv_width)


def make_adapter_config(in_features, out_features, n_adapters, max_rank, dtype) -> cdrge_adapter_config:
    return cdrge_adapter_config(CDRGE_ABI_VERSION, _OPERATOR_DTYPES.get(dtype, dtype), in_features, out_features,
                                n_adapters, max_rank)


def make_distill_config(vocab, top_k, n_models, temperature, dtype) -> cdrge_distill_config:
    return cdrge_distill_config(CDRGE_ABI_VERSION, _OPERATOR_DTYPES.get(dtype, dtype), vocab, top_k, n_models,
                                temperature)


def make_delta_config(n_heads, n_groups, key_dim, value_dim, dtype, q_scale=None, norm_eps=1e-6) -> cdrge_delta_config:
    """q_scale None: key_dim^-0.5."""
    return cdrge_delta_config(CDRGE_ABI_VERSION, _OPERATOR_DTYPES.get(dtype, dtype), n_heads, value_dim, n_groups, key_dim,
                              max(key_dim, 1) ** -0.5 if q_scale is None else q_scale, norm_eps)


def make_score_config(vocab, top_k, temperature, dtype) -> cdrge_score_config:
    return cdrge_score_config(CDRGE_ABI_VERSION, _OPERATOR_DTYPES.get(dtype, dtype), vocab, top_k, temperature)


def make_mx_config(in_features, out_features, dtype) -> cdrge_mx_config:
    return cdrge_mx_config(CDRGE_ABI_VERSION, _OPERATOR_DTYPES.get(dtype, dtype), in_features, out_features)


def config_from_preset(p) -> cdrge_config:
    return make_config(p.n_layers, p.vocab, p.embed, p.hidden, p.batch, p.seq_len, p.n_probes, p.dtype,
                       p.eps, p.lr, p.base_seed, p.probes_per_chunk)


_lib = None

EXPORTS = {
    "cdrge_param_count": (ctypes.c_int64, [ctypes.c_void_p]),
    "cdrge_check_config": (ctypes.c_int, [ctypes.c_void_p]),
    "cdrge_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)]),
    "cdrge_probe_seeds": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]),
    "cdrge_init": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "cdrge_probe_losses": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p,
                                          ctypes.c_void_p]),
    "cdrge_update": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]),
    "cdrge_step": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]),
    "cdrge_sync_status": (ctypes.c_int, [ctypes.c_void_p]),
    "cdrge_destroy": (None, [ctypes.c_void_p]),
    "cdrge_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "cdrge_last_error_detail": (ctypes.c_char_p, []),
    "cdrge_set_timing": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "cdrge_get_timing": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_double),
                                        ctypes.POINTER(ctypes.c_int64), ctypes.c_int]),
    "cdrge_get_work": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_double)]),
    "cdrge_timed_kernel": (ctypes.c_char_p, [ctypes.c_void_p, ctypes.c_int]),
    "cdrge_probe_losses_io": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint64,
                                             ctypes.c_void_p, ctypes.c_void_p]),
    "cdrge_step_io": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint64,
                                     ctypes.c_void_p]),
    "cdrge_step_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint64,
                                          ctypes.c_void_p, ctypes.c_void_p]),
    "cdrge_noalloc_max_workspace_bytes": (ctypes.c_size_t, []),
    "cdrge_scan_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                                  ctypes.POINTER(ctypes.c_size_t)]),
    "cdrge_scan_prompt": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_size_t, ctypes.c_void_p]),
    "cdrge_scan_step": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "cdrge_adapter_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]),
    "cdrge_adapter_project": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                             ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "cdrge_distill_losses": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_void_p]),
    "cdrge_distill_grad": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "cdrge_delta_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                                   ctypes.POINTER(ctypes.c_size_t)]),
    "cdrge_delta_prompt": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_size_t, ctypes.c_void_p]),
    "cdrge_delta_step": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "cdrge_token_scores": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p]),
    "cdrge_token_scores_grad": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_int64, ctypes.c_void_p]),
    "cdrge_mx_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "cdrge_mx_dequantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "cdrge_mx_workspace_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]),
    "cdrge_mx_project": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_void_p]),
}


def lib():
    """Loads libcdrge.so (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        # The caller's device buffers and streams come from torch's HIP runtime; importing torch
        # first makes the loader bind libcdrge.so to that same runtime (same soname) instead of
        # starting a second one.
        import torch  # noqa: F401
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(status: int, where: str):
    if status != 0:
        detail = lib().cdrge_last_error_detail().decode() if status in (3, 4) else ""
        raise CdrgeError(status, f"{where} {detail}".strip())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# ---- entry points, same names as the C ABI ------------------------------------------------------

def cdrge_param_count(cfg: cdrge_config) -> int:
    return int(lib().cdrge_param_count(ctypes.byref(cfg)))


def cdrge_check_config(cfg: cdrge_config) -> int:
    return int(lib().cdrge_check_config(ctypes.byref(cfg)))


def cdrge_workspace_bytes(cfg: cdrge_config) -> int:
    out = ctypes.c_size_t()
    _check(lib().cdrge_workspace_bytes(ctypes.byref(cfg), ctypes.byref(out)), "cdrge_workspace_bytes")
    return int(out.value)


def cdrge_probe_seeds(cfg: cdrge_config, step: int):
    import numpy as np
    out = np.zeros(cfg.n_probes, dtype=np.uint64)
    _check(lib().cdrge_probe_seeds(ctypes.byref(cfg), step, out.ctypes.data_as(ctypes.c_void_p)),
           "cdrge_probe_seeds")
    return out


def cdrge_init(cfg: cdrge_config, params, workspace, stream=None) -> ctypes.c_void_p:
    ctx = ctypes.c_void_p()
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().cdrge_init(ctypes.byref(ctx), ctypes.byref(cfg), _ptr(params), _ptr(workspace), nbytes,
                            _stream_handle(stream)), "cdrge_init")
    return ctx


def cdrge_probe_losses(ctx, tokens, step: int, losses, seq_losses=None):
    _check(lib().cdrge_probe_losses(ctx, _ptr(tokens), step, _ptr(losses), _ptr(seq_losses)), "cdrge_probe_losses")


def cdrge_update(ctx, step: int, losses):
    _check(lib().cdrge_update(ctx, step, _ptr(losses)), "cdrge_update")


def cdrge_step(ctx, tokens, step: int, losses):
    _check(lib().cdrge_step(ctx, _ptr(tokens), step, _ptr(losses)), "cdrge_step")


def cdrge_probe_losses_io(ctx, inputs, targets, step: int, losses, seq_losses=None):
    _check(lib().cdrge_probe_losses_io(ctx, _ptr(inputs), _ptr(targets), step, _ptr(losses), _ptr(seq_losses)),
           "cdrge_probe_losses_io")


def cdrge_step_io(ctx, inputs, targets, step: int, losses):
    _check(lib().cdrge_step_io(ctx, _ptr(inputs), _ptr(targets), step, _ptr(losses)), "cdrge_step_io")


def cdrge_sync_status(ctx) -> int:
    return int(lib().cdrge_sync_status(ctx))


def cdrge_destroy(ctx):
    lib().cdrge_destroy(ctx)


def cdrge_status_string(status: int) -> str:
    return lib().cdrge_status_string(status).decode()


def cdrge_last_error_detail() -> str:
    return lib().cdrge_last_error_detail().decode()


def cdrge_set_timing(ctx, enable: bool):
    _check(lib().cdrge_set_timing(ctx, int(enable)), "cdrge_set_timing")


def cdrge_get_timing(ctx, kind: int, reset: bool = False):
    ms = ctypes.c_double()
    n = ctypes.c_int64()
    _check(lib().cdrge_get_timing(ctx, kind, ctypes.byref(ms), ctypes.byref(n), int(reset)), "cdrge_get_timing")
    return ms.value, n.value


def cdrge_get_work(ctx, kind: int) -> float:
    w = ctypes.c_double()
    _check(lib().cdrge_get_work(ctx, kind, ctypes.byref(w)), "cdrge_get_work")
    return w.value


def cdrge_timed_kernel(ctx, kind: int) -> str:
    return lib().cdrge_timed_kernel(ctx, kind).decode()


def cdrge_step_noalloc(cfg: cdrge_config, params, tokens, step: int, losses, stream=None):
    _check(lib().cdrge_step_noalloc(ctypes.byref(cfg), _ptr(params), _ptr(tokens), step, _ptr(losses),
                                    _stream_handle(stream)), "cdrge_step_noalloc")


def cdrge_noalloc_max_workspace_bytes() -> int:
    return int(lib().cdrge_noalloc_max_workspace_bytes())


class Context:
    """Owns a context plus its torch-allocated parameter and workspace buffers on the GPU."""

    def __init__(self, cfg: cdrge_config, params, device="cuda", stream=None):
        import torch
        self.cfg = cfg
        self.d = cdrge_param_count(cfg)
        if params.numel() != self.d:
            raise ValueError(f"params has {params.numel()} elements, the configuration needs {self.d}")
        want = torch.float32 if cfg.dtype == CDRGE_F32 else torch.int16
        if params.dtype != want or not params.is_cuda or not params.is_contiguous():
            raise ValueError("params must be a contiguous CUDA tensor of float32 (fp32) or int16 bf16 bits")
        self.params = params
        nbytes = cdrge_workspace_bytes(cfg)
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=params.device)
        self.stream = stream
        self.ctx = cdrge_init(cfg, params, self.workspace, stream)
        self.losses = torch.empty(2 * cfg.n_probes, dtype=torch.float32, device=params.device)

    def probe_losses(self, tokens, step: int, seq_losses=None):
        cdrge_probe_losses(self.ctx, tokens, step, self.losses, seq_losses)
        return self.losses

    def update(self, step: int, losses=None):
        cdrge_update(self.ctx, step, self.losses if losses is None else losses)

    def step(self, tokens, step: int):
        cdrge_step(self.ctx, tokens, step, self.losses)
        return self.losses

    def probe_losses_io(self, inputs, targets, step: int, seq_losses=None):
        cdrge_probe_losses_io(self.ctx, inputs, targets, step, self.losses, seq_losses)
        return self.losses

    def step_io(self, inputs, targets, step: int):
        cdrge_step_io(self.ctx, inputs, targets, step, self.losses)
        return self.losses

    def sync_status(self) -> int:
        return cdrge_sync_status(self.ctx)

    def close(self):
        if self.ctx:
            cdrge_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- operators of a population of models ---------------------------------------------------------
#
# The C entry points take structures and pointers; the classes below hold an operator's weights and
# check the tensors of a call (type, shape, device, rows whose elements are adjacent) before their
# pointers cross the boundary. A call runs on torch's current stream of the tensors' device unless
# one is given, allocates its workspace there through torch, and keeps nothing for the next call.

def cdrge_scan_workspace_bytes(cfg: cdrge_scan_config, n_tokens: int, n_seqs: int) -> int:
    out = ctypes.c_size_t()
    _check(lib().cdrge_scan_workspace_bytes(ctypes.byref(cfg), n_tokens, n_seqs, ctypes.byref(out)),
           "cdrge_scan_workspace_bytes")
    return int(out.value)


def cdrge_scan_prompt(cfg, weights: cdrge_scan_weights, io: cdrge_scan_io, workspace, stream: int):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().cdrge_scan_prompt(ctypes.byref(cfg), ctypes.byref(weights), ctypes.byref(io), _ptr(workspace), nbytes,
                                   stream), "cdrge_scan_prompt")


def cdrge_scan_step(cfg, weights: cdrge_scan_weights, io: cdrge_scan_io, stream: int):
    _check(lib().cdrge_scan_step(ctypes.byref(cfg), ctypes.byref(weights), ctypes.byref(io), stream), "cdrge_scan_step")


def cdrge_adapter_workspace_bytes(cfg: cdrge_adapter_config, n_rows: int) -> int:
    out = ctypes.c_size_t()
    _check(lib().cdrge_adapter_workspace_bytes(ctypes.byref(cfg), n_rows, ctypes.byref(out)),
           "cdrge_adapter_workspace_bytes")
    return int(out.value)


def cdrge_adapter_project(cfg, weights: cdrge_adapter_weights, n_rows, x, row_adapter, row_scale, y, workspace,
                          stream: int):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().cdrge_adapter_project(ctypes.byref(cfg), ctypes.byref(weights), n_rows, x.data_ptr(), _row_stride(x),
                                       _ptr(row_adapter), _ptr(row_scale), y.data_ptr(), _row_stride(y),
                                       _ptr(workspace), nbytes, stream), "cdrge_adapter_project")


def cdrge_distill_losses(cfg, logits, ids, teacher, row_losses, losses, stream: int):
    _check(lib().cdrge_distill_losses(ctypes.byref(cfg), logits.shape[0], logits.data_ptr(), _row_stride(logits),
                                      ids.data_ptr(), teacher.data_ptr(), row_losses.data_ptr(), _ptr(losses), stream),
           "cdrge_distill_losses")


def cdrge_distill_grad(cfg, logits, ids, teacher, row_grad, row_losses, losses, dlogits, stream: int):
    _check(lib().cdrge_distill_grad(ctypes.byref(cfg), logits.shape[0], logits.data_ptr(), _row_stride(logits),
                                    ids.data_ptr(), teacher.data_ptr(), _ptr(row_grad), row_losses.data_ptr(),
                                    _ptr(losses), dlogits.data_ptr(), _row_stride(dlogits), stream),
           "cdrge_distill_grad")


def cdrge_delta_workspace_bytes(cfg: cdrge_delta_config, n_tokens: int, n_seqs: int) -> int:
    out = ctypes.c_size_t()
    _check(lib().cdrge_delta_workspace_bytes(ctypes.byref(cfg), n_tokens, n_seqs, ctypes.byref(out)),
           "cdrge_delta_workspace_bytes")
    return int(out.value)


def cdrge_delta_prompt(cfg, weights: cdrge_delta_weights, io: cdrge_delta_io, workspace, stream: int):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().cdrge_delta_prompt(ctypes.byref(cfg), ctypes.byref(weights), ctypes.byref(io), _ptr(workspace), nbytes,
                                    stream), "cdrge_delta_prompt")


def cdrge_delta_step(cfg, weights: cdrge_delta_weights, io: cdrge_delta_io, stream: int):
    _check(lib().cdrge_delta_step(ctypes.byref(cfg), ctypes.byref(weights), ctypes.byref(io), stream), "cdrge_delta_step")


def cdrge_token_scores(cfg, logits, tokens, logprobs, entropy, top_ids, top_logprobs, stream: int):
    _check(lib().cdrge_token_scores(ctypes.byref(cfg), logits.shape[0], logits.data_ptr(), _row_stride(logits), _ptr(tokens),
                                    _ptr(logprobs), _ptr(entropy), _ptr(top_ids), _ptr(top_logprobs), stream),
           "cdrge_token_scores")


def cdrge_token_scores_grad(cfg, logits, tokens, d_logprob, d_entropy, dlogits, stream: int):
    _check(lib().cdrge_token_scores_grad(ctypes.byref(cfg), logits.shape[0], logits.data_ptr(), _row_stride(logits),
                                         _ptr(tokens), _ptr(d_logprob), _ptr(d_entropy), dlogits.data_ptr(),
                                         _row_stride(dlogits), stream), "cdrge_token_scores_grad")


def cdrge_mx_quantize(cfg, x, codes, scales, stream: int):
    _check(lib().cdrge_mx_quantize(ctypes.byref(cfg), x.shape[0], x.data_ptr(), _row_stride(x), codes.data_ptr(),
                                   scales.data_ptr(), stream), "cdrge_mx_quantize")


def cdrge_mx_dequantize(cfg, codes, scales, x, stream: int):
    _check(lib().cdrge_mx_dequantize(ctypes.byref(cfg), x.shape[0], codes.data_ptr(), scales.data_ptr(), x.data_ptr(),
                                     _row_stride(x), stream), "cdrge_mx_dequantize")


def cdrge_mx_workspace_bytes(cfg: cdrge_mx_config, n_rows: int) -> int:
    out = ctypes.c_size_t()
    _check(lib().cdrge_mx_workspace_bytes(ctypes.byref(cfg), n_rows, ctypes.byref(out)), "cdrge_mx_workspace_bytes")
    return int(out.value)


def cdrge_mx_project(cfg, w_codes, w_scales, bias, n_rows, x, y, workspace, stream: int):
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().cdrge_mx_project(ctypes.byref(cfg), w_codes.data_ptr(), w_scales.data_ptr(), _ptr(bias), n_rows, x.data_ptr(),
                                  _row_stride(x), y.data_ptr(), _row_stride(y), _ptr(workspace), nbytes, stream),
           "cdrge_mx_project")


def _row_stride(t) -> int:
    # a single row may have any stride, also one below its length; the library wants at least that
    n = t.shape[1]
    stride = t.stride(0)
    return stride if stride > n else n


def _refuse(name, t, dtype, shape, index, rows):
    """Says what is wrong with an argument that _rows or _whole has found wrong."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have the shape {shape}, not {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the operator on cuda:{index}")
    if rows:
        raise ValueError(f"{name} needs rows of adjacent elements that do not overlap, not strides {t.stride()}")
    raise ValueError(f"{name} must be contiguous")


def _whole(name, t, dtype, shape, index) -> int:
    """Checks a contiguous argument of the shape, type and device; returns its pointer. The checks are written for the
    common case: they are a good part of a small call's time."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(name, t, dtype, shape, index, False)
    return t.data_ptr()


def _rows(name, t, dtype, shape, index) -> int:
    """The same for a matrix whose rows may lie further apart than their length."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        _refuse(name, t, dtype, shape, index, True)
    if not t.is_contiguous():
        n, width = shape
        row, col = t.stride()
        if (col != 1 and width > 1 and n > 0) or (row < width and n > 1):
            _refuse(name, t, dtype, shape, index, True)
    return t.data_ptr()


class _Operator:
    """What the operators share: the element type, the device, and running on its stream."""

    def __init__(self, cfg, device):
        import torch
        self.cfg = cfg
        if cfg.dtype not in (CDRGE_F32, CDRGE_BF16):
            raise CdrgeError(1, type(self).__name__)
        self.dtype = torch.float32 if cfg.dtype == CDRGE_F32 else torch.bfloat16
        self.device = device
        self.index = device.index
        self._cfg = ctypes.addressof(cfg)
        self._torch = torch
        self._lib = lib()
        self._current_device = torch._C._cuda_getDevice
        self._current_stream = torch._C._cuda_getCurrentRawStream
        self._sizes = {}

    def _bytes(self, query, *sizes) -> int:
        """The workspace of a call of these sizes, asked once for each of the last few hundred."""
        n = self._sizes.get(sizes)
        if n is None:
            if len(self._sizes) >= 256:
                self._sizes.clear()
            n = self._sizes[sizes] = query(self.cfg, *sizes)
        return n

    def _run(self, call, nbytes, stream):
        """call(workspace or None, stream handle) on the operator's device. The workspace belongs to the call's stream,
        so that torch gives its memory to nobody before the call has run."""
        torch = self._torch
        if stream is None and self.index == self._current_device():
            ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None
            call(ws, self._current_stream(self.index))
            return
        with torch.cuda.device(self.device):
            on = torch.cuda.current_stream() if stream is None else stream
            if on.device != self.device:
                raise ValueError(f"the stream is on {on.device}, the operator on {self.device}")
            with torch.cuda.stream(on):
                ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None
                call(ws, on.cuda_stream)


def _cuda_device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _gpu(device):
    import torch
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError("the operator runs on a GPU")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


# cdrge_scan_io as bytes: building them is quicker than filling a ctypes structure, and they belong to one call
_SCAN_IO = struct.Struct("@" + "Pq" * 4 + "qii" + "P" * 7)
assert _SCAN_IO.size == ctypes.sizeof(cdrge_scan_io)


class ScanLayer(_Operator):
    """Selective scan with its short causal convolution (cdrge_scan_prompt, cdrge_scan_step).

    conv_weight [channels, conv_width] and conv_bias [channels] or None in the layer's type; decay, skip and dt_bias
    [n_heads] in float32, the latter two or None. channels = n_heads * head_dim + 2 * n_groups * state_dim.
    """

    def __init__(self, cfg: cdrge_scan_config, conv_weight, conv_bias, decay, skip=None, dt_bias=None):
        super().__init__(cfg, _cuda_device(conv_weight, "conv_weight"))
        torch = self._torch
        cdrge_scan_workspace_bytes(cfg, 0, 1)  # raises for a configuration that is not valid or supported
        self.width = cfg.n_heads * cfg.head_dim
        self.channels = self.width + 2 * cfg.n_groups * cfg.state_dim
        self._held = (conv_weight, conv_bias, decay, skip, dt_bias)
        f, heads, at = torch.float32, (cfg.n_heads,), self.index
        self.weights = cdrge_scan_weights(
            _whole("conv_weight", conv_weight, self.dtype, (self.channels, cfg.conv_width), at),
            None if conv_bias is None else _whole("conv_bias", conv_bias, self.dtype, (self.channels,), at),
            _whole("decay", decay, f, heads, at), None if skip is None else _whole("skip", skip, f, heads, at),
            None if dt_bias is None else _whole("dt_bias", dt_bias, f, heads, at))
        self._weights = ctypes.addressof(self.weights)
        self._state_shapes = (cfg.conv_width, self.channels), (cfg.n_heads, cfg.head_dim, cfg.state_dim)

    def _io(self, xbc, dt, y, n_seqs, z, offsets, slots, positions, conv_in, ssm_in, conv_out, ssm_out):
        at, n, t, heads, width = self.index, xbc.shape[0], self.dtype, self.cfg.n_heads, self.width
        i32 = self._torch.int32
        p_xbc = _rows("xbc", xbc, t, (n, self.channels), at)
        p_dt = _rows("dt", dt, t, (n, heads), at)
        p_y = _rows("y", y, t, (n, width), at)
        p_z, z_stride = (0, 0) if z is None else (_rows("z", z, t, (n, width), at), _row_stride(z))
        p_offsets = 0 if offsets is None else _whole("offsets", offsets, i32, (n_seqs + 1,), at)
        p_slots = 0 if slots is None else _whole("slots", slots, i32, (n_seqs,), at)
        p_positions = 0 if positions is None else _whole("positions", positions, i32, (n_seqs,), at)
        p_ci = p_co = p_si = p_so = n_slots = 0
        if conv_in is not None and ssm_in is not None:
            n_slots = ssm_in.shape[0]
            conv, ssm = self._state_shapes
            f = self._torch.float32
            p_ci = p_co = _whole("the convolution's state", conv_in, t, (n_slots, *conv), at)
            p_si = p_so = _whole("the scan's state", ssm_in, f, (n_slots, *ssm), at)
            if conv_out is not None:
                p_co = _whole("conv_out", conv_out, t, (n_slots, *conv), at)
            if ssm_out is not None:
                p_so = _whole("ssm_out", ssm_out, f, (n_slots, *ssm), at)
        elif conv_in is not None or ssm_in is not None:
            raise ValueError("the convolution's state and the scan's are given together or not at all")
        elif conv_out is not None or ssm_out is not None:
            raise ValueError("an output state needs the states that are read")
        return _SCAN_IO.pack(p_xbc, _row_stride(xbc), p_dt, _row_stride(dt), p_z, z_stride, p_y, _row_stride(y), n,
                             n_seqs, n_slots, p_offsets, p_slots, p_positions, p_ci, p_co, p_si, p_so)

    def prompt(self, xbc, dt, y, n_seqs, z=None, offsets=None, slots=None, positions=None, conv_state=None,
               ssm_state=None, conv_out=None, ssm_out=None, stream=None):
        """Whole or continued prompts: rows offsets[i] .. offsets[i + 1] - 1 (or equal shares of the rows) belong to
        sequence i. Writes y, and the states in place unless conv_out and ssm_out are given. Returns y."""
        io = self._io(xbc, dt, y, n_seqs, z, offsets, slots, positions, conv_state, ssm_state, conv_out, ssm_out)
        tokens = xbc.shape[0]
        short = offsets is None and ssm_state is None and 0 < tokens <= 16 * n_seqs  # these need no workspace
        n = 0 if short else self._bytes(cdrge_scan_workspace_bytes, tokens, n_seqs)
        call = self._lib.cdrge_scan_prompt
        self._run(lambda ws, s: _check(call(self._cfg, self._weights, io, 0 if ws is None else ws.data_ptr(), n, s),
                                       "cdrge_scan_prompt"), n, stream)
        return y

    def step(self, xbc, dt, y, positions, conv_state, ssm_state, z=None, slots=None, conv_out=None, ssm_out=None,
             stream=None):
        """One token of each sequence, row i at place positions[i] of the sequence in slot slots[i] (negative: padding).
        Writes y, and the states in place unless conv_out and ssm_out are given. Returns y."""
        n = xbc.shape[0]
        io = self._io(xbc, dt, y, n, z, None, slots, positions, conv_state, ssm_state, conv_out, ssm_out)
        if n:
            call = self._lib.cdrge_scan_step
            self._run(lambda ws, s: _check(call(self._cfg, self._weights, io, s), "cdrge_scan_step"), 0, stream)
        return y


class AdapterProjection(_Operator):
    """A projection shared by all rows with a low-rank adapter by row (cdrge_adapter_project).

    weight [out, in] (its rows may lie apart), bias [out] or None, down [n_adapters, max_rank, in], up [n_adapters, out,
    max_rank] in the operator's type; ranks int32 [n_adapters] or None.
    """

    def __init__(self, cfg: cdrge_adapter_config, weight, bias=None, down=None, up=None, ranks=None):
        super().__init__(cfg, _cuda_device(weight, "weight"))
        cdrge_adapter_workspace_bytes(cfg, 0)
        K, O, A, R = cfg.in_features, cfg.out_features, cfg.n_adapters, cfg.max_rank
        t, at = self.dtype, self.index
        self._held = (weight, bias, down, up, ranks)
        p = [_rows("weight", weight, t, (O, K), at), None, None, None, None]
        if bias is not None:
            p[1] = _whole("bias", bias, t, (O,), at)
        if A > 0:
            if down is None or up is None:
                raise ValueError("adapters need their down and up weights")
            p[2:] = (_whole("down", down, t, (A, R, K), at), _whole("up", up, t, (A, O, R), at),
                     None if ranks is None else _whole("ranks", ranks, self._torch.int32, (A,), at))
        self.weights = cdrge_adapter_weights(p[0], _row_stride(weight), *p[1:])
        self._weights = ctypes.addressof(self.weights)

    def project(self, x, row_adapter, y, row_scale=None, stream=None):
        """y[r] = weight x[r] + bias + row_scale[r] up_a (down_a x[r]), a = row_adapter[r] (negative, or row_adapter
        None: no adapter). Returns y."""
        n, cfg, torch, at, t = x.shape[0], self.cfg, self._torch, self.index, self.dtype
        p_x = _rows("x", x, t, (n, cfg.in_features), at)
        p_y = _rows("y", y, t, (n, cfg.out_features), at)
        p_who = 0 if row_adapter is None else _whole("row_adapter", row_adapter, torch.int32, (n,), at)
        p_scale = 0 if row_scale is None else _whole("row_scale", row_scale, torch.float32, (n,), at)
        nbytes = self._bytes(cdrge_adapter_workspace_bytes, n)
        call = self._lib.cdrge_adapter_project
        x_stride, y_stride = _row_stride(x), _row_stride(y)
        self._run(lambda ws, s: _check(call(self._cfg, self._weights, n, p_x, x_stride, p_who, p_scale, p_y, y_stride,
                                            0 if ws is None else ws.data_ptr(), nbytes, s), "cdrge_adapter_project"),
                  nbytes, stream)
        return y


class DistillLoss(_Operator):
    """Distillation from a teacher's top logits (cdrge_distill_losses, cdrge_distill_grad)."""

    def __init__(self, cfg: cdrge_distill_config, device=None):
        super().__init__(cfg, _gpu(device))

    def _inputs(self, logits, ids, teacher, row_losses, losses):
        n, cfg, at, f = logits.shape[0], self.cfg, self.index, self._torch.float32
        return (self._cfg, n, _rows("logits", logits, self.dtype, (n, cfg.vocab), at), _row_stride(logits),
                _whole("ids", ids, self._torch.int32, (n, cfg.top_k), at),
                _whole("teacher", teacher, f, (n, cfg.top_k), at),
                _whole("row_losses", row_losses, f, (n,), at),
                0 if losses is None else _whole("losses", losses, f, (cfg.n_models,), at))

    def losses(self, logits, ids, teacher, row_losses, losses=None, stream=None):
        """Fills row_losses [rows] and, if given, losses [n_models], the means by model (NaN where no row is scored)."""
        args = self._inputs(logits, ids, teacher, row_losses, losses)
        call = self._lib.cdrge_distill_losses
        self._run(lambda ws, s: _check(call(*args, s), "cdrge_distill_losses"), 0, stream)
        return row_losses

    def grad(self, logits, ids, teacher, row_grad, row_losses, losses, dlogits, stream=None):
        """The losses, and dlogits[r] = row_grad[r] d row_loss_r / d logits[r] (row_grad None: 1; losses may be None).
        dlogits may be logits itself. Returns dlogits."""
        args = self._inputs(logits, ids, teacher, row_losses, losses)
        n = logits.shape[0]
        p_up = 0 if row_grad is None else _whole("row_grad", row_grad, self._torch.float32, (n,), self.index)
        p_d = _rows("dlogits", dlogits, self.dtype, (n, self.cfg.vocab), self.index)
        d_stride = _row_stride(dlogits)
        call = self._lib.cdrge_distill_grad
        self._run(lambda ws, s: _check(call(*args[:6], p_up, *args[6:], p_d, d_stride, s), "cdrge_distill_grad"), 0,
                  stream)
        return dlogits


# cdrge_delta_io as bytes, as _SCAN_IO
_DELTA_IO = struct.Struct("@" + "Pq" * 6 + "qii" + "P" * 5)
assert _DELTA_IO.size == ctypes.sizeof(cdrge_delta_io)


class DeltaLayer(_Operator):
    """Gated delta rule (cdrge_delta_prompt, cdrge_delta_step). decay and dt_bias [n_heads] in float32, the latter or None.
    """

    def __init__(self, cfg: cdrge_delta_config, decay, dt_bias=None):
        super().__init__(cfg, _cuda_device(decay, "decay"))
        cdrge_delta_workspace_bytes(cfg, 0, 1)  # raises for a configuration that is not valid or supported
        f, heads, at = self._torch.float32, (cfg.n_heads,), self.index
        self.keys, self.values = cfg.n_groups * cfg.key_dim, cfg.n_heads * cfg.value_dim
        self._held = (decay, dt_bias)
        self.weights = cdrge_delta_weights(_whole("decay", decay, f, heads, at),
                                           None if dt_bias is None else _whole("dt_bias", dt_bias, f, heads, at))
        self._weights = ctypes.addressof(self.weights)
        self._state_shape = (cfg.n_heads, cfg.value_dim, cfg.key_dim)

    def _io(self, q, k, v, dt, beta, y, n_seqs, offsets, slots, positions, state, state_out):
        at, n, t, heads = self.index, q.shape[0], self.dtype, self.cfg.n_heads
        i32, f = self._torch.int32, self._torch.float32
        keys, values = (n, self.keys), (n, self.values)
        p_in = p_out = n_slots = 0
        if state is not None:
            n_slots = state.shape[0]
            p_in = p_out = _whole("the state", state, f, (n_slots, *self._state_shape), at)
            if state_out is not None:
                p_out = _whole("state_out", state_out, f, (n_slots, *self._state_shape), at)
        elif state_out is not None:
            raise ValueError("an output state needs the state that is read")
        return _DELTA_IO.pack(
            _rows("q", q, t, keys, at), _row_stride(q), _rows("k", k, t, keys, at), _row_stride(k),
            _rows("v", v, t, values, at), _row_stride(v), _rows("dt", dt, t, (n, heads), at), _row_stride(dt),
            _rows("beta", beta, t, (n, heads), at), _row_stride(beta), _rows("y", y, t, values, at), _row_stride(y),
            n, n_seqs, n_slots, 0 if offsets is None else _whole("offsets", offsets, i32, (n_seqs + 1,), at),
            0 if slots is None else _whole("slots", slots, i32, (n_seqs,), at),
            0 if positions is None else _whole("positions", positions, i32, (n_seqs,), at), p_in, p_out)

    def prompt(self, q, k, v, dt, beta, y, n_seqs, offsets=None, slots=None, positions=None, state=None, state_out=None,
               stream=None):
        """Whole or continued prompts: rows offsets[i] .. offsets[i + 1] - 1 (or equal shares of the rows) belong to
        sequence i. Writes y, and the state in place unless state_out is given. Returns y."""
        io = self._io(q, k, v, dt, beta, y, n_seqs, offsets, slots, positions, state, state_out)
        n = self._bytes(cdrge_delta_workspace_bytes, q.shape[0], n_seqs)
        call = self._lib.cdrge_delta_prompt
        self._run(lambda ws, s: _check(call(self._cfg, self._weights, io, 0 if ws is None else ws.data_ptr(), n, s),
                                       "cdrge_delta_prompt"), n, stream)
        return y

    def step(self, q, k, v, dt, beta, y, positions, state, slots=None, state_out=None, stream=None):
        """One token of each sequence, row i at place positions[i] of the sequence in slot slots[i] (negative: padding).
        Writes y, and the state in place unless state_out is given. Returns y."""
        n = q.shape[0]
        io = self._io(q, k, v, dt, beta, y, n, None, slots, positions, state, state_out)
        if n:
            call = self._lib.cdrge_delta_step
            self._run(lambda ws, s: _check(call(self._cfg, self._weights, io, s), "cdrge_delta_step"), 0, stream)
        return y


class TokenScores(_Operator):
    """Log probabilities of given tokens, entropy and top alternatives (cdrge_token_scores, cdrge_token_scores_grad)."""

    def __init__(self, cfg: cdrge_score_config, device=None):
        super().__init__(cfg, _gpu(device))

    def scores(self, logits, tokens, logprobs, entropy=None, top_ids=None, top_logprobs=None, stream=None):
        """Fills logprobs and, if given, entropy [rows], and top_ids (int32) and top_logprobs [rows, top_k], which are
        needed unless top_k is 0. tokens and logprobs may be None together. Returns logprobs."""
        n, cfg, at, f, i32 = logits.shape[0], self.cfg, self.index, self._torch.float32, self._torch.int32
        top = (n, cfg.top_k)
        args = (self._cfg, n, _rows("logits", logits, self.dtype, (n, cfg.vocab), at), _row_stride(logits),
                0 if tokens is None else _whole("tokens", tokens, i32, (n,), at),
                0 if logprobs is None else _whole("logprobs", logprobs, f, (n,), at),
                0 if entropy is None else _whole("entropy", entropy, f, (n,), at),
                0 if top_ids is None else _whole("top_ids", top_ids, i32, top, at),
                0 if top_logprobs is None else _whole("top_logprobs", top_logprobs, f, top, at))
        call = self._lib.cdrge_token_scores
        self._run(lambda ws, s: _check(call(*args, s), "cdrge_token_scores"), 0, stream)
        return logprobs

    def grad(self, logits, tokens, d_logprob, d_entropy, dlogits, stream=None):
        """dlogits[r] = d_logprob[r] d logprob_r / d logits[r] + d_entropy[r] d entropy_r / d logits[r]; either factor may
        be None. dlogits may be logits itself. Returns dlogits."""
        n, cfg, at, f = logits.shape[0], self.cfg, self.index, self._torch.float32
        args = (self._cfg, n, _rows("logits", logits, self.dtype, (n, cfg.vocab), at), _row_stride(logits),
                0 if tokens is None else _whole("tokens", tokens, self._torch.int32, (n,), at),
                0 if d_logprob is None else _whole("d_logprob", d_logprob, f, (n,), at),
                0 if d_entropy is None else _whole("d_entropy", d_entropy, f, (n,), at),
                _rows("dlogits", dlogits, self.dtype, (n, cfg.vocab), at), _row_stride(dlogits))
        call = self._lib.cdrge_token_scores_grad
        self._run(lambda ws, s: _check(call(*args, s), "cdrge_token_scores_grad"), 0, stream)
        return dlogits


class MxFormat(_Operator):
    """Rows in microscaled 4-bit floating point and back (cdrge_mx_quantize, cdrge_mx_dequantize)."""

    def __init__(self, cfg: cdrge_mx_config, device=None):
        super().__init__(cfg, _gpu(device))
        cdrge_mx_workspace_bytes(cfg, 0)
        self.blocks = (cfg.in_features + 31) // 32

    def empty(self, n_rows: int):
        """codes and scales for n_rows rows, not filled."""
        e, u8 = self._torch.empty, self._torch.uint8
        return e((n_rows, 16 * self.blocks), dtype=u8, device=self.device), e((n_rows, self.blocks), dtype=u8, device=self.device)

    def _args(self, x, codes, scales):
        n, at, u8 = x.shape[0], self.index, self._torch.uint8
        return (n, _rows("x", x, self.dtype, (n, self.cfg.in_features), at), _row_stride(x),
                _whole("codes", codes, u8, (n, 16 * self.blocks), at), _whole("scales", scales, u8, (n, self.blocks), at))

    def quantize(self, x, codes, scales, stream=None):
        """Fills codes and scales from the rows of x. Returns both."""
        n, p_x, x_stride, p_codes, p_scales = self._args(x, codes, scales)
        call = self._lib.cdrge_mx_quantize
        self._run(lambda ws, s: _check(call(self._cfg, n, p_x, x_stride, p_codes, p_scales, s), "cdrge_mx_quantize"), 0, stream)
        return codes, scales

    def dequantize(self, codes, scales, x, stream=None):
        """Fills the rows of x with the values that codes and scales stand for. Returns x."""
        n, p_x, x_stride, p_codes, p_scales = self._args(x, codes, scales)
        call = self._lib.cdrge_mx_dequantize
        self._run(lambda ws, s: _check(call(self._cfg, n, p_codes, p_scales, p_x, x_stride, s), "cdrge_mx_dequantize"), 0, stream)
        return x


class MxProjection(_Operator):
    """A projection by weights in microscaled 4-bit floating point (cdrge_mx_project): codes and scales as MxFormat makes
    them of the [out, in] weights, bias [out] in the operator's type or None."""

    def __init__(self, cfg: cdrge_mx_config, codes, scales, bias=None):
        super().__init__(cfg, _cuda_device(codes, "codes"))
        cdrge_mx_workspace_bytes(cfg, 0)
        O, blocks, at, u8 = cfg.out_features, (cfg.in_features + 31) // 32, self.index, self._torch.uint8
        self._held = (codes, scales, bias)
        self._weights = (_whole("codes", codes, u8, (O, 16 * blocks), at), _whole("scales", scales, u8, (O, blocks), at),
                         0 if bias is None else _whole("bias", bias, self.dtype, (O,), at))

    def project(self, x, y, stream=None):
        """y[r] = weight Q(x[r]) + bias, with Q the row in four bits. Returns y."""
        n, cfg, at, t = x.shape[0], self.cfg, self.index, self.dtype
        p_x = _rows("x", x, t, (n, cfg.in_features), at)
        p_y = _rows("y", y, t, (n, cfg.out_features), at)
        nbytes = self._bytes(cdrge_mx_workspace_bytes, n)
        call = self._lib.cdrge_mx_project
        x_stride, y_stride = _row_stride(x), _row_stride(y)
        self._run(lambda ws, s: _check(call(self._cfg, *self._weights, n, p_x, x_stride, p_y, y_stride,
                                            0 if ws is None else ws.data_ptr(), nbytes, s), "cdrge_mx_project"),
                  nbytes, stream)
        return y
