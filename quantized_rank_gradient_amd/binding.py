"""Python binding of libqgalore.so (ctypes): argument marshalling only.

Every step of the optimizer runs in the library's gfx950 kernels; this module checks dtypes,
shapes and devices of torch tensors, passes their device pointers and the current HIP stream
across the C ABI, and turns status codes into exceptions. There is no fallback: if the
library is missing, loading it raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgalore.so")

GROUP = 256

c_int64, c_uint32, c_int32, c_float, c_void_p, c_size_t, c_uint64 = (
    ctypes.c_int64, ctypes.c_uint32, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p,
    ctypes.c_size_t, ctypes.c_uint64)

STATUS = {0: "QG_OK", 1: "QG_ERR_NULL", 2: "QG_ERR_SHAPE", 3: "QG_ERR_ALIGN",
          4: "QG_ERR_WORKSPACE", 5: "QG_ERR_ARG", 6: "QG_ERR_HIP", 7: "QG_ERR_NO_DEVICE"}


class LayerDesc(ctypes.Structure):
    _fields_ = [("m", c_int64), ("n", c_int64), ("r", c_int64), ("layer_id", c_uint32),
                ("lr", c_float), ("beta1", c_float), ("beta2", c_float), ("eps", c_float),
                ("alpha", c_float), ("M_scale", c_void_p), ("V_scale", c_void_p),
                ("R_out", c_void_p), ("U_out", c_void_p), ("workspace", c_void_p),
                ("workspace_bytes", c_size_t), ("stream", c_void_p), ("p_format", c_int32),
                ("dequant_mode", c_int32)]


class Layer(ctypes.Structure):
    _fields_ = [("desc", LayerDesc), ("G", c_void_p), ("W_q", c_void_p), ("W_scale", c_void_p),
                ("P_q", c_void_p), ("P_scale", c_void_p), ("M_q", c_void_p), ("V_q", c_void_p)]


class Proj(ctypes.Structure):
    _fields_ = [("m", c_int64), ("r", c_int64), ("q", c_void_p), ("scale", c_void_p),
                ("format", c_int32)]


class LinearDesc(ctypes.Structure):
    _fields_ = [("T", c_int64), ("m", c_int64), ("n", c_int64), ("act", c_int32),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("stream", c_void_p)]


class NormDesc(ctypes.Structure):
    _fields_ = [("T", c_int64), ("n", c_int64), ("dtype", c_int32), ("center", c_int32),
                ("eps", c_float), ("workspace", c_void_p), ("workspace_bytes", c_size_t),
                ("stream", c_void_p)]


class MuonDesc(ctypes.Structure):
    _fields_ = [("m", c_int64), ("n", c_int64), ("lr", c_float), ("momentum", c_float),
                ("weight_decay", c_float), ("alpha", c_float), ("nesterov", c_int32),
                ("ns_steps", c_int32), ("ns_a", c_float), ("ns_b", c_float), ("ns_c", c_float),
                ("eps", c_float), ("workspace", c_void_p), ("workspace_bytes", c_size_t),
                ("stream", c_void_p)]


class MuonLayerDesc(ctypes.Structure):
    _fields_ = [("G", c_void_p), ("M", c_void_p), ("W_q", c_void_p), ("W_scale", c_void_p),
                ("layer_id", c_uint32)]


class Grad(ctypes.Structure):
    _fields_ = [("g", c_void_p), ("out", c_void_p), ("n", c_int64), ("dtype", c_int32)]


class ClipDesc(ctypes.Structure):
    _fields_ = [("kind", c_int32), ("zero_nonfinite", c_int32), ("max_norm", c_float),
                ("eps", c_float), ("workspace", c_void_p), ("workspace_bytes", c_size_t),
                ("stream", c_void_p)]


class ResnormDesc(ctypes.Structure):
    _fields_ = [("T", c_int64), ("n", c_int64), ("per", c_int64), ("dtype", c_int32),
                ("center", c_int32), ("gate_act", c_int32), ("alpha", c_float), ("eps", c_float),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("stream", c_void_p)]


class ResnormParams(ctypes.Structure):
    _fields_ = [(k, c_void_p) for k in ("gamma1", "beta1", "gamma2", "beta2", "rho", "z")]


class ResnormGrads(ctypes.Structure):
    _fields_ = [(k, c_void_p) for k in ("du", "dx", "dz", "drho", "dgamma1", "dbeta1", "dgamma2",
                                        "dbeta2")]


class Fp8Desc(ctypes.Structure):
    _fields_ = [("rows", c_int64), ("cols", c_int64), ("source", c_int32), ("format", c_int32),
                ("block", c_int32), ("stream", c_void_p)]


class Fp8MmDesc(ctypes.Structure):
    _fields_ = [("M", c_int64), ("N", c_int64), ("K", c_int64), ("a_format", c_int32),
                ("b_block", c_int32), ("out_dtype", c_int32), ("workspace", c_void_p),
                ("workspace_bytes", c_size_t), ("stream", c_void_p)]


class Fp8LinearDesc(ctypes.Structure):
    _fields_ = [("T", c_int64), ("m", c_int64), ("n", c_int64), ("format", c_int32),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("stream", c_void_p)]


# projection storage formats (qg_p_format)
P_FORMATS = {"int4": 0, "int8": 1, "bf16": 2}
# activations of a linear layer (qg_act)
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
# of a block's gate (qg_gate_act)
GATES = {"none": 0, "sigmoid": 1, "tanh": 2}
# norms of a set of gradients (qg_grad_kind)
GRAD_NORMS = {"l2": 0, "max": 1}
# 8-bit floating point formats (qg_fp8_format) and their torch types
FP8_FORMATS = {"e4m3": 0, "e5m2": 1}
FP8_DTYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_BLOCK = 128
# where an INT4 projection is dequantized (qg_dequant_mode)
DEQUANT_MODES = {"auto": 0, "inline": 1, "pass": 2}


class Sched(ctypes.Structure):
    _fields_ = [("delta", c_int64), ("next_refresh", c_int64), ("count", c_int64),
                ("gamma", c_float), ("last_cossim", c_float)]


EXPORTS = {
    "qgalore_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64]),
    "qgalore_layer_workspace_bytes": (c_size_t, [ctypes.POINTER(LayerDesc)]),
    "qgalore_step": (c_int32, [ctypes.POINTER(LayerDesc), c_void_p, c_void_p, c_void_p, c_void_p,
                               c_void_p, c_void_p, c_void_p, c_int64, c_uint64]),
    "qgalore_step_noalloc": (c_int32, [ctypes.POINTER(LayerDesc), c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_uint64]),
    "qgalore_plan_create": (c_int32, [ctypes.POINTER(Layer), c_int32, ctypes.POINTER(c_void_p)]),
    "qgalore_plan_workspace_bytes": (c_size_t, [c_void_p]),
    "qgalore_plan_step": (c_int32, [c_void_p, c_int64, c_uint64, c_void_p, c_size_t, c_void_p]),
    "qgalore_plan_destroy": (c_int32, [c_void_p]),
    "qgalore_plan_enable_timing": (c_int32, [c_void_p, c_int32]),
    "qgalore_plan_cache_proj": (c_int32, [c_void_p, c_int32]),
    "qgalore_plan_proj_changed": (c_int32, [c_void_p, c_int32]),
    "qgalore_plan_kernel_times": (c_int32, [c_void_p, ctypes.POINTER(c_float),
                                           ctypes.POINTER(c_int32)]),
    "qgalore_cossim_workspace_bytes": (c_size_t, [c_int64, c_int64]),
    "qgalore_cossim_async": (c_int32, [ctypes.POINTER(Proj), ctypes.POINTER(Proj), c_void_p,
                                       c_size_t, c_void_p, c_void_p]),
    "qgalore_cossim_batch_workspace_bytes": (c_size_t, [c_int64, c_int32]),
    "qgalore_cossim_batch": (c_int32, [ctypes.POINTER(Proj), ctypes.POINTER(Proj), c_int32,
                                       c_void_p, c_size_t, c_void_p, c_void_p]),
    "qgalore_cossim": (c_int32, [ctypes.POINTER(Proj), ctypes.POINTER(Proj), c_void_p, c_size_t,
                                 c_void_p, ctypes.POINTER(c_float)]),
    "qgalore_quantize_proj": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p, c_void_p]),
    "qgalore_quantize_proj_int8": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p,
                                             c_void_p]),
    "qgalore_refresh_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64, c_int32]),
    "qgalore_refresh_proj": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int32,
                                       c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_size_t, c_void_p]),
    "qgalore_int8_linear_fwd": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_int64,
                                          c_int64, c_void_p, c_void_p]),
    "qgalore_int8_linear_bwd_data": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_int64,
                                               c_int64, c_void_p, c_void_p]),
    "qgalore_linear_bwd_weight": (c_int32, [c_void_p, c_void_p, c_int64, c_int64, c_int64,
                                            c_void_p, c_void_p]),
    "qgalore_int8_linear_act_fwd_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64]),
    "qgalore_int8_linear_act_bwd_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64]),
    "qgalore_int8_linear_act_fwd": (c_int32, [ctypes.POINTER(LinearDesc)] + [c_void_p] * 7),
    "qgalore_int8_linear_act_bwd": (c_int32, [ctypes.POINTER(LinearDesc)] + [c_void_p] * 8),
    "qgalore_norm_bwd_workspace_bytes": (c_size_t, [c_int64, c_int64]),
    "qgalore_norm_fwd": (c_int32, [ctypes.POINTER(NormDesc)] + [c_void_p] * 6),
    "qgalore_norm_bwd": (c_int32, [ctypes.POINTER(NormDesc)] + [c_void_p] * 8),
    "qgalore_muon_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int32]),
    "qgalore_muon_step": (c_int32, [ctypes.POINTER(MuonDesc), ctypes.POINTER(MuonLayerDesc),
                                    c_int32, c_int64, c_uint64]),
    "qgalore_orthogonalize": (c_int32, [ctypes.POINTER(MuonDesc), ctypes.POINTER(c_void_p),
                                        ctypes.POINTER(c_void_p), c_int32]),
    "qgalore_grad_workspace_bytes": (c_size_t, []),
    "qgalore_grad_norm": (c_int32, [ctypes.POINTER(ClipDesc), ctypes.POINTER(Grad), c_int32,
                                    c_void_p, c_void_p]),
    "qgalore_grad_clip": (c_int32, [ctypes.POINTER(ClipDesc), ctypes.POINTER(Grad), c_int32,
                                    c_void_p, c_void_p]),
    "qgalore_resnorm_bwd_workspace_bytes": (c_size_t, [ctypes.POINTER(ResnormDesc)]),
    "qgalore_resnorm_fwd": (c_int32, [ctypes.POINTER(ResnormDesc), ctypes.POINTER(ResnormParams)]
                            + [c_void_p] * 5),
    "qgalore_resnorm_bwd": (c_int32, [ctypes.POINTER(ResnormDesc), ctypes.POINTER(ResnormParams)]
                            + [c_void_p] * 5 + [ctypes.POINTER(ResnormGrads)]),
    "qgalore_fp8_quantize": (c_int32, [ctypes.POINTER(Fp8Desc)] + [c_void_p] * 6),
    "qgalore_fp8_dequantize": (c_int32, [ctypes.POINTER(Fp8Desc)] + [c_void_p] * 3),
    "qgalore_fp8_matmul": (c_int32, [ctypes.POINTER(Fp8MmDesc)] + [c_void_p] * 5),
    "qgalore_fp8_matmul_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64]),
    "qgalore_fp8_linear_fwd_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64]),
    "qgalore_fp8_linear_bwd_workspace_bytes": (c_size_t, [c_int64, c_int64, c_int64]),
    "qgalore_fp8_linear_fwd": (c_int32, [ctypes.POINTER(Fp8LinearDesc)] + [c_void_p] * 4),
    "qgalore_fp8_linear_bwd": (c_int32, [ctypes.POINTER(Fp8LinearDesc)] + [c_void_p] * 7),
    "qgalore_sched_init": (c_int32, [ctypes.POINTER(Sched), c_int64, c_float]),
    "qgalore_sched_due": (c_int32, [ctypes.POINTER(Sched), c_int64]),
    "qgalore_sched_refresh": (c_int32, [ctypes.POINTER(Sched), c_int64, c_float,
                                        ctypes.POINTER(c_int32)]),
    "qgalore_mfma_probe": (c_int32, [c_void_p, c_int64, c_void_p, c_int32, c_int32, c_void_p]),
    "qgalore_status_str": (ctypes.c_char_p, [c_int32]),
    "qgalore_last_error": (ctypes.c_char_p, []),
    "qgalore_version": (ctypes.c_char_p, []),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libqgalore.so (built in-tree by build.py); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python quantized_rank_gradient_amd/build.py`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


class QgError(RuntimeError):
    def __init__(self, status: int, where: str):
        L = lib()
        text = L.qgalore_status_str(status).decode()
        if status == 6:
            text += ": " + L.qgalore_last_error().decode()
        super().__init__(f"{where}: {STATUS.get(status, status)} ({text})")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != 0:
        raise QgError(status, where)


def n_groups(numel: int) -> int:
    return -(-int(numel) // GROUP)


def _ptr(t, dtype, shape=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


@dataclasses.dataclass
class LayerTensors:
    """One linear layer's optimizer state on the GPU (see include/qgalore.h for layouts)."""
    layer_id: int
    G: torch.Tensor          # bf16 m x n
    Wq: torch.Tensor         # int8 m x n
    Ws: torch.Tensor         # fp32 [groups(m*n)]
    Pq: torch.Tensor         # int4: uint8 [ceil(m*r/2)]; int8: int8 m*r; bf16: bf16 m*r
    Ps: torch.Tensor         # fp32 [groups(m*r)] (None for bf16)
    Mq: torch.Tensor         # int8 r x n
    Ms: torch.Tensor         # fp32 [groups(r*n)]
    Vq: torch.Tensor         # int8 r x n
    Vs: torch.Tensor         # fp32 [groups(r*n)]
    r: int
    p_format: str = "int4"   # storage format of P: "int4", "int8" or "bf16"

    @property
    def m(self) -> int:
        return int(self.Wq.shape[0])

    @property
    def n(self) -> int:
        return int(self.Wq.shape[1])


def _proj_codes(Pq, m: int, r: int, fmt: str):
    """Pointer to a projection's codes (or bf16 values) in format fmt, checked."""
    if fmt == "int4":
        return _ptr(Pq, torch.uint8, ((m * r + 1) // 2,), "P_q")
    if fmt == "int8":
        return _ptr(Pq, torch.int8, (m * r,), "P_q")
    if fmt == "bf16":
        return _ptr(Pq.reshape(-1) if Pq is not None else None, torch.bfloat16, (m * r,), "P_q")
    raise ValueError(f"unknown projection format {fmt!r}")


def _fill_desc(d: LayerDesc, L: LayerTensors, hp: dict, R_out=None, U_out=None,
               dequant: str = "auto"):
    m, n, r = L.m, L.n, L.r
    d.m, d.n, d.r = m, n, r
    d.layer_id = L.layer_id
    d.lr, d.beta1, d.beta2 = hp.get("lr", 1e-3), hp.get("beta1", 0.9), hp.get("beta2", 0.999)
    d.eps, d.alpha = hp.get("eps", 1e-8), hp.get("alpha", 0.25)
    d.M_scale = _ptr(L.Ms, torch.float32, (n_groups(r * n),), "Ms")
    d.V_scale = _ptr(L.Vs, torch.float32, (n_groups(r * n),), "Vs")
    d.R_out = _ptr(R_out, torch.float32, (r, n), "R_out")
    d.U_out = _ptr(U_out, torch.float32, (m, n), "U_out")
    d.p_format = P_FORMATS[L.p_format]
    d.dequant_mode = DEQUANT_MODES[dequant]
    ptrs = dict(G=_ptr(L.G, torch.bfloat16, (m, n), "G"),
                W_q=_ptr(L.Wq, torch.int8, (m, n), "Wq"),
                W_scale=_ptr(L.Ws, torch.float32, (n_groups(m * n),), "Ws"),
                P_q=_proj_codes(L.Pq, m, r, L.p_format),
                P_scale=_ptr(L.Ps, torch.float32, (n_groups(m * r),), "Ps"),
                M_q=_ptr(L.Mq, torch.int8, (r, n), "Mq"),
                V_q=_ptr(L.Vq, torch.int8, (r, n), "Vq"))
    return ptrs


def workspace_bytes(m: int, n: int, r: int) -> int:
    return int(lib().qgalore_workspace_bytes(m, n, r))


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def step(L: LayerTensors, t: int, seed: int, hp: dict | None = None, workspace=None,
         R_out=None, U_out=None, stream=None, dequant: str = "auto") -> None:
    """One optimizer step of one layer (asynchronous on the current stream). `dequant`:
    where an INT4 projection is dequantized ("auto", "inline", "pass"; qg_dequant_mode)."""
    hp = hp or {}
    d = LayerDesc()
    ptrs = _fill_desc(d, L, hp, R_out, U_out, dequant)
    need = int(lib().qgalore_layer_workspace_bytes(ctypes.byref(d)))
    if workspace is None:
        workspace = alloc_workspace(need, L.Wq.device)
    d.workspace = _ptr(workspace, torch.uint8, None, "workspace")
    d.workspace_bytes = workspace.numel()
    d.stream = _stream(stream)
    _check(lib().qgalore_step(ctypes.byref(d), ptrs["G"], ptrs["W_q"], ptrs["W_scale"],
                              ptrs["P_q"], ptrs["P_scale"], ptrs["M_q"], ptrs["V_q"], int(t),
                              int(seed) & (2 ** 64 - 1)), "qgalore_step")


# size of the library's own scratch array used by step_noalloc (QG_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 64 << 20


def step_noalloc(L: LayerTensors, t: int, seed: int, hp: dict | None = None, R_out=None,
                 U_out=None, stream=None, dequant: str = "auto") -> None:
    """qgalore_step_noalloc: one layer's step with the library's fixed scratch array instead
    of a workspace (no device allocation anywhere on this path)."""
    hp = hp or {}
    d = LayerDesc()
    ptrs = _fill_desc(d, L, hp, R_out, U_out, dequant)
    d.stream = _stream(stream)
    _check(lib().qgalore_step_noalloc(ctypes.byref(d), ptrs["G"], ptrs["W_q"], ptrs["W_scale"],
                                      ptrs["P_q"], ptrs["P_scale"], ptrs["M_q"], ptrs["V_q"],
                                      int(t), int(seed) & (2 ** 64 - 1)), "qgalore_step_noalloc")


class Plan:
    """A grouped step over many layers: one launch per kernel for the whole set."""

    def __init__(self, layers: list, hp: dict | None = None, per_layer_hp: list | None = None,
                 R_out: list | None = None, U_out: list | None = None, dequant="auto"):
        """`dequant`: one qg_dequant_mode name for every layer, or a list with one per layer."""
        hp = hp or {}
        arr = (Layer * len(layers))()
        self._keep = list(layers) + list(R_out or []) + list(U_out or [])
        for k, L in enumerate(layers):
            h = per_layer_hp[k] if per_layer_hp else hp
            dq = dequant if isinstance(dequant, str) else dequant[k]
            ptrs = _fill_desc(arr[k].desc, L, h, R_out[k] if R_out else None,
                              U_out[k] if U_out else None, dq)
            for name, val in ptrs.items():
                setattr(arr[k], name, val)
        handle = c_void_p()
        _check(lib().qgalore_plan_create(arr, len(layers), ctypes.byref(handle)),
               "qgalore_plan_create")
        self._h = handle
        self.workspace_bytes = int(lib().qgalore_plan_workspace_bytes(handle))
        self.workspace = None

    def step(self, t: int, seed: int, workspace=None, stream=None) -> None:
        if workspace is None:
            if self.workspace is None:
                self.workspace = alloc_workspace(self.workspace_bytes, self._keep[0].Wq.device)
            workspace = self.workspace
        _check(lib().qgalore_plan_step(self._h, int(t), int(seed) & (2 ** 64 - 1),
                                       _ptr(workspace, torch.uint8, None, "workspace"),
                                       workspace.numel(), _stream(stream)), "qgalore_plan_step")

    def cache_proj(self, enable: bool = True) -> None:
        """Keep dequantized projections between steps (qgalore_plan_cache_proj); the caller
        then reports every projection it rewrites with proj_changed()."""
        _check(lib().qgalore_plan_cache_proj(self._h, 1 if enable else 0),
               "qgalore_plan_cache_proj")

    def proj_changed(self, layer: int) -> None:
        _check(lib().qgalore_plan_proj_changed(self._h, int(layer)), "qgalore_plan_proj_changed")

    def enable_timing(self, max_steps: int) -> None:
        _check(lib().qgalore_plan_enable_timing(self._h, int(max_steps)),
               "qgalore_plan_enable_timing")

    def kernel_times(self):
        """Mean (dequant, projection, Adam, back-projection) kernel milliseconds over the
        recorded steps, and the number of steps recorded."""
        out = (c_float * 4)()
        steps = c_int32(0)
        _check(lib().qgalore_plan_kernel_times(self._h, out, ctypes.byref(steps)),
               "qgalore_plan_kernel_times")
        return [float(x) for x in out], int(steps.value)

    def close(self) -> None:
        if self._h:
            _check(lib().qgalore_plan_destroy(self._h), "qgalore_plan_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _proj(Pq, Ps, m, r, fmt="int4") -> Proj:
    p = Proj()
    p.m, p.r = m, r
    p.q = _proj_codes(Pq, m, r, fmt)
    p.scale = _ptr(Ps, torch.float32, (n_groups(m * r),), "P_scale")
    p.format = P_FORMATS[fmt]
    return p


def cossim_workspace_bytes(m: int, r: int) -> int:
    return int(lib().qgalore_cossim_workspace_bytes(m, r))


def cossim_async(Pq_new, Ps_new, Pq_old, Ps_old, m: int, r: int, out: torch.Tensor,
                 workspace=None, stream=None, fmt: str = "int4") -> None:
    """CosSim of two stored projections into out[0] (device fp32), asynchronously."""
    a, b = _proj(Pq_new, Ps_new, m, r, fmt), _proj(Pq_old, Ps_old, m, r, fmt)
    if workspace is None:
        workspace = alloc_workspace(cossim_workspace_bytes(m, r), Pq_new.device)
    _check(lib().qgalore_cossim_async(ctypes.byref(a), ctypes.byref(b),
                                      _ptr(workspace, torch.uint8, None, "workspace"),
                                      workspace.numel(), _stream(stream),
                                      _ptr(out, torch.float32, None, "out")),
           "qgalore_cossim_async")


def cossim_batch_workspace_bytes(r: int, count: int) -> int:
    return int(lib().qgalore_cossim_batch_workspace_bytes(r, count))


def cossim_batch(pairs, r: int, out: torch.Tensor, workspace=None, stream=None) -> None:
    """pairs: list of (Pq_new, Ps_new, Pq_old, Ps_old, m[, format]); out[k] (device fp32)
    receives CosSim of pair k, asynchronously. All pairs share the rank r."""
    n = len(pairs)
    A = (Proj * n)()
    Bp = (Proj * n)()
    for k, pr in enumerate(pairs):
        qn, sn, qo, so, m = pr[:5]
        fmt = pr[5] if len(pr) > 5 else "int4"
        A[k] = _proj(qn, sn, m, r, fmt)
        Bp[k] = _proj(qo, so, m, r, fmt)
    if workspace is None:
        workspace = alloc_workspace(cossim_batch_workspace_bytes(r, n), pairs[0][0].device)
    _check(lib().qgalore_cossim_batch(A, Bp, n, _ptr(workspace, torch.uint8, None, "workspace"),
                                      workspace.numel(), _stream(stream),
                                      _ptr(out, torch.float32, None, "out")),
           "qgalore_cossim_batch")


def cossim(Pq_new, Ps_new, Pq_old, Ps_old, m: int, r: int, workspace=None, stream=None,
           fmt: str = "int4") -> float:
    a, b = _proj(Pq_new, Ps_new, m, r, fmt), _proj(Pq_old, Ps_old, m, r, fmt)
    if workspace is None:
        workspace = alloc_workspace(cossim_workspace_bytes(m, r), Pq_new.device)
    out = c_float()
    _check(lib().qgalore_cossim(ctypes.byref(a), ctypes.byref(b),
                                _ptr(workspace, torch.uint8, None, "workspace"),
                                workspace.numel(), _stream(stream), ctypes.byref(out)),
           "qgalore_cossim")
    return float(out.value)


def quantize_proj(P: torch.Tensor, stream=None, fmt: str = "int4"):
    """Group quantization of an fp32 m x r projection -> (P_q, P_scale): INT4 (uint8 packed
    codes), INT8 (int8 codes), or for "bf16" the bf16 values (a cast; no scales)."""
    m, r = P.shape
    src = _ptr(P, torch.float32, (m, r), "P")
    if fmt == "bf16":
        return P.to(torch.bfloat16).reshape(-1).contiguous(), None
    Ps = torch.empty(n_groups(m * r), dtype=torch.float32, device=P.device)
    if fmt == "int8":
        Pq = torch.empty(m * r, dtype=torch.int8, device=P.device)
        _check(lib().qgalore_quantize_proj_int8(src, m, r, Pq.data_ptr(), Ps.data_ptr(),
                                                _stream(stream)), "qgalore_quantize_proj_int8")
        return Pq, Ps
    if fmt != "int4":
        raise ValueError(f"unknown projection format {fmt!r}")
    Pq = torch.empty((m * r + 1) // 2, dtype=torch.uint8, device=P.device)
    _check(lib().qgalore_quantize_proj(src, m, r, Pq.data_ptr(), Ps.data_ptr(), _stream(stream)),
           "qgalore_quantize_proj")
    return Pq, Ps


def mfma_probe(operands: torch.Tensor, out: torch.Tensor, grid: int, iters: int,
               stream=None) -> float:
    """Launch the MFMA calibration kernel on bf16 `operands` (see qgalore_mfma_probe);
    returns the flops the launch performs."""
    if operands.dtype != torch.bfloat16 or not operands.is_contiguous():
        raise TypeError("operands must be a contiguous bf16 tensor")
    if out.dtype != torch.float32 or out.numel() < grid * 256:
        raise ValueError("out must hold grid * 256 float32 values")
    _check(lib().qgalore_mfma_probe(operands.data_ptr(), operands.numel(), out.data_ptr(), grid,
                                    iters, _stream(stream)), "qgalore_mfma_probe")
    return float(grid) * 4 * iters * 16 * 32768


def refresh_workspace_bytes(m: int, n: int, r: int, oversample: int = 8) -> int:
    return int(lib().qgalore_refresh_workspace_bytes(m, n, r, oversample))


def refresh_proj(G: torch.Tensor, r: int, Omega: torch.Tensor, power_iters: int = 2,
                 P_out=None, sigma_out=None, workspace=None, stream=None):
    """New projection of the gradient G (bf16 m x n): the r leading left singular vectors by
    the library's randomized range finder with the caller's sketch Omega (bf16 n x k,
    k = r + oversample), quantized to INT4 -> (P_q, P_scale). P_out (fp32 m x r) and
    sigma_out (fp32 r) optionally receive P before quantization and the singular values."""
    m, n = G.shape
    k = Omega.shape[1]
    g = _ptr(G, torch.bfloat16, (m, n), "G")
    om = _ptr(Omega, torch.bfloat16, (n, k), "Omega")
    Pq = torch.empty((m * r + 1) // 2, dtype=torch.uint8, device=G.device)
    Ps = torch.empty(n_groups(m * r), dtype=torch.float32, device=G.device)
    if workspace is None:
        nbytes = refresh_workspace_bytes(m, n, r, k - r)
        if nbytes == 0:
            raise ValueError(f"refresh of a {m} x {n} gradient at rank {r} with sketch width "
                             f"{k} is not supported")
        workspace = alloc_workspace(nbytes, G.device)
    _check(lib().qgalore_refresh_proj(
        g, m, n, r, om, k - r, int(power_iters), Pq.data_ptr(), Ps.data_ptr(),
        _ptr(P_out, torch.float32, (m, r), "P_out"), _ptr(sigma_out, torch.float32, (r,), "sigma_out"),
        _ptr(workspace, torch.uint8, None, "workspace"), workspace.numel(), _stream(stream)),
        "qgalore_refresh_proj")
    return Pq, Ps


def int8_linear_fwd(X: torch.Tensor, Wq: torch.Tensor, Ws: torch.Tensor, out=None,
                    stream=None) -> torch.Tensor:
    """Y = X W~^T (bf16 T x m) for the INT8 weight Wq (m x n) with group scales Ws."""
    T, n = X.shape
    m = Wq.shape[0]
    Y = out if out is not None else torch.empty((T, m), dtype=torch.bfloat16, device=X.device)
    _check(lib().qgalore_int8_linear_fwd(
        _ptr(X, torch.bfloat16, (T, n), "X"), _ptr(Wq, torch.int8, (m, n), "Wq"),
        _ptr(Ws, torch.float32, (n_groups(m * n),), "Ws"), T, m, n,
        _ptr(Y, torch.bfloat16, (T, m), "Y"), _stream(stream)), "qgalore_int8_linear_fwd")
    return Y


def int8_linear_bwd_data(dY: torch.Tensor, Wq: torch.Tensor, Ws: torch.Tensor, out=None,
                         stream=None) -> torch.Tensor:
    """dX = dY W~ (bf16 T x n)."""
    T, m = dY.shape
    n = Wq.shape[1]
    dX = out if out is not None else torch.empty((T, n), dtype=torch.bfloat16, device=dY.device)
    _check(lib().qgalore_int8_linear_bwd_data(
        _ptr(dY, torch.bfloat16, (T, m), "dY"), _ptr(Wq, torch.int8, (m, n), "Wq"),
        _ptr(Ws, torch.float32, (n_groups(m * n),), "Ws"), T, m, n,
        _ptr(dX, torch.bfloat16, (T, n), "dX"), _stream(stream)), "qgalore_int8_linear_bwd_data")
    return dX


def linear_bwd_weight(dY: torch.Tensor, X: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """G = dY^T X (bf16 m x n): the weight gradient the optimizer step takes."""
    T, m = dY.shape
    n = X.shape[1]
    G = out if out is not None else torch.empty((m, n), dtype=torch.bfloat16, device=dY.device)
    _check(lib().qgalore_linear_bwd_weight(
        _ptr(dY, torch.bfloat16, (T, m), "dY"), _ptr(X, torch.bfloat16, (T, n), "X"), T, m, n,
        _ptr(G, torch.bfloat16, (m, n), "G"), _stream(stream)), "qgalore_linear_bwd_weight")
    return G


# the raw handle of a device's current stream, without a Stream object where torch has the call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


class _on:
    """The one device of `tensors` as the current one and `stream` (None: that device's current
    stream) as its current stream, so that memory taken inside belongs to the stream that the
    kernels use; yields the stream's handle. Refuses tensors of different devices and a stream
    of another device."""
    __slots__ = ("index", "stream", "stack")

    def __init__(self, tensors, stream):
        index = None
        try:
            for t in tensors:
                if t is not None:
                    i = t.get_device()   # -1: not on a GPU
                    if i != index:
                        if index is not None or i < 0:
                            raise ValueError("tensors must be on one GPU (got "
                                             + ", ".join(sorted({str(t.device) for t in tensors
                                                                 if t is not None})) + ")")
                        index = i
        except AttributeError:
            raise TypeError(f"a torch.Tensor is wanted (got {type(t).__name__})") from None
        if index is None:
            raise ValueError("no tensor given")
        if stream is not None and stream.device.index != index:
            raise ValueError(f"stream of {stream.device}, tensors on cuda:{index}")
        self.index, self.stream, self.stack = index, stream, None

    def __enter__(self):
        if self.stream is None and self.index == torch.cuda.current_device():
            return _raw_stream(self.index)
        self.stack = contextlib.ExitStack()
        self.stack.enter_context(torch.cuda.device(self.index))
        if self.stream is None:
            return _raw_stream(self.index)
        self.stack.enter_context(torch.cuda.stream(self.stream))
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.stack is not None:
            self.stack.close()
        return False


def _arg(t, dtype, shape, name):
    """_ptr for a tensor whose device _on has checked (one look at the usual case)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    return _ptr(t, dtype, shape, name)


def _scratch(d, workspace, nbytes: int, device):
    """Points descriptor d at the workspace (allocated where there is none) and returns it. The caller
    holds it until the library's call has returned: freed before, its memory could go to a tensor of
    another thread on the same stream while this call's kernels are not launched yet."""
    if workspace is None:
        if nbytes == 0:
            return None
        workspace = alloc_workspace(nbytes, device)
    d.workspace = _ptr(workspace, torch.uint8, None, "workspace")
    d.workspace_bytes = workspace.numel()
    return workspace


def _act(act: str) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def int8_linear_act_fwd(X: torch.Tensor, Wq: torch.Tensor, Ws: torch.Tensor, bias=None,
                        residual=None, act: str = "none", keep_z: bool = False, out=None,
                        z_out=None, workspace=None, stream=None):
    """Y = act(X W~^T + bias) + residual (bf16 T x m) for the INT8 weight Wq (m x n) with group
    scales Ws; with keep_z (or z_out) also Z = X W~^T + bias in bf16: returns Y, or (Y, Z)."""
    T, n = X.shape
    m = Wq.shape[0]
    d = LinearDesc(T, m, n, _act(act))
    with _on((X, Wq, Ws, bias, residual, out, z_out, workspace), stream) as d.stream:
        args = (_arg(X, torch.bfloat16, (T, n), "X"),)
        Y = out if out is not None else X.new_empty((T, m))
        Z = z_out if z_out is not None or not keep_z else X.new_empty((T, m))
        args += (_arg(Wq, torch.int8, (m, n), "Wq"),
                _arg(Ws, torch.float32, (n_groups(m * n),), "Ws"),
                _arg(bias, torch.float32, (m,), "bias"),
                _arg(residual, torch.bfloat16, (T, m), "residual"),
                _arg(Y, torch.bfloat16, (T, m), "out"), _arg(Z, torch.bfloat16, (T, m), "z_out"))
        workspace = _scratch(
            d, workspace, lib().qgalore_int8_linear_act_fwd_workspace_bytes(T, m, n), X.device)
        _check(lib().qgalore_int8_linear_act_fwd(ctypes.byref(d), *args),
               "qgalore_int8_linear_act_fwd")
    return Y if Z is None else (Y, Z)


def int8_linear_act_bwd(dY: torch.Tensor, X=None, Wq=None, Ws=None, Z=None, act: str = "none",
                        bias: bool = False, dX=None, G=None, dbias=None, need_dX: bool = True,
                        need_G: bool = True, workspace=None, stream=None):
    """Gradients of int8_linear_act_fwd: (dX, G, dbias), with None for what is not asked for (dbias
    comes with bias=True). Z is the forward pass's, needed with an activation; X is needed for G,
    Wq and Ws for dX. The residual's gradient is dY."""
    T, m = dY.shape
    need_dX, need_G = need_dX or dX is not None, need_G or G is not None
    if need_G and X is None:
        raise ValueError("G needs X")
    if need_dX and (Wq is None or Ws is None):
        raise ValueError("dX needs Wq and Ws")
    if X is None and Wq is None:
        n = 8   # dbias alone: any width
    else:
        n = (X if X is not None else Wq).shape[1]
    d = LinearDesc(T, m, n, _act(act))
    with _on((dY, X, Wq, Ws, Z, dX, G, dbias, workspace), stream) as d.stream:
        args = (_arg(dY, torch.bfloat16, (T, m), "dY"),)
        if need_dX and dX is None:
            dX = dY.new_empty((T, n))
        if need_G and G is None:
            G = dY.new_empty((m, n))
        if bias and dbias is None:
            dbias = dY.new_empty((m,), dtype=torch.float32)
        args += (_arg(Z, torch.bfloat16, (T, m), "Z"),
                _arg(X, torch.bfloat16, (T, n), "X"), _arg(Wq, torch.int8, (m, n), "Wq"),
                _arg(Ws, torch.float32, (n_groups(m * n),), "Ws"),
                _arg(dX, torch.bfloat16, (T, n), "dX"), _arg(G, torch.bfloat16, (m, n), "G"),
                _arg(dbias, torch.float32, (m,), "dbias"))
        workspace = _scratch(
            d, workspace, lib().qgalore_int8_linear_act_bwd_workspace_bytes(T, m, n), dY.device)
        _check(lib().qgalore_int8_linear_act_bwd(ctypes.byref(d), *args),
               "qgalore_int8_linear_act_bwd")
    return dX, G, dbias


def _norm_desc(X: torch.Tensor, eps: float, center: bool) -> NormDesc:
    if X.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"the norm takes bf16 or fp32 (got {X.dtype})")
    T, n = X.shape
    return NormDesc(T, n, 0 if X.dtype == torch.bfloat16 else 1, 1 if center else 0, eps)


def norm_fwd(X: torch.Tensor, gamma: torch.Tensor, beta=None, eps: float = 1e-5,
             center: bool = True, out=None, mean=None, rstd=None, stream=None):
    """Layer norm of the rows of X (T x n, bf16 or fp32), or with center=False the norm by the root
    mean square: (Y, mean, rstd), mean None without center."""
    d = _norm_desc(X, eps, center)
    T, n = X.shape
    with _on((X, gamma, beta, out, mean, rstd), stream) as d.stream:
        args = (_arg(X, X.dtype, (T, n), "X"), _arg(gamma, torch.float32, (n,), "gamma"))
        Y = out if out is not None else torch.empty_like(X)
        if center and mean is None:
            mean = gamma.new_empty((T,))
        if rstd is None:
            rstd = torch.empty_like(mean) if center else gamma.new_empty((T,))
        _check(lib().qgalore_norm_fwd(
            ctypes.byref(d), *args, _arg(beta, torch.float32, (n,), "beta"),
            _arg(Y, X.dtype, (T, n), "out"), _arg(mean, torch.float32, (T,), "mean"),
            _arg(rstd, torch.float32, (T,), "rstd")), "qgalore_norm_fwd")
    return Y, mean, rstd


def norm_bwd(dY: torch.Tensor, X: torch.Tensor, gamma: torch.Tensor, mean, rstd: torch.Tensor,
             center: bool = True, need_dbeta: bool | None = None, dX=None, dgamma=None, dbeta=None,
             workspace=None, stream=None):
    """Gradients of norm_fwd: (dX, dgamma, dbeta), dbeta by default with center only."""
    d = _norm_desc(X, 0.0, center)
    T, n = X.shape
    with _on((dY, X, gamma, mean, rstd, dX, dgamma, dbeta, workspace), stream) as d.stream:
        args = (_arg(dY, X.dtype, (T, n), "dY"), _arg(X, X.dtype, (T, n), "X"),
                _arg(gamma, torch.float32, (n,), "gamma"))
        if dX is None:
            dX = torch.empty_like(X)
        if dgamma is None:
            dgamma = torch.empty_like(gamma)
        if dbeta is None and (center if need_dbeta is None else need_dbeta):
            dbeta = torch.empty_like(gamma)
        args += (_arg(mean, torch.float32, (T,), "mean"), _arg(rstd, torch.float32, (T,), "rstd"),
                _arg(dX, X.dtype, (T, n), "dX"), _arg(dgamma, torch.float32, (n,), "dgamma"),
                _arg(dbeta, torch.float32, (n,), "dbeta"))
        workspace = _scratch(d, workspace, lib().qgalore_norm_bwd_workspace_bytes(T, n), X.device)
        _check(lib().qgalore_norm_bwd(ctypes.byref(d), *args), "qgalore_norm_bwd")
    return dX, dgamma, dbeta


def _gate(act: str) -> int:
    if act not in GATES:
        raise ValueError(f"unknown gate {act!r}: one of {', '.join(GATES)}")
    return GATES[act]


def _resnorm(X, post, pre, gate, gate_act, per, rho, alpha, eps, center):
    """The descriptor and the tensors of the parameters of residual_norm_fwd and _bwd."""
    if X.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"the norms take bf16 or fp32 (got {X.dtype})")
    T, n = X.shape
    if gate is not None and per < 1:
        raise ValueError(f"per must be at least 1 (got {per})")
    d = ResnormDesc(T, n, per if gate is not None else 1, 0 if X.dtype == torch.bfloat16 else 1,
                    1 if center else 0, _gate(gate_act), alpha, eps)
    g1, b1 = post if post is not None else (None, None)
    g2, b2 = pre if pre is not None else (None, None)
    return d, (g1, b1, g2, b2, rho, gate)


def _resnorm_params(d, vecs, dtype) -> ResnormParams:
    n, f32 = (d.n,), torch.float32
    g1, b1, g2, b2, rho, gate = vecs
    return ResnormParams(
        None if g1 is None else _arg(g1, f32, n, "gamma1"),
        None if b1 is None else _arg(b1, f32, n, "beta1"),
        None if g2 is None else _arg(g2, f32, n, "gamma2"),
        None if b2 is None else _arg(b2, f32, n, "beta2"),
        None if rho is None else _arg(rho, f32, n, "rho"),
        None if gate is None else _arg(gate, dtype, (-(-d.T // d.per), d.n), "gate"))


def residual_norm_fwd(U: torch.Tensor, X: torch.Tensor, post=None, pre=None, gate=None,
                      gate_act: str = "none", per: int = 1, rho=None, alpha: float = 1.0,
                      eps: float = 1e-5, center: bool = False, out=None, y_out=None, stats=None,
                      stream=None):
    """Behind a block and before the next: p = norm(U) by post = (gamma, beta or None), or U itself
    without; H = alpha X + rho act(gate) p; Y = norm(H) by pre = (gamma, beta or None), or None. U and
    X are T x n, bf16 or fp32; rho fp32 n; gate has a row for every `per` tokens, gate_act none,
    sigmoid or tanh. center: layer norms, else by the root mean square. Returns (H, Y, stats), stats
    (fp32 4 x T) for the backward pass."""
    d, vecs = _resnorm(X, post, pre, gate, gate_act, per, rho, alpha, eps, center)
    T, n = X.shape
    with _on((U, X, *vecs, out, y_out, stats), stream) as d.stream:
        p = _resnorm_params(d, vecs, X.dtype)
        args = (_arg(U, X.dtype, X.shape, "U"), _arg(X, X.dtype, X.shape, "X"))
        H = out if out is not None else torch.empty_like(X)
        Y = None
        if pre is not None:
            Y = y_out if y_out is not None else torch.empty_like(X)
        elif y_out is not None:
            raise ValueError("y_out needs pre")
        if stats is None:
            stats = X.new_empty((4, T), dtype=torch.float32)
        _check(lib().qgalore_resnorm_fwd(
            ctypes.byref(d), ctypes.byref(p), *args, _arg(H, X.dtype, X.shape, "out"),
            None if Y is None else _arg(Y, X.dtype, X.shape, "y_out"),
            _arg(stats, torch.float32, (4, T), "stats")), "qgalore_resnorm_fwd")
    return H, Y, stats


@dataclasses.dataclass
class ResidualNormGrads:
    """Gradients of residual_norm_fwd; None for what its call does not have."""
    dU: torch.Tensor
    dX: torch.Tensor
    dgate: torch.Tensor | None
    drho: torch.Tensor | None
    dpost: tuple             # (dgamma, dbeta)
    dpre: tuple              # (dgamma, dbeta)


def residual_norm_bwd(dH, dY, U, H, stats: torch.Tensor, post=None, pre=None,
                      gate=None, gate_act: str = "none", per: int = 1, rho=None,
                      alpha: float = 1.0, center: bool = False, dU=None, dX=None, dgate=None,
                      workspace=None, stream=None, drho=None, dpost=None,
                      dpre=None) -> ResidualNormGrads:
    """Gradients of residual_norm_fwd, whose parameters are given again, from dH (None: none but
    through Y) and dY (with pre). U may be None without post, gate and rho, whose gradients alone need
    it. A beta's gradient comes where the beta is given. dU, dX, dgate, drho and the pairs dpost and
    dpre (dgamma, dbeta; either may be None) are tensors to write to."""
    if U is None and not (post is None and gate is None and rho is None):
        raise ValueError("post, gate and rho need U")
    like = U if U is not None else dH if dH is not None else dY
    if like is None:
        raise ValueError("none of dH, dY and U")
    d, vecs = _resnorm(like, post, pre, gate, gate_act, per, rho, alpha, 0.0, center)
    g1, b1, g2, b2 = vecs[:4]
    T, n = like.shape
    if pre is not None and (dY is None or H is None):
        raise ValueError("pre needs dY and H")
    if gate is None and dgate is not None:
        raise ValueError("dgate needs gate")
    into = ()   # where the parameters' gradients go
    if drho is not None or dpost is not None or dpre is not None:
        for to, of, name in ((drho, rho, "rho"), (dpost, post, "post"), (dpre, pre, "pre")):
            if to is not None and of is None:
                raise ValueError(f"d{name} needs {name}")
        into = (drho, *(dpost or (None, None)), *(dpre or (None, None)))
    with _on((U, dH, dY, H, stats, *vecs, dU, dX, dgate, *into, workspace),
             stream) as d.stream:
        p = _resnorm_params(d, vecs, like.dtype)

        def rows(t, name):
            return _arg(t, like.dtype, like.shape, name)
        args = (rows(dH, "dH"), rows(dY if pre is not None else None, "dY"), rows(U, "U"),
                rows(H if pre is not None else None, "H"),
                _arg(stats, torch.float32, (4, T), "stats"))
        dU = torch.empty_like(like) if dU is None else dU
        dX = torch.empty_like(like) if dX is None else dX
        if gate is not None and dgate is None:
            dgate = torch.empty_like(gate)
        vec = (rho, g1, b1, g2, b2)
        if into:
            for v, name in zip(into, ("drho", "dgamma1", "dbeta1", "dgamma2", "dbeta2")):
                _arg(v, torch.float32, (n,), name)
            vec = [torch.empty_like(v) if to is None and v is not None else to
                   for to, v in zip(into, vec)]
        else:
            vec = [torch.empty_like(v) if v is not None else None for v in vec]
        g = ResnormGrads(rows(dU, "dU"), rows(dX, "dX"),
                         _arg(dgate, like.dtype, (-(-T // d.per), n), "dgate"),
                         *(v.data_ptr() if v is not None else None for v in vec))
        workspace = _scratch(d, workspace,
                             lib().qgalore_resnorm_bwd_workspace_bytes(ctypes.byref(d)), like.device)
        _check(lib().qgalore_resnorm_bwd(ctypes.byref(d), ctypes.byref(p), *args, ctypes.byref(g)),
               "qgalore_resnorm_bwd")
    return ResidualNormGrads(dU, dX, dgate, vec[0], (vec[1], vec[2]), (vec[3], vec[4]))


def _fp8_format(fmt: str) -> int:
    if fmt not in FP8_FORMATS:
        raise ValueError(f"unknown FP8 format {fmt!r}: one of {', '.join(FP8_FORMATS)}")
    return FP8_FORMATS[fmt]


def _fp8_of(Q: torch.Tensor, name: str) -> str:
    for fmt, dt in FP8_DTYPES.items():
        if Q.dtype is dt:
            return fmt
    raise TypeError(f"{name} must be an FP8 tensor (got {Q.dtype})")


def fp8_pitch(cols: int) -> int:
    """Codes in a row of a quantized matrix: cols rounded up to 16."""
    return -(-int(cols) // 16) * 16


def _fp8_blocks(n: int) -> int:
    return -(-int(n) // FP8_BLOCK)


def fp8_shapes(rows: int, cols: int, block: bool = False):
    """Shapes of the codes and the scales of a rows x cols matrix."""
    return (rows, fp8_pitch(cols)), (_fp8_blocks(cols), _fp8_blocks(rows) if block else rows)


def fp8_quantize(X: torch.Tensor, scales=None, fmt: str = "e4m3", block: bool = False,
                 rows: bool = True, columns: bool = False, out=None, stream=None):
    """FP8 codes of X (bf16, fp32, or INT8 weights with their `scales`) and their fp32 scales, one for
    each run of 128 values or, with block, each block of 128 x 128. rows: (Q, S), runs along X's rows;
    columns: (Qt, St) of the transpose, runs along X's columns; both: (Q, S, Qt, St). See fp8_shapes.
    `out` gives the same tensors to write to."""
    source = {torch.bfloat16: 0, torch.float32: 1, torch.int8: 2}.get(X.dtype)
    if source is None:
        raise TypeError(f"bf16, fp32 or INT8 weights are quantized (got {X.dtype})")
    if (source == 2) != (scales is not None):
        raise ValueError("INT8 weights come with their scales, other values without")
    if not rows and not columns:
        raise ValueError("neither rows nor columns")
    m, n = X.shape
    d = Fp8Desc(m, n, source, _fp8_format(fmt), 1 if block else 0)
    kind, f32 = FP8_DTYPES[fmt], torch.float32
    with _on((X, scales, *out) if out is not None else (X, scales), stream) as d.stream:
        src = _arg(X, X.dtype, (m, n), "X")
        ws = _arg(scales, f32, (n_groups(m * n),), "scales")
        shapes = (fp8_shapes(m, n, block) if rows else ()) + \
            (fp8_shapes(n, m, block) if columns else ())
        if out is None:
            out = [X.new_empty(s, dtype=f32 if i & 1 else kind) for i, s in enumerate(shapes)]
            ptrs = [t.data_ptr() for t in out]
        else:
            if len(out) != len(shapes):
                raise ValueError(f"{len(shapes)} outputs are wanted (got {len(out)})")
            ptrs = [_arg(t, f32 if i & 1 else kind, s, "out")
                    for i, (t, s) in enumerate(zip(out, shapes))]
        if len(ptrs) < 4:
            ptrs = (*ptrs, None, None) if rows else (None, None, *ptrs)
        _check(lib().qgalore_fp8_quantize(ctypes.byref(d), src, ws, *ptrs), "qgalore_fp8_quantize")
    return tuple(out)


def fp8_dequantize(Q: torch.Tensor, S: torch.Tensor, cols: int, block: bool = False,
                   dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """The values of a quantized matrix of `cols` columns, in bf16 or fp32."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"values are bf16 or fp32 (got {dtype})")
    m = Q.shape[0]
    d = Fp8Desc(m, cols, 0 if dtype == torch.bfloat16 else 1, FP8_FORMATS[_fp8_of(Q, "Q")],
                1 if block else 0)
    q, s = fp8_shapes(m, cols, block)
    with _on((Q, S, out), stream) as d.stream:
        args = (_arg(Q, Q.dtype, q, "Q"), _arg(S, torch.float32, s, "S"))
        if out is None:
            out = Q.new_empty((m, cols), dtype=dtype)
        _check(lib().qgalore_fp8_dequantize(ctypes.byref(d), *args,
                                            _arg(out, dtype, (m, cols), "out")),
               "qgalore_fp8_dequantize")
    return out


def fp8_matmul(A: torch.Tensor, SA: torch.Tensor, Bq: torch.Tensor, SB: torch.Tensor, K: int,
               dtype=torch.bfloat16, out=None, workspace=None, stream=None) -> torch.Tensor:
    """A B^T (M x N, bf16 or fp32) of quantized matrices with K values in a row: A in either format
    with runs, Bq in e4m3 with runs or blocks, as SB's shape says. workspace: at least
    qgalore_fp8_matmul_workspace_bytes (None: allocated)."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"the product is bf16 or fp32 (got {dtype})")
    M, N = A.shape[0], Bq.shape[0]
    fmt = FP8_FORMATS[_fp8_of(A, "A")]
    block = tuple(SB.shape) == fp8_shapes(N, K, True)[1]
    d = Fp8MmDesc(M, N, K, fmt, 1 if block else 0, 0 if dtype == torch.bfloat16 else 1)
    (qa, sa), (qb, sb) = fp8_shapes(M, K), fp8_shapes(N, K, block)
    with _on((A, SA, Bq, SB, out, workspace), stream) as d.stream:
        args = (_arg(A, A.dtype, qa, "A"), _arg(SA, torch.float32, sa, "SA"),
                _arg(Bq, torch.float8_e4m3fn, qb, "Bq"), _arg(SB, torch.float32, sb, "SB"))
        if out is None:
            out = A.new_empty((M, N), dtype=dtype)
        workspace = _scratch(d, workspace, lib().qgalore_fp8_matmul_workspace_bytes(M, N, K), A.device)
        _check(lib().qgalore_fp8_matmul(ctypes.byref(d), *args, _arg(out, dtype, (M, N), "out")),
               "qgalore_fp8_matmul")
    return out


def fp8_linear_fwd(X: torch.Tensor, W: torch.Tensor, S: torch.Tensor, out=None, workspace=None,
                   stream=None) -> torch.Tensor:
    """Y = q(X) W^T (bf16 T x m) for an FP8 weight W (m outputs, e4m3) with block scales S, as
    fp8_quantize(..., block=True) gives them; X (bf16 T x n) is quantized within."""
    T, n = X.shape
    m = W.shape[0]
    d = Fp8LinearDesc(T, m, n, 0)
    qw, sw = fp8_shapes(m, n, True)
    with _on((X, W, S, out, workspace), stream) as d.stream:
        args = (_arg(X, torch.bfloat16, (T, n), "X"), _arg(W, torch.float8_e4m3fn, qw, "W"),
                _arg(S, torch.float32, sw, "S"))
        Y = out if out is not None else X.new_empty((T, m))
        workspace = _scratch(d, workspace, lib().qgalore_fp8_linear_fwd_workspace_bytes(T, m, n),
                             X.device)
        _check(lib().qgalore_fp8_linear_fwd(ctypes.byref(d), *args,
                                            _arg(Y, torch.bfloat16, (T, m), "out")),
               "qgalore_fp8_linear_fwd")
    return Y


def fp8_linear_bwd(dY: torch.Tensor, Wt=None, St=None, Xt=None, Sx=None, fmt: str = "e5m2", dX=None,
                   G=None, workspace=None, stream=None):
    """Gradients (dX, G) of fp8_linear_fwd in bf16: dX = q(dY) W with the weight's transpose Wt, St,
    G = q(dY)^T q(X) with the inputs' columns Xt, Sx (fp8_quantize(X, rows=False, columns=True)). dY is
    quantized within, in `fmt`. Without Wt or Xt its gradient is None."""
    T, m = dY.shape
    if (Wt is None) != (St is None) or (Xt is None) != (Sx is None):
        raise ValueError("codes and scales come together")
    if Wt is None and Xt is None:
        raise ValueError("neither Wt nor Xt")
    if (Wt is None and dX is not None) or (Xt is None and G is not None):
        raise ValueError("dX needs Wt and St, G needs Xt and Sx")
    n = (Wt if Wt is not None else Xt).shape[0]
    d = Fp8LinearDesc(T, m, n, _fp8_format(fmt))
    with _on((dY, Wt, St, Xt, Sx, dX, G, workspace), stream) as d.stream:
        (qw, sw), (qx, sx) = fp8_shapes(n, m, True), fp8_shapes(n, T)
        e4m3 = torch.float8_e4m3fn
        args = (_arg(dY, torch.bfloat16, (T, m), "dY"), _arg(Wt, e4m3, qw, "Wt"),
                _arg(St, torch.float32, sw, "St"), _arg(Xt, e4m3, qx, "Xt"),
                _arg(Sx, torch.float32, sx, "Sx"))
        if Wt is not None and dX is None:
            dX = dY.new_empty((T, n))
        if Xt is not None and G is None:
            G = dY.new_empty((m, n))
        workspace = _scratch(d, workspace, lib().qgalore_fp8_linear_bwd_workspace_bytes(T, m, n),
                             dY.device)
        _check(lib().qgalore_fp8_linear_bwd(
            ctypes.byref(d), *args, _arg(dX, torch.bfloat16, (T, n), "dX"),
            _arg(G, torch.bfloat16, (m, n), "G")), "qgalore_fp8_linear_bwd")
    return dX, G


class GradSet:
    """The gradients of a model (bf16 or fp32, contiguous, of any shapes): their norm, and their
    clipping in place or into `out`. kind: l2 or max. nonfinite: with "zero" a norm that is not finite
    makes every clipped gradient 0; otherwise it goes into them by the formula. The tensors must stay
    valid while the object is used; it keeps a workspace of its own, so calls of one object are to be
    ordered (one stream, or events), and it is to live as long as a graph that has captured one."""

    def __init__(self, tensors: list, out=None, kind: str = "l2", eps: float = 1e-6,
                 nonfinite: str = "keep"):
        tensors = list(tensors)
        out = tensors if out is None else list(out)
        if not tensors:
            raise ValueError("no tensors")
        if len(out) != len(tensors):
            raise ValueError(f"{len(tensors)} tensors, {len(out)} outputs")
        if kind not in GRAD_NORMS:
            raise ValueError(f"unknown norm {kind!r}: one of {', '.join(GRAD_NORMS)}")
        if nonfinite not in ("keep", "zero"):
            raise ValueError(f"nonfinite is keep or zero (got {nonfinite!r})")
        with _on((*tensors, *out), None):
            self._arr = (Grad * len(tensors))()
            for a, t, o in zip(self._arr, tensors, out):
                if t.dtype not in (torch.bfloat16, torch.float32):
                    raise TypeError(f"gradients are bf16 or fp32 (got {t.dtype})")
                a.g = _ptr(t, t.dtype, None, "gradient")
                a.out = _ptr(o, t.dtype, t.shape, "out")
                a.n = t.numel()
                a.dtype = 0 if t.dtype == torch.bfloat16 else 1
        self._keep, self.out = tensors, out
        self._desc = ClipDesc(GRAD_NORMS[kind], 1 if nonfinite == "zero" else 0, 0.0, eps)
        self._workspace, self._stream = None, None

    def _call(self, handle):
        w = self._workspace
        if w is None:
            w = self._workspace = alloc_workspace(lib().qgalore_grad_workspace_bytes(),
                                                  self._keep[0].device)
            self._stream = handle
        elif handle != self._stream:   # not to be given away before this call is through
            w.record_stream(torch.cuda.current_stream(w.device))
        d = self._desc
        d.workspace, d.workspace_bytes, d.stream = w.data_ptr(), w.numel(), handle
        return d

    def norm(self, total=None, out=None, stream=None) -> torch.Tensor:
        """The norm (fp32, one element; `out` to write to). total: an fp64 tensor of one element that
        gets the sum of squares, or the maximum, to be joined with other processes' shares."""
        with _on((self._keep[0], total, out), stream) as handle:
            if out is None:
                out = self._keep[0].new_empty((1,), dtype=torch.float32)
            args = (_arg(out, torch.float32, (1,), "out"), _arg(total, torch.float64, (1,), "total"))
            _check(lib().qgalore_grad_norm(ctypes.byref(self._call(handle)), self._arr,
                                           len(self._arr), *args), "qgalore_grad_norm")
        return out[0]

    def clip(self, max_norm: float, total=None, norm=None, stream=None) -> torch.Tensor:
        """Scales the gradients by min(1, max_norm / (norm + eps)), max_norm finite, and returns the norm
        (fp32; `norm`, one element, to write to). total: the fp64 total to take in place of these gradients' own."""
        with _on((self._keep[0], total, norm), stream) as handle:
            if norm is None:
                norm = self._keep[0].new_empty((1,), dtype=torch.float32)
            args = (_arg(total, torch.float64, (1,), "total"), _arg(norm, torch.float32, (1,), "norm"))
            d = self._call(handle)
            d.max_norm = max_norm
            _check(lib().qgalore_grad_clip(ctypes.byref(d), self._arr, len(self._arr), *args),
                   "qgalore_grad_clip")
        return norm[0]


def grad_norm(tensors: list, kind: str = "l2", stream=None) -> torch.Tensor:
    """The norm of all values of a list of gradients (fp32)."""
    return GradSet(tensors, kind=kind).norm(stream=stream)


def clip_gradients(tensors: list, max_norm: float, out=None, kind: str = "l2", eps: float = 1e-6,
                   nonfinite: str = "keep", stream=None) -> torch.Tensor:
    """Clips a list of gradients by their joint norm, in place or into `out`; returns the norm."""
    return GradSet(tensors, out, kind, eps, nonfinite).clip(max_norm, stream=stream)


# the Newton-Schulz polynomial a x + b x^3 + c x^5 of Muon: five steps take singular values from
# about 0.01 on into [0.7, 1.2]
MUON_COEF = (3.4445, -4.7750, 2.0315)


@dataclasses.dataclass
class MuonLayer:
    """One layer of the orthogonalised update (see include/qgalore.h for layouts)."""
    layer_id: int
    G: torch.Tensor          # bf16 m x n
    Wq: torch.Tensor         # int8 m x n
    Ws: torch.Tensor         # fp32 [groups(m*n)]
    M: torch.Tensor          # fp32 m x n momentum


def muon_workspace_bytes(m: int, n: int, count: int = 1) -> int:
    return int(lib().qgalore_muon_workspace_bytes(m, n, count))


def _muon_desc(m: int, n: int, hp: dict) -> MuonDesc:
    d = MuonDesc()
    d.m, d.n = m, n
    d.lr, d.momentum = hp.get("lr", 0.02), hp.get("momentum", 0.95)
    d.weight_decay, d.nesterov = hp.get("weight_decay", 0.0), int(hp.get("nesterov", True))
    d.alpha = hp.get("alpha", math.sqrt(max(1.0, m / n)))
    d.ns_steps, d.eps = int(hp.get("ns_steps", 5)), hp.get("eps", 1e-7)
    d.ns_a, d.ns_b, d.ns_c = hp.get("coef", MUON_COEF)
    return d


def _overlap(tensors) -> bool:
    """Whether any two of these contiguous tensors share memory."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors)
    return any(a[1] > b[0] for a, b in zip(spans, spans[1:]))


def _muon_workspace(d: MuonDesc, workspace, count: int, device):
    if workspace is None:
        nbytes = muon_workspace_bytes(d.m, d.n, count)
        if nbytes == 0:
            raise ValueError(f"{count} matrices of {d.m} x {d.n} are not supported")
        workspace = alloc_workspace(nbytes, device)
    d.workspace = _arg(workspace, torch.uint8, None, "workspace")
    d.workspace_bytes = workspace.numel()
    return workspace


class Muon:
    """The orthogonalised update of a set of layers of any shapes: layers of one shape go through
    one call. The tensors named by `layers` must stay valid while the object is used. `hp`: lr,
    momentum, nesterov, weight_decay, alpha (default: sqrt(max(1, m / n)) for each shape), ns_steps,
    coef, eps."""

    def __init__(self, layers: list, hp: dict | None = None):
        if not layers:
            raise ValueError("no layers")
        self._keep = list(layers)
        self._calls = []
        self.workspace, self.workspace_bytes = None, 0
        shapes = {}
        for L in layers:
            shapes.setdefault(tuple(L.Wq.shape), []).append(L)
        self._tensors = [t for L in layers for t in (L.G, L.Wq, L.Ws, L.M)]
        if _overlap([L.Wq for L in layers]) or _overlap([L.M for L in layers]):
            raise ValueError("two layers share a weight or a momentum")
        for (m, n), group in shapes.items():
            arr = (MuonLayerDesc * len(group))()
            for k, L in enumerate(group):
                arr[k].G = _ptr(L.G, torch.bfloat16, (m, n), "G")
                arr[k].M = _ptr(L.M, torch.float32, (m, n), "M")
                arr[k].W_q = _ptr(L.Wq, torch.int8, (m, n), "Wq")
                arr[k].W_scale = _ptr(L.Ws, torch.float32, (n_groups(m * n),), "Ws")
                arr[k].layer_id = L.layer_id
            nbytes = muon_workspace_bytes(m, n, len(group))
            if nbytes == 0:
                raise ValueError(f"layers of {m} x {n} are not supported")
            self.workspace_bytes = max(self.workspace_bytes, nbytes)
            self._calls.append((_muon_desc(m, n, hp or {}), arr, len(group)))
        with _on(self._tensors, None):
            pass

    def step(self, t: int, seed: int, workspace=None, stream=None) -> None:
        """One update of every layer (asynchronous). Without a workspace the object allocates its
        own and keeps it: steps of one object are then to be ordered (one stream, or events), and the
        object is to live as long as a graph that has captured one."""
        with _on((self._tensors[0], workspace), stream) as handle:
            if workspace is None:
                if self.workspace is None:
                    self.workspace = alloc_workspace(self.workspace_bytes, self._tensors[0].device)
                    self._stream = handle
                elif handle != self._stream:   # not to be given away before this step is through
                    self.workspace.record_stream(torch.cuda.current_stream(self.workspace.device))
                workspace = self.workspace
            ws = _ptr(workspace, torch.uint8, None, "workspace")
            for d, arr, count in self._calls:
                d.workspace, d.workspace_bytes, d.stream = ws, workspace.numel(), handle
                _check(lib().qgalore_muon_step(ctypes.byref(d), arr, count, int(t),
                                               int(seed) & (2 ** 64 - 1)), "qgalore_muon_step")


def muon_step(L: MuonLayer, t: int, seed: int, hp: dict | None = None, workspace=None,
              stream=None) -> None:
    """One orthogonalised update of one layer (asynchronous on the current stream)."""
    m, n = L.Wq.shape
    d = _muon_desc(m, n, hp or {})
    one = MuonLayerDesc(_arg(L.G, torch.bfloat16, (m, n), "G"),
                        _arg(L.M, torch.float32, (m, n), "M"),
                        _arg(L.Wq, torch.int8, (m, n), "Wq"),
                        _arg(L.Ws, torch.float32, (n_groups(m * n),), "Ws"), L.layer_id)
    with _on((L.G, L.M, L.Wq, L.Ws, workspace), stream) as d.stream:
        workspace = _muon_workspace(d, workspace, 1, L.Wq.device)
        _check(lib().qgalore_muon_step(ctypes.byref(d), ctypes.byref(one), 1, int(t),
                                       int(seed) & (2 ** 64 - 1)), "qgalore_muon_step")


def orthogonalize(Gs: list, steps: int = 5, coef=MUON_COEF, eps: float = 1e-7, out=None,
                  workspace=None, stream=None) -> list:
    """The orthogonalised matrices (bf16) of a list of bf16 matrices of one shape."""
    if not Gs:
        raise ValueError("no matrices")
    m, n = Gs[0].shape
    count = len(Gs)
    d = _muon_desc(m, n, dict(ns_steps=steps, coef=coef, eps=eps))
    with _on((*Gs, *(out or ()), workspace), stream) as d.stream:
        if out is None:
            out = [torch.empty_like(G, memory_format=torch.contiguous_format) for G in Gs]
        if len(out) != count:
            raise ValueError(f"{count} matrices, {len(out)} outputs")
        src = (c_void_p * count)(*(_arg(G, torch.bfloat16, (m, n), "G") for G in Gs))
        dst = (c_void_p * count)(*(_arg(O, torch.bfloat16, (m, n), "out") for O in out))
        workspace = _muon_workspace(d, workspace, count, Gs[0].device)
        _check(lib().qgalore_orthogonalize(ctypes.byref(d), src, dst, count),
               "qgalore_orthogonalize")
    return out


class Schedule:
    """Per-layer refresh bookkeeping (host-side, in the library)."""

    def __init__(self, delta0: int, gamma: float = 0.4):
        self._s = Sched()
        _check(lib().qgalore_sched_init(ctypes.byref(self._s), int(delta0), float(gamma)),
               "qgalore_sched_init")

    def due(self, t: int) -> bool:
        return bool(lib().qgalore_sched_due(ctypes.byref(self._s), int(t)))

    def refresh(self, t: int, cs: float | None) -> bool:
        doubled = c_int32(0)
        _check(lib().qgalore_sched_refresh(ctypes.byref(self._s), int(t),
                                           float("nan") if cs is None else float(cs),
                                           ctypes.byref(doubled)), "qgalore_sched_refresh")
        return bool(doubled.value)

    @property
    def delta(self) -> int:
        return int(self._s.delta)

    @property
    def next_refresh(self) -> int:
        return int(self._s.next_refresh)

    @property
    def count(self) -> int:
        return int(self._s.count)

    @property
    def last_cossim(self) -> float:
        v = float(self._s.last_cossim)
        return v if not math.isnan(v) else float("nan")
