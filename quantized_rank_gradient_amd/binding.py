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


# projection storage formats (qg_p_format)
P_FORMATS = {"int4": 0, "int8": 1, "bf16": 2}
# activations of a linear layer (qg_act)
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
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
