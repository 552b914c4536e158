"""Python binding of the B200 fused MoE expert layer (``libmoe_b200.so``).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. PyTorch provides device memory and streams. The functions carry the C
entry points' names (see ``include/moe.h``); each takes and returns torch
tensors on the current CUDA device and launches on the current stream.

There is no fallback: if the shared library is missing the import fails.
Build it with ``python mixture_experts_layer_21_b200/build.py``.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass, field

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_b200.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: run `python mixture_experts_layer_21_b200/build.py`")

_lib = ctypes.CDLL(LIB_PATH)

MOE_OK = 0
STATUS = ["MOE_OK", "MOE_ERR_INVALID_ARG", "MOE_ERR_UNSUPPORTED", "MOE_ERR_ALIGNMENT",
          "MOE_ERR_WORKSPACE_TOO_SMALL", "MOE_ERR_CUDA", "MOE_ERR_DEVICE", "MOE_ERR_TIMEOUT",
          "MOE_ERR_NOT_PREPARED"]
ACT = {"silu": 0, "situ": 1, "swigluoai": 2}
SCORING = {"softmax": 0, "sigmoid": 1}
GROUP_SCORE = {"max": 0, "top2": 1}
QUANT = {None: 0, "mxfp8": 1, "mxfp4": 2}
WFMT = {"bf16": 0, "mxfp4": 1, "nvfp4": 2}

# Every symbol include/moe.h declares.
EXPORTS = ["moe_status_string", "moe_version", "moe_route_topk", "moe_permute_workspace_size",
           "moe_permute", "moe_grouped_gemm_workspace_size", "moe_grouped_gemm", "moe_act_and_mul",
           "moe_combine", "moe_quantize_nvfp4", "moe_prepared_weight_bytes", "moe_prepare_weights",
           "moe_forward_workspace_size", "moe_forward", "moe_get_device_error", "moe_permute_noalloc",
           "moe_permute_noalloc_status", "moe_grouped_gemm_nvfp4", "moe_quantize_mxfp8", "moe_route_topk_grouped",
           "moe_bias_act_and_mul", "moe_forward_workspace_size_args", "moe_route_scored", "moe_add_rmsnorm",
           "moe_quantize_mxfp4", "moe_grouped_gemm_mxfp4", "moe_grouped_gemm_mxfp4_room",
           "moe_grouped_gemm_mxfp4_rows_size"]


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = STATUS[status] if 0 <= status < len(STATUS) else str(status)
        super().__init__(f"{where}: {name}")


class moe_weight_t(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("G", ctypes.c_int32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("data", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("alpha", ctypes.c_void_p), ("kdata", ctypes.c_void_p), ("kscale", ctypes.c_void_p),
                ("kalpha", ctypes.c_void_p)]


class moe_act_params_t(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("situ_alpha", ctypes.c_float), ("situ_beta", ctypes.c_float)]


class moe_act_ex_t(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("situ_alpha", ctypes.c_float), ("situ_beta", ctypes.c_float),
                ("swiglu_alpha", ctypes.c_float), ("swiglu_beta", ctypes.c_float),
                ("swiglu_limit", ctypes.c_float)]


class moe_rmsnorm_args_t(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("x_is_f32", ctypes.c_int32), ("weight_is_f32", ctypes.c_int32),
                ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64),
                ("residual_out_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("eps", ctypes.c_float), ("quant", ctypes.c_int32), ("residual_out", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("deq", ctypes.c_void_p)]


class moe_route_args_t(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("topk_ids", ctypes.c_void_p),
                ("topk_w", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("in_is_bf16", ctypes.c_int32),
                ("T", ctypes.c_int32), ("E", ctypes.c_int32), ("topk", ctypes.c_int32), ("scoring", ctypes.c_int32),
                ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32), ("group_score", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("routed_scaling_factor", ctypes.c_float)]


# The two argument structures in one pack each, a fraction of the time that a ctypes object takes to
# fill: what a one-token call spends on the host is most of its time.
_ROUTE_ARGS = struct.Struct("PPPPqiiiiiiiiif")
_RMSNORM_ARGS = struct.Struct("PPPiiiiqqqqfiPPPPP")


class moe_forward_args_t(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("router_logits", ctypes.c_void_p),
                ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("B", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("replica_src", ctypes.c_void_p),
                ("w_gate", moe_weight_t), ("w_up", moe_weight_t), ("w_down", moe_weight_t),
                ("act", moe_act_params_t), ("apply_topk_in_fc1", ctypes.c_int32),
                ("act_quant", ctypes.c_int32), ("out", ctypes.c_void_p),
                ("topk_ids_out", ctypes.c_void_p), ("topk_w_out", ctypes.c_void_p),
                ("T_max", ctypes.c_int32), ("stage_events", ctypes.c_void_p),
                ("routing", ctypes.c_int32), ("routing_bias", ctypes.c_void_p),
                ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("routed_scaling_factor", ctypes.c_float),
                ("topk_ids_in", ctypes.c_void_p), ("topk_w_in", ctypes.c_void_p),
                ("apply_router_weight_on_input", ctypes.c_int32),
                ("swiglu_alpha", ctypes.c_float), ("swiglu_beta", ctypes.c_float),
                ("swiglu_limit", ctypes.c_float),
                ("bias_gate", ctypes.c_void_p), ("bias_up", ctypes.c_void_p), ("bias_down", ctypes.c_void_p)]

ROUTING = {"renormalize": 0, "deepseek_v3": 1, "given": 2}

MOE_FWD_STAGE_EVENTS = 7


_P, _I, _S, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
_sig = {
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_version": (ctypes.c_char_p, []),
    "moe_route_topk": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_permute_workspace_size": (_S, [_I, _I, _I, _I]),
    "moe_permute": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _I, _P, _S, _P]),
    "moe_grouped_gemm_workspace_size": (_S, [_I, ctypes.POINTER(moe_weight_t)]),
    "moe_grouped_gemm": (_I, [_P, _I, ctypes.POINTER(moe_weight_t), _P, _P, _P, _S, _P]),
    "moe_act_and_mul": (_I, [_P, _P, _P, _I, _I, moe_act_params_t, _P, _P]),
    "moe_combine": (_I, [_P, _P, _P, _I, _I, _I, _P, _P]),
    "moe_quantize_nvfp4": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "moe_prepared_weight_bytes": (_S, [ctypes.POINTER(moe_weight_t)]),
    "moe_prepare_weights": (_I, [ctypes.POINTER(moe_weight_t), _P, _S, _P]),
    "moe_forward_workspace_size": (_S, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "moe_forward": (_I, [ctypes.POINTER(moe_forward_args_t), _P, _S, _P]),
    "moe_get_device_error": (_I, [_P, _P]),
    "moe_permute_noalloc": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _I, _P]),
    "moe_permute_noalloc_status": (_I, [_P]),
    "moe_grouped_gemm_nvfp4": (_I, [_P, _P, _P, _I, ctypes.POINTER(moe_weight_t), _P, _P, _P, _S, _P]),
    "moe_quantize_mxfp8": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_route_topk_grouped": (_I, [_P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P]),
    "moe_bias_act_and_mul": (_I, [_P, _P, _I, _P, _P, _P, _I, _P, _I, _I, ctypes.POINTER(moe_act_ex_t), _P, _P]),
    "moe_forward_workspace_size_args": (_S, [ctypes.POINTER(moe_forward_args_t)]),
    "moe_route_scored": (_I, [_P, _P]),      # moe_route_args_t*
    "moe_add_rmsnorm": (_I, [_P, _P]),       # moe_rmsnorm_args_t*
    "moe_quantize_mxfp4": (_I, [_P, _I, _L, _I, _I, _P, _P, _P, _P]),
    "moe_grouped_gemm_mxfp4": (_I, [_P, _P, _I, _P, _I, ctypes.POINTER(moe_weight_t), _P, _P, _P, _P, _S, _P]),
    "moe_grouped_gemm_mxfp4_room": (_I, [_P, _P, _I, _P, _I, ctypes.POINTER(moe_weight_t), _P, _P, _P, _S, _P, _S, _P]),
    "moe_grouped_gemm_mxfp4_rows_size": (_S, [_I, ctypes.POINTER(moe_weight_t)]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype, _f.argtypes = _res, _args


def lib() -> ctypes.CDLL:
    return _lib


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _on(stream, make, *args, **kw) -> torch.Tensor:
    """A tensor that a call makes for itself or its caller: memory of the stream that the call launches on,
    filled in that stream's order. A block of the current stream's could still be read or written there."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


_error_words: dict[int, torch.Tensor] = {}


def _error_word(dev: int) -> torch.Tensor:
    """The error word of the calls on a device that get no workspace and need none but for it: one that
    outlives them, so that moe_get_device_error() can read it. The first error stays until it is read."""
    t = _error_words.get(dev)
    if t is None:
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("ws: the first call on a device needs one while a graph is captured")
        with torch.cuda.device(dev):
            t = torch.zeros(256, dtype=torch.uint8, device=f"cuda:{dev}")
            torch.cuda.current_stream().synchronize()  # zero before a kernel on any stream
        t = _error_words.setdefault(dev, t)
    return t


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoEError(status, where)


def _launch_device(t: torch.Tensor) -> int:
    """The device of a call, that of its first tensor: the kernels run on the current device."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"need tensors on the current CUDA device, got {t.device}")
    return dev


def _launch_stream(dev: int, stream) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _want(t, name: str, shape, dtype, dev: int, dense: bool = True) -> int:
    """A tensor argument of this shape and type on this device; rows contiguous, and dense unless the
    call takes a row stride. Returns the elements between rows, 0 where they follow one another."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        if t.is_contiguous():
            return 0
        if not dense and (t.shape[1] <= 1 or t.stride(1) == 1) and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1]):
            return t.stride(0) if t.shape[0] > 1 else 0
        raise ValueError(f"{name}: need {'a contiguous tensor' if dense else 'contiguous rows that do not overlap'}, "
                         f"got strides {t.stride()}")
    raise ValueError(f"{name}: need {tuple(shape)} {dtype} on cuda:{dev}, got {tuple(t.shape)} {t.dtype} on {t.device}")


def _output(out, name: str, like, shape, dtype, dev: int, stream, dense: bool = True):
    """The caller's output of that name, checked, or a new one; and its row stride."""
    t = out.get(name)
    if t is None:
        return _on(stream, torch.empty, shape, dtype=dtype, device=like.device), 0
    return t, _want(t, name, shape, dtype, dev, dense)


def _float_type(t, name: str) -> torch.dtype:
    if t.dtype is torch.bfloat16 or t.dtype is torch.float32:
        return t.dtype
    raise ValueError(f"{name}: need bf16 or fp32, got {t.dtype}")


def version() -> str:
    return _lib.moe_version().decode()


def status_string(s: int) -> str:
    return _lib.moe_status_string(s).decode()


# ---------------------------------------------------------------------------- weights

@dataclass
class Weight:
    """One projection's weights on the device plus their prepared kernel-format copy.

    ``data``: bf16 [G,N,K] or uint8 packed e2m1 [G,N,K/2]; ``scale``: uint8 e8m0
    [G,N,K/32] (MXFP4) or e4m3 [G,N,K/16] (NVFP4); ``alpha``: fp32 [G] or None.
    """

    fmt: str
    data: torch.Tensor
    scale: torch.Tensor | None = None
    alpha: torch.Tensor | None = None
    prepared: torch.Tensor | None = None
    desc: moe_weight_t = field(default_factory=moe_weight_t)

    def __post_init__(self):
        d = self.desc
        d.fmt = WFMT[self.fmt]
        d.G, d.N = self.data.shape[0], self.data.shape[1]
        d.K = self.data.shape[2] * (1 if self.fmt == "bf16" else 2)
        d.data, d.scale, d.alpha = _ptr(self.data), _ptr(self.scale), _ptr(self.alpha)

    @property
    def desc_ref(self):
        return ctypes.byref(self.desc)

    @property
    def G(self):
        return self.desc.G

    @property
    def N(self):
        return self.desc.N

    @property
    def K(self):
        return self.desc.K

    @classmethod
    def from_host(cls, ws, device="cuda") -> "Weight":
        """From a ``workloads.WeightSet`` (CPU) to the device."""
        mv = lambda t: None if t is None else t.to(device, non_blocking=False).contiguous()
        return cls(ws.fmt, mv(ws.data), mv(ws.scale), mv(ws.alpha))


def moe_prepare_weights(w: Weight, stream=None) -> Weight:
    """S0: kernel-format copy of FP4 weights (no-op for BF16). Synchronises."""
    if w.fmt == "bf16":
        return w
    nbytes = _lib.moe_prepared_weight_bytes(ctypes.byref(w.desc))
    w.prepared = _on(stream, torch.empty, nbytes, dtype=torch.uint8, device=w.data.device)
    _check(_lib.moe_prepare_weights(ctypes.byref(w.desc), _ptr(w.prepared), nbytes, _stream(stream)),
           "moe_prepare_weights")
    _error_word(w.prepared.get_device())  # made here, it is there when a product is captured
    return w


# ---------------------------------------------------------------------------- steps

def moe_route_topk(logits: torch.Tensor, topk: int, ids=None, w=None, stream=None):
    T, E = logits.shape
    ids = ids if ids is not None else _on(stream, torch.empty, T, topk, dtype=torch.int32, device=logits.device)
    w = w if w is not None else _on(stream, torch.empty, T, topk, dtype=torch.float32, device=logits.device)
    _check(_lib.moe_route_topk(_ptr(logits), T, E, topk, _ptr(ids), _ptr(w), _stream(stream)),
           "moe_route_topk")
    return ids, w


def moe_route_topk_grouped(logits: torch.Tensor, topk: int, n_group: int, topk_group: int, bias=None,
                           routed_scaling_factor: float = 1.0, ids=None, w=None, stream=None):
    """DeepSeekV3 routing (grouped top-k on sigmoid scores, bias for selection only)."""
    T, E = logits.shape
    ids = ids if ids is not None else _on(stream, torch.empty, T, topk, dtype=torch.int32, device=logits.device)
    w = w if w is not None else _on(stream, torch.empty, T, topk, dtype=torch.float32, device=logits.device)
    _check(_lib.moe_route_topk_grouped(_ptr(logits), _ptr(bias), T, E, topk, n_group, topk_group,
                                       routed_scaling_factor, _ptr(ids), _ptr(w), _stream(stream)),
           "moe_route_topk_grouped")
    return ids, w


def moe_route_scored(logits: torch.Tensor, topk: int, scoring: str = "softmax", bias=None, n_group: int = 1,
                     topk_group: int = 1, group_score: str = "max", renormalize: bool = True,
                     routed_scaling_factor: float = 1.0, ids=None, w=None, stream=None):
    """Routing by softmax or sigmoid scores, with a selection bias (fp32 [E]), groups kept by their
    best ("max") or two best ("top2") experts, and raw or renormalised weights. logits fp32 or bf16
    [T,E], rows in any stride; a logit of -inf masks its expert."""
    T, E = logits.shape
    dev = _launch_device(logits)
    dt = _float_type(logits, "logits")
    stride = _want(logits, "logits", (T, E), dt, dev, False) or E
    if bias is not None:
        _want(bias, "bias", (E,), torch.float32, dev)
    if ids is None:
        ids = _on(stream, torch.empty, T, topk, dtype=torch.int32, device=logits.device)
    else:
        _want(ids, "ids", (T, topk), torch.int32, dev)
    if w is None:
        w = _on(stream, torch.empty, T, topk, dtype=torch.float32, device=logits.device)
    else:
        _want(w, "w", (T, topk), torch.float32, dev)
    a = _ROUTE_ARGS.pack(logits.data_ptr(), 0 if bias is None else bias.data_ptr(), ids.data_ptr(), w.data_ptr(),
                         stride, dt is torch.bfloat16, T, E, topk, SCORING[scoring], n_group, topk_group,
                         GROUP_SCORE[group_score], renormalize, routed_scaling_factor)
    _check(_lib.moe_route_scored(a, _launch_stream(dev, stream)), "moe_route_scored")
    return ids, w


def moe_add_rmsnorm(x: torch.Tensor, weight=None, residual=None, eps: float = 1e-6, quant: str | None = None,
                    want_y: bool = True, deq: bool = False, out=None, stream=None):
    """r = x + residual; y = r / sqrt(mean(r^2) + eps) * weight; y optionally quantised to "mxfp8" or
    "mxfp4" rows. x bf16 or fp32 [T,H], residual bf16 [T,H], weight bf16 or fp32 [H] (rows of x and
    residual in any stride of a multiple of 8 elements; tensors 16-byte aligned).
    ``out``: optional dict of caller-allocated outputs (any of residual, y, codes, scales, deq; the
    rows of residual and y may be strided, residual may be the input's own tensor); the others are
    allocated here. Returns a dict with those five, None where not asked for: ``residual`` (bf16
    rows of r) comes with a residual, ``y`` (bf16) with want_y, ``codes`` and ``scales`` with quant,
    ``deq`` (bf16, the values they stand for) with deq."""
    T, H = x.shape
    dev = _launch_device(x)
    out = out or {}
    bf16, shape = torch.bfloat16, (T, H)
    xt = _float_type(x, "x")
    sx = _want(x, "x", shape, xt, dev, False)
    y = r = codes = scales = d = None
    sres = sr = sy = pres = pw = pr = py = pc = ps = pd = w32 = 0
    if residual is not None:
        sres, pres = _want(residual, "residual", shape, bf16, dev, False), residual.data_ptr()
        r, sr = _output(out, "residual", x, shape, bf16, dev, stream, False)
        pr = r.data_ptr()
    if weight is not None:
        wt = _float_type(weight, "weight")
        _want(weight, "weight", (H,), wt, dev)
        pw, w32 = weight.data_ptr(), wt is not bf16
    if want_y:
        y, sy = _output(out, "y", x, shape, bf16, dev, stream, False)
        py = y.data_ptr()
    q = QUANT[quant]
    if q:
        codes, _ = _output(out, "codes", x, (T, H // 2) if q == 2 else shape, torch.uint8, dev, stream)
        scales, _ = _output(out, "scales", x, (T, H // 32), torch.uint8, dev, stream)
        pc, ps = codes.data_ptr(), scales.data_ptr()
        if deq:
            d, _ = _output(out, "deq", x, shape, bf16, dev, stream)
            pd = d.data_ptr()
    elif deq:
        raise ValueError("deq needs quant")
    a = _RMSNORM_ARGS.pack(x.data_ptr(), pres, pw, xt is not bf16, w32, T, H, sx, sres, sr, sy, eps, q, pr, py, pc, ps, pd)
    _check(_lib.moe_add_rmsnorm(a, _launch_stream(dev, stream)), "moe_add_rmsnorm")
    return dict(residual=r, y=y, codes=codes, scales=scales, deq=d)


def permute_workspace(T: int, topk: int, E: int, B: int, device="cuda") -> torch.Tensor:
    n = _lib.moe_permute_workspace_size(T, topk, E, B)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def moe_permute(topk_ids, topk_w, E: int, B: int = 0, replica_src=None, x=None, M_alloc=None,
                ws=None, stream=None, out=None):
    """``out``: optional dict of caller-allocated outputs (any of cu_seqlens, perm_token,
    perm_w, inv_perm, x_perm [M_alloc,H]); the others are allocated here."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    NvS = T * k
    out = out or {}
    M_alloc = NvS if M_alloc is None else M_alloc
    ws = ws if ws is not None else _on(stream, permute_workspace, T, k, E, B, dev)
    def buf(name, shape, dtype):
        t = out.get(name)
        return t if t is not None else _on(stream, torch.empty, shape, dtype=dtype, device=dev)

    cu = buf("cu_seqlens", (E + B,), torch.int32)
    perm_token = buf("perm_token", (NvS,), torch.int32)
    perm_w = buf("perm_w", (NvS,), torch.float32)
    inv = buf("inv_perm", (T, k), torch.int32)
    x_perm = None
    H = 0
    if x is not None:
        H = x.shape[1]
        x_perm = out.get("x_perm")
        if x_perm is None:
            x_perm = _on(stream, torch.zeros, M_alloc, H, dtype=x.dtype, device=dev)
        M_alloc = x_perm.shape[0]
    _check(_lib.moe_permute(_ptr(topk_ids), _ptr(topk_w), T, k, E, B, _ptr(replica_src), _ptr(x), H,
                            _ptr(cu), _ptr(perm_token), _ptr(perm_w), _ptr(inv), _ptr(x_perm), M_alloc,
                            _ptr(ws), ws.numel(), _stream(stream)), "moe_permute")
    return dict(cu_seqlens=cu, perm_token=perm_token, perm_w=perm_w, inv_perm=inv, x_perm=x_perm, ws=ws)


def moe_grouped_gemm(a: torch.Tensor, w: Weight, cu_seqlens: torch.Tensor, out=None, ws=None,
                     stream=None) -> torch.Tensor:
    M = a.shape[0]
    out = out if out is not None else _on(stream, torch.empty, M, w.N, dtype=torch.bfloat16, device=a.device)
    if ws is None:
        n = _lib.moe_grouped_gemm_workspace_size(M, ctypes.byref(w.desc))
        ws = _on(stream, torch.zeros, n, dtype=torch.uint8, device=a.device)
    _check(_lib.moe_grouped_gemm(_ptr(a), M, ctypes.byref(w.desc), _ptr(cu_seqlens), _ptr(out),
                                 _ptr(ws), ws.numel(), _stream(stream)), "moe_grouped_gemm")
    return out


def moe_grouped_gemm_nvfp4(a_codes: torch.Tensor, a_sb: torch.Tensor, a_s: torch.Tensor, w: Weight,
                           cu_seqlens: torch.Tensor, out=None, ws=None, stream=None) -> torch.Tensor:
    """Block-scaled grouped GEMM on NVFP4 activations (codes [M,K/2], e4m3 scales [M,K/16],
    row scales [M]) and prepared NVFP4 weights; bf16 out [M,N]. Without ``ws`` errors go to the device's
    own error word, which moe_get_device_error() reads."""
    M = a_codes.shape[0]
    out = out if out is not None else _on(stream, torch.empty, M, w.N, dtype=torch.bfloat16, device=a_codes.device)
    ws = ws if ws is not None else _error_word(a_codes.get_device())
    _check(_lib.moe_grouped_gemm_nvfp4(_ptr(a_codes), _ptr(a_sb), _ptr(a_s), M, ctypes.byref(w.desc),
                                       _ptr(cu_seqlens), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_grouped_gemm_nvfp4")
    return out


def moe_grouped_gemm_mxfp4(a_codes: torch.Tensor, a_scales: torch.Tensor, w: Weight, cu_seqlens: torch.Tensor,
                           row_idx=None, out=None, ws=None, stream=None) -> torch.Tensor:
    """Block-scaled grouped GEMM on MXFP4 activations (codes [R,K/2], e8m0 scales [R,K/32]) and
    prepared MXFP4 weights. row_idx (int32 [M]): row r of the segments is row row_idx[r] of a (the
    permutation's perm_token), segments of many rows being gathered before the product into memory
    allocated here; without it the R rows are in segment order. bf16 out [M,N]. What the kernel finds (an
    index or a segment end out of range, a wait that ran out) is in ``ws`` (256 bytes, zeroed once), without
    it in the device's own error word: moe_get_device_error(ws) or moe_get_device_error()."""
    R, dev, u8 = a_codes.shape[0], _launch_device(a_codes), torch.uint8
    K, N = w.K, w.N
    _want(a_codes, "a_codes", (R, K // 2), u8, dev)
    _want(a_scales, "a_scales", (R, K // 32), u8, dev)
    _want(cu_seqlens, "cu_seqlens", (w.G,), torch.int32, dev)
    if w.data.get_device() != dev:
        raise ValueError(f"w: need weights on cuda:{dev}, got {w.data.device}")
    M, rows, room = R, None, 0
    if row_idx is not None:
        M = row_idx.shape[0]
        _want(row_idx, "row_idx", (M,), torch.int32, dev)
        room = _lib.moe_grouped_gemm_mxfp4_rows_size(M, w.desc_ref)
        if room:
            rows = _on(stream, torch.empty, room, dtype=u8, device=a_codes.device)
    if out is None:
        out = _on(stream, torch.empty, M, N, dtype=torch.bfloat16, device=a_codes.device)
    else:
        _want(out, "out", (M, N), torch.bfloat16, dev)
    if ws is None:
        ws = _error_word(dev)
    elif ws.get_device() != dev:
        raise ValueError(f"ws: need a workspace on cuda:{dev}, got {ws.device}")
    _check(_lib.moe_grouped_gemm_mxfp4_room(a_codes.data_ptr(), a_scales.data_ptr(), R, _ptr(row_idx), M, w.desc_ref,
                                            cu_seqlens.data_ptr(), out.data_ptr(), _ptr(rows), room, ws.data_ptr(),
                                            ws.numel(), _launch_stream(dev, stream)), "moe_grouped_gemm_mxfp4")
    return out


def act_params(act: str = "silu", situ_alpha: float = 1.0, situ_beta: float = 1.0) -> moe_act_params_t:
    return moe_act_params_t(ACT[act], situ_alpha, situ_beta)


def moe_act_and_mul(gate, up, perm_w=None, act: str = "silu", situ_alpha=1.0, situ_beta=1.0, out=None,
                    stream=None):
    M, I = gate.shape
    out = out if out is not None else _on(stream, torch.empty_like, gate)
    _check(_lib.moe_act_and_mul(_ptr(gate), _ptr(up), _ptr(perm_w), M, I,
                                act_params(act, situ_alpha, situ_beta), _ptr(out), _stream(stream)),
           "moe_act_and_mul")
    return out


def act_ex(act: str = "silu", situ_alpha: float = 1.0, situ_beta: float = 1.0, swiglu_alpha: float = 1.702,
           swiglu_beta: float = 1.0, swiglu_limit: float | None = 7.0) -> moe_act_ex_t:
    """Activation and parameters; ``swiglu_limit=None`` means no clamp (+inf)."""
    lim = float("inf") if swiglu_limit is None else swiglu_limit
    return moe_act_ex_t(ACT[act], situ_alpha, situ_beta, swiglu_alpha, swiglu_beta, lim)


def moe_bias_act_and_mul(gate, up, cu_seqlens, bias_gate=None, bias_up=None, perm_w=None, act: str = "silu",
                         situ_alpha=1.0, situ_beta=1.0, swiglu_alpha=1.702, swiglu_beta=1.0, swiglu_limit=7.0,
                         out=None, stream=None):
    """S4 with per-expert biases (fp32 [G,I]) and any activation, SWIGLUOAI included. gate/up
    bf16 or fp32 [M,I]; bf16 out [M,I]; rows past cu_seqlens[-1] come out zero."""
    M, I = gate.shape
    out = out if out is not None else _on(stream, torch.empty, M, I, dtype=torch.bfloat16, device=gate.device)
    a = act_ex(act, situ_alpha, situ_beta, swiglu_alpha, swiglu_beta, swiglu_limit)
    _check(_lib.moe_bias_act_and_mul(_ptr(gate), _ptr(up), 1 if gate.dtype == torch.float32 else 0, _ptr(bias_gate),
                                     _ptr(bias_up), _ptr(cu_seqlens), cu_seqlens.numel(), _ptr(perm_w), M, I,
                                     ctypes.byref(a), _ptr(out), _stream(stream)), "moe_bias_act_and_mul")
    return out


def moe_combine(y_perm, inv_perm, topk_w=None, out=None, stream=None):
    T, k = inv_perm.shape
    H = y_perm.shape[1]
    out = out if out is not None else _on(stream, torch.empty, T, H, dtype=torch.bfloat16, device=y_perm.device)
    _check(_lib.moe_combine(_ptr(y_perm), _ptr(inv_perm), _ptr(topk_w), T, k, H, _ptr(out),
                            _stream(stream)), "moe_combine")
    return out


def moe_quantize_nvfp4(x: torch.Tensor, deq: bool = True, stream=None):
    R, K = x.shape
    dev = x.device
    codes = _on(stream, torch.empty, R, K // 2, dtype=torch.uint8, device=dev)
    sb = _on(stream, torch.empty, R, K // 16, dtype=torch.uint8, device=dev)
    s = _on(stream, torch.empty, R, dtype=torch.float32, device=dev)
    d = _on(stream, torch.empty, R, K, dtype=torch.float16, device=dev) if deq else None
    _check(_lib.moe_quantize_nvfp4(_ptr(x), 1 if x.dtype == torch.float32 else 0, R, K, _ptr(codes),
                                   _ptr(sb), _ptr(s), _ptr(d), _stream(stream)), "moe_quantize_nvfp4")
    return codes, sb, s, d


def moe_quantize_mxfp8(x: torch.Tensor, stream=None):
    """Dynamic MXFP8 quantisation of rows (bf16 or fp32 [R,K]): e4m3 codes [R,K] and e8m0
    scales [R,K/32]."""
    R, K = x.shape
    codes = _on(stream, torch.empty, R, K, dtype=torch.uint8, device=x.device)
    scales = _on(stream, torch.empty, R, K // 32, dtype=torch.uint8, device=x.device)
    _check(_lib.moe_quantize_mxfp8(_ptr(x), 1 if x.dtype == torch.float32 else 0, R, K, _ptr(codes), _ptr(scales),
                                   _stream(stream)), "moe_quantize_mxfp8")
    return codes, scales


def moe_quantize_mxfp4(x: torch.Tensor, deq: bool = False, out=None, stream=None):
    """MXFP4 quantisation of rows (bf16 or fp32 [R,K], rows a multiple of 8 elements apart): packed e2m1 codes [R,K/2],
    e8m0 scales [R,K/32] and, with deq, the bf16 values they stand for [R,K] (else None). ``out``:
    optional dict of caller-allocated outputs (any of codes, scales, deq)."""
    R, K = x.shape
    dev = _launch_device(x)
    out = out or {}
    xt = _float_type(x, "x")
    stride = _want(x, "x", (R, K), xt, dev, False) or K
    codes, _ = _output(out, "codes", x, (R, K // 2), torch.uint8, dev, stream)
    scales, _ = _output(out, "scales", x, (R, K // 32), torch.uint8, dev, stream)
    d = _output(out, "deq", x, (R, K), torch.bfloat16, dev, stream)[0] if deq else None
    _check(_lib.moe_quantize_mxfp4(x.data_ptr(), xt is torch.float32, stride, R, K, codes.data_ptr(), scales.data_ptr(),
                                   _ptr(d), _launch_stream(dev, stream)), "moe_quantize_mxfp4")
    return codes, scales, d


def forward_workspace(T_max, H, I, E, B, topk, wfmt="bf16", act_quant=0, device="cuda") -> torch.Tensor:
    n = _lib.moe_forward_workspace_size(T_max, H, I, E, B, topk, WFMT[wfmt], act_quant)
    return torch.zeros(n, dtype=torch.uint8, device=device)


class MoEForward:
    """The fused layer with its weights and a pre-sized workspace (no per-call allocation
    besides the output, which the caller may also pass)."""

    def __init__(self, w_gate: Weight, w_up: Weight, w_down: Weight, E: int, topk: int, B: int = 0,
                 replica_src=None, act: str = "silu", situ_alpha=1.0, situ_beta=1.0,
                 act_quant: int = 0, apply_topk_in_fc1: bool = True, T_max: int = 1,
                 routing: str = "renormalize", routing_bias=None, n_group: int = 1, topk_group: int = 1,
                 routed_scaling_factor: float = 1.0, apply_router_weight_on_input: bool = False,
                 swiglu_alpha: float = 1.702, swiglu_beta: float = 1.0, swiglu_limit: float | None = 7.0,
                 biases=None):
        """``biases``: None, or (bias_gate [E+B,I], bias_up [E+B,I], bias_down [E+B,H]) fp32
        device tensors, each of which may be None; the GEMMs' epilogues apply them."""
        for w in (w_gate, w_up, w_down):
            if w.fmt != "bf16" and w.prepared is None:
                moe_prepare_weights(w)
        self.w_gate, self.w_up, self.w_down = w_gate, w_up, w_down
        self.E, self.topk, self.B = E, topk, B
        self.H, self.I = w_gate.K, w_gate.N
        self.replica_src = replica_src
        self.act = act_params(act, situ_alpha, situ_beta)
        self.act_quant = act_quant
        self.apply_topk_in_fc1 = apply_topk_in_fc1
        self.T_max = T_max
        self.args = moe_forward_args_t()
        a = self.args
        a.swiglu_alpha, a.swiglu_beta = swiglu_alpha, swiglu_beta
        a.swiglu_limit = float("inf") if swiglu_limit is None else swiglu_limit
        self.biases = tuple(biases) if biases is not None else (None, None, None)
        a.bias_gate, a.bias_up, a.bias_down = (_ptr(b) for b in self.biases)
        if act == "swigluoai" or any(b is not None for b in self.biases):
            a.T_max, a.H, a.I, a.E, a.B, a.topk = T_max, self.H, self.I, E, B, topk
            a.w_gate, a.act, a.act_quant = w_gate.desc, self.act, act_quant
            n = _lib.moe_forward_workspace_size_args(ctypes.byref(a))
            self.ws = torch.zeros(n, dtype=torch.uint8, device=w_gate.data.device)
        else:
            self.ws = forward_workspace(T_max, self.H, self.I, E, B, topk, w_gate.fmt, act_quant,
                                        w_gate.data.device)
        self._made_on = torch.cuda.current_stream(self.ws.device) if self.ws.is_cuda else None
        self.args.routing = ROUTING[routing]
        self.routing_bias = routing_bias
        self.args.n_group, self.args.topk_group = n_group, topk_group
        self.args.routed_scaling_factor = routed_scaling_factor
        self.args.apply_router_weight_on_input = 1 if apply_router_weight_on_input else 0

    def __call__(self, x, router_logits=None, out=None, topk_ids=None, topk_w=None, stream=None,
                 stage_events=None, topk_ids_in=None, topk_w_in=None):
        """``stage_events``: None, or a list of MOE_FWD_STAGE_EVENTS entries, each None (not
        recorded) or a torch.cuda.Event created with enable_timing and recorded once (so that
        its handle exists). ``topk_ids_in``/``topk_w_in``: the given top-k of routing "given"."""
        T = x.shape[0]
        if stage_events is not None:
            if len(stage_events) != MOE_FWD_STAGE_EVENTS:
                raise ValueError(f"need {MOE_FWD_STAGE_EVENTS} events")
            self._ev = (ctypes.c_void_p * MOE_FWD_STAGE_EVENTS)(
                *[None if e is None else e.cuda_event for e in stage_events])
            self.args.stage_events = ctypes.cast(self._ev, ctypes.c_void_p)
        else:
            self.args.stage_events = None
        out = out if out is not None else _on(stream, torch.empty, T, self.H, dtype=torch.bfloat16, device=x.device)
        if stream is not None:
            if self._made_on is not None and not torch.cuda.is_current_stream_capturing():
                self._made_on.synchronize()  # the workspace is free and zeroed before another stream has it
                self._made_on = None
            self.ws.record_stream(stream)  # and not handed out again before this call is done
        a = self.args
        a.x, a.router_logits = _ptr(x), _ptr(router_logits)
        a.T, a.H, a.I, a.E, a.B, a.topk = T, self.H, self.I, self.E, self.B, self.topk
        a.replica_src = _ptr(self.replica_src)
        a.w_gate, a.w_up, a.w_down = self.w_gate.desc, self.w_up.desc, self.w_down.desc
        a.act = self.act
        a.apply_topk_in_fc1 = 1 if self.apply_topk_in_fc1 else 0
        a.act_quant = self.act_quant
        a.out = _ptr(out)
        a.topk_ids_out, a.topk_w_out = _ptr(topk_ids), _ptr(topk_w)
        a.T_max = self.T_max
        a.routing_bias = _ptr(self.routing_bias)
        a.topk_ids_in, a.topk_w_in = _ptr(topk_ids_in), _ptr(topk_w_in)
        _check(_lib.moe_forward(ctypes.byref(a), _ptr(self.ws), self.ws.numel(), _stream(stream)),
               "moe_forward")
        return out

    def device_error(self, stream=None) -> int:
        return _lib.moe_get_device_error(_ptr(self.ws), _stream(stream))

    def graph(self, x, router_logits=None, out=None, warmup: int = 1, **kw):
        """One forward on these buffers captured into a CUDA graph; ``graph.replay()`` reruns the
        layer on whatever x / router_logits (and the given top-k, if any) then hold and writes
        ``out``. ``warmup`` eager calls on a side stream come first: they also set the library's
        one-time host state (kernel attributes, the SM count), which must not be set up during
        capture. Returns ``(graph, out)``."""
        T = x.shape[0]
        out = out if out is not None else torch.empty(T, self.H, dtype=torch.bfloat16, device=x.device)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(warmup):
                self(x, router_logits, out=out, **kw)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self(x, router_logits, out=out, **kw)
        return g, out


def moe_forward(x, router_logits, w_gate: Weight, w_up: Weight, w_down: Weight, E: int, topk: int,
                B: int = 0, replica_src=None, act="silu", situ_alpha=1.0, situ_beta=1.0, act_quant=0,
                apply_topk_in_fc1=True, topk_ids=None, topk_w=None):
    layer = MoEForward(w_gate, w_up, w_down, E, topk, B, replica_src, act, situ_alpha, situ_beta,
                       act_quant, apply_topk_in_fc1, T_max=max(1, x.shape[0]))
    out = layer(x, router_logits, topk_ids=topk_ids, topk_w=topk_w)
    return out, layer


def moe_get_device_error(ws: torch.Tensor | None = None, stream=None) -> int:
    """Waits for the stream, then reads and clears the error word of a workspace; without one, that of the
    calls on the current device that were given no workspace (moe_grouped_gemm_mxfp4 and _nvfp4)."""
    if ws is None:
        ws = _error_word(torch.cuda.current_device())
    return _lib.moe_get_device_error(_ptr(ws), _stream(stream))
