"""Python binding of liblmoe, the sm_100a LatentMoE layer-forward library.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels (include/lmoe.h).  PyTorch supplies device memory and streams.  The
functions keep the C names; ``LatentMoE`` is a small convenience wrapper that
owns a handle and a cached workspace and returns the four outputs of the
"Stable LatentMoE" contract as a dict.

Importing fails loudly (ImportError) when the library has not been built:
``python latent_space_routed_b200/build.py``.  There is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading
from typing import Dict, NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "liblmoe.so")

LMOE_OK, LMOE_ERR_INVALID_ARG, LMOE_ERR_UNSUPPORTED, LMOE_ERR_OOM, LMOE_ERR_CUDA, LMOE_ERR_DEVICE_TIMEOUT, \
    LMOE_ERR_WORKSPACE = range(7)
LMOE_F32, LMOE_BF16 = 0, 1
LMOE_ACT_SWIGLU, LMOE_ACT_SITU = 0, 1

STATUS_NAMES = {0: "LMOE_OK", 1: "LMOE_ERR_INVALID_ARG", 2: "LMOE_ERR_UNSUPPORTED", 3: "LMOE_ERR_OOM",
                4: "LMOE_ERR_CUDA", 5: "LMOE_ERR_DEVICE_TIMEOUT", 6: "LMOE_ERR_WORKSPACE"}

# lmoe_workspace_region ids
REGION = {"scores": 0, "p32": 1, "counts": 2, "offsets": 3, "slot_of": 4, "perm_tok": 5, "Z": 6, "H": 7,
          "Y": 8, "HS": 9, "status": 10, "cutoff": 11, "Zp": 12, "Zp4": 13, "Zp4_scales": 14, "H4": 15, "H4_scales": 16}

EXPORTS = ("lmoe_config_from_base", "lmoe_create", "lmoe_workspace_size", "lmoe_forward", "lmoe_host_workspace_size",
           "lmoe_forward_host", "lmoe_forward_noalloc", "lmoe_create_mx4", "lmoe_few_workspace_size", "lmoe_forward_few",
           "lmoe_mx4_quantize", "lmoe_mx4_dequantize", "lmoe_mx4_gemm", "lmoe_mx4_gemm_check", "lmoe_debug_inject", "lmoe_set_bias", "lmoe_qb_histogram", "lmoe_qb_bias_update", "lmoe_set_stage_events", "lmoe_launch_count", "lmoe_workspace_region", "lmoe_check_device", "lmoe_check_device_host",
           "lmoe_last_error", "lmoe_destroy")


class LmoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class lmoe_config(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("l", ctypes.c_int32), ("f", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("f_shared", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("eps", ctypes.c_float), ("dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("gate_cap", ctypes.c_float), ("up_cap", ctypes.c_float), ("gemm", ctypes.c_int32),
                ("standard", ctypes.c_int32)]


class lmoe_mx4_experts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("G", "G_scales", "U", "U_scales", "D", "D_scales")]


class lmoe_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("W_r", "b", "W_down", "W_up", "G", "U", "D", "Gs", "Us", "Ds")]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python latent_space_routed_b200/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "lmoe_config_from_base": (I32, [I32, I32, I32, I32, I32, I32, ctypes.c_char_p, ctypes.POINTER(lmoe_config)]),
        "lmoe_create": (I32, [ctypes.POINTER(lmoe_config), ctypes.POINTER(lmoe_weights), P, ctypes.POINTER(P)]),
        "lmoe_create_mx4": (I32, [ctypes.POINTER(lmoe_config), ctypes.POINTER(lmoe_weights),
                                  ctypes.POINTER(lmoe_mx4_experts), P, ctypes.POINTER(P)]),
        "lmoe_few_workspace_size": (I32, [P, I64, ctypes.POINTER(SZ)]),
        "lmoe_forward_few": (I32, [P, P, I64, P, P, P, P, P, SZ, P]),
        "lmoe_mx4_quantize": (I32, [P, I32, I64, I64, I64, P, P, P]),
        "lmoe_mx4_gemm": (I32, [P, P, I64, P, P, I64, I64, P, I32, I32, P, I64, P, SZ, P]),
        "lmoe_mx4_gemm_check": (I32, [P, P]),
        "lmoe_mx4_dequantize": (I32, [P, P, I64, I64, I32, P, I64, P]),
        "lmoe_workspace_size": (I32, [P, I64, ctypes.POINTER(SZ)]),
        "lmoe_forward": (I32, [P, P, I64, P, P, P, P, P, SZ, P]),
        "lmoe_host_workspace_size": (I32, [P, I64, ctypes.POINTER(SZ)]),
        "lmoe_forward_host": (I32, [P, P, I64, P, P, P, P, P, SZ, P]),
        "lmoe_forward_noalloc": (I32, [P, P, I64, P, P, P, P, P]),
        "lmoe_debug_inject": (I32, [I32, I32]),
        "lmoe_set_bias": (I32, [P, P, P]),
        "lmoe_qb_histogram": (I32, [P, P, I64, I32, ctypes.c_float, ctypes.c_float, P, P]),
        "lmoe_qb_bias_update": (I32, [P, P, I32, ctypes.c_float, ctypes.c_float, I64, P, P]),
        "lmoe_set_stage_events": (I32, [P, P, I32]),
        "lmoe_launch_count": (I32, [P, I64, ctypes.POINTER(I32)]),
        "lmoe_workspace_region": (I32, [P, I64, I32, ctypes.POINTER(SZ), ctypes.POINTER(SZ)]),
        "lmoe_check_device": (I32, [P, I64, P, P]),
        "lmoe_check_device_host": (I32, [P, I64, P, P]),
        "lmoe_last_error": (ctypes.c_char_p, []),
        "lmoe_destroy": (None, [P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def _check(status: int):
    if status != LMOE_OK:
        raise LmoeError(status, _lib.lmoe_last_error().decode())


_cuda_available = functools.lru_cache(maxsize=None)(torch.cuda.is_available)


def _stream(stream) -> Optional[int]:
    if stream is None:      # (the raw handle: a Stream object costs microseconds per call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()) if _cuda_available() else None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr()
    return int(t)


# ------------------------------------------------------------------ C names
def lmoe_last_error() -> str:
    return _lib.lmoe_last_error().decode()


def lmoe_config_from_base(d, m, N, K, alpha, n_shared, variant) -> lmoe_config:
    cfg = lmoe_config()
    _check(_lib.lmoe_config_from_base(d, m, N, K, alpha, n_shared, variant.encode(), ctypes.byref(cfg)))
    return cfg


def make_config(d, l, f, E, k, f_shared, n_shared=2, eps=1e-6, dtype=LMOE_BF16, act=LMOE_ACT_SWIGLU,
                gate_cap=4.0, up_cap=25.0, gemm=0, standard=0) -> lmoe_config:
    return lmoe_config(d, l, f, E, k, f_shared, n_shared, eps, dtype, act, gate_cap, up_cap, gemm, standard)


def lmoe_create(cfg: lmoe_config, weights: Dict[str, torch.Tensor], stream=None) -> int:
    w = lmoe_weights(*[_ptr(weights.get(n)) for n in ("W_r", "b", "W_down", "W_up", "G", "U", "D", "Gs", "Us", "Ds")])
    h = ctypes.c_void_p()
    _check(_lib.lmoe_create(ctypes.byref(cfg), ctypes.byref(w), _stream(stream), ctypes.byref(h)))
    return h.value


def lmoe_create_mx4(cfg: lmoe_config, weights: Dict[str, torch.Tensor], experts: Dict[str, "Mx4"], stream=None) -> int:
    w = lmoe_weights(*[_ptr(weights.get(n)) if n not in ("G", "U", "D") else None
                       for n in ("W_r", "b", "W_down", "W_up", "G", "U", "D", "Gs", "Us", "Ds")])
    x4 = lmoe_mx4_experts(*[_ptr(t) for n in ("G", "U", "D") for t in (experts[n].codes, experts[n].scales)])
    h = ctypes.c_void_p()
    _check(_lib.lmoe_create_mx4(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(x4), _stream(stream), ctypes.byref(h)))
    return h.value


def lmoe_few_workspace_size(h: int, T: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.lmoe_few_workspace_size(h, T, ctypes.byref(n)))
    return n.value


def lmoe_forward_few(h, x, T, output, selected_experts, mixture_weights, latent_routed_aggregate, workspace, ws_bytes,
                     stream=None):
    _check(_lib.lmoe_forward_few(h, _ptr(x), T, _ptr(output), _ptr(selected_experts), _ptr(mixture_weights),
                                 _ptr(latent_routed_aggregate), _ptr(workspace), ws_bytes, _stream(stream)))


def lmoe_mx4_quantize(x, dtype, rows, cols, ld, codes, scales, stream=None):
    _check(_lib.lmoe_mx4_quantize(_ptr(x), dtype, rows, cols, ld, _ptr(codes), _ptr(scales), _stream(stream)))


def lmoe_mx4_dequantize(codes, scales, rows, cols, dtype, y, ld, stream=None):
    _check(_lib.lmoe_mx4_dequantize(_ptr(codes), _ptr(scales), rows, cols, dtype, _ptr(y), ld, _stream(stream)))


LMOE_MX4_GEMM_WORKSPACE_BYTES = 256


def lmoe_mx4_gemm(a_codes, a_scales, M, w_codes, w_scales, N, K, offsets, E, dtype, out, ldo, workspace, ws_bytes,
                  stream=None):
    _check(_lib.lmoe_mx4_gemm(_ptr(a_codes), _ptr(a_scales), M, _ptr(w_codes), _ptr(w_scales), N, K, _ptr(offsets), E,
                              dtype, _ptr(out), ldo, _ptr(workspace), ws_bytes, _stream(stream)))


def lmoe_mx4_gemm_check(workspace, stream=None):
    _check(_lib.lmoe_mx4_gemm_check(_ptr(workspace), _stream(stream)))


def lmoe_destroy(h: int):
    _lib.lmoe_destroy(h)


def lmoe_workspace_size(h: int, T: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.lmoe_workspace_size(h, T, ctypes.byref(n)))
    return n.value


def lmoe_host_workspace_size(h: int, T: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.lmoe_host_workspace_size(h, T, ctypes.byref(n)))
    return n.value


def lmoe_forward(h, x, T, output, selected_experts, mixture_weights, latent_routed_aggregate, workspace, ws_bytes,
                 stream=None):
    _check(_lib.lmoe_forward(h, _ptr(x), T, _ptr(output), _ptr(selected_experts), _ptr(mixture_weights),
                             _ptr(latent_routed_aggregate), _ptr(workspace), ws_bytes, _stream(stream)))


def lmoe_forward_host(h, x_host, T, output_host, selected_experts_host, mixture_weights_host,
                      latent_routed_aggregate_host, workspace, ws_bytes, stream=None):
    _check(_lib.lmoe_forward_host(h, _ptr(x_host), T, _ptr(output_host), _ptr(selected_experts_host),
                                  _ptr(mixture_weights_host), _ptr(latent_routed_aggregate_host), _ptr(workspace),
                                  ws_bytes, _stream(stream)))


LMOE_NOALLOC_WORKSPACE_BYTES = 64 << 20
LMOE_INJECT_STALL_NEXT_GEMM, LMOE_INJECT_FAIL_ALLOC, LMOE_INJECT_STALL_NEXT_FEW, LMOE_INJECT_STALL_NEXT_MX4 = 1, 2, 3, 4
LMOE_FEW_MAX_T = 8


def lmoe_debug_inject(what, arg=0):
    """Failure-detection test hooks (see include/lmoe.h)."""
    _check(_lib.lmoe_debug_inject(what, arg))



def lmoe_forward_noalloc(h, x, T, output, selected_experts, mixture_weights, latent_routed_aggregate, stream=None):
    """lmoe_forward on the library's built-in 64 MiB scratch area (no caller
    workspace, no allocation); see include/lmoe.h for its rules."""
    _check(_lib.lmoe_forward_noalloc(h, _ptr(x), T, _ptr(output), _ptr(selected_experts), _ptr(mixture_weights),
                                     _ptr(latent_routed_aggregate), _stream(stream)))


def lmoe_set_bias(h, b, stream=None):
    _check(_lib.lmoe_set_bias(h, _ptr(b), _stream(stream)))


def lmoe_qb_histogram(h, workspace, T, bins, lo, hi, hist, stream=None):
    _check(_lib.lmoe_qb_histogram(h, _ptr(workspace), T, bins, lo, hi, _ptr(hist), _stream(stream)))


def lmoe_qb_bias_update(h, hist, bins, lo, hi, target, bias_out, stream=None):
    _check(_lib.lmoe_qb_bias_update(h, _ptr(hist), bins, lo, hi, target, _ptr(bias_out), _stream(stream)))


LMOE_NUM_STAGES = 11
STAGE_NAMES = ("router", "topk", "scan", "dispatch", "down_proj", "permute", "gate_up", "down_combine",
               "combine_norm", "shared_gate_up", "final")


def lmoe_set_stage_events(h, events, n):
    """events: a ctypes array of cudaEvent_t handles (kept alive by the caller), or None."""
    _check(_lib.lmoe_set_stage_events(h, events, n))


def lmoe_launch_count(h, T) -> int:
    n = ctypes.c_int32()
    _check(_lib.lmoe_launch_count(h, T, ctypes.byref(n)))
    return n.value


def lmoe_workspace_region(h, T, region):
    off, n = ctypes.c_size_t(), ctypes.c_size_t()
    rid = REGION[region] if isinstance(region, str) else int(region)
    _check(_lib.lmoe_workspace_region(h, T, rid, ctypes.byref(off), ctypes.byref(n)))
    return off.value, n.value


def lmoe_check_device(h, T, workspace, stream=None):
    _check(_lib.lmoe_check_device(h, T, _ptr(workspace), _stream(stream)))


def lmoe_check_device_host(h, T, workspace, stream=None):
    _check(_lib.lmoe_check_device_host(h, T, _ptr(workspace), _stream(stream)))


# ------------------------------------------------------------------ convenience wrapper
_TORCH_DT = {LMOE_F32: torch.float32, LMOE_BF16: torch.bfloat16}


_LM_DT = {torch.float32: LMOE_F32, torch.bfloat16: LMOE_BF16}


class Mx4(NamedTuple):
    """A microscaled 4-bit tensor (see include/lmoe.h): codes [..., cols / 2] and scales [..., cols / 32], uint8."""
    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def shape(self):
        return (*self.codes.shape[:-1], 2 * self.codes.shape[-1])

    def check(self, what: str, device: Optional[torch.device] = None) -> "Mx4":
        c, s = self.codes, self.scales
        if c.dtype != torch.uint8 or s.dtype != torch.uint8:
            raise TypeError(f"{what}: codes and scales must be uint8, got {c.dtype} and {s.dtype}")
        if c.dim() < 1 or c.shape[-1] % 16 or tuple(s.shape) != (*c.shape[:-1], c.shape[-1] // 16):
            raise ValueError(f"{what}: codes [..., cols / 2] and scales [..., cols / 32] do not match: "
                             f"{tuple(c.shape)}, {tuple(s.shape)}")
        if not c.is_cuda or c.device != s.device:
            raise ValueError(f"{what}: codes and scales must be on one CUDA device")
        if device is not None and c.device != device:
            raise ValueError(f"{what} must be on {device}, not {c.device}")
        if not c.is_contiguous() or not s.is_contiguous():
            raise ValueError(f"{what}: codes and scales must be contiguous")
        return self


def _with(device, stream):
    """`device` and `stream`, where they are not the current ones, made current for what is inside: copies and
    allocations are then ordered with the kernel."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            handle = _stream(stream)
            stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        return torch.cuda.stream(stream)
    return contextlib.nullcontext() if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def mx4_quantize(x: torch.Tensor, stream=None) -> Mx4:
    """x [..., cols] (fp32 or bf16 on a CUDA device, cols a multiple of 32) in 4 bits."""
    if x.dtype not in _LM_DT:
        raise TypeError(f"fp32 or bf16 expected, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError("x must be on a CUDA device")
    if x.dim() < 1:
        raise ValueError("x needs a last dimension")
    cols, lead = x.shape[-1], x.shape[:-1]
    if cols % 32:
        raise ValueError(f"the last dimension {cols} is not a multiple of 32")
    per16 = 16 // x.element_size()
    with _with(x.device, stream):
        # a matrix whose rows are whole and 16-byte aligned is read as it lies; anything else is laid out first
        x2 = x if x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= cols and x.stride(0) % per16 == 0 \
            else x.reshape(-1, cols).contiguous() if x.numel() else x
        if x2.data_ptr() % 16:
            x2 = x2.clone(memory_format=torch.contiguous_format)
        q = Mx4(torch.empty((*lead, cols // 2), dtype=torch.uint8, device=x.device),
                torch.empty((*lead, cols // 32), dtype=torch.uint8, device=x.device))
        if x.numel():
            lmoe_mx4_quantize(x2, _LM_DT[x.dtype], x2.shape[0], cols, x2.stride(0) if x2.shape[0] > 1 else cols,
                              q.codes, q.scales)
    return q


def mx4_dequantize(q: Mx4, dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The values of a 4-bit tensor, exact in either type."""
    if dtype not in _LM_DT:
        raise TypeError(f"fp32 or bf16 expected, got {dtype}")
    q.check("q")
    cols = 2 * q.codes.shape[-1]
    with _with(q.codes.device, stream):
        y = torch.empty(q.shape, dtype=dtype, device=q.codes.device)
        if y.numel():
            lmoe_mx4_dequantize(q.codes, q.scales, y.numel() // cols, cols, _LM_DT[dtype], y, cols)
    return y


def mx4_gemm_workspace(device=None) -> torch.Tensor:
    """A workspace for mx4_gemm calls that follow one another on one stream."""
    return torch.zeros(LMOE_MX4_GEMM_WORKSPACE_BYTES, dtype=torch.uint8,
                       device=torch.device("cuda", torch.cuda.current_device()) if device is None else device)


# status words of mx4_gemm calls without a workspace: device index -> stream -> workspace
_mx4_words: Dict[int, Dict[int, torch.Tensor]] = {}


def _mx4_word(device: torch.device) -> torch.Tensor:
    """The status word of the current stream (of `device`).  Words only ever gain bits, so calls may share one; a
    captured call takes one that exists, since its own would be zeroed by every replay."""
    words = _mx4_words.setdefault(device.index, {})
    key = _stream(None)
    if key not in words:
        if torch.cuda.is_current_stream_capturing():
            return next(iter(words.values())) if words else mx4_gemm_workspace(device)
        words.setdefault(key, mx4_gemm_workspace(device))      # (two threads may be here)
    return words[key]


def mx4_gemm_check(device=None):
    """Wait for the device (the current one by default), then raise LmoeError (LMOE_ERR_DEVICE_TIMEOUT) if a bounded
    wait gave up in an mx4_gemm call on it that had no ``workspace``; their outputs are then invalid.  (A call that
    was captured before any other had been made on its device has no word here: give such a call a workspace.)"""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        torch.cuda.synchronize()
        failed = None
        for word in list(_mx4_words.get(torch.cuda.current_device(), {}).values()):
            try:
                lmoe_mx4_gemm_check(word)
            except LmoeError as e:
                failed = e
    if failed is not None:
        raise failed


def mx4_gemm(a: Mx4, w: Mx4, offsets: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
             out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """a [M, K] times w [N, K] transposed, in 4 bits with fp32 sums; with offsets [E + 1] (int32, on the device)
    rows offsets[e] to offsets[e + 1] of a times w[e] of w [E, N, K].  ``out`` [M, N] (its dtype counts then) may
    have a row stride; without it, rows that belong to no expert are zero.  ``mx4_gemm_check`` reports a wait that
    gave up, ``lmoe_mx4_gemm_check`` that of a call with a ``workspace``."""
    a.check("a"), w.check("w")
    if a.codes.dim() != 2 or w.codes.dim() != (2 if offsets is None else 3):
        raise ValueError("a must be [M, K] and w [N, K], or [E, N, K] with offsets")
    M, K = a.shape
    N = w.shape[-2]
    if w.shape[-1] != K:
        raise ValueError(f"K differs: {K} and {w.shape[-1]}")
    dev = a.codes.device
    E = 1 if offsets is None else w.shape[0]
    if offsets is not None and (offsets.dtype != torch.int32 or offsets.shape != (E + 1,) or offsets.device != dev
                                or not offsets.is_contiguous()):
        raise ValueError(f"offsets must be a contiguous int32 tensor [{E + 1}] on {dev}")
    if (dtype if out is None else out.dtype) not in _LM_DT:
        raise TypeError(f"fp32 or bf16 expected, got {dtype if out is None else out.dtype}")
    if out is None:
        make = torch.empty if offsets is None else torch.zeros
        with _with(dev, stream):
            out = make(M, N, dtype=dtype, device=dev)
    if out.shape != (M, N) or (N > 1 and out.stride(1) != 1) or (M > 1 and out.stride(0) < N):
        raise ValueError(f"out must be [{M}, {N}] with whole rows")
    if w.codes.device != dev or out.device != dev or (workspace is not None and workspace.device != dev):
        raise ValueError(f"all tensors must be on {dev}")
    with _with(dev, stream):
        ws = _mx4_word(dev) if workspace is None else workspace
        lmoe_mx4_gemm(a.codes, a.scales, M, w.codes, w.scales, N, K, offsets, E, _LM_DT[out.dtype], out,
                      out.stride(0) if M > 1 else N, ws, ws.numel() * ws.element_size())
    return out


class LatentMoE:
    """A LatentMoE layer on the current CUDA device.

    ``weights`` holds W_r [E, d] fp32, b [E] fp32, W_down [l, d], W_up [d, l],
    G, U [E, f, l], D [E, l, f], Gs, Us [2, f_s, d], Ds [2, d, f_s] (CUDA
    tensors; copied and repacked at construction, so they may be freed after).
    G, U and D may all be ``Mx4`` tensors of the same shapes: the routed experts
    are then held and computed in 4 bits.
    ``layer(x)`` with x [..., d] returns the dict of the "Stable LatentMoE"
    contract: output [..., d], selected_experts [..., k] int32,
    mixture_weights [..., k], latent_routed_aggregate [..., l].
    """

    def __init__(self, cfg: lmoe_config, weights: Dict[str, torch.Tensor], stream=None):
        self.cfg = cfg
        self.dtype = _TORCH_DT[cfg.dtype]
        dev = torch.device("cuda", torch.cuda.current_device())
        self.mx4 = any(isinstance(weights[n], Mx4) for n in ("G", "U", "D"))
        if self.mx4:
            shapes = {"G": (cfg.E, cfg.f, cfg.l), "U": (cfg.E, cfg.f, cfg.l), "D": (cfg.E, cfg.l, cfg.f)}
            for n, shape in shapes.items():
                if not isinstance(weights[n], Mx4):
                    raise TypeError("G, U and D must all be Mx4 tensors, or none of them")
                if weights[n].check(n, dev).shape != shape:
                    raise ValueError(f"{n}: shape {weights[n].shape} != {shape}")
        w = {}
        for n in ("W_r", "b", "W_down", "W_up", "G", "U", "D", "Gs", "Us", "Ds"):
            if cfg.standard and n in ("W_down", "W_up"):
                continue                 # the standard-MoE form has no projections
            if isinstance(weights[n], Mx4):
                continue
            want = torch.float32 if n in ("W_r", "b") else self.dtype
            w[n] = weights[n].to(device=dev, dtype=want).contiguous()
        if self.mx4:
            self.handle = lmoe_create_mx4(cfg, w, {n: weights[n] for n in shapes}, stream)
        else:
            self.handle = lmoe_create(cfg, w, stream)
        self.device = dev
        self._ws = None
        self._few_ws = {}
        self._captured_ws = []

    def close(self):
        if getattr(self, "handle", None):
            lmoe_destroy(self.handle)
            self.handle = None

    def __del__(self):  # pragma: no cover
        try:
            self.close()
        except Exception:
            pass

    def workspace(self, T: int, host: bool = False) -> torch.Tensor:
        n = lmoe_host_workspace_size(self.handle, T) if host else lmoe_workspace_size(self.handle, T)
        if self._ws is None or self._ws.numel() < n:
            self._ws = torch.empty(max(n, 256), dtype=torch.uint8, device=self.device)
        return self._ws

    def empty_outputs(self, T: int, device=None, pin: bool = False):
        c = self.cfg
        dev = self.device if device is None else device
        kw = dict(device=dev, pin_memory=pin) if str(dev) == "cpu" else dict(device=dev)
        return {"output": torch.empty(T, c.d, dtype=self.dtype, **kw),
                "selected_experts": torch.empty(T, c.k, dtype=torch.int32, **kw),
                "mixture_weights": torch.empty(T, c.k, dtype=self.dtype, **kw),
                "latent_routed_aggregate": torch.empty(T, c.l, dtype=self.dtype, **kw)}

    def forward_into(self, x: torch.Tensor, out: Dict[str, torch.Tensor], stream=None):
        T = x.shape[0]
        ws = self.workspace(T)
        lmoe_forward(self.handle, x, T, out["output"], out["selected_experts"], out["mixture_weights"],
                     out["latent_routed_aggregate"], ws, ws.numel(), stream)
        return out

    def few_workspace(self, T: int, stream=None) -> torch.Tensor:
        """The workspace that forward_few_into takes by itself for T tokens: one for each stream and thread, whose
        calls follow one another (two threads' calls on one stream may not: each is a memset and a kernel)."""
        key = (T, _stream(stream), threading.get_ident())
        ws = self._few_ws.get(key)
        if ws is None:
            ws = self._few_ws[key] = self._new_few_workspace(T, stream)
        return ws

    def _new_few_workspace(self, T: int, stream) -> torch.Tensor:
        with _with(self.device, stream):
            return torch.empty(max(lmoe_few_workspace_size(self.handle, T), 256), dtype=torch.uint8, device=self.device)

    def forward_few_into(self, x: torch.Tensor, out: Dict[str, torch.Tensor], workspace: Optional[torch.Tensor] = None,
                         stream=None):
        """The layer for x [T, d] of 1 to 8 tokens in one kernel, into the four output tensors (x that
        is not 16-byte aligned is copied first).

        ``workspace`` (``lmoe_few_workspace_size`` bytes) must not be shared by calls that may overlap on the
        GPU.  Without it, calls outside a capture use ``few_workspace``, and each captured call gets a buffer of
        its own, which the layer keeps (a graph may replay beside anything): give a graph of many calls one."""
        T, c, dev = x.shape[0], self.cfg, self.device
        if x.dim() != 2 or x.shape[1] != c.d or x.dtype != self.dtype or not x.is_contiguous() or x.device != dev:
            raise ValueError(f"x must be a contiguous {self.dtype} tensor [T, {c.d}] on {dev}")
        for name, cols, dtype in (("output", c.d, self.dtype), ("selected_experts", c.k, torch.int32),
                                  ("mixture_weights", c.k, self.dtype), ("latent_routed_aggregate", c.l, self.dtype)):
            t = out[name]
            if t.dtype != dtype or t.numel() < T * cols or not t.is_contiguous() or t.device != dev:
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of {T} x {cols} values or more on {dev}")
        if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be a contiguous tensor on {dev}")
        if x.data_ptr() % 16:
            with contextlib.nullcontext() if stream is None else _with(self.device, stream):
                x = x.clone()
        handle = _stream(stream)
        ws = self._few_workspace_of_call(T, stream, handle) if workspace is None else workspace
        lmoe_forward_few(self.handle, x, T, out["output"], out["selected_experts"], out["mixture_weights"],
                         out["latent_routed_aggregate"], ws, ws.numel() * ws.element_size(), handle)
        return out

    def _few_workspace_of_call(self, T: int, stream, handle: int) -> torch.Tensor:
        if stream is None:
            capturing = torch.cuda.is_current_stream_capturing()
        else:
            with _with(self.device, stream):
                capturing = torch.cuda.is_current_stream_capturing()
        if not capturing:
            ws = self._few_ws.get((T, handle, threading.get_ident()))
            return self.few_workspace(T, stream) if ws is None else ws
        self._captured_ws.append(self._new_few_workspace(T, stream))
        return self._captured_ws[-1]

    def forward_few(self, x: torch.Tensor, stream=None) -> Dict[str, torch.Tensor]:
        """``layer(x)`` for at most 8 tokens, in one kernel."""
        return self._call(x, self.forward_few_into, stream)

    def _call(self, x: torch.Tensor, forward_into, stream) -> Dict[str, torch.Tensor]:
        c = self.cfg
        if x.shape[-1] != c.d:
            raise ValueError(f"last dim {x.shape[-1]} != d={c.d}")
        lead = x.shape[:-1]
        with contextlib.nullcontext() if stream is None else _with(self.device, stream):
            x2 = x.reshape(-1, c.d).to(device=self.device, dtype=self.dtype).contiguous()
            out = forward_into(x2, self.empty_outputs(x2.shape[0]), stream=stream)
        return {"output": out["output"].reshape(*lead, c.d),
                "selected_experts": out["selected_experts"].reshape(*lead, c.k),
                "mixture_weights": out["mixture_weights"].reshape(*lead, c.k),
                "latent_routed_aggregate": out["latent_routed_aggregate"].reshape(*lead, c.l)}

    def __call__(self, x: torch.Tensor, stream=None) -> Dict[str, torch.Tensor]:
        return self._call(x, self.forward_into, stream)

    def forward_host(self, x_host: torch.Tensor, out_host: Dict[str, torch.Tensor], stream=None):
        """Host buffers in and out (pinned for async copies); copies are inside the library call."""
        T = x_host.shape[0]
        ws = self.workspace(T, host=True)
        lmoe_forward_host(self.handle, x_host, T, out_host["output"], out_host["selected_experts"],
                          out_host["mixture_weights"], out_host["latent_routed_aggregate"], ws, ws.numel(), stream)
        return out_host

    def region(self, T: int, name: str, dtype: torch.dtype, shape) -> torch.Tensor:
        """View of one intermediate in the workspace of the last forward of T tokens."""
        off, n = lmoe_workspace_region(self.handle, T, name)
        ws = self.workspace(T)
        return ws[off:off + n].view(dtype).reshape(shape)

    def check_device(self, T: int, stream=None):
        lmoe_check_device(self.handle, T, self.workspace(T), stream)

    def check_device_host(self, T: int, stream=None):
        """lmoe_check_device after forward_host of T tokens."""
        lmoe_check_device_host(self.handle, T, self.workspace(T, host=True), stream)

    def launch_count(self, T: int) -> int:
        return lmoe_launch_count(self.handle, T)

    def set_bias(self, b: torch.Tensor, stream=None):
        """Replace the selection bias with b [E] (device fp32)."""
        lmoe_set_bias(self.handle, b, stream)

    def qb_histogram(self, T: int, hist: torch.Tensor, bins: int, lo: float, hi: float, stream=None):
        """Add the last forward's (T tokens) Quantile-Balancing margin histogram to hist [E, bins] int32."""
        lmoe_qb_histogram(self.handle, self.workspace(T), T, bins, lo, hi, hist, stream)
        return hist

    def qb_bias_update(self, hist: torch.Tensor, bins: int, lo: float, hi: float, target: int, stream=None):
        """The next step's bias [E] fp32 from an accumulated histogram (apply with set_bias)."""
        out = torch.empty(self.cfg.E, dtype=torch.float32, device=self.device)
        lmoe_qb_bias_update(self.handle, hist, bins, lo, hi, target, out, stream)
        return out


def config_for(workload, gemm: int = 0, act: int = LMOE_ACT_SWIGLU) -> lmoe_config:
    """lmoe_config from an lmoe_inputs.Workload."""
    return make_config(workload.d, workload.l, workload.f, workload.E, workload.k, workload.f_s,
                       workload.n_shared, workload.eps, LMOE_F32 if workload.dtype == "f32" else LMOE_BF16, act,
                       4.0, 25.0, gemm, 1 if getattr(workload, "standard", False) else 0)
