"""Four-over-six NVFP4 quantization for AMD MI355X (gfx950).

Python binding of the HIP library ``libfos.so`` (C ABI in ``include/fos.h``).
The functions carry the C entry points' names and only marshal arguments:
PyTorch supplies device memory (outputs are ``torch.empty`` on the input's
device) and the current stream; every step of the quantizer runs in the HIP
kernels. There is no fallback: if the library is missing or the device is not
a gfx950, the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfos.so")

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
RECIPES = {"nvfp4": 0, "4over6": 1}
BLOCKS = {"1x16": 0, "16x16": 1}
GRANS = {"tensor": 0, "row": 1}
METRICS = {"mae": 0, "mse": 1}
PRECS = {"exact": 0, "fp16": 1}
ORDERS = {"tree": 0, "seq": 1}
AMAX_GRANS = {"tensor": 0, "row": 1, "band16": 2}
OPERAND_GRANS = {"tensor": 0, "row": 1, "group": 2}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
OPERAND_E4M3, OPERAND_NVFP4 = 3, 4  # FOS_E4M3, FOS_NVFP4

STATUS_TILE_NONUNIFORM = 1
STATUS_BAD_OFFS = 2
STATUS_BARRIER_TIMEOUT = 4
STATUS_BAD_INDEX = 8
STATUS_BAD_CACHE = 16
FUSED_WORKSPACE_BYTES = 16384  # FOS_FUSED_WORKSPACE_BYTES
FUSED_MAX_GROUPS = 256  # FOS_FUSED_MAX_GROUPS


class FosError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"fos error {code}: {msg}")
        self.code = code


class _Config(ctypes.Structure):
    _fields_ = [("recipe", ctypes.c_int32), ("block", ctypes.c_int32), ("scale_gran", ctypes.c_int32),
                ("err_metric", ctypes.c_int32), ("err_prec", ctypes.c_int32), ("e4m3_bound", ctypes.c_int32),
                ("err_order", ctypes.c_int32)]


class _Desc(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("amax", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("K", ctypes.c_int64)]


class _Operand(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("block_scales", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("type", ctypes.c_int32), ("gran", ctypes.c_int32)]


class _Epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("bias_dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


_P = ctypes.c_void_p
_F = ctypes.c_float
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SIGS = {
    "fos_abi_version": (_I, []),
    "fos_status_string": (ctypes.c_char_p, [_I]),
    "fos_last_error": (ctypes.c_char_p, []),
    "fos_set_barrier_poll_limit": (_I, [_I]),
    "fos_set_phase_timestamps": (_I, [_P, _I64, _P]),
    "fos_amax": (_I, [_P, _I, _I64, _I64, _I, _P, _P]),
    "fos_quantize": (_I, [_P, _I, _I64, _I64, _P, ctypes.POINTER(_Config), _P, _P, _P, _P, _P]),
    "fos_qdq": (_I, [_P, _I, _I64, _I64, _P, ctypes.POINTER(_Config), _P, _P]),
    "fos_qdq_list": (_I, [_I, _P, _I, ctypes.POINTER(_Config), _P]),
    "fos_qdq_list_fused": (_I, [_I, _P, _I, ctypes.POINTER(_Config), _P, _P, _P, _P]),
    "nvfp4_dequantize": (_I, [_P, _P, _I64, _I64, _P, _I, _I, _P, _P]),
    "fos_quantize_grouped": (_I, [_P, _I, _I64, _I64, _P, _I, _P, ctypes.POINTER(_Config), _P, _P, _P, _P, _P]),
    "fos_quantize_fused": (_I, [_P, _I, _I64, _I64, ctypes.POINTER(_Config), _P, _P, _P, _P, _P, _P, _P]),
    "fos_qdq_fused": (_I, [_P, _I, _I64, _I64, ctypes.POINTER(_Config), _P, _P, _P, _P, _P]),
    "fos_quantize_columnwise": (_I, [_P, _I, _I64, _I64, _P, ctypes.POINTER(_Config), _P, _P, _P, _P]),
    "fos_quantize_grouped_fused": (_I, [_P, _I, _I64, _I64, _P, _I, ctypes.POINTER(_Config), _P, _P, _P, _P, _P, _P,
                                        _P]),
    "fos_quantize_grouped_fused_noalloc": (_I, [_P, _I, _I64, _I64, _P, _I, ctypes.POINTER(_Config), _P, _P, _P, _P,
                                                _P, _P]),
    "fos_linear_workspace": (_I64, [_I64, _I64, _I64, _I]),
    "fos_linear": (_I, [_P, _P, _I64, _I64, _I64, _P, _P, _I, _P, _I64, _P]),
    "fos_linear_grouped": (_I, [_P, _P, _P, _I, _I64, _I64, _I64, _P, _P, _I, _P, _I64, _P, _P]),
    "fos_rmsnorm_quantize": (_I, [_P, _I, _I64, _I64, _P, _P, _I, _F, _P, _P, _P, _P, _P]),
    "fos_balance_workspace": (_I64, [_I64, _I]),
    "fos_balance_loss": (_I, [_P, _I, _I64, _I, _P, _I, _I, _P, _F, _I, _P, _P, _P, _P, _P, _I64, _P, _P]),
    "fos_balance_loss_backward": (_I, [_P, _P, _I, _I64, _I, _P, _P, _P, _P]),
    "fos_kv_append": (_I, [_P, _P, _I, _I64, _I64, _I64, _P, _P, ctypes.POINTER(_Config), _P, _P, _P, _P]),
    "fos_kv_attention": (_I, [_P, _I, _I64, _I, _I64, _P, _P, _F, _I, _I64, _P, _P, _P, _I64, _P, _P]),
    "fos_kv_attention_workspace": (_I64, [_I64, _I, _I64, _I64, _I, _I, _I, _I64]),
    "fos_kv_weights": (_I, [_P, _I, _I64, _I, _I64, _P, _P, _F, _I, _I64, _P, _P, _P, _P]),
    "fos_kv_evict": (_I, [_P, _P, _I, _I, _I, _P, _P, _I64, _P, _P]),
    "fos_kv_evict_workspace": (_I64, [_I64, _I, _I, _I]),
}
EXPORTS = tuple(_SIGS)

_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libfos.so (fails loudly when it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"{p} is not built; run `python -m nvfp4_adaptive_block_amd.build`")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(rc: int):
    if rc != 0:
        lib = load_library()
        raise FosError(rc, lib.fos_last_error().decode())


def config(recipe="4over6", block="1x16", scale_gran="tensor", err_metric="mse", err_prec="exact",
           bound=448, err_order="tree") -> _Config:
    return _Config(RECIPES[recipe], BLOCKS[block], GRANS[scale_gran], METRICS[err_metric], PRECS[err_prec],
                   int(bound), ORDERS[err_order])


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(x: torch.Tensor, name: str):
    if not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fos_amax(x: torch.Tensor, gran: str = "tensor", out: torch.Tensor | None = None) -> torch.Tensor:
    """NaN-dropping amax per tensor ([1]), per row ([M]) or per 16-row band ([M])."""
    _need(x, "x")
    M, K = x.shape
    if out is None:
        out = torch.empty(1 if gran == "tensor" else M, dtype=torch.float32, device=x.device)
    with torch.cuda.device(x.device):
        _check(load_library().fos_amax(_ptr(x), DTYPES[x.dtype], M, K, AMAX_GRANS[gran], _ptr(out),
                                       _stream(x.device)))
    return out


def fos_quantize(x: torch.Tensor, amax: torch.Tensor, *, codes=None, scales=None, sdec=None, status=None,
                 **knobs):
    """Quantize x[M, K]. Returns (codes uint8[M, K/2], scales uint8[M, K/16],
    sdec float32[1 or M])."""
    _need(x, "x")
    M, K = x.shape
    cfg = config(**knobs)
    dev = x.device
    if codes is None:
        codes = torch.empty(M, K // 2, dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(M, K // 16, dtype=torch.uint8, device=dev)
    if sdec is None:
        sdec = torch.empty(M if knobs.get("scale_gran", "tensor") == "row" else 1, dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(load_library().fos_quantize(_ptr(x), DTYPES[x.dtype], M, K, _ptr(amax), ctypes.byref(cfg),
                                           _ptr(codes), _ptr(scales), _ptr(sdec), _ptr(status), _stream(dev)))
    return codes, scales, sdec


def set_barrier_poll_limit(polls: int) -> int:
    """Polls a fused call's grid barrier makes before giving up (process-wide,
    for calls enqueued from now on); returns the previous limit."""
    prev = load_library().fos_set_barrier_poll_limit(int(polls))
    if prev < 0:
        raise ValueError(f"poll limit must be >= 0, got {polls}")
    return prev


def set_phase_timestamps(buf: torch.Tensor | None) -> int:
    """Diagnostics: the one-read fused kernels enqueued from now on write, per
    wave, four real-time-counter values (start, loads landed, barrier
    released, end) to buf (int64 [waves, 4] on the device); None stops it.
    Returns the counter's rate in kHz."""
    khz = ctypes.c_int(0)
    if buf is None:
        _check(load_library().fos_set_phase_timestamps(None, 0, ctypes.byref(khz)))
    else:
        if buf.dtype != torch.int64 or buf.dim() != 2 or buf.shape[1] != 4 or not buf.is_contiguous():
            raise ValueError("buf must be a contiguous int64 [waves, 4] tensor")
        with torch.cuda.device(buf.device):
            _check(load_library().fos_set_phase_timestamps(ctypes.c_void_p(buf.data_ptr()), buf.shape[0],
                                                           ctypes.byref(khz)))
    return khz.value


def _dev(device) -> torch.device:
    dev = torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    return dev


# Default workspaces and status words of the fused calls, one of each per
# (device, stream): calls on one stream run one after another and may share
# them; calls on different streams may overlap and must not.
_workspaces: dict = {}
_status_words: dict = {}


def _stream_key(device, stream=None):
    dev = _dev(device)
    s = torch.cuda.current_stream(dev) if stream is None else stream
    return dev, int(s.cuda_stream)


def fused_workspace(device, stream=None) -> torch.Tensor:
    """The zero-initialised workspace the fused calls use on `device` and
    `stream` (default: the device's current stream) when the caller passes
    none."""
    key = _stream_key(device, stream)
    if key not in _workspaces:
        _workspaces[key] = torch.zeros(FUSED_WORKSPACE_BYTES, dtype=torch.uint8, device=key[0])
    return _workspaces[key]


def fused_status_word(device, stream=None) -> torch.Tensor:
    """The device int32 status word the fused calls on `device` and `stream`
    OR their FOS_STATUS_* bits into when the caller passes none. Bits stay
    set until read with fused_status()."""
    key = _stream_key(device, stream)
    if key not in _status_words:
        _status_words[key] = torch.zeros(1, dtype=torch.int32, device=key[0])
    return _status_words[key]


def fused_status(device=None, stream=None, clear: bool = True) -> int:
    """Synchronize `stream` and return the status bits the fused calls on it
    have set since the last read (clearing them unless clear=False)."""
    dev = _dev(device if device is not None else "cuda")
    word = fused_status_word(dev, stream)
    s = torch.cuda.current_stream(dev) if stream is None else stream
    s.synchronize()
    v = int(word.item())
    if clear and v:
        with torch.cuda.stream(s):
            word.zero_()
        s.synchronize()
    return v


def _fused_done(dev, status, own_status: bool, check: bool):
    """After a fused call: with check, synchronize and raise on a barrier
    timeout (the outputs are then incomplete)."""
    if not check:
        return
    torch.cuda.current_stream(dev).synchronize()
    v = int(status.item())
    if own_status and v:
        status.zero_()
        torch.cuda.current_stream(dev).synchronize()
    if v & STATUS_BARRIER_TIMEOUT:
        raise FosError(-1, "fused call: the grid barrier timed out; outputs are incomplete "
                           "(another long-running kernel held part of the device)")


def fos_quantize_fused(x: torch.Tensor, *, codes=None, scales=None, amax=None, sdec=None, status=None,
                       workspace=None, check=False, **knobs):
    """Amax (per tensor, or per row with scale_gran="row") and quantize in
    one launch. Returns (codes, scales, amax float32[1 or M], sdec float32[1
    or M]). Without `workspace` / `status` the current stream's own are used
    (fused_workspace, fused_status_word); with check=True the call
    synchronizes and raises FosError if the grid barrier timed out."""
    _need(x, "x")
    M, K = x.shape
    cfg = config(**knobs)
    dev = x.device
    n_amax = M if knobs.get("scale_gran", "tensor") == "row" else 1
    if codes is None:
        codes = torch.empty(M, K // 2, dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(M, K // 16, dtype=torch.uint8, device=dev)
    if amax is None:
        amax = torch.empty(n_amax, dtype=torch.float32, device=dev)
    if sdec is None:
        sdec = torch.empty(n_amax, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = fused_workspace(dev)
    own = status is None
    if own:
        status = fused_status_word(dev)
    with torch.cuda.device(dev):
        _check(load_library().fos_quantize_fused(_ptr(x), DTYPES[x.dtype], M, K, ctypes.byref(cfg), _ptr(codes),
                                                 _ptr(scales), _ptr(amax), _ptr(sdec), _ptr(workspace),
                                                 _ptr(status), _stream(dev)))
    _fused_done(dev, status, own, check)
    return codes, scales, amax, sdec


def fos_qdq_fused(x: torch.Tensor, *, out=None, amax=None, status=None, workspace=None, check=False, **knobs):
    """Per-tensor amax and fused quantize-dequantize in one launch (two when
    the tensor does not fit on chip). Returns (y, amax float32[1]).
    `workspace`, `status` and `check` as for fos_quantize_fused."""
    _need(x, "x")
    M, K = x.shape
    cfg = config(**knobs)
    dev = x.device
    y = torch.empty_like(x) if out is None else out
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = fused_workspace(dev)
    own = status is None
    if own:
        status = fused_status_word(dev)
    with torch.cuda.device(dev):
        _check(load_library().fos_qdq_fused(_ptr(x), DTYPES[x.dtype], M, K, ctypes.byref(cfg), _ptr(y), _ptr(amax),
                                            _ptr(workspace), _ptr(status), _stream(dev)))
    _fused_done(dev, status, own, check)
    return y, amax


def fos_quantize_columnwise(x: torch.Tensor, amax: torch.Tensor, *, codes=None, scales=None, sdec=None, **knobs):
    """Quantize the transpose of x[M, K] without materialising it. Returns
    (codes uint8[K, M/2], scales uint8[K, M/16], sdec float32[1])."""
    _need(x, "x")
    M, K = x.shape
    cfg = config(**knobs)
    dev = x.device
    if codes is None:
        codes = torch.empty(K, M // 2, dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(K, M // 16, dtype=torch.uint8, device=dev)
    if sdec is None:
        sdec = torch.empty(1, dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(load_library().fos_quantize_columnwise(_ptr(x), DTYPES[x.dtype], M, K, _ptr(amax), ctypes.byref(cfg),
                                                      _ptr(codes), _ptr(scales), _ptr(sdec), _stream(dev)))
    return codes, scales, sdec


def fos_qdq(x: torch.Tensor, amax: torch.Tensor, *, out=None, **knobs) -> torch.Tensor:
    """Fused quantize-dequantize: y has x's dtype and shape."""
    _need(x, "x")
    M, K = x.shape
    cfg = config(**knobs)
    y = torch.empty_like(x) if out is None else out
    with torch.cuda.device(x.device):
        _check(load_library().fos_qdq(_ptr(x), DTYPES[x.dtype], M, K, _ptr(amax), ctypes.byref(cfg), _ptr(y),
                                      _stream(x.device)))
    return y


def fos_qdq_list(xs: Sequence[torch.Tensor], amaxes: Sequence[torch.Tensor], *, outs=None, **knobs):
    """Fused quantize-dequantize over a list of rank-2 tensors of one dtype."""
    if len(xs) != len(amaxes):
        raise ValueError("xs and amaxes differ in length")
    if not xs:
        return []
    dev = xs[0].device
    ys = [torch.empty_like(x) for x in xs] if outs is None else list(outs)
    descs = (_Desc * len(xs))()
    for i, (x, a, y) in enumerate(zip(xs, amaxes, ys)):
        _need(x, f"xs[{i}]")
        if x.dtype != xs[0].dtype or x.device != dev:
            raise ValueError("all tensors of a list share one dtype and device")
        descs[i] = _Desc(x.data_ptr(), y.data_ptr(), a.data_ptr(), x.shape[0], x.shape[1])
    cfg = config(**knobs)
    with torch.cuda.device(dev):
        _check(load_library().fos_qdq_list(len(xs), ctypes.cast(descs, ctypes.c_void_p), DTYPES[xs[0].dtype],
                                           ctypes.byref(cfg), _stream(dev)))
    return ys


def fos_qdq_list_fused(xs: Sequence[torch.Tensor], *, outs=None, amax=None, workspace=None, status=None,
                       check=False, **knobs):
    """Every tensor's amax and the fused quantize-dequantize of the list in one
    launch. Returns (ys, amax float32[n]). `workspace`, `status` and `check`
    as for fos_quantize_fused."""
    if not xs:
        return [], None
    dev = xs[0].device
    ys = [torch.empty_like(x) for x in xs] if outs is None else list(outs)
    if amax is None:
        amax = torch.empty(len(xs), dtype=torch.float32, device=dev)
    descs = (_Desc * len(xs))()
    for i, (x, y) in enumerate(zip(xs, ys)):
        _need(x, f"xs[{i}]")
        if x.dtype != xs[0].dtype or x.device != dev:
            raise ValueError("all tensors of a list share one dtype and device")
        descs[i] = _Desc(x.data_ptr(), y.data_ptr(), None, x.shape[0], x.shape[1])
    cfg = config(**knobs)
    if workspace is None:
        workspace = fused_workspace(dev)
    own = status is None
    if own:
        status = fused_status_word(dev)
    with torch.cuda.device(dev):
        _check(load_library().fos_qdq_list_fused(len(xs), ctypes.cast(descs, ctypes.c_void_p), DTYPES[xs[0].dtype],
                                                 ctypes.byref(cfg), _ptr(amax), _ptr(workspace), _ptr(status),
                                                 _stream(dev)))
    _fused_done(dev, status, own, check)
    return ys, amax


def nvfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, sdec: torch.Tensor, scale_gran: str = "tensor",
                     out_dtype: torch.dtype = torch.bfloat16, out=None) -> torch.Tensor:
    """Standard NVFP4 decode of codes[M, K/2] and scales[M, K/16]."""
    _need(codes, "codes")
    M, K = codes.shape[0], codes.shape[1] * 2
    y = torch.empty(M, K, dtype=out_dtype, device=codes.device) if out is None else out
    with torch.cuda.device(codes.device):
        _check(load_library().nvfp4_dequantize(_ptr(codes), _ptr(scales), M, K, _ptr(sdec), GRANS[scale_gran],
                                               DTYPES[out_dtype], _ptr(y), _stream(codes.device)))
    return y


def fos_quantize_grouped(x: torch.Tensor, offs: torch.Tensor, group_amax: torch.Tensor, *, codes=None, scales=None,
                         group_sdec=None, status=None, **knobs):
    """Quantize a packed token tensor of G groups (cumulative end offsets
    ``offs``) with per-group amaxes in one launch. Returns (codes, scales,
    group_sdec)."""
    _need(x, "x")
    M, K = x.shape
    dev = x.device
    G = offs.numel()
    cfg = config(**knobs)
    if codes is None:
        codes = torch.empty(M, K // 2, dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(M, K // 16, dtype=torch.uint8, device=dev)
    if group_sdec is None:
        group_sdec = torch.empty(G, dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(load_library().fos_quantize_grouped(_ptr(x), DTYPES[x.dtype], M, K, _ptr(offs), G, _ptr(group_amax),
                                                   ctypes.byref(cfg), _ptr(codes), _ptr(scales), _ptr(group_sdec),
                                                   _ptr(status), _stream(dev)))
    return codes, scales, group_sdec


def fos_quantize_grouped_fused(x: torch.Tensor, offs: torch.Tensor, *, codes=None, scales=None, group_amax=None,
                               group_sdec=None, status=None, workspace=None, check=False, **knobs):
    """Group amaxes and the grouped quantize in one launch. Returns (codes,
    scales, group_amax float32[G], group_sdec float32[G]). `workspace`,
    `status` and `check` as for fos_quantize_fused."""
    _need(x, "x")
    M, K = x.shape
    dev = x.device
    G = offs.numel()
    cfg = config(**knobs)
    if codes is None:
        codes = torch.empty(M, K // 2, dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(M, K // 16, dtype=torch.uint8, device=dev)
    if group_amax is None:
        group_amax = torch.empty(G, dtype=torch.float32, device=dev)
    if group_sdec is None:
        group_sdec = torch.empty(G, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = fused_workspace(dev)
    own = status is None
    if own:
        status = fused_status_word(dev)
    with torch.cuda.device(dev):
        _check(load_library().fos_quantize_grouped_fused(_ptr(x), DTYPES[x.dtype], M, K, _ptr(offs), G,
                                                         ctypes.byref(cfg), _ptr(codes), _ptr(scales),
                                                         _ptr(group_amax), _ptr(group_sdec), _ptr(workspace),
                                                         _ptr(status), _stream(dev)))
    _fused_done(dev, status, own, check)
    return codes, scales, group_amax, group_sdec


def fos_quantize_grouped_fused_noalloc(x: torch.Tensor, offs: torch.Tensor, *, codes, scales, group_amax,
                                       group_sdec=None, status=None, **knobs):
    """fos_quantize_grouped_fused with the library-held workspace (the C call
    allocates nothing). The caller passes every output buffer. Calls on
    different streams of one device must not overlap."""
    _need(x, "x")
    M, K = x.shape
    dev = x.device
    cfg = config(**knobs)
    with torch.cuda.device(dev):
        _check(load_library().fos_quantize_grouped_fused_noalloc(_ptr(x), DTYPES[x.dtype], M, K, _ptr(offs),
                                                                 offs.numel(), ctypes.byref(cfg), _ptr(codes),
                                                                 _ptr(scales), _ptr(group_amax), _ptr(group_sdec),
                                                                 _ptr(status), _stream(dev)))
    return codes, scales, group_amax, group_sdec


# ------------------------------------------------- operators around the quantizer
#
# A call on one token takes the GPU a few microseconds, less than careless
# argument handling takes the host: these bindings pass plain integers to
# ctypes, compare each tensor's properties once and switch devices only where
# the current one is another.
#
# Like the quantizer's, their outputs are outside autograd's graph, whatever the
# inputs require; only fos_balance_loss's loss is in it.


def _mismatch(t, name, device, shape, dtype):
    _need(t, name)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _match(t, name: str, device, shape=None, dtype=None) -> int:
    """Address of a tensor that the C call takes as a bare pointer, checked."""
    if (t.device != device or not t.is_contiguous() or (shape is not None and t.shape != shape)
            or (dtype is not None and t.dtype != dtype)):
        _mismatch(t, name, device, shape, dtype)
    return t.data_ptr()


def _status_pointer(status, device):
    """Address of the status word. A tensor without elements has none, and would be
    taken for no status."""
    if status.numel() < 1:
        raise ValueError("status must hold a value")
    return _match(status, "status", device, None, torch.int32)


# The current stream's handle without a Stream object (2 us less a call) where
# this torch has the function.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(dev, fn, *args):
    """fn(*args, current stream of dev) with dev current; raises on an error code."""
    index = dev.index
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(index))
    if rc:
        _check(rc)


def _float_type(t, name: str) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    return code


def _scale_pointer(scale, gran: str, rows: int, groups: int | None, name: str, device) -> int:
    if gran not in OPERAND_GRANS or (gran == "group" and groups is None):
        raise ValueError(f"{name}: unknown scale granularity {gran!r}")
    want = 1 if gran == "tensor" else rows if gran == "row" else groups
    if scale.numel() != want:
        raise ValueError(f"{name}'s scale must hold {want} value(s) (per {gran}), got {scale.numel()}")
    return _match(scale, f"{name}'s scale", device, None, torch.float32)


def _activation_operand(x, gran, groups):
    """(_Operand, M, K, device) of a bf16/fp16 tensor, an (E4M3 values,
    scales) pair or a (codes, block scales, S_dec) triple."""
    if isinstance(x, torch.Tensor):
        _need(x, "x")
        if x.dim() != 2 or x.dtype not in (torch.bfloat16, torch.float16):
            raise ValueError(f"x must be a bf16 or fp16 [M, K] tensor, got {x.dtype} {list(x.shape)}")
        M, K = x.shape
        return _Operand(x.data_ptr(), None, None, DTYPES[x.dtype], 0), M, K, x.device
    if not isinstance(x, (tuple, list)) or len(x) not in (2, 3):
        raise ValueError("x must be a tensor, (q, scale) or (codes, scales, sdec)")
    data = x[0]
    _need(data, "x")
    if data.dim() != 2:
        raise ValueError(f"x must be rank 2, got {list(data.shape)}")
    dev = data.device
    M, width = data.shape
    if len(x) == 2:
        if data.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise ValueError(f"x's values must be float8_e4m3fn, got {data.dtype}")
        gran = gran or "row"
        scale = _scale_pointer(x[1], gran, M, groups, "x", dev)
        return _Operand(data.data_ptr(), None, scale, OPERAND_E4M3, OPERAND_GRANS[gran]), M, width, dev
    K = 2 * width
    gran = gran or "tensor"
    return (_Operand(_match(data, "x's codes", dev, None, torch.uint8),
                     _match(x[1], "x's block scales", dev, (M, K // 16), torch.uint8),
                     _scale_pointer(x[2], gran, M, groups, "x", dev), OPERAND_NVFP4, OPERAND_GRANS[gran]), M, K, dev)


def _linear(x, w, offs, bias, act, residual, out_dtype, out, x_gran, w_gran, workspace, status):
    codes, scales, sdec = w
    G = None if offs is None else offs.numel()
    xo, M, K, dev = _activation_operand(x, x_gran, G)
    if codes.dim() != (2 if G is None else 3):
        raise ValueError(f"w's codes must have shape {['N', K // 2] if G is None else [G, 'N', K // 2]}, "
                         f"got {list(codes.shape)}")
    N = codes.shape[-2]
    lead = (N,) if G is None else (G, N)
    wo = _Operand(_match(codes, "w's codes", dev, (*lead, K // 2), torch.uint8),
                  _match(scales, "w's block scales", dev, (*lead, K // 16), torch.uint8),
                  _scale_pointer(sdec, w_gran, N * (G or 1), G, "w", dev), OPERAND_NVFP4, OPERAND_GRANS[w_gran])
    if out is not None:
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = x.dtype if isinstance(x, torch.Tensor) else torch.bfloat16
    out_code = DTYPES.get(out_dtype)
    if out_code is None:
        raise ValueError(f"unsupported output dtype {out_dtype}")
    if act not in ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}")
    epi = None
    if bias is not None or residual is not None or act != "none":
        epi = ctypes.byref(_Epilogue(None if bias is None else _match(bias, "bias", dev, lead),
                                     None if residual is None else _match(residual, "residual", dev, (M, N),
                                                                          out_dtype),
                                     0 if bias is None else _float_type(bias, "bias"), ACTIVATIONS[act]))
    y = torch.empty(M, N, dtype=out_dtype, device=dev) if out is None else out
    yp = y.data_ptr() if out is None else _match(out, "out", dev, (M, N))
    lib = load_library()
    need = lib.fos_linear_workspace(M, N, K, G or 0)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    work, room = (None, 0) if workspace is None else (_match(workspace, "workspace", dev),
                                                      workspace.numel() * workspace.element_size())
    if G is None:
        _call(dev, lib.fos_linear, ctypes.byref(xo), ctypes.byref(wo), M, N, K, epi, yp, out_code, work, room)
    else:
        _call(dev, lib.fos_linear_grouped, ctypes.byref(xo), ctypes.byref(wo),
              _match(offs, "offs", dev, (G,), torch.int32), G, M, N, K, epi, yp, out_code, work, room,
              None if status is None else _status_pointer(status, dev))
    return y


def fos_linear(x, w, *, bias=None, act: str = "none", residual=None, out_dtype=None, out=None, x_gran=None,
               w_gran: str = "tensor", workspace=None) -> torch.Tensor:
    """act(x @ dequantize(w).T + bias) + residual, [M, N].

    x: a bf16 or fp16 tensor [M, K]; (q, scale) of fos_rmsnorm_quantize (E4M3,
    a scale per row); or (codes, scales, sdec) of fos_quantize. w: (codes,
    scales, sdec) of fos_quantize for a weight [N, K], or of
    fos_quantize_columnwise for the backward product. ``x_gran`` and ``w_gran``
    say what one float32 scale covers ("tensor" or "row"; E4M3 rows default to
    "row"). out_dtype defaults to x's, or bf16 for a quantized x. A workspace
    (fos_linear_workspace bytes) is allocated when none is passed."""
    return _linear(x, w, None, bias, act, residual, out_dtype, out, x_gran, w_gran, workspace, None)


def fos_linear_grouped(x, w, offs: torch.Tensor, *, bias=None, act: str = "none", residual=None, out_dtype=None,
                       out=None, x_gran=None, w_gran: str = "tensor", workspace=None, status=None) -> torch.Tensor:
    """fos_linear of each group of rows with its own weight, in one launch:
    rows [offs[g-1], offs[g]) of x take w[g] (codes [G, N, K/2], scales [G, N,
    K/16], sdec [1], [G] with w_gran="group" or [G * N] with w_gran="row") and
    bias[g]; rows at or past offs[-1] come out as zero."""
    _need(offs, "offs")
    return _linear(x, w, offs, bias, act, residual, out_dtype, out, x_gran, w_gran, workspace, status)


def fos_linear_workspace(M: int, N: int, K: int, G: int = 0) -> int:
    """Bytes of workspace of fos_linear (G = 0) or fos_linear_grouped."""
    need = load_library().fos_linear_workspace(M, N, K, G)
    if need < 0:
        raise ValueError(f"unsupported sizes M={M} N={N} K={K} G={G}")
    return need


def fos_rmsnorm_quantize(x: torch.Tensor, weight: torch.Tensor, *, residual=None, eps: float = 1e-6, q=None,
                         scale=None, h=None, y=None):
    """RMS norm of x + residual, [M, K], with an 8-bit output. Returns (q
    float8_e4m3fn[M, K], scale float32[M], h): q * scale is the normalised row
    and h = x + residual in x's dtype (x itself without a residual). Pass
    ``y`` (x's shape and dtype) to have the unquantized norm written too."""
    _need(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be rank 2, got {list(x.shape)}")
    shape = x.shape
    M, K = shape
    dev, dtype = x.device, x.dtype
    code, wp, rp = _float_type(x, "x"), _match(weight, "weight", dev, (K,)), None
    if residual is not None:
        rp = _match(residual, "residual", dev, shape, dtype)
        if h is None:
            h = torch.empty_like(x)
    hp = None if h is None else _match(h, "h", dev, shape, dtype)
    yp = None if y is None else _match(y, "y", dev, shape, dtype)
    if q is None:
        q = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=dev)
    if scale is None:
        scale = torch.empty(M, dtype=torch.float32, device=dev)
    _call(dev, load_library().fos_rmsnorm_quantize, x.data_ptr(), code, M, K, rp, wp, _float_type(weight, "weight"),
          eps, _match(q, "q", dev, shape, torch.float8_e4m3fn), _match(scale, "scale", dev, (M,), torch.float32), hp,
          yp)
    return q, scale, x if h is None else h


def _mask_pointer(mask, T, dev):
    if mask is None:
        return None
    if mask.dtype not in (torch.bool, torch.uint8):
        raise ValueError(f"mask must be bool or uint8, got {mask.dtype}")
    return _match(mask, "mask", dev, (T,))


def fos_balance_loss(logits: torch.Tensor, idx: torch.Tensor, *, coef: float = 0.01, mask=None, align: int = 16,
                     loss=None, counts=None, offs=None, slope=None, workspace=None, status=None):
    """Load-balance loss of router logits [T, E] and the chosen experts idx
    [T, k] (int32 or int64, -1 for a dropped assignment). Returns (loss
    float32[1], counts int32[E], offs int32[E], slope float32[E]): the
    assignments per expert, the end offsets of groups padded to multiples of
    ``align`` (what the grouped calls take), and what the backward call needs.

    Where gradients are recorded and the logits require one, the loss (unless it
    is a buffer that the caller passes) is differentiable with respect to them,
    once, by fos_balance_loss_backward; the other outputs are constants."""
    if logits.requires_grad and loss is None and torch.is_grad_enabled():
        return _BalanceLoss.apply(logits, idx, coef, mask, align, counts, offs, slope, workspace, status)
    _need(logits, "logits")
    _need(idx, "idx")
    if logits.dim() != 2 or idx.dim() != 2 or idx.shape[0] != logits.shape[0]:
        raise ValueError(f"logits [T, E] and idx [T, k] expected, got {list(logits.shape)} and {list(idx.shape)}")
    T, E = logits.shape
    dev = logits.device
    code = _float_type(logits, "logits")
    if idx.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"idx must be int32 or int64, got {idx.dtype}")
    if loss is None:
        loss = torch.empty(1, dtype=torch.float32, device=dev)
    if counts is None:
        counts = torch.empty(E, dtype=torch.int32, device=dev)
    if offs is None:
        offs = torch.empty(E, dtype=torch.int32, device=dev)
    if slope is None:
        slope = torch.empty(E, dtype=torch.float32, device=dev)
    lib = load_library()
    if workspace is None:
        workspace = torch.empty(max(0, lib.fos_balance_workspace(T, E)), dtype=torch.uint8, device=dev)
    _call(dev, lib.fos_balance_loss, logits.data_ptr(), code, T, E, _match(idx, "idx", dev),
          8 if idx.dtype == torch.int64 else 4, idx.shape[1], _mask_pointer(mask, T, dev), coef, align,
          _match(loss, "loss", dev, (1,), torch.float32), _match(counts, "counts", dev, (E,), torch.int32),
          _match(offs, "offs", dev, (E,), torch.int32), _match(slope, "slope", dev, (E,), torch.float32),
          _match(workspace, "workspace", dev), workspace.numel() * workspace.element_size(),
          None if status is None else _status_pointer(status, dev))
    return loss, counts, offs, slope


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, idx, coef, mask, align, counts, offs, slope, workspace, status):
        # a slope of the caller's may be written again before the backward pass
        outs = fos_balance_loss(logits, idx, coef=coef, mask=mask, align=align, counts=counts, offs=offs,
                                workspace=workspace, status=status)
        ctx.save_for_backward(logits, outs[3], mask)
        if slope is not None:
            _match(slope, "slope", logits.device, outs[3].shape, torch.float32)
            outs = (*outs[:3], slope.copy_(outs[3]))
        ctx.mark_non_differentiable(*outs[1:])
        return outs

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss, *_):
        logits, slope, mask = ctx.saved_tensors
        return fos_balance_loss_backward(dloss.contiguous(), logits, slope, mask=mask), *(None,) * 9


def fos_balance_workspace(T: int, E: int) -> int:
    """Bytes of workspace of fos_balance_loss."""
    need = load_library().fos_balance_workspace(T, E)
    if need < 0:
        raise ValueError(f"unsupported sizes T={T} E={E}")
    return need


def fos_balance_loss_backward(dloss: torch.Tensor, logits: torch.Tensor, slope: torch.Tensor, *, mask=None,
                              out=None) -> torch.Tensor:
    """Gradient of fos_balance_loss with respect to its logits, times dloss
    (float32[1]); ``slope`` and ``mask`` as in the forward call."""
    _need(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits must be rank 2, got {list(logits.shape)}")
    T, E = logits.shape
    dev = logits.device
    code = _float_type(logits, "logits")
    if dloss.numel() != 1:
        raise ValueError("dloss must hold one value")
    d = torch.empty_like(logits) if out is None else out
    _call(dev, load_library().fos_balance_loss_backward, _match(dloss, "dloss", dev, None, torch.float32),
          logits.data_ptr(), code, T, E, _mask_pointer(mask, T, dev),
          _match(slope, "slope", dev, (E,), torch.float32), _match(d, "out", dev, (T, E), logits.dtype))
    return d


# ------------------------------------------------------------- key/value cache
#
# One side of the cache is (codes uint8[pages, H, P, D/2], scales uint8[pages, H, P,
# D/16], sdec float32[pages, H, P]): pages of P rows for each of H heads, a row as
# fos_quantize writes it with scale_gran="row". table int32[B, W] holds the pages of
# each sequence in order, lens int32[B] its tokens, those of the call included, and
# offs int32[B] the end row of each sequence's tokens among the packed ones.


# A fos_kv_cache, packed: a ctypes structure of the same fields takes three times as long
# to fill. An instance of bytes is passed as its address.
_KV_CACHE = struct.Struct("8Pq5i4x")


def _kv_device(index):
    return torch.device("cuda", index) if index >= 0 else torch.device("cpu")


def _kv_at(t, name, index, shape, dtype) -> int:
    """Address of a contiguous tensor on device `index`, checked."""
    if t.get_device() != index or t.dtype is not dtype or not t.is_contiguous() or t.shape != shape:
        _mismatch(t, name, _kv_device(index), shape, dtype)
    return t.data_ptr()


def _kv_cache(k, v, table, lens):
    """(packed fos_kv_cache, device index, B, W, H, P, D); v may be None."""
    codes, scales, sdec = k
    index = codes.get_device()
    if index < 0:
        raise ValueError("the cache must be on a device")
    shape = codes.shape
    if len(shape) != 4:
        raise ValueError(f"k_cache's codes must have shape ['pages', 'H', 'P', 'D / 2'], got {list(shape)}")
    pages, H, P, half = shape
    of_scales, of_sdec = (pages, H, P, half // 8), (pages, H, P)
    at = [_kv_at(codes, "k_cache's codes", index, shape, torch.uint8),
          _kv_at(scales, "k_cache's scales", index, of_scales, torch.uint8),
          _kv_at(sdec, "k_cache's sdec", index, of_sdec, torch.float32)]
    if v is None:
        at += at
    else:
        codes, scales, sdec = v
        at += (_kv_at(codes, "v_cache's codes", index, shape, torch.uint8),
               _kv_at(scales, "v_cache's scales", index, of_scales, torch.uint8),
               _kv_at(sdec, "v_cache's sdec", index, of_sdec, torch.float32))
    if table.dim() != 2:
        raise ValueError(f"table must have shape ['B', 'W'], got {list(table.shape)}")
    B, W = table.shape
    return (_KV_CACHE.pack(*at, _kv_at(table, "table", index, (B, W), torch.int32),
                           _kv_at(lens, "lens", index, (B,), torch.int32), pages, B, W, H, P, 2 * half),
            index, B, W, H, P, 2 * half)


def _kv_tokens(x, name, index, heads, D):
    """Address and token stride of [T, heads, D] rows, whose tokens may lie apart."""
    shape = x.shape
    if len(shape) != 3 or shape[2] != D or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must have shape ['T', {heads or 'heads'}, {D}], got {list(shape)}")
    if x.get_device() != index:
        raise ValueError(f"{name} is on {x.device}, expected cuda:{index}")
    T, n, _ = shape
    apart, between, inner = x.stride()
    if T * n and (inner != 1 or (n > 1 and between != D)):
        raise ValueError(f"{name}'s tokens must be contiguous, got strides {[apart, between, inner]}")
    return x.data_ptr(), apart if T > 1 else n * D


def _kv_call(index, fn, *args):
    """fn(*args, current stream of the device) with the device current; raises on an error code."""
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc:
        _check(rc)


def _kv_room(workspace, need, index):
    """(address, bytes, tensor) of a workspace: the caller's, or a new one."""
    if workspace is None:
        if need <= 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=_kv_device(index))
        return workspace.data_ptr(), need, workspace
    if workspace.get_device() != index or not workspace.is_contiguous():
        _mismatch(workspace, "workspace", _kv_device(index), None, None)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _kv_ints(**values):
    """Sizes that the library takes in 32 bits, of which ctypes would drop the others."""
    for name, v in values.items():
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"{name}={v} is out of range")


def _kv_status(status, index):
    return None if status is None else _status_pointer(status, _kv_device(index))


def fos_kv_cache(pages: int, heads: int, page: int, dim: int, device="cuda"):
    """An empty side of a cache, (codes, scales, sdec), for `pages` pages of
    `page` rows of `dim` values for each of `heads` heads."""
    return (torch.zeros(pages, heads, page, dim // 2, dtype=torch.uint8, device=device),
            torch.zeros(pages, heads, page, dim // 16, dtype=torch.uint8, device=device),
            torch.zeros(pages, heads, page, dtype=torch.float32, device=device))


@functools.lru_cache(maxsize=None)
def _kv_config(**knobs):
    return ctypes.byref(config(scale_gran="row", **knobs))


def fos_kv_append(k: torch.Tensor, v: torch.Tensor, offs: torch.Tensor, k_cache, v_cache, table: torch.Tensor,
                  lens: torch.Tensor, *, values: bool = False, k_out=None, v_out=None, status=None, **knobs):
    """Quantize the rows k and v [T, H, D] of new tokens into the pages of their
    sequences: rows [offs[b-1], offs[b]) are the last of sequence b's lens[b]
    tokens. Tokens may lie apart (parts of a wider row). Returns (k_out, v_out),
    what the cache then holds for these rows in k's dtype, with values=True or
    where the outputs are passed, else None. ``knobs`` as for fos_quantize
    (1x16 blocks, a float32 scale per row)."""
    cache, index, B, _, H, _, D = _kv_cache(k_cache, v_cache, table, lens)
    kp, k_stride = _kv_tokens(k, "k", index, H, D)
    vp, v_stride = _kv_tokens(v, "v", index, H, D)
    shape, dtype = k.shape, k.dtype
    code = _float_type(k, "k")
    if v.shape != shape or v.dtype is not dtype:
        raise ValueError(f"v must be {dtype} {list(shape)} as k is, got {v.dtype} {list(v.shape)}")
    if values:
        k_out = torch.empty(shape, dtype=dtype, device=k.device) if k_out is None else k_out
        v_out = torch.empty(shape, dtype=dtype, device=k.device) if v_out is None else v_out
    _kv_call(index, load_library().fos_kv_append, kp, vp, code, shape[0], k_stride, v_stride,
             _kv_at(offs, "offs", index, (B,), torch.int32), cache, _kv_config(**knobs),
             None if k_out is None else _kv_at(k_out, "k_out", index, shape, dtype),
             None if v_out is None else _kv_at(v_out, "v_out", index, shape, dtype), _kv_status(status, index))
    return k_out, v_out


def _kv_queries(q, index, D):
    if q.dtype is not torch.bfloat16 and q.dtype is not torch.float16:
        raise ValueError(f"q must be bf16 or fp16, got {q.dtype}")
    return _kv_tokens(q, "q", index, None, D)


@functools.lru_cache(maxsize=4096)
def _kv_attention_room(*sizes) -> int:
    return load_library().fos_kv_attention_workspace(*sizes)


def fos_kv_attention(q: torch.Tensor, offs: torch.Tensor, k_cache, v_cache, table: torch.Tensor, lens: torch.Tensor, *,
                     scale: float | None = None, causal: bool = True, max_len: int = 0, out=None, lse=None,
                     workspace=None, status=None):
    """Attention of the queries q [T, Hq, D] (bf16 or fp16; Hq a multiple of the
    cache's heads; tokens may lie apart) of the sequences' last tokens over the
    cache, in which these tokens' keys already are. Returns (out [T, Hq, D], lse
    float32[T, Hq]). scale defaults to D ** -0.5; causal lets a token see what
    stands before it and itself; max_len (what the caller knows lens to be at
    most; default: what the table holds) shapes the launch. Queries that see no
    key, and rows past offs[-1], have out 0 and lse -inf."""
    cache, index, B, W, H, P, D = _kv_cache(k_cache, v_cache, table, lens)
    qp, stride = _kv_queries(q, index, D)
    shape, dtype = q.shape, q.dtype
    T, Hq, _ = shape
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)
        to_out = out.data_ptr()
    else:
        to_out = _kv_at(out, "out", index, shape, dtype)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
        to_lse = lse.data_ptr()
    else:
        to_lse = _kv_at(lse, "lse", index, (T, Hq), torch.float32)
    need = 0 if workspace is not None else _kv_attention_room(T, Hq, B, W, H, P, D, max_len)
    work, room, workspace = _kv_room(workspace, need, index)
    _kv_call(index, load_library().fos_kv_attention, qp, DTYPES[dtype], T, Hq, stride,
             _kv_at(offs, "offs", index, (B,), torch.int32), cache, D ** -0.5 if scale is None else scale, causal,
             max_len, to_out, to_lse, work, room, _kv_status(status, index))
    return out, lse


def fos_kv_attention_workspace(T: int, Hq: int, B: int, W: int, H: int, P: int, D: int, max_len: int = 0) -> int:
    """Bytes of workspace of fos_kv_attention for T tokens of Hq query heads on a
    cache of H heads, with a table [B, W] of pages of P rows of D values."""
    _kv_ints(Hq=Hq, H=H, P=P, D=D)
    need = load_library().fos_kv_attention_workspace(T, Hq, B, W, H, P, D, max_len)
    if need < 0:
        raise ValueError(f"unsupported sizes T={T} Hq={Hq} B={B} W={W} H={H} P={P} D={D}")
    return need


def fos_kv_weights(q: torch.Tensor, offs: torch.Tensor, k_cache, table: torch.Tensor, lens: torch.Tensor,
                   lse: torch.Tensor, acc: torch.Tensor, *, scale: float | None = None, causal: bool = True,
                   max_len: int = 0, status=None) -> torch.Tensor:
    """Add to acc float32[B, H, W * P], per cached key, the attention weights that
    the queries q give it, summed over the new tokens and the query heads of each
    of the cache's; lse [T, Hq] of fos_kv_attention. q, offs and lse may be those
    of each sequence's last tokens only. Returns acc; places at or past lens[b] are
    left as they are."""
    cache, index, B, W, H, P, D = _kv_cache(k_cache, None, table, lens)
    qp, stride = _kv_queries(q, index, D)
    T, Hq, _ = q.shape
    _kv_call(index, load_library().fos_kv_weights, qp, DTYPES[q.dtype], T, Hq, stride,
             _kv_at(offs, "offs", index, (B,), torch.int32), cache, D ** -0.5 if scale is None else scale, causal, max_len,
             _kv_at(lse, "lse", index, (T, Hq), torch.float32), _kv_at(acc, "acc", index, (B, H, W * P), torch.float32),
             _kv_status(status, index))
    return acc


def fos_kv_evict(acc: torch.Tensor, k_cache, v_cache, table: torch.Tensor, lens: torch.Tensor, budget: int, *,
                 sinks: int = 0, recent: int = 0, new_lens=None, workspace=None, status=None) -> torch.Tensor:
    """Cut sequences of more than `budget` tokens to that many, each head on its own:
    the first `sinks` rows, the last `recent` rows and, of those between, the ones
    with the largest acc float32[B, H, W * P] stay. Kept rows, and their acc, move
    into the places that others gave up; the last rows end at the new length in
    their order. Returns new_lens int32[B], min(lens, budget); lens itself is left."""
    _kv_ints(budget=budget, sinks=sinks, recent=recent)
    cache, index, B, W, H, P, _ = _kv_cache(k_cache, v_cache, table, lens)
    lib = load_library()
    if new_lens is None:
        new_lens = torch.empty_like(lens)
        to_lens = new_lens.data_ptr()
    else:
        to_lens = _kv_at(new_lens, "new_lens", index, (B,), torch.int32)
    need = 0 if workspace is not None else lib.fos_kv_evict_workspace(B, H, budget, recent)
    work, room, workspace = _kv_room(workspace, need, index)
    _kv_call(index, lib.fos_kv_evict, cache, _kv_at(acc, "acc", index, (B, H, W * P), torch.float32), budget, sinks,
             recent, to_lens, work, room, _kv_status(status, index))
    return new_lens


def fos_kv_evict_workspace(B: int, H: int, budget: int, recent: int = 0) -> int:
    """Bytes of workspace of fos_kv_evict."""
    _kv_ints(H=H, budget=budget, recent=recent)
    need = load_library().fos_kv_evict_workspace(B, H, budget, recent)
    if need < 0:
        raise ValueError(f"unsupported sizes B={B} H={H} budget={budget} recent={recent}")
    return need
