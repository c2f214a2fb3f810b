"""Python binding of the DeltaLog C ABI (``include/deltalog.h``).

Argument marshalling only: every function here has the name of the C entry
point it calls and passes plain device pointers, sizes and a CUDA stream
through ctypes.  All arithmetic runs in the CUDA kernels of
``libdeltalog.so``.  Torch tensors are accepted as the carriers of device
memory (their ``data_ptr()``); the binding checks their dtype, device, size
and contiguity so that the C library never sees a buffer smaller than the
layout it is told about.

Importing this module loads the library and fails loudly when it has not
been built (``python -m linear_attention_recurrent_deltalog_b200.build``):
there is no fallback path.
"""

from __future__ import annotations

import ctypes
import dataclasses
import functools
import os
import struct
from typing import Optional, Sequence

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdeltalog.so")

# enums (mirror deltalog.h)
DL_GDN, DL_KDA, DL_RWKV6, DL_GDN2 = 0, 1, 2, 3
DL_F32, DL_BF16 = 0, 1
DL_OK = 0
DL_ERR_ARG, DL_ERR_ALIGN, DL_ERR_LOG_FULL = -1, -2, -3
DL_ERR_CUDA, DL_ERR_UNSUPPORTED, DL_ERR_DEVICE = -4, -5, -6
DL_MERGE_FULL, DL_MERGE_ALL = 0, 1
DL_FLAG_FUSED_MERGE = 1
DL_FLAG_KLA = 4
DL_FLAG_BASE_Q8 = 8
DL_E4M3 = 2
DL_CONV_SILU = 1
DL_SSM_SOFTPLUS = 1

VARIANT_IDS = {"gdn": DL_GDN, "kda": DL_KDA, "rwkv6": DL_RWKV6, "gdn2": DL_GDN2}
DTYPE_IDS = {"f32": DL_F32, "bf16": DL_BF16}
OUT_DTYPE_IDS = {**DTYPE_IDS, "e4m3": DL_E4M3}
_TORCH_IN = {DL_F32: torch.float32, DL_BF16: torch.bfloat16, DL_E4M3: torch.float8_e4m3fn}


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with "
            "`python -m linear_attention_recurrent_deltalog_b200.build` (there is no CPU fallback)")
    return ctypes.CDLL(_LIB_PATH)


_lib = _load()


class dl_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("variant", "B", "H", "d_k", "d_v", "L", "in_dtype", "flags", "step_split")] + \
        [("kla_eps", ctypes.c_float)]


class dl_conv_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("C", "W", "in_dtype", "flags")]


class dl_ssm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("H", "G", "d_k", "d_v", "in_dtype", "flags")]


class dl_ssm_io(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "dt", "a", "d", "dt_bias", "o")] + \
        [(n, ctypes.c_int64) for n in ("ldq", "ldk", "ldv", "lddt", "ldo")]


class dl_norm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("D", "in_dtype", "out_dtype", "block")] + \
        [("eps", ctypes.c_float)]


_pack_ssm_io = struct.Struct("=8Q5q").pack  # dl_ssm_io's layout, quicker than the Structure
assert struct.calcsize("=8Q5q") == ctypes.sizeof(dl_ssm_io)

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_SZ = ctypes.POINTER(ctypes.c_size_t)
_CFG = ctypes.POINTER(dl_config)
_CONV = ctypes.POINTER(dl_conv_config)
_SSM = ctypes.POINTER(dl_ssm_config)
_NORM = ctypes.POINTER(dl_norm_config)

_SIGS = {
    "dl_state_bytes": (_I, [_CFG, _SZ, _SZ, _SZ]),
    "dl_state_create": (_I, [_CFG, _P, _P, _P, ctypes.POINTER(_P)]),
    "dl_state_reset": (_I, [_P, _P, ctypes.POINTER(ctypes.c_int32), _P]),
    "dl_state_load_seqs": (_I, [_P, _I, ctypes.POINTER(ctypes.c_int32), _P, _P]),
    "dl_decode_step": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "dl_merge": (_I, [_P, _I, _P]),
    "dl_materialize": (_I, [_P, _P, _P]),
    "dl_eager_step": (_I, [_CFG, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "dl_conv_prompt": (_I, [_CONV, _I, _P, _P, _L, _P, _P, _P, _P, _P, _L, _P]),
    "dl_conv_step": (_I, [_CONV, _I, _P, _L, _P, _P, _P, _P, _L, _P]),
    "dl_ssm_bytes": (_I, [_SSM, _I, _P, _SZ]),
    "dl_ssm_prompt": (_I, [_SSM, _I, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "dl_ssm_step": (_I, [_SSM, _I, _P, _P, _P]),
    "dl_norm": (_I, [_NORM, _L, _P, _L, _P, _L, _P, _P, _L, _P, _L, _P, _P]),
    "dl_state_fill": (_I, [_P, ctypes.POINTER(ctypes.c_int32)]),
    "dl_state_destroy": (_I, [_P]),
    "dl_device_error": (_I, [_P, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32),
                             _I, _P]),
    "dl_selftest_wait_timeout": (_I, [ctypes.POINTER(ctypes.c_int32), _P]),
    "dl_launch_count": (ctypes.c_uint64, []),
    "dl_status_string": (ctypes.c_char_p, [_I]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)
LIB_PATH = _LIB_PATH


class DeltaLogError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {dl_status_string(status)} ({status})")


def _check(status: int, call: str) -> int:
    if status < 0:
        raise DeltaLogError(status, call)
    return status


def dl_status_string(status: int) -> str:
    return _lib.dl_status_string(int(status)).decode()


def dl_launch_count() -> int:
    return int(_lib.dl_launch_count())


def dl_selftest_wait_timeout(stream=None) -> int:
    """Runs the bounded-wait failure path once; returns the recorded code."""
    code = ctypes.c_int32()
    _check(_lib.dl_selftest_wait_timeout(ctypes.byref(code), _stream(stream)),
           "dl_selftest_wait_timeout")
    return code.value


# ----------------------------------------------------------------- config

@dataclasses.dataclass(frozen=True)
class Config:
    """Python mirror of ``dl_config``."""

    variant: str
    B: int
    H: int
    d_k: int
    d_v: int
    L: int
    in_dtype: str = "bf16"
    fused_merge: bool = False
    step_split: int = 0
    kla_eps: Optional[float] = None  # set: beta carries the KLA gate eta
    base: str = "f32"                # "f32", or "q8": int8 codes + row scales

    def c(self) -> dl_config:
        if self.base not in ("f32", "q8"):
            raise ValueError(f"base must be 'f32' or 'q8', not {self.base!r}")
        flags = (DL_FLAG_FUSED_MERGE if self.fused_merge else 0) | \
            (DL_FLAG_KLA if self.kla_eps is not None else 0) | \
            (DL_FLAG_BASE_Q8 if self.base == "q8" else 0)
        return dl_config(VARIANT_IDS[self.variant], self.B, self.H, self.d_k, self.d_v, self.L,
                         DTYPE_IDS[self.in_dtype], flags, self.step_split,
                         0.0 if self.kla_eps is None else float(self.kla_eps))

    @property
    def heads(self) -> int:
        return self.B * self.H

    @property
    def torch_in_dtype(self) -> torch.dtype:
        return _TORCH_IN[DTYPE_IDS[self.in_dtype]]


@dataclasses.dataclass(frozen=True)
class ConvConfig:
    """Python mirror of ``dl_conv_config``: a depthwise causal convolution of
    ``W`` taps over ``C`` channels."""

    C: int
    W: int
    in_dtype: str = "bf16"
    silu: bool = True

    @functools.cached_property
    def c(self) -> dl_conv_config:
        return dl_conv_config(self.C, self.W, DTYPE_IDS[self.in_dtype],
                              DL_CONV_SILU if self.silu else 0)

    @functools.cached_property
    def ref(self):
        return ctypes.byref(self.c)

    @functools.cached_property
    def torch_in_dtype(self) -> torch.dtype:
        return _TORCH_IN[DTYPE_IDS[self.in_dtype]]


@dataclasses.dataclass(frozen=True)
class SsmConfig:
    """Python mirror of ``dl_ssm_config``: ``H`` heads of d_v x d_k states, q
    and k shared by the heads of each of ``G`` groups."""

    H: int
    G: int
    d_k: int
    d_v: int
    in_dtype: str = "bf16"
    softplus: bool = True

    @functools.cached_property
    def c(self) -> dl_ssm_config:
        return dl_ssm_config(self.H, self.G, self.d_k, self.d_v, DTYPE_IDS[self.in_dtype],
                             DL_SSM_SOFTPLUS if self.softplus else 0)

    @functools.cached_property
    def ref(self):
        return ctypes.byref(self.c)

    @functools.cached_property
    def torch_in_dtype(self) -> torch.dtype:
        return _TORCH_IN[DTYPE_IDS[self.in_dtype]]


@dataclasses.dataclass(frozen=True)
class NormConfig:
    """Python mirror of ``dl_norm_config``: rows of ``D``; ``out_dtype`` "f32",
    "bf16" or "e4m3", the last with one scale per ``block`` (128) channels or
    per row (0)."""

    D: int
    in_dtype: str = "bf16"
    out_dtype: str = "bf16"
    block: int = 0
    eps: float = 1e-6

    @functools.cached_property
    def c(self) -> dl_norm_config:
        return dl_norm_config(self.D, DTYPE_IDS[self.in_dtype], OUT_DTYPE_IDS[self.out_dtype],
                              self.block, float(self.eps))

    @functools.cached_property
    def ref(self):
        return ctypes.byref(self.c)

    @functools.cached_property
    def torch_in_dtype(self) -> torch.dtype:
        return _TORCH_IN[DTYPE_IDS[self.in_dtype]]

    @functools.cached_property
    def torch_out_dtype(self) -> torch.dtype:
        return _TORCH_IN[OUT_DTYPE_IDS[self.out_dtype]]

    @functools.cached_property
    def scales_per_row(self) -> int:
        return -(-self.D // self.block) if self.block else 1


# ----------------------------------------------------------------- marshalling

def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _cuda_calls():
    """-> (current device's index, handle of a device's current stream), by torch's quick forms where
    it has them: current_stream() builds a Stream object per call."""
    return (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
            getattr(torch._C, "_cuda_getCurrentRawStream",
                    lambda dev: torch.cuda.current_stream(dev).cuda_stream))


_current_device, _current_stream = _cuda_calls()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream(_current_device()) if torch.cuda.is_initialized() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _need(t, name: str, numel: int, dtype: torch.dtype) -> None:
    """Buffer checks that keep every kernel access inside the tensor."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        if isinstance(t, int):
            return
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, need {numel}")


def _flat(t, name: str, numel: int, dtype: torch.dtype) -> Optional[int]:
    """The same for a tensor (or None); returns its address."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.numel() >= numel and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    _need(t, name, numel, dtype)
    return t.data_ptr()


def _check_step_tensors(cfg: Config, q, k, v, decay, beta, bonus, o) -> None:
    BH, dk, dv = cfg.heads, cfg.d_k, cfg.d_v
    tin = cfg.torch_in_dtype
    _need(q, "q", BH * dk, tin)
    _need(k, "k", BH * dk, tin)
    _need(v, "v", BH * dv, tin)
    _need(decay, "decay", BH * (1 if cfg.variant == "gdn" else dk), torch.float32)
    if cfg.variant == "rwkv6":
        _need(bonus, "bonus", cfg.H * dk, torch.float32)
    elif cfg.variant == "gdn2":           # beta: erase gate; bonus: write gate
        _need(beta, "beta", BH * dk, torch.float32)
        _need(bonus, "bonus", BH * dv, torch.float32)
    else:
        _need(beta, "beta", BH, torch.float32)
    _need(o, "o", BH * dv, torch.float32)


def _rows(t, name: str, rows: int, cols: int, dtype: torch.dtype) -> int:
    """Checks a tensor of at least ``rows`` rows of ``cols`` elements and
    returns its row stride: [rows, cols], or [rows, a, b] with a * b = cols,
    whose rows may lie apart but are contiguous themselves."""
    try:  # the common case first: the checks cost as much as a small kernel
        if t.dtype is dtype:
            n, width = t.shape
            ld, unit = t.stride()
            if width == cols and unit == 1 and n >= rows and (ld >= cols or n <= 1):
                return ld if n > 1 else cols  # a single row's stride is never used
    except (AttributeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    shape, ld = t.shape, t.stride()
    n = shape[0] if shape else 0
    if len(shape) == 2:
        ok = shape[1] == cols and (ld[1] == 1 or cols == 1)
    else:
        ok = len(shape) == 3 and shape[1] * shape[2] == cols and \
            (n == 0 or t[0].is_contiguous())
    if not ok:
        raise ValueError(f"{name}: expected rows of {cols} contiguous elements, got shape "
                         f"{tuple(shape)} with strides {ld}")
    if n < rows:
        raise ValueError(f"{name}: {n} rows, need {rows}")
    if n <= 1:
        return cols
    if ld[0] < cols:
        raise ValueError(f"{name}: rows overlap (stride {ld[0]}, {cols} elements)")
    return ld[0]


def _on_device(names: str, *tensors) -> Optional[int]:
    """Every tensor (or None) on the current CUDA device, whose stream the call uses."""
    dev = _current_device() if torch.cuda.is_initialized() else None
    for t in tensors:
        if t is not None and t.get_device() != dev:
            name = names.split()[[x is t for x in tensors].index(True)]
            raise ValueError(f"{name}: must be on the current CUDA device, not {t.device}")
    return dev


def _stream_on(dev: int, stream) -> int:
    """The given stream's handle, or the current one's of the current device ``dev``, to which a
    given one has to belong (a bare handle does not say)."""
    if stream is None:
        return _current_stream(dev)
    if getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"stream: must belong to the current CUDA device {dev}, not {stream}")
    return _stream(stream)


def _workspace(nbytes: int, device, stream) -> torch.Tensor:
    """Memory for one call on ``stream``, from that stream's pool: what it held before and what it
    is given to afterwards then run before and after the call."""
    if stream is None or nbytes == 0:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = _stream(stream)
        if stream == 2:  # the per-thread default stream: another one in every thread
            raise ValueError("workspace: needed on the per-thread default stream")
        # 0 and 1 both name the legacy default stream
        stream = torch.cuda.default_stream(device) if stream < 2 else \
            torch.cuda.ExternalStream(stream, device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


_INT32 = np.dtype(np.int32)


def _starts(starts):
    """-> (address of a host int32 array, n, rows, the array): sequence s holds rows starts[s] ..
    starts[s+1] - 1."""
    a = starts if isinstance(starts, np.ndarray) else np.asarray(starts)
    if a.ndim != 1 or a.size < 1 or a.dtype.kind not in "iu":
        raise ValueError("starts: expected n + 1 integers on the host")
    if a.dtype is not _INT32 or not a.flags.c_contiguous:
        if int(a.min()) < 0 or int(a.max()) > 0x7fffffff:
            raise ValueError("starts: must fit int32 and be >= 0")
        a = np.ascontiguousarray(a, dtype=np.int32)
    return a.__array_interface__["data"][0], a.size - 1, int(a[-1]), a


# ----------------------------------------------------------------- C entry points

def dl_state_bytes(cfg: Config):
    """-> (base_bytes, log_bytes, meta_bytes)"""
    b, l, m = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    c = cfg.c()
    _check(_lib.dl_state_bytes(ctypes.byref(c), ctypes.byref(b), ctypes.byref(l), ctypes.byref(m)),
           "dl_state_bytes")
    return b.value, l.value, m.value


def dl_state_create(cfg: Config, base, log, meta) -> int:
    sizes = dl_state_bytes(cfg)
    for t, n, name in zip((base, log, meta), sizes, ("base", "log", "meta")):
        if isinstance(t, torch.Tensor) and t.numel() * t.element_size() < n:
            raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, need {n}")
    h = _P()
    c = cfg.c()
    _check(_lib.dl_state_create(ctypes.byref(c), _ptr(base), _ptr(log), _ptr(meta),
                                ctypes.byref(h)), "dl_state_create")
    return h.value


def dl_state_reset(handle: int, cfg: Config, S0=None, fill0: Optional[Sequence[int]] = None,
                   stream=None) -> None:
    _need(S0, "S0", cfg.heads * cfg.d_v * cfg.d_k, torch.float32)
    arr = None
    if fill0 is not None:
        if len(fill0) != cfg.B:
            raise ValueError("fill0 must have B entries")
        arr = (ctypes.c_int32 * cfg.B)(*[int(x) for x in fill0])
    _check(_lib.dl_state_reset(handle, _ptr(S0), arr, _stream(stream)), "dl_state_reset")


def dl_state_load_seqs(handle: int, cfg: Config, seqs: Sequence[int], S=None, stream=None) -> None:
    n = len(seqs)
    _need(S, "S", n * cfg.H * cfg.d_v * cfg.d_k, torch.float32)
    arr = (ctypes.c_int32 * max(n, 1))(*[int(x) for x in seqs])
    _check(_lib.dl_state_load_seqs(handle, n, arr, _ptr(S), _stream(stream)), "dl_state_load_seqs")


def dl_decode_step(handle: int, cfg: Config, q, k, v, decay, beta, bonus, o, stream=None) -> None:
    _check_step_tensors(cfg, q, k, v, decay, beta, bonus, o)
    _check(_lib.dl_decode_step(handle, _ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(beta),
                               _ptr(bonus), _ptr(o), _stream(stream)), "dl_decode_step")


def dl_merge(handle: int, mode: int = DL_MERGE_FULL, stream=None) -> None:
    _check(_lib.dl_merge(handle, int(mode), _stream(stream)), "dl_merge")


def dl_materialize(handle: int, cfg: Config, S_out, stream=None) -> None:
    _need(S_out, "S_out", cfg.heads * cfg.d_v * cfg.d_k, torch.float32)
    _check(_lib.dl_materialize(handle, _ptr(S_out), _stream(stream)), "dl_materialize")


def dl_eager_step(cfg: Config, S, q, k, v, decay, beta, bonus, o, stream=None) -> None:
    _need(S, "S", cfg.heads * cfg.d_v * cfg.d_k, torch.float32)
    _check_step_tensors(cfg, q, k, v, decay, beta, bonus, o)
    c = cfg.c()
    _check(_lib.dl_eager_step(ctypes.byref(c), _ptr(S), _ptr(q), _ptr(k), _ptr(v), _ptr(decay),
                              _ptr(beta), _ptr(bonus), _ptr(o), _stream(stream)), "dl_eager_step")


def dl_conv_prompt(cfg: ConvConfig, starts, x, w, bias, h0, h1, y, stream=None) -> None:
    """y = short causal convolution of packed sequences; ``h0`` (or None) and
    ``h1`` (or None, or ``h0``) are the states [n, W-1, C] before and after."""
    at, n, rows, keep = _starts(starts)
    C, W, t = cfg.C, cfg.W, cfg.torch_in_dtype
    ldx = _rows(x, "x", rows, C, t)
    ldy = _rows(y, "y", rows, C, t)
    if w is None:
        raise TypeError("w: expected a torch.Tensor")
    pw = _flat(w, "w", C * W, torch.float32)
    pb = _flat(bias, "bias", C, torch.float32)
    ph0 = _flat(h0, "h0", n * (W - 1) * C, t)
    ph1 = _flat(h1, "h1", n * (W - 1) * C, t)
    dev = _on_device("x w bias h0 h1 y", x, w, bias, h0, h1, y)
    rc = _lib.dl_conv_prompt(cfg.ref, n, at, x.data_ptr(), ldx, pw, pb, ph0, ph1,
                             y.data_ptr(), ldy, _stream_on(dev, stream))
    if rc:
        _check(rc, "dl_conv_prompt")


def dl_conv_step(cfg: ConvConfig, x, w, bias, h, y, stream=None) -> None:
    """One token of each of x.shape[0] sequences; the state ``h`` is updated in place."""
    B = x.shape[0]
    C, W, t = cfg.C, cfg.W, cfg.torch_in_dtype
    ldx = _rows(x, "x", B, C, t)
    ldy = _rows(y, "y", B, C, t)
    if w is None or h is None:
        raise TypeError("w, h: expected a torch.Tensor")
    pw = _flat(w, "w", C * W, torch.float32)
    pb = _flat(bias, "bias", C, torch.float32)
    ph = _flat(h, "h", B * (W - 1) * C, t)
    dev = _on_device("x w bias h y", x, w, bias, h, y)
    rc = _lib.dl_conv_step(cfg.ref, B, x.data_ptr(), ldx, pw, pb, ph, y.data_ptr(), ldy,
                           _stream_on(dev, stream))
    if rc:
        _check(rc, "dl_conv_step")


def dl_ssm_bytes(cfg: SsmConfig, starts) -> int:
    """Bytes of workspace ``dl_ssm_prompt`` needs for these lengths."""
    at, n, _, keep = _starts(starts)
    b = ctypes.c_size_t()
    _check(_lib.dl_ssm_bytes(cfg.ref, n, at, ctypes.byref(b)),
           "dl_ssm_bytes")
    return b.value


def _ssm_io(cfg: SsmConfig, rows: int, n: int, q, k, v, dt, a, d, dt_bias, o, S0, S1):
    """-> (dl_ssm_io as bytes, addresses of S0 and S1, the device)"""
    t, H, f32 = cfg.torch_in_dtype, cfg.H, torch.float32
    nk, nv = cfg.G * cfg.d_k, H * cfg.d_v
    ldq, ldk = _rows(q, "q", rows, nk, t), _rows(k, "k", rows, nk, t)
    ldv, ldo = _rows(v, "v", rows, nv, t), _rows(o, "o", rows, nv, t)
    lddt = _rows(dt, "dt", rows, H, f32)
    if a is None:
        raise TypeError("a: expected a torch.Tensor")
    pa, pd, pb = _flat(a, "a", H, f32), _flat(d, "d", H, f32), _flat(dt_bias, "dt_bias", H, f32)
    p0 = _flat(S0, "S0", n * nv * cfg.d_k, f32)
    p1 = _flat(S1, "S1", n * nv * cfg.d_k, f32)
    dev = _on_device("q k v dt a d dt_bias o S0 S1", q, k, v, dt, a, d, dt_bias, o, S0, S1)
    return _pack_ssm_io(q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(), pa, pd or 0,
                        pb or 0, o.data_ptr(), ldq, ldk, ldv, lddt, ldo), p0, p1, dev


def dl_ssm_prompt(cfg: SsmConfig, starts, q, k, v, dt, a, d, dt_bias, S0, S1, o, workspace=None,
                  stream=None) -> None:
    """Selective state space scan of packed sequences; ``S0`` (or None) and
    ``S1`` (or None, or ``S0``) are the states [n, H, d_v, d_k] before and
    after.  ``workspace``: a uint8 tensor of ``dl_ssm_bytes`` (allocated for
    the call, on its stream, when None)."""
    at, n, rows, keep = _starts(starts)
    io, p0, p1, dev = _ssm_io(cfg, rows, n, q, k, v, dt, a, d, dt_bias, o, S0, S1)
    on = _stream_on(dev, stream)
    if workspace is None:
        workspace = _workspace(dl_ssm_bytes(cfg, keep), q.device, stream)
    elif not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace: expected a torch.Tensor")
    nb = workspace.numel() * workspace.element_size()
    if not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    _on_device("workspace", workspace)
    rc = _lib.dl_ssm_prompt(cfg.ref, n, at, io, p0, p1,
                            workspace.data_ptr() if nb else None, nb, on)
    if rc:
        _check(rc, "dl_ssm_prompt")


def dl_ssm_step(cfg: SsmConfig, q, k, v, dt, a, d, dt_bias, S, o, stream=None) -> None:
    """One token of each of q.shape[0] sequences; the state ``S`` [B, H, d_v,
    d_k] is updated in place."""
    B = q.shape[0]
    if S is None:
        raise TypeError("S: expected a torch.Tensor")
    io, p, _, dev = _ssm_io(cfg, B, B, q, k, v, dt, a, d, dt_bias, o, S, None)
    rc = _lib.dl_ssm_step(cfg.ref, B, io, p, _stream_on(dev, stream))
    if rc:
        _check(rc, "dl_ssm_step")


def dl_norm(cfg: NormConfig, x, w, out, res=None, res_out=None, scales=None, stream=None) -> None:
    """out = RMS norm of x (+ res), times w; ``res_out`` takes x + res.  An
    "e4m3" output needs ``scales`` [rows, cfg.scales_per_row]."""
    rows, D, t = x.shape[0], cfg.D, cfg.torch_in_dtype
    ldx = _rows(x, "x", rows, D, t)
    ldo = _rows(out, "out", rows, D, cfg.torch_out_dtype)
    ldr = ldro = D
    pr = pro = None
    if res is not None:
        ldr, pr = _rows(res, "res", rows, D, t), res.data_ptr()
    if res_out is not None:
        ldro, pro = _rows(res_out, "res_out", rows, D, t), res_out.data_ptr()
    if w is None:
        raise TypeError("w: expected a torch.Tensor")
    pw = _flat(w, "w", D, torch.float32)
    if scales is None and cfg.out_dtype == "e4m3":
        raise TypeError("scales: expected a torch.Tensor for an e4m3 output")
    ps = _flat(scales, "scales", rows * cfg.scales_per_row, torch.float32)
    dev = _on_device("x w out res res_out scales", x, w, out, res, res_out, scales)
    rc = _lib.dl_norm(cfg.ref, rows, x.data_ptr(), ldx, pr, ldr, pw, pro, ldro, out.data_ptr(), ldo,
                      ps, _stream_on(dev, stream))
    if rc:
        _check(rc, "dl_norm")


def dl_state_fill(handle: int, cfg: Config):
    arr = (ctypes.c_int32 * cfg.B)()
    _check(_lib.dl_state_fill(handle, arr), "dl_state_fill")
    return list(arr)


def dl_state_destroy(handle: Optional[int]) -> None:
    _check(_lib.dl_state_destroy(handle), "dl_state_destroy")


def dl_device_error(handle: Optional[int], clear: bool = False, stream=None):
    code, head = ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.dl_device_error(handle, ctypes.byref(code), ctypes.byref(head), int(clear),
                                _stream(stream)), "dl_device_error")
    return code.value, head.value


# ----------------------------------------------------------------- convenience

class DeltaLogState:
    """A state whose three buffers are torch device tensors (allocation is
    torch's; the library only borrows them)."""

    def __init__(self, cfg: Config, device="cuda"):
        self.cfg = cfg
        nb, nl, nm = dl_state_bytes(cfg)
        self.base = torch.empty(nb // 4, dtype=torch.float32, device=device)
        self.log = torch.empty(nl, dtype=torch.uint8, device=device)
        self.meta = torch.empty(nm, dtype=torch.uint8, device=device)
        self.handle = dl_state_create(cfg, self.base, self.log, self.meta)

    def reset(self, S0=None, fill0=None, stream=None) -> None:
        dl_state_reset(self.handle, self.cfg, S0, fill0, stream)

    def load_seqs(self, seqs, S=None, stream=None) -> None:
        dl_state_load_seqs(self.handle, self.cfg, seqs, S, stream)

    def step(self, q, k, v, decay, beta=None, bonus=None, o=None, stream=None):
        if o is None:
            o = torch.empty(self.cfg.heads * self.cfg.d_v, dtype=torch.float32, device=self.base.device)
        dl_decode_step(self.handle, self.cfg, q, k, v, decay, beta, bonus, o, stream)
        return o

    def merge(self, mode: int = DL_MERGE_FULL, stream=None) -> None:
        dl_merge(self.handle, mode, stream)

    def materialize(self, out=None, stream=None):
        if out is None:
            out = torch.empty(self.cfg.heads * self.cfg.d_v * self.cfg.d_k, dtype=torch.float32,
                              device=self.base.device)
        dl_materialize(self.handle, self.cfg, out, stream)
        return out

    def fill(self):
        return dl_state_fill(self.handle, self.cfg)

    # An int8 base in the layout deltalog.h documents: codes [B*H, d_v, d_k]
    # with each row's 16-byte chunks stored XOR-swizzled (chunk ^ (row mod 8)
    # for d_k = 128, chunk ^ ((row / 2) mod 4) for d_k = 64), then the fp32
    # row scales [B*H, d_v] at the next 256-byte boundary.
    def _scale_offset(self) -> int:
        n = self.cfg.heads * self.cfg.d_v * self.cfg.d_k
        return (n + 255) // 256 * 256

    def _q8_perm(self) -> torch.Tensor:
        """Physical position of each logical (row, c) code within a head."""
        if getattr(self, "_perm", None) is None:
            dv, dk = self.cfg.d_v, self.cfg.d_k
            r = torch.arange(dv).view(dv, 1)
            c = torch.arange(dk).view(1, dk)
            sw = (r & 7) if dk == 128 else ((r >> 1) & 3)
            self._perm = (r * dk + (((c >> 4) ^ sw) << 4) + (c & 15)).reshape(-1).to(self.base.device)
        return self._perm

    def base_codes_raw(self) -> torch.Tensor:
        """The stored int8 codes [B*H, d_v*d_k] in their swizzled order (a view)."""
        if self.cfg.base != "q8":
            raise ValueError("base_codes_raw: the base is fp32")
        c = self.cfg
        return self.base.view(torch.uint8)[:c.heads * c.d_v * c.d_k].view(torch.int8).view(
            c.heads, c.d_v * c.d_k)

    def base_codes(self, heads=None) -> torch.Tensor:
        """The codes of `heads` (all when None) in logical order [n, d_v, d_k] (a copy)."""
        raw = self.base_codes_raw()
        if heads is not None:
            raw = raw.index_select(0, torch.as_tensor(heads, device=raw.device))
        return raw[:, self._q8_perm()].view(-1, self.cfg.d_v, self.cfg.d_k)

    def set_base_codes(self, heads, codes: torch.Tensor) -> None:
        """Writes logical-order codes [n, d_v, d_k] of `heads` into the base."""
        raw = self.base_codes_raw()
        heads = torch.as_tensor(heads, device=raw.device)
        tmp = torch.empty((heads.numel(), raw.shape[1]), dtype=torch.int8, device=raw.device)
        tmp[:, self._q8_perm()] = codes.reshape(heads.numel(), -1).to(device=raw.device,
                                                                      dtype=torch.int8)
        raw.index_copy_(0, heads, tmp)

    def base_scales(self) -> torch.Tensor:
        """The fp32 row scales [B*H, d_v] (a view)."""
        if self.cfg.base != "q8":
            raise ValueError("base_scales: the base is fp32")
        c = self.cfg
        off = self._scale_offset()
        raw = self.base.view(torch.uint8)
        return raw[off:off + c.heads * c.d_v * 4].view(torch.float32).view(c.heads, c.d_v)

    def device_error(self, clear: bool = False, stream=None):
        return dl_device_error(self.handle, clear, stream)

    def close(self) -> None:
        if self.handle is not None:
            dl_state_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
