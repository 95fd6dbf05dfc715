"""SketchSSM windowed linear-attention decode for AMD Instinct MI355X (gfx950).

A thin ctypes binding over ``libsketchssm.so`` (C ABI in
``include/sketchssm.h``). Each function here marshals its arguments and calls
the library entry point of the same name; every step of the decode path runs
in the library's HIP kernels. Tensors are PyTorch device tensors (PyTorch
provides memory and streams only) or raw device addresses as ``int``; a call
whose pointers and stream are all ``int`` goes straight to the library (the
library still checks the arguments, but not their sizes).

If the library has not been built this module raises on import: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Union

__all__ = [
    "Dims", "SSMError", "MAMBA2", "GDN", "KDA", "IN_BF16", "IN_F32", "RULES",
    "abi_version", "buffer_append", "window_update_refresh", "sketch_decode_step",
    "full_read_decode_step", "recurrent_decode_step", "window_update_refresh_ranked",
    "sketch_decode_step_ranked", "rank_offsets", "window_update_refresh_varlen",
    "sketch_decode_step_varlen", "decode_step_varlen", "window_update_refresh_ls",
    "sketch_decode_step_ls", "scan_sizes", "scan_plan", "scan_forward", "scan_backward",
    "window_plan", "ConvDims", "conv_sizes", "conv_forward", "conv_backward", "conv_step",
    "SelectiveDims", "selective_sizes", "selective_forward", "selective_backward",
    "selective_step", "NormDims", "gated_norm_sizes", "gated_norm", "gated_norm_backward",
    "fit_basis", "stream_probe", "SKETCH_F32", "SKETCH_BF16", "LIB_PATH", "HEADER",
    "declared_symbols", "numel", "library",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsketchssm.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "sketchssm.h")

MAMBA2, GDN, KDA = 0, 1, 2
RULES = {"mamba2": MAMBA2, "gdn": GDN, "kda": KDA}
IN_BF16, IN_F32 = 0, 1
SKETCH_F32, SKETCH_BF16 = 0, 1

STATUS = {0: "SSM_OK", 1: "SSM_E_NULL", 2: "SSM_E_SHAPE", 3: "SSM_E_ALIGN", 4: "SSM_E_RANGE",
          5: "SSM_E_ALIAS", 6: "SSM_E_LAUNCH"}


class SSMError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status
        self.detail = detail


class Dims(ctypes.Structure):
    """ssm_dims: rule, in_dtype, batch, heads, d_k, d_v, window, rank, sketch_dtype."""

    _fields_ = [(n, ctypes.c_int32) for n in
                ("rule", "in_dtype", "batch", "heads", "d_k", "d_v", "window", "rank",
                 "sketch_dtype")]

    @classmethod
    def make(cls, rule, in_dtype, batch, heads, d_k, d_v, window, rank,
             sketch_dtype="f32") -> "Dims":
        if isinstance(rule, str):
            rule = RULES[rule]
        if isinstance(in_dtype, str):
            in_dtype = {"bf16": IN_BF16, "f32": IN_F32}[in_dtype]
        if isinstance(sketch_dtype, str):
            sketch_dtype = {"f32": SKETCH_F32, "bf16": SKETCH_BF16}[sketch_dtype]
        return cls(rule, in_dtype, batch, heads, d_k, d_v, window, rank, sketch_dtype)

    def __repr__(self):
        return "Dims(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


_IN_DTYPES = {"bf16": IN_BF16, "f32": IN_F32}
_ACTIVATIONS = {"none": 0, "silu": 1, "sigmoid": 2}
_GATES = {"none": 0, "after": 1, "before": 2}
CONV_PARTS = 4


def _fields_repr(x):
    vals = ((n, getattr(x, n)) for n, _ in x._fields_)
    return type(x).__name__ + "(" + ", ".join(
        f"{n}={list(v) if isinstance(v, ctypes.Array) else v}" for n, v in vals) + ")"


class ConvDims(ctypes.Structure):
    """ssm_conv_dims: the short convolution of 1 to 4 parts of a layer's inputs."""

    _fields_ = ([(n, ctypes.c_int32) for n in ("in_dtype", "batch", "taps", "activation", "parts")]
                + [("channels", ctypes.c_int32 * CONV_PARTS), ("norm", ctypes.c_int32 * CONV_PARTS),
                   ("scale", ctypes.c_float * CONV_PARTS), ("eps", ctypes.c_float)])
    __repr__ = _fields_repr

    @classmethod
    def make(cls, in_dtype, batch, taps, channels, *, norm=None, scale=None, activation="silu",
             eps=1e-6) -> "ConvDims":
        """channels: of each part. norm: channels of a head that are normalised together, per
        part (0: no norm); scale: what a normalised part is multiplied with."""
        channels = [channels] if isinstance(channels, int) else list(channels)
        n = len(channels)
        norm = [0] * n if norm is None else [int(x) for x in norm]
        scale = [1.0] * n if scale is None else [float(x) for x in scale]
        if not 1 <= n <= CONV_PARTS or len(norm) != n or len(scale) != n:
            raise ValueError(f"{n} parts with {len(norm)} norms and {len(scale)} scales; 1 to {CONV_PARTS} parts")
        d = cls(_IN_DTYPES.get(in_dtype, in_dtype), batch, taps, _ACTIVATIONS.get(activation, activation), n)
        d.channels[:n], d.norm[:n], d.scale[:n], d.eps = channels, norm, scale, eps
        return d


class SelectiveDims(ctypes.Structure):
    """ssm_selective_dims: in_dtype, batch, channels, d_state, groups, softplus."""

    _fields_ = [(n, ctypes.c_int32) for n in
                ("in_dtype", "batch", "channels", "d_state", "groups", "softplus")]
    __repr__ = _fields_repr

    @classmethod
    def make(cls, in_dtype, batch, channels, d_state, *, groups=1, softplus=True) -> "SelectiveDims":
        return cls(_IN_DTYPES.get(in_dtype, in_dtype), batch, channels, d_state, groups, int(softplus))


class NormDims(ctypes.Structure):
    """ssm_norm_dims: the norm of groups of `width` channels with a gate."""

    _fields_ = ([(n, ctypes.c_int32) for n in ("x_dtype", "in_dtype", "groups", "width", "gate",
                                               "activation", "shared", "centred")]
                + [("eps", ctypes.c_float)])
    __repr__ = _fields_repr

    @classmethod
    def make(cls, x_dtype, in_dtype, groups, width, *, gate="after", activation="silu", shared=False,
             centred=False, eps=1e-5) -> "NormDims":
        """gate: "after" or "before" the norm, or "none"; shared: one weight row for all groups."""
        return cls(_IN_DTYPES.get(x_dtype, x_dtype), _IN_DTYPES.get(in_dtype, in_dtype), groups,
                   width, _GATES.get(gate, gate), _ACTIVATIONS.get(activation, activation),
                   int(shared), int(centred), eps)


def _load():
    # The tensors handed to the library come from PyTorch's HIP runtime, and the
    # process must hold exactly one HIP runtime: load torch first so that the
    # library's libamdhip64.so.7 dependency resolves to the copy torch loaded.
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python sketched_recurrent_state_amd/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, dp = ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(Dims)
    lib.ssm_abi_version.restype = i32
    lib.ssm_abi_version.argtypes = []
    lib.ssm_status_string.restype = ctypes.c_char_p
    lib.ssm_status_string.argtypes = [i32]
    lib.ssm_last_error.restype = ctypes.c_char_p
    lib.ssm_last_error.argtypes = []
    lib.ssm_buffer_append.restype = i32
    lib.ssm_buffer_append.argtypes = [dp] + [vp] * 8 + [i32, vp]
    lib.ssm_window_update_refresh.restype = i32
    lib.ssm_window_update_refresh.argtypes = [dp] + [vp] * 7 + [i32, vp]
    lib.ssm_sketch_decode_step.restype = i32
    lib.ssm_sketch_decode_step.argtypes = [dp] + [vp] * 11 + [i32, vp, vp]
    ip = ctypes.POINTER(ctypes.c_int32)
    lib.ssm_window_update_refresh_ranked.restype = i32
    lib.ssm_window_update_refresh_ranked.argtypes = [dp, ip] + [vp] * 7 + [i32, vp]
    lib.ssm_sketch_decode_step_ranked.restype = i32
    lib.ssm_sketch_decode_step_ranked.argtypes = [dp, ip] + [vp] * 11 + [i32, vp, vp]
    lib.ssm_window_update_refresh_varlen.restype = i32
    lib.ssm_window_update_refresh_varlen.argtypes = [dp, i32] + [vp] * 9 + [vp]
    lib.ssm_sketch_decode_step_varlen.restype = i32
    lib.ssm_sketch_decode_step_varlen.argtypes = [dp, i32] + [vp] * 15
    lib.ssm_decode_step_varlen.restype = i32
    lib.ssm_decode_step_varlen.argtypes = [dp, i32, vp, vp, vp, i32] + [vp] * 15 + [vp]
    lib.ssm_recurrent_decode_step.restype = i32
    lib.ssm_recurrent_decode_step.argtypes = [dp] + [vp] * 7 + [vp]
    lib.ssm_full_read_decode_step.restype = i32
    lib.ssm_full_read_decode_step.argtypes = [dp] + [vp] * 10 + [i32, vp, vp]
    lib.ssm_window_update_refresh_ls.restype = i32
    lib.ssm_window_update_refresh_ls.argtypes = [dp] + [vp] * 8 + [i32, vp]
    lib.ssm_sketch_decode_step_ls.restype = i32
    lib.ssm_sketch_decode_step_ls.argtypes = [dp] + [vp] * 11 + [i32, vp, vp]
    lib.ssm_fit_basis.restype = i32
    lib.ssm_fit_basis.argtypes = [dp, vp, i32, vp, vp]
    i64 = ctypes.c_int64
    lib.ssm_scan_sizes.restype = i32
    lib.ssm_scan_sizes.argtypes = [dp, i32] + [ctypes.POINTER(i64)] * 3
    lib.ssm_scan_plan.restype = i32
    lib.ssm_scan_plan.argtypes = [vp, i32, i32, vp, vp]
    lib.ssm_scan_forward.restype = i32
    lib.ssm_scan_forward.argtypes = [dp, i32, vp, i32] + [vp] * 10 + [i64, vp]
    lib.ssm_scan_backward.restype = i32
    lib.ssm_scan_backward.argtypes = [dp, i32] + [vp] * 16 + [i64, vp]
    lib.ssm_window_plan.restype = i32
    lib.ssm_window_plan.argtypes = [dp] + [vp] * 6
    cp, sp, np_ = (ctypes.POINTER(t) for t in (ConvDims, SelectiveDims, NormDims))
    rp = ins = outs = vp  # arrays of rows, as addresses and strides (_flat)
    lp = ctypes.POINTER(i64)
    lib.ssm_conv_sizes.argtypes = [cp, i32, lp]
    lib.ssm_conv_forward.argtypes = [cp, i32, vp, i32, vp, vp, rp, vp, vp, vp, rp, vp]
    lib.ssm_conv_backward.argtypes = [cp, i32, vp, vp, rp, vp, vp, rp, vp, rp, vp, vp, vp, vp, i64, vp]
    lib.ssm_conv_step.argtypes = [cp, i32, vp, rp, vp, vp, vp, rp, vp]
    lib.ssm_selective_sizes.argtypes = [sp, i32, lp, lp]
    lib.ssm_selective_forward.argtypes = [sp, i32, vp, i32, vp, vp, ins, vp, rp, vp, i64, vp]
    lib.ssm_selective_backward.argtypes = [sp, i32, vp, vp, ins, rp, vp, outs, vp, vp, i64, vp]
    lib.ssm_selective_step.argtypes = [sp, i32, vp, ins, vp, rp, vp]
    lib.ssm_gated_norm_sizes.argtypes = [np_, i32, lp]
    lib.ssm_gated_norm.argtypes = [np_, i32, rp, rp, vp, vp, rp, vp]
    lib.ssm_gated_norm_backward.argtypes = [np_, i32, rp, rp, vp, vp, rp, rp, rp, vp, vp, vp, i64, vp]
    for name in ("conv_sizes", "conv_forward", "conv_backward", "conv_step", "selective_sizes",
                 "selective_forward", "selective_backward", "selective_step", "gated_norm_sizes",
                 "gated_norm", "gated_norm_backward"):
        getattr(lib, "ssm_" + name).restype = i32
    lib.ssm_stream_probe.restype = i32
    lib.ssm_stream_probe.argtypes = [vp, ctypes.c_int64, i32, vp]
    return lib


_lib = _load()


def declared_symbols(header: str = HEADER):
    """Function names declared in the C header."""
    import re
    text = open(header).read()
    return sorted(set(re.findall(r"^\s*(?:ssm_status|int32_t|const char\*)\s+(ssm_\w+)\s*\(",
                                 text, re.M)))


def library():
    return _lib


def abi_version() -> int:
    return int(_lib.ssm_abi_version())


# ----------------------------------------------------------------------------
# marshalling
# ----------------------------------------------------------------------------
Ptr = Union["torch.Tensor", int, None]  # noqa: F821


def numel(d: Dims) -> dict:
    """Element count of every array argument for these dimensions."""
    U = d.batch * d.heads
    dstr = d.d_k if d.rule == KDA else 1
    return {
        "state": U * d.d_k * d.d_v, "sketch": U * d.rank * d.d_v, "basis": d.heads * d.rank * d.d_k,
        "read_map": U * d.rank * d.d_k,
        "k_buf": U * d.window * d.d_k, "v_buf": U * d.window * d.d_v,
        "decay_buf": U * d.window * dstr, "beta_buf": U * d.window,
        "q": U * d.d_k, "k_t": U * d.d_k, "v_t": U * d.d_v, "decay_t": U * dstr, "beta_t": U,
        "y": U * d.d_v,
    }


def _addr(x: Ptr, name: str, dtype=None, count: Optional[int] = None) -> Optional[int]:
    """Device address of a tensor (checked: device, contiguity, dtype, size) or int."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError(f"{name}: expected a device tensor")
    if not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if dtype is not None and x.dtype not in dtype:
        raise TypeError(f"{name}: dtype {x.dtype} not in {dtype}")
    if count is not None and x.numel() != count:
        raise ValueError(f"{name}: {x.numel()} elements, the dimensions need {count}")
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        if torch.cuda.is_available():
            return torch.cuda.current_stream().cuda_stream
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _in_types(d: Dims):
    import torch
    return (torch.bfloat16,) if d.in_dtype == IN_BF16 else (torch.float32,)


def _f32():
    import torch
    return (torch.float32,)


def _sk_types(d: Dims, f32):
    """Dtype set of the sketch (None when only raw addresses are passed)."""
    if f32 is None:
        return None
    import torch
    return (torch.bfloat16,) if d.sketch_dtype == SKETCH_BF16 else (torch.float32,)


def _check(status: int):
    if status != 0:
        raise SSMError(status, _lib.ssm_last_error().decode())


def _types(d: Dims, args):
    """Dtype sets only when tensors are passed (raw ints skip the torch import)."""
    if all(a is None or isinstance(a, int) for a in args):
        return None, None
    return _in_types(d), _f32()


def _all_raw(args) -> bool:
    return all(a is None or isinstance(a, int) for a in args)


# ----------------------------------------------------------------------------
# entry points (same names as the C ABI, without the ssm_ prefix)
# ----------------------------------------------------------------------------
def buffer_append(d: Dims, k_t, v_t, decay_t, beta_t, k_buf, v_buf, decay_buf, beta_buf,
                  slot: int, stream=None) -> None:
    if isinstance(stream, int) and _all_raw((k_t, v_t, decay_t, beta_t, k_buf, v_buf, decay_buf,
                                             beta_buf)):
        return _check(_lib.ssm_buffer_append(ctypes.byref(d), k_t, v_t, decay_t, beta_t, k_buf,
                                             v_buf, decay_buf, beta_buf, slot, stream))
    tin, f32 = _types(d, (k_t, v_t, decay_t, beta_t, k_buf, v_buf, decay_buf, beta_buf))
    n = numel(d)
    _check(_lib.ssm_buffer_append(
        ctypes.byref(d), _addr(k_t, "k_t", tin, n["k_t"]), _addr(v_t, "v_t", tin, n["v_t"]),
        _addr(decay_t, "decay_t", f32, n["decay_t"]), _addr(beta_t, "beta_t", f32, n["beta_t"]),
        _addr(k_buf, "k_buf", tin, n["k_buf"]), _addr(v_buf, "v_buf", tin, n["v_buf"]),
        _addr(decay_buf, "decay_buf", f32, n["decay_buf"]), _addr(beta_buf, "beta_buf", f32, n["beta_buf"]),
        int(slot), _stream(stream)))


def window_update_refresh(d: Dims, state, sketch, basis, k_buf, v_buf, decay_buf, beta_buf,
                          n_tokens: int, stream=None) -> None:
    if isinstance(stream, int) and _all_raw((state, sketch, basis, k_buf, v_buf, decay_buf,
                                             beta_buf)):
        return _check(_lib.ssm_window_update_refresh(ctypes.byref(d), state, sketch, basis, k_buf,
                                                     v_buf, decay_buf, beta_buf, n_tokens, stream))
    tin, f32 = _types(d, (state, sketch, basis, k_buf, v_buf, decay_buf, beta_buf))
    n = numel(d)
    _check(_lib.ssm_window_update_refresh(
        ctypes.byref(d), _addr(state, "state", f32, n["state"]), _addr(sketch, "sketch", _sk_types(d, f32), n["sketch"]),
        _addr(basis, "basis", f32, n["basis"]), _addr(k_buf, "k_buf", tin, n["k_buf"]), _addr(v_buf, "v_buf", tin, n["v_buf"]),
        _addr(decay_buf, "decay_buf", f32, n["decay_buf"]), _addr(beta_buf, "beta_buf", f32, n["beta_buf"]),
        int(n_tokens), _stream(stream)))


def sketch_decode_step(d: Dims, sketch, basis, q, k_buf, v_buf, decay_buf, beta_buf, tau: int,
                       y, *, k_t=None, v_t=None, decay_t=None, beta_t=None, stream=None) -> None:
    if isinstance(stream, int) and _all_raw((sketch, basis, q, k_buf, v_buf, decay_buf, beta_buf,
                                             y, k_t, v_t, decay_t, beta_t)):
        return _check(_lib.ssm_sketch_decode_step(ctypes.byref(d), sketch, basis, q, k_t, v_t,
                                                  decay_t, beta_t, k_buf, v_buf, decay_buf,
                                                  beta_buf, tau, y, stream))
    tin, f32 = _types(d, (sketch, basis, q, k_buf, v_buf, decay_buf, beta_buf, y, k_t, v_t))
    n = numel(d)
    _check(_lib.ssm_sketch_decode_step(
        ctypes.byref(d), _addr(sketch, "sketch", _sk_types(d, f32), n["sketch"]), _addr(basis, "basis", f32, n["basis"]),
        _addr(q, "q", tin, n["q"]), _addr(k_t, "k_t", tin, n["k_t"]), _addr(v_t, "v_t", tin, n["v_t"]),
        _addr(decay_t, "decay_t", f32, n["decay_t"]), _addr(beta_t, "beta_t", f32, n["beta_t"]),
        _addr(k_buf, "k_buf", tin, n["k_buf"]), _addr(v_buf, "v_buf", tin, n["v_buf"]),
        _addr(decay_buf, "decay_buf", f32, n["decay_buf"]), _addr(beta_buf, "beta_buf", f32, n["beta_buf"]),
        int(tau), _addr(y, "y", f32, n["y"]), _stream(stream)))


def full_read_decode_step(d: Dims, state, q, k_buf, v_buf, decay_buf, beta_buf, tau: int, y, *,
                          k_t=None, v_t=None, decay_t=None, beta_t=None, stream=None) -> None:
    if isinstance(stream, int) and _all_raw((state, q, k_buf, v_buf, decay_buf, beta_buf, y, k_t,
                                             v_t, decay_t, beta_t)):
        return _check(_lib.ssm_full_read_decode_step(ctypes.byref(d), state, q, k_t, v_t, decay_t,
                                                     beta_t, k_buf, v_buf, decay_buf, beta_buf,
                                                     tau, y, stream))
    tin, f32 = _types(d, (state, q, k_buf, v_buf, decay_buf, beta_buf, y, k_t, v_t))
    n = numel(d)
    _check(_lib.ssm_full_read_decode_step(
        ctypes.byref(d), _addr(state, "state", f32, n["state"]), _addr(q, "q", tin, n["q"]),
        _addr(k_t, "k_t", tin, n["k_t"]), _addr(v_t, "v_t", tin, n["v_t"]),
        _addr(decay_t, "decay_t", f32, n["decay_t"]), _addr(beta_t, "beta_t", f32, n["beta_t"]),
        _addr(k_buf, "k_buf", tin, n["k_buf"]), _addr(v_buf, "v_buf", tin, n["v_buf"]),
        _addr(decay_buf, "decay_buf", f32, n["decay_buf"]), _addr(beta_buf, "beta_buf", f32, n["beta_buf"]),
        int(tau), _addr(y, "y", f32, n["y"]), _stream(stream)))


def recurrent_decode_step(d: Dims, state, q, k_t, v_t, decay_t, beta_t, y, stream=None) -> None:
    if isinstance(stream, int) and _all_raw((state, q, k_t, v_t, decay_t, beta_t, y)):
        return _check(_lib.ssm_recurrent_decode_step(ctypes.byref(d), state, q, k_t, v_t, decay_t,
                                                     beta_t, y, stream))
    tin, f32 = _types(d, (state, q, k_t, v_t, decay_t, beta_t, y))
    n = numel(d)
    _check(_lib.ssm_recurrent_decode_step(
        ctypes.byref(d), _addr(state, "state", f32, n["state"]), _addr(q, "q", tin, n["q"]),
        _addr(k_t, "k_t", tin, n["k_t"]), _addr(v_t, "v_t", tin, n["v_t"]),
        _addr(decay_t, "decay_t", f32, n["decay_t"]), _addr(beta_t, "beta_t", f32, n["beta_t"]),
        _addr(y, "y", f32, n["y"]), _stream(stream)))


def fit_basis(d: Dims, samples, n_samples: int, basis, stream=None) -> None:
    """ssm_fit_basis: per head, the d.rank leading eigenvectors of the samples' uncentred
    second moment as orthonormal rows of basis. samples [H][n_samples][d_k] (d.in_dtype),
    basis [H][rank][d_k] fp32."""
    if isinstance(stream, int) and _all_raw((samples, basis)):
        return _check(_lib.ssm_fit_basis(ctypes.byref(d), samples, int(n_samples), basis, stream))
    tin, f32 = _types(d, (samples, basis))
    _check(_lib.ssm_fit_basis(
        ctypes.byref(d), _addr(samples, "samples", tin, d.heads * int(n_samples) * d.d_k),
        int(n_samples), _addr(basis, "basis", f32, d.heads * d.rank * d.d_k), _stream(stream)))


def stream_probe(buf, n_tiles: int, shape: int, stream=None) -> None:
    """ssm_stream_probe (a measurement aid): stream buf, n_tiles 64 KB fp32 tiles, in place
    in access shape 0 (the window update's order) or 1 (flat runs of two tiles)."""
    ptr = buf if isinstance(buf, int) else _addr(buf, "buf", _f32(), int(n_tiles) * 16384)
    _check(_lib.ssm_stream_probe(ptr, int(n_tiles), int(shape), _stream(stream)))


# ----------------------------------------------------------------------------
# heterogeneous per-head sketch ranks
# ----------------------------------------------------------------------------
def rank_offsets(ranks) -> "ctypes.Array":
    """Host int32 prefix offsets (H + 1 values) for per-head ranks."""
    off = [0]
    for r in ranks:
        off.append(off[-1] + int(r))
    return (ctypes.c_int32 * len(off))(*off)


def _ranked_numel(d: Dims, offsets) -> dict:
    n = numel(d)
    R = int(offsets[d.heads]) if len(offsets) > d.heads else 0
    n["sketch"] = d.batch * R * d.d_v
    n["basis"] = R * d.d_k
    return n


def _offsets_arg(d: Dims, offsets):
    if not isinstance(offsets, ctypes.Array):
        offsets = rank_offsets(offsets) if len(offsets) == d.heads else \
            (ctypes.c_int32 * len(offsets))(*[int(x) for x in offsets])
    if len(offsets) != d.heads + 1:
        raise ValueError(f"rank_offsets: {len(offsets)} entries, need heads + 1 = {d.heads + 1}")
    return offsets


def window_update_refresh_ranked(d: Dims, offsets, state, sketch, basis, k_buf, v_buf,
                                 decay_buf, beta_buf, n_tokens: int, stream=None) -> None:
    """ssm_window_update_refresh_ranked. `offsets`: H + 1 prefix offsets, or H per-head ranks."""
    off = _offsets_arg(d, offsets)
    if isinstance(stream, int) and _all_raw((state, sketch, basis, k_buf, v_buf, decay_buf,
                                             beta_buf)):
        return _check(_lib.ssm_window_update_refresh_ranked(
            ctypes.byref(d), off, state, sketch, basis, k_buf, v_buf, decay_buf, beta_buf,
            n_tokens, stream))
    tin, f32 = _types(d, (state, sketch, basis, k_buf, v_buf, decay_buf, beta_buf))
    n = _ranked_numel(d, off)
    _check(_lib.ssm_window_update_refresh_ranked(
        ctypes.byref(d), off, _addr(state, "state", f32, n["state"]),
        _addr(sketch, "sketch", _sk_types(d, f32), n["sketch"]), _addr(basis, "basis", f32, n["basis"]),
        _addr(k_buf, "k_buf", tin, n["k_buf"]), _addr(v_buf, "v_buf", tin, n["v_buf"]),
        _addr(decay_buf, "decay_buf", f32, n["decay_buf"]),
        _addr(beta_buf, "beta_buf", f32, n["beta_buf"]), int(n_tokens), _stream(stream)))


def sketch_decode_step_ranked(d: Dims, offsets, sketch, basis, q, k_buf, v_buf, decay_buf,
                              beta_buf, tau: int, y, *, k_t=None, v_t=None, decay_t=None,
                              beta_t=None, stream=None) -> None:
    """ssm_sketch_decode_step_ranked. `offsets`: H + 1 prefix offsets, or H per-head ranks."""
    off = _offsets_arg(d, offsets)
    if isinstance(stream, int) and _all_raw((sketch, basis, q, k_buf, v_buf, decay_buf, beta_buf,
                                             y, k_t, v_t, decay_t, beta_t)):
        return _check(_lib.ssm_sketch_decode_step_ranked(
            ctypes.byref(d), off, sketch, basis, q, k_t, v_t, decay_t, beta_t, k_buf, v_buf,
            decay_buf, beta_buf, tau, y, stream))
    tin, f32 = _types(d, (sketch, basis, q, k_buf, v_buf, decay_buf, beta_buf, y, k_t, v_t))
    n = _ranked_numel(d, off)
    _check(_lib.ssm_sketch_decode_step_ranked(
        ctypes.byref(d), off, _addr(sketch, "sketch", _sk_types(d, f32), n["sketch"]),
        _addr(basis, "basis", f32, n["basis"]), _addr(q, "q", tin, n["q"]),
        _addr(k_t, "k_t", tin, n["k_t"]), _addr(v_t, "v_t", tin, n["v_t"]),
        _addr(decay_t, "decay_t", f32, n["decay_t"]), _addr(beta_t, "beta_t", f32, n["beta_t"]),
        _addr(k_buf, "k_buf", tin, n["k_buf"]), _addr(v_buf, "v_buf", tin, n["v_buf"]),
        _addr(decay_buf, "decay_buf", f32, n["decay_buf"]),
        _addr(beta_buf, "beta_buf", f32, n["beta_buf"]), int(tau), _addr(y, "y", f32, n["y"]),
        _stream(stream)))


# ----------------------------------------------------------------------------
# variable-length batches over a pool of slots
# ----------------------------------------------------------------------------
def _pool_numel(d: Dims, num_slots: int) -> dict:
    n = numel(d)
    p = numel(Dims(d.rule, d.in_dtype, num_slots, d.heads, d.d_k, d.d_v, d.window, d.rank))
    for key in ("state", "sketch", "k_buf", "v_buf", "decay_buf", "beta_buf"):
        n[key] = p[key]
    n["rows"] = d.batch
    return n


def _i32():
    import torch
    return (torch.int32,)


def window_update_refresh_varlen(d: Dims, num_slots: int, slot, n_tokens, state, sketch, basis,
                                 k_buf, v_buf, decay_buf, beta_buf, stream=None) -> None:
    """ssm_window_update_refresh_varlen: per-row token counts (device int32 [batch]) and an
    optional slot map (device int32 [batch]) into a pool of num_slots persistent slots."""
    args = (slot, n_tokens, state, sketch, basis, k_buf, v_buf, decay_buf, beta_buf)
    if isinstance(stream, int) and _all_raw(args):
        return _check(_lib.ssm_window_update_refresh_varlen(ctypes.byref(d), int(num_slots), *args,
                                                            stream))
    tin, f32 = _types(d, args)
    i32 = None if tin is None else _i32()
    n = _pool_numel(d, num_slots)
    _check(_lib.ssm_window_update_refresh_varlen(
        ctypes.byref(d), int(num_slots), _addr(slot, "slot", i32, n["rows"]),
        _addr(n_tokens, "n_tokens", i32, n["rows"]), _addr(state, "state", f32, n["state"]),
        _addr(sketch, "sketch", _sk_types(d, f32), n["sketch"]), _addr(basis, "basis", f32, n["basis"]),
        _addr(k_buf, "k_buf", tin, n["k_buf"]), _addr(v_buf, "v_buf", tin, n["v_buf"]),
        _addr(decay_buf, "decay_buf", f32, n["decay_buf"]),
        _addr(beta_buf, "beta_buf", f32, n["beta_buf"]), _stream(stream)))


def sketch_decode_step_varlen(d: Dims, num_slots: int, slot, tau, sketch, basis, q, k_buf, v_buf,
                              decay_buf, beta_buf, y, *, k_t=None, v_t=None, decay_t=None,
                              beta_t=None, stream=None) -> None:
    """ssm_sketch_decode_step_varlen: per-row window positions tau (device int32 [batch])."""
    args = (slot, tau, sketch, basis, q, k_t, v_t, decay_t, beta_t, k_buf, v_buf, decay_buf,
            beta_buf, y)
    if isinstance(stream, int) and _all_raw(args):
        return _check(_lib.ssm_sketch_decode_step_varlen(ctypes.byref(d), int(num_slots), *args,
                                                         stream))
    tin, f32 = _types(d, args)
    i32 = None if tin is None else _i32()
    n = _pool_numel(d, num_slots)
    _check(_lib.ssm_sketch_decode_step_varlen(
        ctypes.byref(d), int(num_slots), _addr(slot, "slot", i32, n["rows"]),
        _addr(tau, "tau", i32, n["rows"]), _addr(sketch, "sketch", _sk_types(d, f32), n["sketch"]),
        _addr(basis, "basis", f32, n["basis"]), _addr(q, "q", tin, n["q"]),
        _addr(k_t, "k_t", tin, n["k_t"]), _addr(v_t, "v_t", tin, n["v_t"]),
        _addr(decay_t, "decay_t", f32, n["decay_t"]), _addr(beta_t, "beta_t", f32, n["beta_t"]),
        _addr(k_buf, "k_buf", tin, n["k_buf"]), _addr(v_buf, "v_buf", tin, n["v_buf"]),
        _addr(decay_buf, "decay_buf", f32, n["decay_buf"]),
        _addr(beta_buf, "beta_buf", f32, n["beta_buf"]), _addr(y, "y", f32, n["y"]),
        _stream(stream)))


def decode_step_varlen(d: Dims, num_slots: int, slot, tau, parity, n_update: int, update_rows,
                       state, sketch0, sketch1, basis, q, k_t, v_t, decay_t, beta_t, k_buf,
                       v_buf, decay_buf, beta_buf, y, stream=None) -> None:
    """ssm_decode_step_varlen: one serving step in one launch. Every row reads y at its own
    window position tau (device int32 [batch]) from sketch0 or sketch1 (parity, device int32
    [batch]) with the current token appended; the n_update rows listed in update_rows (device
    int32) whose window fills (tau == W) also apply the window to the state and store the
    refreshed sketch in the other buffer."""
    args = (slot, tau, parity, update_rows, state, sketch0, sketch1, basis, q, k_t, v_t, decay_t,
            beta_t, k_buf, v_buf, decay_buf, beta_buf, y)
    if isinstance(stream, int) and _all_raw(args):
        return _check(_lib.ssm_decode_step_varlen(
            ctypes.byref(d), int(num_slots), slot, tau, parity, int(n_update), update_rows, state,
            sketch0, sketch1, basis, q, k_t, v_t, decay_t, beta_t, k_buf, v_buf, decay_buf,
            beta_buf, y, stream))
    tin, f32 = _types(d, args)
    i32 = None if tin is None else _i32()
    n = _pool_numel(d, num_slots)
    sk = _sk_types(d, f32)
    _check(_lib.ssm_decode_step_varlen(
        ctypes.byref(d), int(num_slots), _addr(slot, "slot", i32, n["rows"]),
        _addr(tau, "tau", i32, n["rows"]), _addr(parity, "parity", i32, n["rows"]),
        int(n_update), _addr(update_rows, "update_rows", i32, int(n_update) if n_update else None),
        _addr(state, "state", f32, n["state"]), _addr(sketch0, "sketch0", sk, n["sketch"]),
        _addr(sketch1, "sketch1", sk, n["sketch"]), _addr(basis, "basis", f32, n["basis"]),
        _addr(q, "q", tin, n["q"]), _addr(k_t, "k_t", tin, n["k_t"]),
        _addr(v_t, "v_t", tin, n["v_t"]), _addr(decay_t, "decay_t", f32, n["decay_t"]),
        _addr(beta_t, "beta_t", f32, n["beta_t"]), _addr(k_buf, "k_buf", tin, n["k_buf"]),
        _addr(v_buf, "v_buf", tin, n["v_buf"]), _addr(decay_buf, "decay_buf", f32, n["decay_buf"]),
        _addr(beta_buf, "beta_buf", f32, n["beta_buf"]), _addr(y, "y", f32, n["y"]),
        _stream(stream)))


def window_update_refresh_ls(d: Dims, state, sketch_q, read_map, basis, k_buf, v_buf, decay_buf,
                             beta_buf, n_tokens: int, stream=None) -> None:
    """ssm_window_update_refresh_ls: the window update, then the least-squares sketch
    (orthonormal sketch rows sketch_q [N][H][r][d_v] and read_map [N][H][r][d_k])."""
    args = (state, sketch_q, read_map, basis, k_buf, v_buf, decay_buf, beta_buf)
    if isinstance(stream, int) and _all_raw(args):
        return _check(_lib.ssm_window_update_refresh_ls(ctypes.byref(d), *args, n_tokens, stream))
    tin, f32 = _types(d, args)
    n = numel(d)
    _check(_lib.ssm_window_update_refresh_ls(
        ctypes.byref(d), _addr(state, "state", f32, n["state"]),
        _addr(sketch_q, "sketch_q", f32, n["sketch"]),
        _addr(read_map, "read_map", f32, n["read_map"]), _addr(basis, "basis", f32, n["basis"]),
        _addr(k_buf, "k_buf", tin, n["k_buf"]), _addr(v_buf, "v_buf", tin, n["v_buf"]),
        _addr(decay_buf, "decay_buf", f32, n["decay_buf"]),
        _addr(beta_buf, "beta_buf", f32, n["beta_buf"]), int(n_tokens), _stream(stream)))


def sketch_decode_step_ls(d: Dims, sketch_q, read_map, q, k_buf, v_buf, decay_buf, beta_buf,
                          tau: int, y, *, k_t=None, v_t=None, decay_t=None, beta_t=None,
                          stream=None) -> None:
    """ssm_sketch_decode_step_ls: y = sketch_q^T (read_map q~) + R^T q."""
    args = (sketch_q, read_map, q, k_buf, v_buf, decay_buf, beta_buf, y, k_t, v_t, decay_t,
            beta_t)
    if isinstance(stream, int) and _all_raw(args):
        return _check(_lib.ssm_sketch_decode_step_ls(ctypes.byref(d), sketch_q, read_map, q, k_t,
                                                     v_t, decay_t, beta_t, k_buf, v_buf,
                                                     decay_buf, beta_buf, tau, y, stream))
    tin, f32 = _types(d, args)
    n = numel(d)
    _check(_lib.ssm_sketch_decode_step_ls(
        ctypes.byref(d), _addr(sketch_q, "sketch_q", f32, n["sketch"]),
        _addr(read_map, "read_map", f32, n["read_map"]), _addr(q, "q", tin, n["q"]),
        _addr(k_t, "k_t", tin, n["k_t"]), _addr(v_t, "v_t", tin, n["v_t"]),
        _addr(decay_t, "decay_t", f32, n["decay_t"]), _addr(beta_t, "beta_t", f32, n["beta_t"]),
        _addr(k_buf, "k_buf", tin, n["k_buf"]), _addr(v_buf, "v_buf", tin, n["v_buf"]),
        _addr(decay_buf, "decay_buf", f32, n["decay_buf"]),
        _addr(beta_buf, "beta_buf", f32, n["beta_buf"]), int(tau), _addr(y, "y", f32, n["y"]),
        _stream(stream)))


# ----------------------------------------------------------------------------
# whole sequences and serving plans
# ----------------------------------------------------------------------------
# These calls take a few microseconds on the device at small sizes, so their marshalling keeps
# to one look at each tensor, one at the device and one at its stream.
import torch as _torch  # noqa: E402  (loaded above, before the library)

_F32_T, _I32_T = (_torch.float32,), (_torch.int32,)
_IN_T = {IN_BF16: (_torch.bfloat16,), IN_F32: (_torch.float32,)}


# the address of a device's current stream, without a Stream object around it
_stream_of_device = getattr(_torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: _torch.cuda.current_stream(index).cuda_stream)


def _on_device(args, stream, call) -> None:
    """call(stream address) on the device that the tensors among args share: their device
    becomes the current one for the call, and its current stream is the default."""
    index = None
    for a in args:
        if a is None or isinstance(a, int):
            continue
        i = a.get_device()
        if index is None:
            index = i
        elif i != index:
            raise ValueError(f"tensors on different devices: {index}, {i}")
    if index is None:
        return call(_stream(stream))  # raw addresses
    if stream is None:
        stream = _stream_of_device(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if index == _torch.cuda.current_device():
        return call(stream)
    with _torch.cuda.device(index):
        call(stream)


def _count(x, name: str) -> int:
    """A 32-bit argument (ctypes would keep the low 32 bits of a larger one)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name}: {x} is beyond 32 bits")
    return x


def scan_sizes(d: Dims, total_tokens: int) -> tuple:
    """(int32 elements of the plan, workspace bytes of scan_forward, of scan_backward)."""
    got = [ctypes.c_int64() for _ in range(3)]
    total = _count(total_tokens, "total_tokens")
    _check(_lib.ssm_scan_sizes(ctypes.byref(d), total, *map(ctypes.byref, got)))
    return tuple(int(x.value) for x in got)


def scan_plan(lengths, total_tokens: int, plan, *, n_seqs: Optional[int] = None,
              stream=None) -> None:
    """ssm_scan_plan: the plan of a packed batch from its sequences' lengths (int32 [n]).
    plan: int32, 2 (n + 1) + total_tokens // 64 + n elements. n_seqs is needed with raw addresses."""
    n = _count(lengths.numel() if n_seqs is None else n_seqs, "n_seqs")
    total = _count(total_tokens, "total_tokens")
    a = _addr(lengths, "lengths", _I32_T, n)
    b = _addr(plan, "plan", _I32_T, 2 * (n + 1) + total // 64 + n)
    _on_device((lengths, plan), stream,
               lambda s: _check(_lib.ssm_scan_plan(a, n, total, b, s)))


def _packed(d: Dims, total: int, plan, q, k, v, decay, beta):
    """Addresses of a packed batch's arrays."""
    rows, n, tin = total * d.heads, d.batch, _IN_T.get(d.in_dtype)
    return (_addr(plan, "plan", _I32_T, 2 * (n + 1) + total // 64 + n),
            _addr(q, "q", tin, rows * d.d_k), _addr(k, "k", tin, rows * d.d_k),
            _addr(v, "v", tin, rows * d.d_v),
            _addr(decay, "decay", _F32_T, rows * d.d_k if d.rule == KDA else rows),
            _addr(beta, "beta", _F32_T, rows))


def _workspace(workspace, need, args, stream):
    """A workspace and its bytes: the caller's, or one of need() bytes from PyTorch, which owns
    it again, in the call's stream's order, when the call returns."""
    if isinstance(workspace, int):
        raise ValueError("workspace: expected a device tensor or None")
    if workspace is not None:
        _addr(workspace, "workspace")
        return workspace, workspace.numel() * workspace.element_size()
    dev = next((a.device for a in args if a is not None and not isinstance(a, int)), None)
    if dev is None:
        raise ValueError("workspace: raw addresses need a workspace tensor")
    need = need()
    if stream is None:
        ws = _torch.empty(need, dtype=_torch.uint8, device=dev)
    else:
        # from the pool of the stream that uses it: a free block of another stream's may still be
        # in use by what is queued there
        if not isinstance(stream, _torch.cuda.Stream):
            handle = stream if isinstance(stream, int) else stream.cuda_stream
            stream = (_torch.cuda.ExternalStream(handle, device=dev) if handle
                      else _torch.cuda.default_stream(dev))
        if stream.device != dev:
            raise ValueError(f"stream on device {stream.device}, tensors on {dev}")
        with _torch.cuda.stream(stream):
            ws = _torch.empty(need, dtype=_torch.uint8, device=dev)
    return ws, need


def _scan_workspace(workspace, d: Dims, total: int, which: int, args, stream):
    def need():
        got = ctypes.c_int64()
        out = (None, ctypes.byref(got), None) if which == 1 else (None, None, ctypes.byref(got))
        _check(_lib.ssm_scan_sizes(ctypes.byref(d), total, *out))
        return got.value

    return _workspace(workspace, need, args, stream)


def scan_forward(d: Dims, total_tokens: int, plan, q, k, v, decay, beta, state, y, *,
                 state_in=None, slot=None, num_slots: Optional[int] = None, workspace=None,
                 stream=None) -> None:
    """ssm_scan_forward: a packed batch of d.batch sequences through the recurrence; y
    [total_tokens][H][d_v] and the final states [num_slots][H][d_k][d_v] (num_slots defaults to
    d.batch), from state_in (None: zero; may be `state` itself). workspace: a device tensor of
    scan_sizes(...)[1] bytes, or None to take one from PyTorch for the call."""
    total = _count(total_tokens, "total_tokens")
    ns = d.batch if num_slots is None else _count(num_slots, "num_slots")
    p = _packed(d, total, plan, q, k, v, decay, beta)
    states = ns * d.heads * d.d_k * d.d_v
    a = (_addr(slot, "slot", _I32_T, d.batch), _addr(state_in, "state_in", _F32_T, states))
    b = (_addr(state, "state", _F32_T, states), _addr(y, "y", _F32_T, total * d.heads * d.d_v))
    args = (plan, q, k, v, decay, beta, state, y, state_in, slot)
    ws, have = _scan_workspace(workspace, d, total, 1, args, stream)
    _on_device(args + (ws,), stream, lambda s: _check(_lib.ssm_scan_forward(
        ctypes.byref(d), total, p[0], ns, *a, *p[1:], *b, ws.data_ptr(), have, s)))


def scan_backward(d: Dims, total_tokens: int, plan, q, k, v, decay, beta, dy, dq, dk, dv,
                  dlog_decay, dbeta, *, state_in=None, dstate=None, dstate_in=None,
                  workspace=None, stream=None) -> None:
    """ssm_scan_backward: the gradients of scan_forward (dlog_decay is decay * dL/d(decay)).
    workspace: a device tensor of scan_sizes(...)[2] bytes, or None."""
    total = _count(total_tokens, "total_tokens")
    p = _packed(d, total, plan, q, k, v, decay, beta)
    rows, tin = total * d.heads, _IN_T.get(d.in_dtype)
    states = d.batch * d.heads * d.d_k * d.d_v
    s0 = _addr(state_in, "state_in", _F32_T, states)
    b = (_addr(dy, "dy", _F32_T, rows * d.d_v), _addr(dstate, "dstate", _F32_T, states),
         _addr(dq, "dq", tin, rows * d.d_k), _addr(dk, "dk", tin, rows * d.d_k),
         _addr(dv, "dv", tin, rows * d.d_v),
         _addr(dlog_decay, "dlog_decay", _F32_T, rows * d.d_k if d.rule == KDA else rows),
         _addr(dbeta, "dbeta", _F32_T, rows), _addr(dstate_in, "dstate_in", _F32_T, states))
    args = (plan, q, k, v, decay, beta, dy, dq, dk, dv, dlog_decay, dbeta, state_in, dstate,
            dstate_in)
    ws, have = _scan_workspace(workspace, d, total, 2, args, stream)
    _on_device(args + (ws,), stream, lambda s: _check(_lib.ssm_scan_backward(
        ctypes.byref(d), total, p[0], s0, *p[1:], *b, ws.data_ptr(), have, s)))


def window_plan(d: Dims, lengths, tau, parity, update_rows, n_update, stream=None) -> None:
    """ssm_window_plan: tau, parity, update_rows (int32 [d.batch] each) and n_update (one int32)
    of a serving step from the tokens each row has decoded (int32 [d.batch], negative: padding)."""
    n = d.batch
    a = (_addr(lengths, "lengths", _I32_T, n), _addr(tau, "tau", _I32_T, n),
         _addr(parity, "parity", _I32_T, n), _addr(update_rows, "update_rows", _I32_T, n),
         _addr(n_update, "n_update", _I32_T, 1))
    _on_device((lengths, tau, parity, update_rows, n_update), stream,
               lambda s: _check(_lib.ssm_window_plan(ctypes.byref(d), *a, s)))


# ----------------------------------------------------------------------------
# around the recurrence: short convolution, selective recurrence, output norm
# ----------------------------------------------------------------------------
def _row_addr(x, name: str, types, rows: int, width: int) -> tuple:
    """Address and stride of rows of `width` elements: a contiguous tensor, one whose first dimension alone is
    strided (a column range of a larger one), an address of contiguous rows, or None."""
    if x is None:
        return 0, width
    if isinstance(x, int):
        return x, width
    if x.is_cuda and (types is None or x.dtype in types) and x.numel() == rows * width:
        if x.is_contiguous():
            return x.data_ptr(), width
        if x.dim() == 2 and x.stride(1) == 1 and x.shape[0] == rows:
            return x.data_ptr(), x.stride(0) if rows > 1 else width
    if not x.is_cuda:
        raise ValueError(f"{name}: expected a device tensor")
    if types is not None and x.dtype not in types:
        raise TypeError(f"{name}: dtype {x.dtype} not in {types}")
    if x.numel() != rows * width:
        raise ValueError(f"{name}: {x.numel()} elements, the dimensions need {rows} x {width}")
    inner = 1
    for size, stride in zip(reversed(x.shape[1:]), reversed(x.stride()[1:])):
        if size != 1 and stride != inner:
            raise ValueError(f"{name}: expected rows of contiguous elements, got strides {x.stride()}")
        inner *= size
    if x.shape[0] != rows:
        raise ValueError(f"{name}: expected {rows} rows of {width}, got {tuple(x.shape)}")
    return x.data_ptr(), x.stride(0) if rows > 1 else width


# Addresses and strides one after another have the layout of ssm_rows and of the structs made of it; an array
# of integers is built in a fraction of the time of the structs.
_ROWS1, _ROWS4, _INS, _OUTS = (ctypes.c_int64 * n for n in (2, 2 * CONV_PARTS, 13, 13))


def _bytes_of(call, *args) -> int:
    got = ctypes.c_int64()
    _check(call(*args, ctypes.byref(got)))
    return int(got.value)


def _conv_parts(d: ConvDims, xs, name: str, types, rows: int):
    """The parts' rows as an array, and their tensors."""
    if xs is None:
        raise ValueError(f"{name}: expected {d.parts} parts")
    xs = list(xs) if isinstance(xs, (list, tuple)) else [xs]
    if len(xs) != d.parts:
        raise ValueError(f"{name}: {len(xs)} parts, the dimensions have {d.parts}")
    flat = []
    for p, x in enumerate(xs):
        flat += _row_addr(x, name, types, rows, d.channels[p])
    return _ROWS4(*flat), xs


def _conv_width(d: ConvDims) -> int:
    return sum(d.channels[:d.parts])


def conv_sizes(d: ConvDims, total_tokens: int) -> int:
    """Workspace bytes of conv_backward."""
    return _bytes_of(_lib.ssm_conv_sizes, ctypes.byref(d), _count(total_tokens, "total_tokens"))


def _plan_ints(total: int, n: int) -> int:
    return 2 * (n + 1) + total // 64 + n


def conv_forward(d: ConvDims, total_tokens: int, plan, x, weight, bias, y, state=None, *, state_in=None,
                 slot=None, num_slots: Optional[int] = None, stream=None) -> None:
    """ssm_conv_forward: a packed batch of d.batch sequences through the convolution. x, y: a tensor of
    rows per part ([total_tokens][channels]; column ranges of a larger tensor are taken as they are),
    or one tensor for one part. weight [C][taps] fp32, bias [C] fp32 or None. state, state_in: the
    last taps - 1 inputs [num_slots][taps - 1][C] after and before (None: not wanted; zero)."""
    total = _count(total_tokens, "total_tokens")
    ns = d.batch if num_slots is None else _count(num_slots, "num_slots")
    tin, C = _IN_T.get(d.in_dtype), _conv_width(d)
    xr, xs = _conv_parts(d, x, "x", tin, total)
    yr, ys = _conv_parts(d, y, "y", tin, total)
    kept = ns * (d.taps - 1) * C
    a = (_addr(plan, "plan", _I32_T, _plan_ints(total, d.batch)), ns,
         _addr(slot, "slot", _I32_T, d.batch), _addr(state_in, "state_in", tin, kept))
    b = (_addr(weight, "weight", _F32_T, C * d.taps), _addr(bias, "bias", _F32_T, C),
         _addr(state, "state", tin, kept))
    _on_device((plan, weight, bias, state, state_in, slot, *xs, *ys), stream,
               lambda s: _check(_lib.ssm_conv_forward(ctypes.byref(d), total, *a, xr, *b, yr, s)))


def conv_backward(d: ConvDims, total_tokens: int, plan, x, weight, bias, dy, dx, dweight, dbias=None, *,
                  state_in=None, dstate=None, dstate_in=None, workspace=None, stream=None) -> None:
    """ssm_conv_backward: the gradients of conv_forward for dy (and dstate, of the final states).
    workspace: a device tensor of conv_sizes(...) bytes, or None to take one from PyTorch for the call."""
    total = _count(total_tokens, "total_tokens")
    tin, C = _IN_T.get(d.in_dtype), _conv_width(d)
    xr, xs = _conv_parts(d, x, "x", tin, total)
    gr, gs = _conv_parts(d, dy, "dy", tin, total)
    dr, ds = _conv_parts(d, dx, "dx", tin, total)
    kept = d.batch * (d.taps - 1) * C
    a = (_addr(plan, "plan", _I32_T, _plan_ints(total, d.batch)), _addr(state_in, "state_in", tin, kept))
    w = (_addr(weight, "weight", _F32_T, C * d.taps), _addr(bias, "bias", _F32_T, C))
    end = _addr(dstate, "dstate", tin, kept)
    b = (_addr(dweight, "dweight", _F32_T, C * d.taps), _addr(dbias, "dbias", _F32_T, C),
         _addr(dstate_in, "dstate_in", tin, kept))
    args = (plan, weight, bias, state_in, dstate, dweight, dbias, dstate_in, *xs, *gs, *ds)
    ws, have = _workspace(workspace, lambda: conv_sizes(d, total), args, stream)
    _on_device(args + (ws,), stream, lambda s: _check(_lib.ssm_conv_backward(
        ctypes.byref(d), total, *a, xr, *w, gr, end, dr, *b, ws.data_ptr(), have, s)))


def conv_step(d: ConvDims, x, weight, bias, state, y, *, slot=None, num_slots: Optional[int] = None,
              stream=None) -> None:
    """ssm_conv_step: one token of each of d.batch rows; the state is updated in place."""
    ns = d.batch if num_slots is None else _count(num_slots, "num_slots")
    tin, C = _IN_T.get(d.in_dtype), _conv_width(d)
    xr, xs = _conv_parts(d, x, "x", tin, d.batch)
    yr, ys = _conv_parts(d, y, "y", tin, d.batch)
    a = (ns, _addr(slot, "slot", _I32_T, d.batch))
    b = (_addr(weight, "weight", _F32_T, C * d.taps), _addr(bias, "bias", _F32_T, C),
         _addr(state, "state", tin, ns * (d.taps - 1) * C))
    _on_device((weight, bias, state, slot, *xs, *ys), stream,
               lambda s: _check(_lib.ssm_conv_step(ctypes.byref(d), *a, xr, *b, yr, s)))


def _selective_in(d: SelectiveDims, rows: int, x, dt, A, B, C, D, z, dt_bias):
    tin, ch, bc = _IN_T.get(d.in_dtype), d.channels, d.groups * d.d_state
    return _INS(
        *_row_addr(x, "x", tin, rows, ch), *_row_addr(dt, "dt", tin, rows, ch),
        *_row_addr(z, "z", tin, rows, ch), *_row_addr(B, "B", tin, rows, bc),
        *_row_addr(C, "C", tin, rows, bc), _addr(A, "A", _F32_T, ch * d.d_state) or 0,
        _addr(D, "D", _F32_T, ch) or 0, _addr(dt_bias, "dt_bias", _F32_T, ch) or 0)


def selective_sizes(d: SelectiveDims, total_tokens: int) -> tuple:
    """Workspace bytes of (selective_forward, selective_backward)."""
    got = ctypes.c_int64(), ctypes.c_int64()
    _check(_lib.ssm_selective_sizes(ctypes.byref(d), _count(total_tokens, "total_tokens"),
                                    *map(ctypes.byref, got)))
    return tuple(int(x.value) for x in got)


def selective_forward(d: SelectiveDims, total_tokens: int, plan, x, dt, A, B, C, state, out, *, D=None,
                      z=None, dt_bias=None, state_in=None, slot=None, num_slots: Optional[int] = None,
                      workspace=None, stream=None) -> None:
    """ssm_selective_forward: a packed batch of d.batch sequences. x, dt, z, out: rows of d.channels;
    B, C: rows of groups * d_state; A [channels][d_state], D and dt_bias [channels] fp32; final
    states [num_slots][channels][d_state] fp32, from state_in (None: zero; may be `state` itself).
    workspace: a device tensor of selective_sizes(...)[0] bytes, or None."""
    total = _count(total_tokens, "total_tokens")
    ns = d.batch if num_slots is None else _count(num_slots, "num_slots")
    states = ns * d.channels * d.d_state
    ins = _selective_in(d, total, x, dt, A, B, C, D, z, dt_bias)
    o = _ROWS1(*_row_addr(out, "out", _IN_T.get(d.in_dtype), total, d.channels))
    a = (_addr(plan, "plan", _I32_T, _plan_ints(total, d.batch)), ns,
         _addr(slot, "slot", _I32_T, d.batch), _addr(state_in, "state_in", _F32_T, states))
    end = _addr(state, "state", _F32_T, states)
    args = (plan, x, dt, A, B, C, D, z, dt_bias, state, out, state_in, slot)
    ws, have = _workspace(workspace, lambda: selective_sizes(d, total)[0], args, stream)
    _on_device(args + (ws,), stream, lambda s: _check(_lib.ssm_selective_forward(
        ctypes.byref(d), total, *a, ins, end, o, ws.data_ptr(), have, s)))


def selective_backward(d: SelectiveDims, total_tokens: int, plan, x, dt, A, B, C, dout, dx, ddt, dA, dB,
                       dC, *, D=None, z=None, dt_bias=None, dD=None, dz=None, ddt_bias=None,
                       state_in=None, dstate=None, dstate_in=None, workspace=None,
                       stream=None) -> None:
    """ssm_selective_backward: the gradients of selective_forward for dout (and dstate, of the final
    states). dz, dD, ddt_bias go with z, D, dt_bias. workspace: a device tensor of
    selective_sizes(...)[1] bytes, or None."""
    total = _count(total_tokens, "total_tokens")
    tin, ch, bc = _IN_T.get(d.in_dtype), d.channels, d.groups * d.d_state
    states = d.batch * ch * d.d_state
    ins = _selective_in(d, total, x, dt, A, B, C, D, z, dt_bias)
    g = _ROWS1(*_row_addr(dout, "dout", tin, total, ch))
    outs = _OUTS(
        *_row_addr(dx, "dx", tin, total, ch), *_row_addr(ddt, "ddt", tin, total, ch),
        *_row_addr(dz, "dz", tin, total, ch), *_row_addr(dB, "dB", tin, total, bc),
        *_row_addr(dC, "dC", tin, total, bc), _addr(dA, "dA", _F32_T, ch * d.d_state) or 0,
        _addr(dD, "dD", _F32_T, ch) or 0, _addr(ddt_bias, "ddt_bias", _F32_T, ch) or 0)
    a = (_addr(plan, "plan", _I32_T, _plan_ints(total, d.batch)),
         _addr(state_in, "state_in", _F32_T, states))
    end, start = _addr(dstate, "dstate", _F32_T, states), _addr(dstate_in, "dstate_in", _F32_T, states)
    args = (plan, x, dt, A, B, C, dout, dx, ddt, dA, dB, dC, D, z, dt_bias, dD, dz, ddt_bias, state_in,
            dstate, dstate_in)
    ws, have = _workspace(workspace, lambda: selective_sizes(d, total)[1], args, stream)
    _on_device(args + (ws,), stream, lambda s: _check(_lib.ssm_selective_backward(
        ctypes.byref(d), total, *a, ins, g, end, outs, start,
        ws.data_ptr(), have, s)))


def selective_step(d: SelectiveDims, x, dt, A, B, C, state, out, *, D=None, z=None, dt_bias=None,
                   slot=None, num_slots: Optional[int] = None, stream=None) -> None:
    """ssm_selective_step: one token of each of d.batch rows; the state is updated in place."""
    ns = d.batch if num_slots is None else _count(num_slots, "num_slots")
    ins = _selective_in(d, d.batch, x, dt, A, B, C, D, z, dt_bias)
    o = _ROWS1(*_row_addr(out, "out", _IN_T.get(d.in_dtype), d.batch, d.channels))
    a = (ns, _addr(slot, "slot", _I32_T, d.batch))
    s0 = _addr(state, "state", _F32_T, ns * d.channels * d.d_state)
    _on_device((x, dt, A, B, C, state, out, D, z, dt_bias, slot), stream,
               lambda s: _check(_lib.ssm_selective_step(ctypes.byref(d), *a, ins, s0,
                                                        o, s)))


def _norm_in(d: NormDims, rows: int, x, z, weight, bias):
    wide = d.groups * d.width
    own = d.width if d.shared else wide
    return (_ROWS1(*_row_addr(x, "x", _IN_T.get(d.x_dtype), rows, wide)),
            _ROWS1(*_row_addr(z, "z", _IN_T.get(d.in_dtype), rows, wide)),
            _addr(weight, "weight", _F32_T, own), _addr(bias, "bias", _F32_T, own))


def gated_norm_sizes(d: NormDims, rows: int) -> int:
    """Workspace bytes of gated_norm_backward."""
    return _bytes_of(_lib.ssm_gated_norm_sizes, ctypes.byref(d), _count(rows, "rows"))


def gated_norm(d: NormDims, rows: int, x, z, weight, bias, out, stream=None) -> None:
    """ssm_gated_norm: rows of groups * width channels (x in x_dtype, z and out in in_dtype), each group
    normalised, weighted and gated by z (None without a gate). weight, bias (or None) fp32, [groups][width],
    or [width] where shared."""
    rows = _count(rows, "rows")
    xr, zr, w, b = _norm_in(d, rows, x, z, weight, bias)
    o = _ROWS1(*_row_addr(out, "out", _IN_T.get(d.in_dtype), rows, d.groups * d.width))
    _on_device((x, z, weight, bias, out), stream, lambda s: _check(_lib.ssm_gated_norm(
        ctypes.byref(d), rows, xr, zr, w, b, o, s)))


def gated_norm_backward(d: NormDims, rows: int, x, z, weight, bias, dout, dx, dz, dweight, dbias=None, *,
                        workspace=None, stream=None) -> None:
    """ssm_gated_norm_backward: the gradients of gated_norm for dout. workspace: a device tensor of
    gated_norm_sizes(...) bytes, or None."""
    rows = _count(rows, "rows")
    xr, zr, w, b = _norm_in(d, rows, x, z, weight, bias)
    wide, tin = d.groups * d.width, _IN_T.get(d.in_dtype)
    own = d.width if d.shared else wide
    g, dxr, dzr = (_ROWS1(*_row_addr(dout, "dout", tin, rows, wide)),
                   _ROWS1(*_row_addr(dx, "dx", _IN_T.get(d.x_dtype), rows, wide)),
                   _ROWS1(*_row_addr(dz, "dz", tin, rows, wide)))
    dw, db = _addr(dweight, "dweight", _F32_T, own), _addr(dbias, "dbias", _F32_T, own)
    args = (x, z, weight, bias, dout, dx, dz, dweight, dbias)
    ws, have = _workspace(workspace, lambda: gated_norm_sizes(d, rows), args, stream)
    _on_device(args + (ws,), stream, lambda s: _check(_lib.ssm_gated_norm_backward(
        ctypes.byref(d), rows, xr, zr, w, b, g,
        dxr, dzr, dw, db, ws.data_ptr(), have, s)))
