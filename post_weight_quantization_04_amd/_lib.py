"""ctypes binding of ``libgptq_mi355x.so`` (the C ABI in ``include/gptq.h``).

Argument marshalling only: torch tensors are turned into device pointers and
the current HIP stream; every computation happens in the library's kernels.
There is no fallback: if the library is missing or fails to load, every call
raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgptq_mi355x.so")

GPTQ_OK, GPTQ_EINVAL, GPTQ_EUNSUPPORTED, GPTQ_EHIP, GPTQ_EWORKSPACE, GPTQ_ESCRATCH = 0, 1, 2, 3, 4, 5
GPTQ_F16, GPTQ_F32, GPTQ_BF16 = 0, 1, 2

EXPORTS = (
    "gptq_hessian_accumulate",
    "gptq_hessian_set",
    "gptq_hessian_accumulate_chunks",
    "gptq_prepare_hinv_workspace",
    "gptq_prepare_hinv",
    "gptq_prepare_hinv_fp32_workspace",
    "gptq_prepare_hinv_fp32",
    "gptq_prepare_hinv_noalloc",
    "gptq_prepare_hinv_noalloc_max_din",
    "gptq_quantize_layer_workspace",
    "gptq_quantize_layer_split_workspace",
    "gptq_quantize_layer",
    "gptq_quantize_layer_split",
    "gptq_status_string",
    "gptq_packed_words",
    "gptq_pack_codes",
    "gptq_dequantize",
    "gptq_output_error",
    "gptq_propagate",
    "gptq_obq_workspace",
    "gptq_obq_quantize",
    "gptq_fp8_weight",
    "gptq_fp8_activations",
    "gptq_fp8_rms_norm",
    "gptq_fp8_matmul",
    "gptq_fp8_gated_workspace",
    "gptq_fp8_gated",
    "gptq_fp8_matmul_kernel",
    "gptq_fp8_gated_kernel",
    "gptq_packed_matmul",
    "gptq_packed_matmul_kernel",
    "gptq_attention",
    "gptq_cache_store",
    "gptq_cached_attention_workspace",
    "gptq_cached_attention",
    "gptq_kernel_count",
    "gptq_kernel_name",
    "gptq_timing_enable",
    "gptq_timing_read",
)


class GptqError(RuntimeError):
    def __init__(self, fn: str, rc: int, msg: str):
        super().__init__(f"{fn} -> {rc} ({msg})")
        self.rc = rc


_lib: Optional[ctypes.CDLL] = None

_vp, _i64, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library once and declare every signature of ``include/gptq.h``."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(
            f"{path} is missing: build it with `python -m post_weight_quantization_04_amd.build`")
    # torch ships its own HIP runtime under the same soname.  Loading torch
    # first makes the library bind to that one runtime, the one that owns the
    # device memory and streams handed in; loaded the other way round, the
    # process holds two runtimes and every launch on torch's buffers fails.
    import torch  # noqa: F401
    lib = ctypes.CDLL(path)
    sig = {
        "gptq_hessian_accumulate": (_i32, [_vp, _i64, _vp, _i32, _i64, _i64, _vp]),
        "gptq_hessian_set": (_i32, [_vp, _i64, _vp, _i32, _i64, _i64, _vp]),
        "gptq_hessian_accumulate_chunks": (_i32, [_vp, _i64, _vp, _i64, _i32, _i64, _i64, _i32, _vp]),
        "gptq_prepare_hinv_workspace": (_sz, [_i64]),
        "gptq_prepare_hinv": (_i32, [_vp, _i64, ctypes.c_double, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
        "gptq_prepare_hinv_fp32_workspace": (_sz, [_i64]),
        "gptq_prepare_hinv_fp32": (_i32, [_vp, _i64, ctypes.c_double, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
        "gptq_prepare_hinv_noalloc": (_i32, [_vp, _i64, ctypes.c_double, _vp, _vp, _vp, _vp, _vp]),
        "gptq_prepare_hinv_noalloc_max_din": (_i64, []),
        "gptq_quantize_layer_workspace": (_sz, [_i64, _i64, _i64]),
        "gptq_quantize_layer_split_workspace": (_sz, [_i64, _i64, _i64]),
        "gptq_quantize_layer": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp,
                                       _vp, _sz, _vp]),
        "gptq_quantize_layer_split": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp,
                                             _vp, _vp, _sz, _vp]),
        "gptq_status_string": (ctypes.c_char_p, [_i32]),
        "gptq_packed_words": (_i64, [_i64, _i32]),
        "gptq_pack_codes": (_i32, [_vp, _i64, _i64, _i32, _vp, _vp]),
        "gptq_dequantize": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _i64, _vp, _i32, _vp]),
        "gptq_output_error": (_i32, [_vp, _i32, _vp, _vp, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
        "gptq_propagate": (_i32, [_vp, _i32, _i64, _i64, _vp, _i32, _i64, _i64, _vp, _i64, _i32, _vp]),
        "gptq_obq_workspace": (_sz, [_i64]),
        "gptq_obq_quantize": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _sz, _vp]),
        "gptq_fp8_weight": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp]),
        "gptq_fp8_activations": (_i32, [_vp, _i32, _i64, _i64, _i64, _i32, _vp, _i64, _vp, _i64, _vp]),
        "gptq_fp8_rms_norm": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i32, _i64, _i64, ctypes.c_double, _vp,
                                     _i64, _vp, _i64, _vp]),
        "gptq_fp8_matmul": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i32, _i64,
                                   _i32, _i32, _vp]),
        "gptq_fp8_gated_workspace": (_sz, [_i64, _i64]),
        "gptq_fp8_gated": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64,
                                  _vp, _i64, _vp, _sz, _vp]),
        "gptq_fp8_matmul_kernel": (ctypes.c_char_p, [_i64, _i64, _i64, _i32, _i32]),
        "gptq_fp8_gated_kernel": (ctypes.c_char_p, [_i64, _i64, _i64, _i32]),
        "gptq_packed_matmul_kernel": (ctypes.c_char_p, [_i64, _i64, _i64, _i64, _i32, _i32]),
        "gptq_packed_matmul": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _i64, _vp, _i32, _i64, _i64, _vp, _vp, _i64,
                                      _vp, _i32, _i64, _i32, _vp]),
        "gptq_attention": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i32, _i64, _i64,
                                  _i64, _i64, _vp, _i64, _i32, ctypes.c_double, _vp]),
        "gptq_cache_store": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i32, _i64, _i64, _i64, _vp, _vp, _i64, _i64,
                                    _i64, _vp, _i64, _i64, _i64, _i64, _i64, _vp]),
        "gptq_cached_attention_workspace": (_sz, [_i64, _i64, _i64, _i64, _i64, _i64]),
        "gptq_cached_attention": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _vp,
                                         _i64, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _i64, _i32,
                                         ctypes.c_double, _vp, _sz, _vp]),
        "gptq_kernel_count": (_i32, []),
        "gptq_kernel_name": (ctypes.c_char_p, [_i32]),
        "gptq_timing_enable": (_i32, [_i32]),
        "gptq_timing_read": (_i32, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _fp8_names()
    _lib = lib
    return lib


def status_string(rc: int) -> str:
    return load().gptq_status_string(rc).decode()


def _check(fn: str, rc: int) -> None:
    if rc != GPTQ_OK:
        raise GptqError(fn, rc, status_string(rc))


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float16:
        return GPTQ_F16
    if t.dtype == torch.float32:
        return GPTQ_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


# ---------------------------------------------------------------------------
# the three entry points
# ---------------------------------------------------------------------------
def _hessian_call(fn: str, H, X, stream) -> None:
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be 2-D with unit column stride")
    d_in, n = X.shape
    if H.shape != (d_in, d_in):
        raise ValueError("H shape")
    if not X.is_cuda:
        raise ValueError("device tensor expected")
    rc = getattr(load(), fn)(_ptr(H), d_in, X.data_ptr(), _dtype_code(X), n, X.stride(0), _stream(stream))
    _check(fn, rc)


def hessian_accumulate(H, X, stream=None) -> None:
    """``H[lower] += 2 X X^T`` for ``X: [d_in, n]`` (a 2-D view with unit
    column stride; row stride = ``X.stride(0)``)."""
    _hessian_call("gptq_hessian_accumulate", H, X, stream)


def hessian_set(H, X, stream=None) -> None:
    """``H[lower] = 2 X X^T`` (the old values not read; the strictly upper
    triangle not written), for the first token chunk."""
    _hessian_call("gptq_hessian_set", H, X, stream)


def hessian_chunks(H, Xs, set_first: bool = False, stream=None) -> None:
    """``H[lower] (=|+=) sum_c 2 X_c X_c^T`` over a list of token chunks of
    one shape, dtype and row stride (2-D views with unit column stride);
    ``set_first`` writes H from the first chunk instead of adding."""
    Xs = list(Xs)
    if not Xs:
        raise ValueError("no chunks")
    X0 = Xs[0]
    for X in Xs:
        if X.dim() != 2 or X.stride(1) != 1 or not X.is_cuda:
            raise ValueError("chunks must be 2-D device views with unit column stride")
        if X.shape != X0.shape or X.stride(0) != X0.stride(0) or X.dtype != X0.dtype:
            raise ValueError("chunks differ in shape, row stride or dtype")
    d_in, n = X0.shape
    if H.shape != (d_in, d_in):
        raise ValueError("H shape")
    ptrs = (ctypes.c_void_p * len(Xs))(*[X.data_ptr() for X in Xs])
    rc = load().gptq_hessian_accumulate_chunks(_ptr(H), d_in, ctypes.cast(ptrs, ctypes.c_void_p), len(Xs),
                                               _dtype_code(X0), n, X0.stride(0), int(bool(set_first)),
                                               _stream(stream))
    _check("gptq_hessian_accumulate_chunks", rc)


def prepare_hinv_workspace(d_in: int, fp32: bool = False) -> int:
    lib = load()
    return int(lib.gptq_prepare_hinv_fp32_workspace(d_in) if fp32 else lib.gptq_prepare_hinv_workspace(d_in))


def prepare_hinv(H, damp_frac: float, U, dead=None, info=None, lambda_out=None, workspace=None,
                 stream=None, fp32: bool = False) -> None:
    """``gptq_prepare_hinv`` (float64 factorization) or, with ``fp32``,
    ``gptq_prepare_hinv_fp32``."""
    d_in = H.shape[0]
    name = "gptq_prepare_hinv_fp32" if fp32 else "gptq_prepare_hinv"
    rc = getattr(load(), name)(_ptr(H), d_in, float(damp_frac), _ptr(U), _ptr(dead), _ptr(info),
                               _ptr(lambda_out), _ptr(workspace),
                               workspace.numel() * workspace.element_size() if workspace is not None else 0,
                               _stream(stream))
    _check(name, rc)


def prepare_hinv_noalloc(H, damp_frac: float, U, dead=None, info=None, lambda_out=None, stream=None) -> None:
    """``gptq_prepare_hinv`` on the library's fixed device scratch (no workspace, no allocation)."""
    d_in = H.shape[0]
    rc = load().gptq_prepare_hinv_noalloc(_ptr(H), d_in, float(damp_frac), _ptr(U), _ptr(dead), _ptr(info),
                                          _ptr(lambda_out), _stream(stream))
    _check("gptq_prepare_hinv_noalloc", rc)


def prepare_hinv_noalloc_max_din() -> int:
    return int(load().gptq_prepare_hinv_noalloc_max_din())


def quantize_layer_workspace(d_out: int, d_in: int, block_size: int, split: bool = False) -> int:
    name = "gptq_quantize_layer_split_workspace" if split else "gptq_quantize_layer_workspace"
    return int(getattr(load(), name)(d_out, d_in, block_size))


def quantize_layer(W, U, dead, bits: int, group_size: int, block_size: int, codes, scales, zeros,
                   err_row=None, minmax=None, workspace=None, stream=None, split: bool = False) -> None:
    """``gptq_quantize_layer``, or ``gptq_quantize_layer_split`` (the lazy
    trailing update on split-precision bf16 products) with ``split``."""
    d_out, d_in = W.shape
    name = "gptq_quantize_layer_split" if split else "gptq_quantize_layer"
    rc = getattr(load(), name)(_ptr(W), _dtype_code(W), d_out, d_in, _ptr(U), _ptr(dead), int(bits),
                               int(group_size), int(block_size), _ptr(codes), _ptr(scales), _ptr(zeros),
                               _ptr(err_row), _ptr(minmax), _ptr(workspace),
                               workspace.numel() * workspace.element_size() if workspace is not None else 0,
                               _stream(stream))
    _check(name, rc)


# ---------------------------------------------------------------------------
# few-bit storage, dequantization, output error
# ---------------------------------------------------------------------------
def packed_words(d_in: int, bits: int) -> int:
    return int(load().gptq_packed_words(d_in, int(bits)))


def pack_codes(codes, bits: int, packed, stream=None) -> None:
    d_out, d_in = codes.shape
    rc = load().gptq_pack_codes(_ptr(codes), d_out, d_in, int(bits), _ptr(packed), _stream(stream))
    _check("gptq_pack_codes", rc)


def dequantize(packed, bits: int, d_in: int, scales, zeros, group_size: int, out, stream=None) -> None:
    d_out = packed.shape[0]
    rc = load().gptq_dequantize(_ptr(packed), int(bits), d_out, d_in, _ptr(scales), _ptr(zeros), int(group_size),
                                _ptr(out), _dtype_code(out), _stream(stream))
    _check("gptq_dequantize", rc)


def output_error(W, dead, packed, bits: int, scales, zeros, group_size: int, err_row, lam, out_row,
                 stream=None) -> None:
    d_out, d_in = W.shape
    rc = load().gptq_output_error(_ptr(W), _dtype_code(W), _ptr(dead), _ptr(packed), int(bits), _ptr(scales),
                                  _ptr(zeros), int(group_size), d_out, d_in, _ptr(err_row), _ptr(lam),
                                  _ptr(out_row), _stream(stream))
    _check("gptq_output_error", rc)


def propagate(W_hat, X, Y, activation: int = 0, stream=None) -> None:
    """``Y = act(W_hat X)``: ``W_hat [d_out, d_in]`` f16 contiguous, ``X
    [d_in, n]`` and ``Y [d_out, n]`` f16 2-D views with unit column stride
    (row strides ``X.stride(0)``, ``Y.stride(0)``); activation 0 none, 1 ReLU."""
    for t in (X, Y):
        if t.dim() != 2 or t.stride(1) != 1 or not t.is_cuda:
            raise ValueError("X and Y must be 2-D device views with unit column stride")
    d_out, d_in = W_hat.shape
    n = X.shape[1]
    if X.shape[0] != d_in or Y.shape != (d_out, n):
        raise ValueError("shapes")
    rc = load().gptq_propagate(_ptr(W_hat), _dtype_code(W_hat), d_out, d_in, X.data_ptr(), _dtype_code(X), n,
                               X.stride(0), Y.data_ptr(), Y.stride(0), int(activation), _stream(stream))
    _check("gptq_propagate", rc)


def obq_workspace(d_in: int) -> int:
    return int(load().gptq_obq_workspace(int(d_in)))


def obq_quantize(W, U, dead, bits: int, codes, scales, zeros, order=None, loss=None, workspace=None,
                 stream=None) -> None:
    d_out, d_in = W.shape
    rc = load().gptq_obq_quantize(_ptr(W), _dtype_code(W), d_out, d_in, _ptr(U), _ptr(dead), int(bits),
                                  _ptr(codes), _ptr(scales), _ptr(zeros), _ptr(order), _ptr(loss),
                                  _ptr(workspace),
                                  workspace.numel() * workspace.element_size() if workspace is not None else 0,
                                  _stream(stream))
    _check("gptq_obq_quantize", rc)


# ---------------------------------------------------------------------------
# 8-bit operands: e4m3 values [rows, ld] (ld a multiple of 16, zeros behind
# the columns up to a multiple of 128) and float32 scales, as include/gptq.h
# lays them out.  `values` may be float8_e4m3fn or uint8.
#
# One decoded token's kernel takes 3 to 6 us, so these calls are written to
# cost the host less: tensors are read once each, by the accessors that do not
# build new objects (asking whether a tensor is contiguous costs a third of
# reading its strides), the names used by every call are set by load(), and
# outputs that the caller made for the call (``made``, contiguous, of the right
# type, shape and device) are not checked.
# ---------------------------------------------------------------------------
_fp8_codes = {}          # torch type -> gptq_dtype
_fp8_eights = ()         # types of the 8-bit values
_fp8_scale = None        # type of the scales
_int32 = None
_fp8_current = None      # () -> index of the current device
_fp8_current_stream = None  # (device index) -> handle of its current stream


def _fp8_names() -> None:
    global _fp8_codes, _fp8_eights, _fp8_scale, _int32, _fp8_current, _fp8_current_stream
    import torch
    _int32 = torch.int32
    _fp8_codes = {torch.float16: GPTQ_F16, torch.float32: GPTQ_F32, torch.bfloat16: GPTQ_BF16}
    _fp8_eights = (torch.float8_e4m3fn, torch.uint8)
    _fp8_scale = torch.float32
    _fp8_current = torch._C._cuda_getDevice
    _fp8_current_stream = torch._C._cuda_getCurrentRawStream


def _fp8_dtype(t) -> int:
    code = _fp8_codes.get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return code


def _fp8_device(t) -> int:
    """Index of the device of ``t``, which has to be the current one (the
    library launches there)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("device tensor expected")
    if dev != _fp8_current():
        raise ValueError(f"tensors on cuda:{dev}, but the current device is cuda:{_fp8_current()}")
    return dev


def _fp8_stream(dev: int, stream) -> int:
    if stream is None:
        return _fp8_current_stream(dev)
    if stream.device.index != dev:
        raise ValueError(f"tensors on cuda:{dev}, stream on {stream.device}")
    return stream.cuda_stream


def _fp8_ld(t, rows: int, cols: int, what: str) -> int:
    """Row stride of a 2-D view with unit column stride."""
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what} must have unit column stride")
    # the stride of a single row is never used, and torch leaves it arbitrary
    return ld if rows > 1 else max(ld, cols)


def _fp8_matrix(t, dev: int, what: str):
    """(pointer, row stride, rows, columns) of a 2-D view on device ``dev``
    with unit column stride."""
    shape = t.shape
    if len(shape) != 2 or t.get_device() != dev:
        raise ValueError(f"{what} must be a 2-D view on cuda:{dev} with unit column stride")
    rows, cols = shape
    return t.data_ptr(), cols if t.is_contiguous() else _fp8_ld(t, rows, cols, what), rows, cols


def _fp8_operand(values, scales, cols: int, by_row: bool, dev: int, what: str):
    """(values pointer, ld, scales pointer, lds, rows) of an 8-bit matrix of
    ``cols`` columns: a scale per row and 128 columns (``by_row``), or per 128
    x 128 block."""
    shape, sshape = values.shape, scales.shape
    if (values.dtype not in _fp8_eights or scales.dtype is not _fp8_scale or len(shape) != 2 or len(sshape) != 2
            or values.get_device() != dev or scales.get_device() != dev):
        raise ValueError(f"{what}: values must be a 2-D float8_e4m3fn view and scales a 2-D float32 view on cuda:{dev}, "
                         f"both with unit column stride")
    rows, held = shape
    lead, along = sshape
    nb = (cols + 127) >> 7
    if held < nb << 7:
        raise ValueError(f"{what}: {held} stored columns hold fewer than {cols} rounded up to 128")
    if (lead < nb or along < rows) if by_row else (lead < (rows + 127) >> 7 or along < nb):
        raise ValueError(f"{what}: scales {(lead, along)} for {rows} x {cols}")
    return (values.data_ptr(), held if values.is_contiguous() else _fp8_ld(values, rows, held, what),
            scales.data_ptr(), along if scales.is_contiguous() else _fp8_ld(scales, lead, along, what), rows)


def _fp8_made(values, scales, cols: int, along: int, dev: int):
    if values.get_device() != dev:
        raise ValueError(f"outputs on another device than cuda:{dev}")
    return values.data_ptr(), (cols + 127) >> 7 << 7, scales.data_ptr(), along


def fp8_weight(W, values, scales, stream=None) -> None:
    """``W [d_out, d_in]`` to 8 bits, a scale per 128 x 128 block."""
    lib = _lib or load()
    dev = _fp8_device(W)
    wp, ldw, d_out, d_in = _fp8_matrix(W, dev, "W")
    vp, ld, sp, lds, rows = _fp8_operand(values, scales, d_in, False, dev, "out")
    if rows != d_out:
        raise ValueError("rows of the output")
    rc = lib.gptq_fp8_weight(wp, _fp8_dtype(W), d_out, d_in, ldw, vp, ld, sp, lds, _fp8_stream(dev, stream))
    if rc:
        _check("gptq_fp8_weight", rc)


def fp8_activations(X, values, scales, channel_major: bool = False, stream=None, made: bool = False) -> None:
    """``X [n, d]`` (or ``[d, n]`` with ``channel_major``) to 8 bits, a scale
    per token and 128 channels."""
    lib = _lib or load()
    dev = _fp8_device(X)
    xp, ldx, n, d = _fp8_matrix(X, dev, "X")
    if channel_major:
        n, d = d, n
    if made:
        vp, ld, sp, lds = _fp8_made(values, scales, d, n, dev)
    else:
        vp, ld, sp, lds, rows = _fp8_operand(values, scales, d, True, dev, "out")
        if rows != n:
            raise ValueError("rows of the output")
    rc = lib.gptq_fp8_activations(xp, _fp8_dtype(X), n, d, ldx, 1 if channel_major else 0, vp, ld, sp, lds,
                                  _fp8_stream(dev, stream))
    if rc:
        _check("gptq_fp8_activations", rc)


def fp8_rms_norm(x, gain, eps: float, values, scales, residual=None, sum_out=None, stream=None, made: bool = False,
                 sum_made: bool = False) -> None:
    """``h = x + residual``; ``h / sqrt(mean(h^2) + eps) * gain`` to 8 bits;
    ``sum_out = h``."""
    lib = _lib or load()
    dev = _fp8_device(x)
    xp, ldx, n, d = _fp8_matrix(x, dev, "x")
    kind, shape = x.dtype, x.shape
    rp, ldr, op, ldo = None, 0, None, 0
    if residual is not None:
        if residual.shape != shape or residual.dtype != kind:
            raise ValueError("residual must have the shape and type of x")
        rp, ldr, _, _ = _fp8_matrix(residual, dev, "residual")
    if sum_made:
        op, ldo = sum_out.data_ptr(), d
    elif sum_out is not None:
        if sum_out.shape != shape or sum_out.dtype != kind:
            raise ValueError("sum_out must have the shape and type of x")
        op, ldo, _, _ = _fp8_matrix(sum_out, dev, "sum_out")
    if gain.shape != shape[1:] or gain.dtype != kind or gain.get_device() != dev or not gain.is_contiguous():
        raise ValueError("gain must be a contiguous vector of x's type, one value per channel")
    if made:
        vp, ld, sp, lds = _fp8_made(values, scales, d, n, dev)
    else:
        vp, ld, sp, lds, rows = _fp8_operand(values, scales, d, True, dev, "out")
        if rows != n:
            raise ValueError("rows of the output")
    rc = lib.gptq_fp8_rms_norm(xp, ldx, rp, ldr, op, ldo, gain.data_ptr(), _fp8_dtype(x), n, d, eps, vp, ld, sp,
                               lds, _fp8_stream(dev, stream))
    if rc:
        _check("gptq_fp8_rms_norm", rc)


def fp8_matmul(wq, ws, xq, xs, d_in: int, Y, channel_major: bool = False, activation: int = 0, stream=None) -> None:
    """``Y = act(X W^T)`` of 8-bit operands; ``Y [n, d_out]``, or ``[d_out,
    n]`` with ``channel_major``; activation 0 none, 1 ReLU."""
    lib = _lib or load()
    dev = _fp8_device(Y)
    yp, ldy, y0, y1 = _fp8_matrix(Y, dev, "Y")
    wp, ldw, wsp, ldws, d_out = _fp8_operand(wq, ws, d_in, False, dev, "weights")
    xp, ldx, xsp, ldxs, n = _fp8_operand(xq, xs, d_in, True, dev, "activations")
    if (y0 != d_out or y1 != n) if channel_major else (y0 != n or y1 != d_out):
        raise ValueError("shape of Y")
    rc = lib.gptq_fp8_matmul(wp, ldw, wsp, ldws, d_out, d_in, xp, ldx, xsp, ldxs, n, yp, _fp8_dtype(Y), ldy,
                             1 if channel_major else 0, activation, _fp8_stream(dev, stream))
    if rc:
        _check("gptq_fp8_matmul", rc)


def fp8_gated_workspace(n: int, d_ff: int) -> int:
    return load().gptq_fp8_gated_workspace(n, d_ff)


def fp8_gated(gq, gs, uq, us, xq, xs, d_in: int, values, scales, workspace=None, stream=None,
              made: bool = False) -> None:
    """``silu(X G^T) * (X U^T)`` of 8-bit operands, written in 8 bits."""
    lib = _lib or load()
    dev = _fp8_device(values)
    gp, ldw, gsp, ldws, d_ff = _fp8_operand(gq, gs, d_in, False, dev, "gate")
    up, ldu, usp, ldus, up_rows = _fp8_operand(uq, us, d_in, False, dev, "up")
    if up_rows != d_ff or (ldu != ldw and d_ff > 1) or (ldus != ldws and d_ff > 128):
        raise ValueError("gate and up must have one shape and strides")
    xp, ldx, xsp, ldxs, n = _fp8_operand(xq, xs, d_in, True, dev, "activations")
    if made:
        vp, ld, sp, lds = _fp8_made(values, scales, d_ff, n, dev)
    else:
        vp, ld, sp, lds, rows = _fp8_operand(values, scales, d_ff, True, dev, "out")
        if rows != n:
            raise ValueError("rows of the output")
    room = 0
    if workspace is not None:
        if workspace.get_device() != dev:
            raise ValueError("workspace on another device")
        room = workspace.numel() * workspace.element_size()
    rc = lib.gptq_fp8_gated(gp, gsp, up, usp, ldw, ldws, d_ff, d_in, xp, ldx, xsp, ldxs, n, vp, ld, sp, lds,
                            _ptr(workspace), room, _fp8_stream(dev, stream))
    if rc:
        _check("gptq_fp8_gated", rc)


def fp8_matmul_kernel(n: int, d_out: int, d_in: int, dtype, compute_units: int = 0) -> Optional[str]:
    """Which kernel a product of these sizes and output type runs on, on a
    device of ``compute_units`` CUs (0: the current one)."""
    name = load().gptq_fp8_matmul_kernel(d_out, d_in, n, _fp8_codes.get(dtype, -1), compute_units)
    return name.decode() if name else None


def fp8_gated_kernel(n: int, d_ff: int, d_in: int, compute_units: int = 0) -> Optional[str]:
    """Which kernel a gated block of these sizes runs on."""
    name = load().gptq_fp8_gated_kernel(d_ff, d_in, n, compute_units)
    return name.decode() if name else None


# ---------------------------------------------------------------------------
# Products with packed weights, attention and the paged cache.  As above, these
# calls are written to cost the host little: they take as long as a small call's
# kernel.
# ---------------------------------------------------------------------------
ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3}


def _whole_numbers(t, dev: int, what: str):
    """(pointer, row stride) of a 1-D or 2-D int32 tensor on device ``dev``,
    its last dimension contiguous."""
    if t.dtype is not _int32 or t.get_device() != dev:
        raise ValueError(f"{what} must be int32 on cuda:{dev}")
    if not t.is_contiguous() and (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{what} must be contiguous in its last dimension")
    if len(t.shape) == 1:
        return t.data_ptr(), 0
    rows, cols = t.shape
    return t.data_ptr(), t.stride(0) if rows > 1 else cols


def packed_matmul(packed, bits: int, d_in: int, scales, zeros, group_size: int, X, Y, bias=None, residual=None,
                  activation: int = 0, stream=None) -> None:
    """``Y = act(X W^T + bias) + residual`` over packed codes, ``X [n, d_in]``
    and ``Y [n, d_out]`` 2-D views with unit column stride."""
    lib = _lib or load()
    dev = _fp8_device(Y)
    yp, ldy, n, d_out = _fp8_matrix(Y, dev, "Y")
    xp, ldx, n_x, d_x = _fp8_matrix(X, dev, "X")
    if n_x != n or d_x != d_in:
        raise ValueError(f"X is {n_x} x {d_x}, the product {n} x {d_in}")
    groups = d_in // group_size if group_size > 0 else 1
    shape, kind = scales.shape, Y.dtype
    if (packed.dtype is not _int32 or packed.get_device() != dev or not packed.is_contiguous()
            or len(packed.shape) != 2 or packed.shape[0] != d_out
            or packed.shape[1] != max((d_in * bits + 31) >> 5, 1)):
        raise ValueError(f"packed must be a contiguous int32 [{d_out}, {max((d_in * bits + 31) >> 5, 1)}] on cuda:{dev}")
    if (len(shape) != 2 or shape[0] != d_out or shape[1] != groups or zeros.shape != shape or scales.dtype is not _fp8_scale
            or zeros.dtype is not _int32 or scales.get_device() != dev or zeros.get_device() != dev
            or not scales.is_contiguous() or not zeros.is_contiguous()):
        raise ValueError(f"scales (float32) and zeros (int32) must be contiguous [{d_out}, {groups}] on cuda:{dev}")
    bp, rp, ldr = None, None, 0
    if bias is not None:
        if bias.shape != Y.shape[1:] or bias.dtype != kind or bias.get_device() != dev or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous vector of Y's type, one value per output")
        bp = bias.data_ptr()
    if residual is not None:
        if residual.shape != Y.shape or residual.dtype != kind:
            raise ValueError("residual must have the shape and type of Y")
        rp, ldr, _, _ = _fp8_matrix(residual, dev, "residual")
    rc = lib.gptq_packed_matmul(packed.data_ptr(), bits, d_out, d_in, scales.data_ptr(), zeros.data_ptr(), group_size,
                                xp, _fp8_dtype(X), n, ldx, bp, rp, ldr, yp, _fp8_dtype(Y), ldy, activation,
                                _fp8_stream(dev, stream))
    if rc:
        _check("gptq_packed_matmul", rc)


def packed_matmul_kernel(n: int, d_out: int, d_in: int, group_size: int = 0, aligned: bool = True,
                         compute_units: int = 0) -> Optional[str]:
    """Which kernel a product with packed weights of these sizes runs on, where
    rows of X start 16-byte aligned or not."""
    name = load().gptq_packed_matmul_kernel(d_out, d_in, group_size, n, aligned, compute_units)
    return name.decode() if name else None


def _heads_of(t, dev: int, kind, what: str):
    """(pointer, token stride, head stride, tokens, heads, d) of a [tokens,
    heads, d] view on device ``dev`` with unit last stride."""
    shape = t.shape
    if len(shape) != 3 or t.dtype is not kind or t.get_device() != dev:
        raise ValueError(f"{what} must be a 3-D {kind} view on cuda:{dev}")
    n, heads, d = shape
    if t.is_contiguous():
        return t.data_ptr(), heads * d, d, n, heads, d
    token, head, step = t.stride()
    if step != 1 and d > 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    # strides that are never used, and that torch leaves arbitrary
    if heads <= 1:
        head = d
    if n <= 1:
        token = max(d, 8)
    return t.data_ptr(), token, head, n, heads, d


def _pages_of(t, dev: int, kind, what: str):
    """(pointer, page, head and row strides) of a [pages, heads, rows, d] view."""
    shape = t.shape
    if len(shape) != 4 or t.dtype is not kind or t.get_device() != dev:
        raise ValueError(f"{what} must be a 4-D {kind} view on cuda:{dev}")
    pages, heads, rows, d = shape
    if t.is_contiguous():
        return t.data_ptr(), heads * rows * d, rows * d, d
    page, head, row, step = t.stride()
    if step != 1 and d > 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    return t.data_ptr(), page if pages > 1 else max(d, 8), head if heads > 1 else d, row if rows > 1 else d


def attention(q, k, v, starts, out, causal: bool, scale: float, stream=None) -> None:
    """Attention over packed prompts: ``q``, ``out`` [n, heads, d], ``k``, ``v``
    [n, kv_heads, d], ``starts`` [n_seqs + 1] int32 or None (one sequence)."""
    lib = _lib or load()
    dev, kind = _fp8_device(q), q.dtype
    qp, qt, qh, n, heads, d = _heads_of(q, dev, kind, "q")
    kp, kt, kh, n_k, kv_heads, d_k = _heads_of(k, dev, kind, "k")
    vp, vt, vh, n_v, heads_v, d_v = _heads_of(v, dev, kind, "v")
    op, ot, oh, n_o, heads_o, d_o = _heads_of(out, dev, kind, "out")
    if n_k != n or n_v != n or n_o != n or heads_v != kv_heads or heads_o != heads or d_k != d or d_v != d or d_o != d:
        raise ValueError("q and out must have one shape, k and v too, with q's tokens and head size")
    sp, seqs = None, 1
    if starts is not None:
        if len(starts.shape) != 1 or starts.shape[0] < 1:
            raise ValueError("starts must be a vector of one value per sequence and one more")
        sp, _ = _whole_numbers(starts, dev, "starts")
        seqs = starts.shape[0] - 1
    rc = lib.gptq_attention(qp, qt, qh, kp, kt, kh, vp, vt, vh, op, ot, oh, _fp8_dtype(q), n, heads, kv_heads, d, sp,
                            seqs, 1 if causal else 0, scale, _fp8_stream(dev, stream))
    if rc:
        _check("gptq_attention", rc)


def cache_store(k, v, slots, keys, values, stream=None) -> None:
    """``keys[page, :, row] = k[t]``, ``values[page, :, row] = v[t]`` for
    ``slots[t] = page * page_size + row``."""
    lib = _lib or load()
    dev, kind = _fp8_device(k), k.dtype
    kp, kt, kh, n, kv_heads, d = _heads_of(k, dev, kind, "k")
    vp, vt, vh, n_v, heads_v, d_v = _heads_of(v, dev, kind, "v")
    cp, c0, c1, c2 = _pages_of(keys, dev, kind, "keys")
    wp, w0, w1, w2 = _pages_of(values, dev, kind, "values")
    pages, cached, page_size, d_c = keys.shape
    if n_v != n or heads_v != kv_heads or d_v != d or values.shape != keys.shape or cached != kv_heads or d_c != d:
        raise ValueError("k and v must have one shape, keys and values too, with the heads and head size of k")
    if slots.shape != k.shape[:1]:
        raise ValueError("slots must be a vector of one value per token")
    sp, _ = _whole_numbers(slots, dev, "slots")
    rc = lib.gptq_cache_store(kp, kt, kh, vp, vt, vh, _fp8_dtype(k), n, kv_heads, d, sp, cp, c0, c1, c2, wp, w0, w1, w2,
                              pages, page_size, _fp8_stream(dev, stream))
    if rc:
        _check("gptq_cache_store", rc)


def cached_attention_workspace(n_seqs: int, heads: int, kv_heads: int, d: int, max_pages: int, page_size: int) -> int:
    return load().gptq_cached_attention_workspace(n_seqs, heads, kv_heads, d, max_pages, page_size)


def cached_attention(q, keys, values, table, lengths, out, scale: float, workspace=None, stream=None) -> None:
    """Attention of one new token a sequence: ``q``, ``out`` [n_seqs, heads, d],
    ``table`` [n_seqs, max_pages] and ``lengths`` [n_seqs] int32."""
    lib = _lib or load()
    dev, kind = _fp8_device(q), q.dtype
    qp, qt, qh, n, heads, d = _heads_of(q, dev, kind, "q")
    op, ot, oh, n_o, heads_o, d_o = _heads_of(out, dev, kind, "out")
    cp, c0, c1, c2 = _pages_of(keys, dev, kind, "keys")
    wp, w0, w1, w2 = _pages_of(values, dev, kind, "values")
    pages, kv_heads, page_size, d_c = keys.shape
    if n_o != n or heads_o != heads or d_o != d or values.shape != keys.shape or d_c != d:
        raise ValueError("q and out must have one shape, keys and values too, with one head size")
    if len(table.shape) != 2 or table.shape[0] != n or lengths.shape != q.shape[:1]:
        raise ValueError("table must have a row, and lengths a value, per sequence")
    tp, ldt = _whole_numbers(table, dev, "table")
    lp, _ = _whole_numbers(lengths, dev, "lengths")
    room = 0
    if workspace is not None:
        if workspace.get_device() != dev:
            raise ValueError("workspace on another device")
        room = workspace.numel() * workspace.element_size()
    rc = lib.gptq_cached_attention(qp, qt, qh, cp, c0, c1, c2, wp, w0, w1, w2, pages, page_size, tp, ldt,
                                   table.shape[1], lp, n, heads, kv_heads, d, op, ot, oh, _fp8_dtype(q), scale,
                                   _ptr(workspace), room, _fp8_stream(dev, stream))
    if rc:
        _check("gptq_cached_attention", rc)


# ---------------------------------------------------------------------------
# kernel timing
# ---------------------------------------------------------------------------
def kernel_names() -> Tuple[str, ...]:
    lib = load()
    return tuple(lib.gptq_kernel_name(i).decode() for i in range(lib.gptq_kernel_count()))


def timing_enable(name: Optional[str]) -> None:
    idx = -1 if name is None else kernel_names().index(name)
    _check("gptq_timing_enable", load().gptq_timing_enable(idx))


def timing_read() -> Tuple[float, int]:
    ms = ctypes.c_double()
    n = ctypes.c_int64()
    _check("gptq_timing_read", load().gptq_timing_read(ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value
