"""ctypes binding for libhadq (include/hadq.h).  Argument marshalling only.

The entry points keep the C names.  Tensors are passed as raw device
pointers; every step of the rotation and quantization runs in libhadq's CUDA
kernels.  There is no fallback: if ``libhadq.so`` is missing or the CUDA call
fails, a ``HadqError`` is raised.

    codes, scales = hadq_rotate_quant(x, block=0, fmt="int4", group=128)

``x`` is any contiguous fp32 / bf16 CUDA tensor; its last dimension is n
(the rotated dimension), all leading dimensions are rows.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libhadq.so")

HADQ_OK, HADQ_ERR_INVALID_ARG, HADQ_ERR_UNSUPPORTED, HADQ_ERR_MISALIGNED, HADQ_ERR_CUDA = range(5)
HADQ_F32, HADQ_BF16 = 0, 1
FMTS = {"int4": 0, "int8": 1, "mxfp4": 2, "nvfp4": 3, "mxfp4_blocked": 4, "nvfp4_blocked": 5}
HADQ_SIGNS_AFTER, HADQ_SIGNS_BEFORE = 0, 1
SIDES = {"after": HADQ_SIGNS_AFTER, "before": HADQ_SIGNS_BEFORE}
EXPORTS = (
    "hadq_rotate", "hadq_rotate_inverse", "hadq_rotate_quant", "hadq_rotate_quant_host",
    "hadq_codes_bytes", "hadq_scales_bytes", "hadq_status_string", "hadq_last_error", "hadq_version",
    "hadq_device_faults", "hadq_rotate_quant_host_static", "hadq_rotate_signed", "hadq_rotate_quant_signed",
    "hadq_rotate_quant_nvfp4", "hadq_set_impl", "hadq_get_impl", "hadq_codebook",
    "hadq_rotate_rpbh", "hadq_rotate_quant_rpbh", "hadq_rotate_quant_codebook",
    "hadq_rmsnorm_quant", "hadq_matmul_int8", "hadq_kv4_append", "hadq_kv4_attention",
    "hadq_kv4_attention_workspace",
)
IMPLS = {"auto": 0, "butterfly": 1, "tensor": 2}

_lock = threading.Lock()
_lib = None


class HadqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libhadq status {status}: {message}")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libhadq.so once and declare the C signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise HadqError(-1, f"{path} is not built; run `python -m hadamard_rotation_bit_b200.build`")
        lib = ctypes.CDLL(path)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.hadq_rotate.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp]
        lib.hadq_rotate_inverse.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp]
        lib.hadq_rotate_quant.argtypes = [vp, i32, i64, i64, i64, i32, i64, vp, vp, vp]
        lib.hadq_rotate_quant_host.argtypes = [vp, i32, i64, i64, i64, i32, i64, vp, vp, vp, vp, vp, vp]
        for f in ("hadq_rotate", "hadq_rotate_inverse", "hadq_rotate_quant", "hadq_rotate_quant_host"):
            getattr(lib, f).restype = i32
        lib.hadq_codes_bytes.argtypes = [i64, i64, i32]
        lib.hadq_codes_bytes.restype = i64
        lib.hadq_scales_bytes.argtypes = [i64, i64, i32, i64]
        lib.hadq_scales_bytes.restype = i64
        lib.hadq_status_string.argtypes = [i32]
        lib.hadq_status_string.restype = ctypes.c_char_p
        lib.hadq_last_error.argtypes = []
        lib.hadq_last_error.restype = ctypes.c_char_p
        lib.hadq_version.argtypes = []
        lib.hadq_version.restype = i32
        lib.hadq_device_faults.argtypes = [i32]
        lib.hadq_device_faults.restype = i32
        lib.hadq_rotate_quant_host_static.argtypes = [vp, i32, i64, i64, i64, i32, i64, vp, vp, vp]
        lib.hadq_rotate_quant_host_static.restype = i32
        lib.hadq_rotate_signed.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp, i32, vp]
        lib.hadq_rotate_signed.restype = i32
        lib.hadq_rotate_quant_signed.argtypes = [vp, i32, i64, i64, i64, vp, i32, i32, i64, vp, vp, vp]
        lib.hadq_rotate_quant_signed.restype = i32
        lib.hadq_rotate_quant_nvfp4.argtypes = [vp, i32, i64, i64, i64, ctypes.c_float, vp, vp, vp]
        lib.hadq_rotate_quant_nvfp4.restype = i32
        lib.hadq_set_impl.argtypes = [i32]
        lib.hadq_set_impl.restype = i32
        lib.hadq_get_impl.argtypes = []
        lib.hadq_get_impl.restype = i32
        lib.hadq_codebook.argtypes = [i64, i32, vp, vp]
        lib.hadq_codebook.restype = i32
        lib.hadq_rotate_rpbh.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp, i32, vp]
        lib.hadq_rotate_rpbh.restype = i32
        lib.hadq_rotate_quant_rpbh.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, i64, vp, vp, vp]
        lib.hadq_rotate_quant_rpbh.restype = i32
        lib.hadq_rotate_quant_codebook.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, vp, vp, vp, vp]
        lib.hadq_rotate_quant_codebook.restype = i32
        f32 = ctypes.c_float
        lib.hadq_rmsnorm_quant.argtypes = [vp, i32, i64, i64, vp, vp, f32, vp, vp, vp, vp]
        lib.hadq_matmul_int8.argtypes = [vp, vp, i64, vp, vp, i64, i64, vp, vp, i32, vp]
        lib.hadq_kv4_append.argtypes = [vp, i64, vp, i64, i32, i64, i64, i64, i64, i64, vp, i64, i64, vp, vp, vp, vp, vp]
        lib.hadq_kv4_attention.argtypes = [vp, i64, i32, i64, i64, i64, i64, i64, i64, i64, vp, vp, vp, vp, i64, i64,
                                           vp, i64, vp, f32, vp, vp, i64, vp]
        for f in ("hadq_rmsnorm_quant", "hadq_matmul_int8", "hadq_kv4_append", "hadq_kv4_attention"):
            getattr(lib, f).restype = i32
        lib.hadq_kv4_attention_workspace.argtypes = [i64, i64, i64, i64, i64, i64]
        lib.hadq_kv4_attention_workspace.restype = i64
        _lib = lib
        return lib


def _check(status: int) -> None:
    if status != HADQ_OK:
        lib = load_library()
        msg = lib.hadq_last_error().decode() or lib.hadq_status_string(status).decode()
        raise HadqError(status, msg)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return HADQ_F32
    if t == torch.bfloat16:
        return HADQ_BF16
    raise HadqError(HADQ_ERR_INVALID_ARG, f"unsupported dtype {t} (float32 or bfloat16)")


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _on_device(name: str, t: torch.Tensor, dev: torch.device) -> None:
    """The C ABI takes device pointers: a host tensor here would be read or
    written by the kernel through a host address."""
    if not t.is_cuda:
        raise HadqError(HADQ_ERR_INVALID_ARG, f"{name} must be a CUDA tensor (got {t.device})")
    if t.device != dev:
        raise HadqError(HADQ_ERR_INVALID_ARG, f"{name} is on {t.device}, x on {dev}")


def _on_host(name: str, t: torch.Tensor) -> None:
    if t.is_cuda:
        raise HadqError(HADQ_ERR_INVALID_ARG, f"{name} must be a host tensor (got {t.device})")


def _holds(name: str, t: torch.Tensor, nbytes: int) -> None:
    """A caller-supplied buffer must be contiguous and at least nbytes long:
    the C ABI receives only its address."""
    if not t.is_contiguous():
        raise HadqError(HADQ_ERR_INVALID_ARG, f"{name} must be contiguous")
    if t.numel() * t.element_size() < nbytes:
        raise HadqError(HADQ_ERR_INVALID_ARG,
                        f"{name} holds {t.numel() * t.element_size()} bytes, the call writes {nbytes}")


def _quant_outputs(lib, rows: int, n: int, fmt: str, group: int, codes, scales, dev) -> None:
    if fmt not in FMTS:
        raise HadqError(HADQ_ERR_INVALID_ARG, f"unknown fmt {fmt!r}")
    for name, t, nbytes in (("codes", codes, int(lib.hadq_codes_bytes(rows, n, FMTS[fmt]))),
                            ("scales", scales, int(lib.hadq_scales_bytes(rows, n, FMTS[fmt], group)))):
        if dev is None:
            _on_host(name, t)
        else:
            _on_device(name, t, dev)
        _holds(name, t, nbytes)


def _rows_n(x: torch.Tensor):
    if not x.is_contiguous():
        raise HadqError(HADQ_ERR_INVALID_ARG, "tensors must be contiguous")
    n = x.shape[-1] if x.dim() else 1
    return (x.numel() // n if n else 0), n


def hadq_device_faults(clear: bool = True) -> int:
    """Fault bits of kernels whose bounded waits ran out (0 = none)."""
    return int(load_library().hadq_device_faults(1 if clear else 0))


def hadq_set_impl(impl: str) -> str:
    """Choose the implementation for the shapes both cover ("auto", "tensor"
    or "butterfly", see include/hadq.h); returns the previous choice."""
    lib = load_library()
    if impl not in IMPLS:
        raise HadqError(HADQ_ERR_INVALID_ARG, f"unknown impl {impl!r}")
    prev = hadq_get_impl()
    _check(lib.hadq_set_impl(IMPLS[impl]))
    return prev


def hadq_get_impl() -> str:
    code = int(load_library().hadq_get_impl())
    return {v: k for k, v in IMPLS.items()}[code]


def hadq_codebook(d: int, bits: int):
    """The library's unit-sphere Lloyd-Max codebook for rows of length d:
    (centroids, thresholds) as float64 numpy arrays (see include/hadq.h)."""
    import numpy as np
    lib = load_library()
    c = np.empty(1 << bits, dtype=np.float64)
    t = np.empty(max(1, (1 << bits) - 1), dtype=np.float64)
    _check(lib.hadq_codebook(int(d), int(bits), c.ctypes.data, t.ctypes.data))
    return c, t[: (1 << bits) - 1]


def codes_nbytes(rows: int, n: int, fmt: str) -> int:
    return int(load_library().hadq_codes_bytes(rows, n, FMTS[fmt]))


def scales_nbytes(rows: int, n: int, fmt: str, group: int) -> int:
    return int(load_library().hadq_scales_bytes(rows, n, FMTS[fmt], group))


def output_shapes(rows: int, n: int, fmt: str, group: int):
    """(codes shape, codes dtype, scales shape, scales dtype) of hadq_rotate_quant."""
    if fmt == "int4":
        return (rows, n // 2), torch.uint8, (rows, n // group), torch.float16
    if fmt == "int8":
        return (rows, n), torch.int8, (rows,), torch.float32
    if fmt == "mxfp4":
        return (rows, n // 2), torch.uint8, (rows, n // 32), torch.uint8
    if fmt == "nvfp4":
        return (rows, n // 2), torch.uint8, (rows, n // 16), torch.uint8
    if fmt in ("mxfp4_blocked", "nvfp4_blocked"):
        # the tiled GEMM scale layout: rows padded to 128, stored as 128 x 4 tiles
        blk = 32 if fmt == "mxfp4_blocked" else 16
        return (rows, n // 2), torch.uint8, ((rows + 127) // 128 * 128, n // blk), torch.uint8
    raise HadqError(HADQ_ERR_INVALID_ARG, f"unknown fmt {fmt!r}")


def hadq_rotate(x: torch.Tensor, block: int = 0, out: torch.Tensor | None = None,
                out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """out = x . diag(H_b) / sqrt(b) along the last dimension (see include/hadq.h)."""
    lib = load_library()
    rows, n = _rows_n(x)
    _on_device("x", x, x.device)
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    _on_device("out", out, x.device)
    _holds("out", out, rows * n * out.element_size())
    _check(lib.hadq_rotate(x.data_ptr(), _dtype_code(x.dtype), rows, n, block, out.data_ptr(),
                           _dtype_code(out.dtype), _stream_handle(stream)))
    return out


def hadq_rotate_inverse(x: torch.Tensor, block: int = 0, out: torch.Tensor | None = None,
                        out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """Inverse rotation (the same symmetric, involutory operation)."""
    lib = load_library()
    rows, n = _rows_n(x)
    _on_device("x", x, x.device)
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    _on_device("out", out, x.device)
    _holds("out", out, rows * n * out.element_size())
    _check(lib.hadq_rotate_inverse(x.data_ptr(), _dtype_code(x.dtype), rows, n, block, out.data_ptr(),
                                   _dtype_code(out.dtype), _stream_handle(stream)))
    return out


def hadq_rotate_quant(x: torch.Tensor, block: int = 0, fmt: str = "int4", group: int = 128,
                      codes: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """Rotate and quantize in one pass; returns (codes, scales) (see include/hadq.h)."""
    lib = load_library()
    rows, n = _rows_n(x)
    _on_device("x", x, x.device)
    cs, cd, ss, sd = output_shapes(rows, n, fmt, group if fmt == "int4" else 32)
    if codes is None:
        codes = torch.empty(cs, dtype=cd, device=x.device)
    if scales is None:
        scales = torch.empty(ss, dtype=sd, device=x.device)
    _quant_outputs(lib, rows, n, fmt, group, codes, scales, x.device)
    _check(lib.hadq_rotate_quant(x.data_ptr(), _dtype_code(x.dtype), rows, n, block, FMTS[fmt], group,
                                 codes.data_ptr(), scales.data_ptr(), _stream_handle(stream)))
    return codes, scales


def hadq_rotate_quant_host(x_host: torch.Tensor, block: int, fmt: str, group: int,
                           codes_host: torch.Tensor, scales_host: torch.Tensor,
                           x_dev: torch.Tensor, codes_dev: torch.Tensor, scales_dev: torch.Tensor,
                           stream=None) -> None:
    """Host-buffer form: copy in, rotate+quantize, copy out, all enqueued on `stream`."""
    lib = load_library()
    rows, n = _rows_n(x_host)
    _on_host("x_host", x_host)
    _quant_outputs(lib, rows, n, fmt, group, codes_host, scales_host, None)
    _on_device("x_dev", x_dev, x_dev.device)
    _holds("x_dev", x_dev, rows * n * x_host.element_size())
    _quant_outputs(lib, rows, n, fmt, group, codes_dev, scales_dev, x_dev.device)
    _check(lib.hadq_rotate_quant_host(x_host.data_ptr(), _dtype_code(x_host.dtype), rows, n, block, FMTS[fmt], group,
                                      codes_host.data_ptr(), scales_host.data_ptr(), x_dev.data_ptr(),
                                      codes_dev.data_ptr(), scales_dev.data_ptr(), _stream_handle(stream)))


def hadq_rotate_quant_host_static(x_host: torch.Tensor, block: int, fmt: str, group: int,
                                  codes_host: torch.Tensor, scales_host: torch.Tensor, stream=None) -> None:
    """Host buffers only: the library stages through its own static device
    array (32 MiB per GPU), so this call allocates no device memory."""
    lib = load_library()
    rows, n = _rows_n(x_host)
    _on_host("x_host", x_host)
    _quant_outputs(lib, rows, n, fmt, group, codes_host, scales_host, None)
    _check(lib.hadq_rotate_quant_host_static(x_host.data_ptr(), _dtype_code(x_host.dtype), rows, n, block, FMTS[fmt],
                                             group, codes_host.data_ptr(), scales_host.data_ptr(),
                                             _stream_handle(stream)))


def _signs_ptr(signs: torch.Tensor | None, dev: torch.device, b: int) -> int | None:
    if signs is None:
        return None
    if signs.dtype != torch.int8 or not signs.is_contiguous():
        raise HadqError(HADQ_ERR_INVALID_ARG, "signs must be a contiguous int8 tensor")
    _on_device("signs", signs, dev)
    _holds("signs", signs, b)
    return signs.data_ptr()


def _block_len(n: int, block: int) -> int:
    """b of the call (block 0 or -1: the whole row)."""
    return n if block in (0, -1) or block >= n else block


def hadq_rotate_signed(x: torch.Tensor, signs: torch.Tensor, side: str = "after", block: int = 0,
                       out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                       stream=None) -> torch.Tensor:
    """Random Hadamard rotation: every block times H_b diag(s) / sqrt(b)
    (side "after") or diag(s) H_b / sqrt(b) (side "before"); ``signs`` holds
    the b int8 signs on the device (see include/hadq.h)."""
    lib = load_library()
    rows, n = _rows_n(x)
    _on_device("x", x, x.device)
    sp = _signs_ptr(signs, x.device, _block_len(n, block))
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    _on_device("out", out, x.device)
    _holds("out", out, rows * n * out.element_size())
    _check(lib.hadq_rotate_signed(x.data_ptr(), _dtype_code(x.dtype), rows, n, block, sp,
                                  SIDES[side], out.data_ptr(), _dtype_code(out.dtype), _stream_handle(stream)))
    return out


def hadq_rotate_quant_signed(x: torch.Tensor, signs: torch.Tensor, side: str = "after", block: int = 0,
                             fmt: str = "int4", group: int = 128, codes: torch.Tensor | None = None,
                             scales: torch.Tensor | None = None, stream=None):
    """Random Hadamard rotation and quantization in one pass; returns (codes, scales)."""
    lib = load_library()
    rows, n = _rows_n(x)
    _on_device("x", x, x.device)
    sp = _signs_ptr(signs, x.device, _block_len(n, block))
    cs, cd, ss, sd = output_shapes(rows, n, fmt, group if fmt == "int4" else 32)
    if codes is None:
        codes = torch.empty(cs, dtype=cd, device=x.device)
    if scales is None:
        scales = torch.empty(ss, dtype=sd, device=x.device)
    _quant_outputs(lib, rows, n, fmt, group, codes, scales, x.device)
    _check(lib.hadq_rotate_quant_signed(x.data_ptr(), _dtype_code(x.dtype), rows, n, block, sp,
                                        SIDES[side], FMTS[fmt], group, codes.data_ptr(), scales.data_ptr(),
                                        _stream_handle(stream)))
    return codes, scales


def hadq_rotate_quant_nvfp4(x: torch.Tensor, tensor_scale: float = 1.0, block: int = 0,
                            codes: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """Rotate and quantize to NVFP4 with a per-tensor scale; returns (codes, E4M3 scales)."""
    lib = load_library()
    rows, n = _rows_n(x)
    _on_device("x", x, x.device)
    cs, cd, ss, sd = output_shapes(rows, n, "nvfp4", 16)
    if codes is None:
        codes = torch.empty(cs, dtype=cd, device=x.device)
    if scales is None:
        scales = torch.empty(ss, dtype=sd, device=x.device)
    _quant_outputs(lib, rows, n, "nvfp4", 16, codes, scales, x.device)
    _check(lib.hadq_rotate_quant_nvfp4(x.data_ptr(), _dtype_code(x.dtype), rows, n, block, float(tensor_scale),
                                       codes.data_ptr(), scales.data_ptr(), _stream_handle(stream)))
    return codes, scales


def _rpbh_ptrs(perm, signs, dev, n):
    if perm is None or signs is None:
        raise HadqError(HADQ_ERR_INVALID_ARG, "RPBH needs perm (int32) and signs (int8)")
    if perm.dtype != torch.int32 or signs.dtype != torch.int8:
        raise HadqError(HADQ_ERR_INVALID_ARG, "perm must be int32 and signs int8")
    for name, t, nb in (("perm", perm, 4 * n), ("signs", signs, n)):
        _on_device(name, t, dev)
        _holds(name, t, nb)
    return perm.data_ptr(), signs.data_ptr()


def hadq_rotate_rpbh(x: torch.Tensor, perm: torch.Tensor, signs: torch.Tensor, block: int = 0,
                     out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None, stream=None):
    """RPBH rotation: x[..., perm] * signs, then the block rotation (see include/hadq.h)."""
    lib = load_library()
    rows, n = _rows_n(x)
    _on_device("x", x, x.device)
    pp, sp = _rpbh_ptrs(perm, signs, x.device, n)
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    _on_device("out", out, x.device)
    _holds("out", out, rows * n * out.element_size())
    _check(lib.hadq_rotate_rpbh(x.data_ptr(), _dtype_code(x.dtype), rows, n, block, pp, sp, out.data_ptr(),
                                _dtype_code(out.dtype), _stream_handle(stream)))
    return out


def hadq_rotate_quant_rpbh(x: torch.Tensor, perm: torch.Tensor, signs: torch.Tensor, block: int = 0,
                           fmt: str = "int4", group: int = 128, codes: torch.Tensor | None = None,
                           scales: torch.Tensor | None = None, stream=None):
    """RPBH rotation and quantization in one pass; returns (codes, scales)."""
    lib = load_library()
    rows, n = _rows_n(x)
    _on_device("x", x, x.device)
    pp, sp = _rpbh_ptrs(perm, signs, x.device, n)
    cs, cd, ss, sd = output_shapes(rows, n, fmt, group if fmt == "int4" else 32)
    if codes is None:
        codes = torch.empty(cs, dtype=cd, device=x.device)
    if scales is None:
        scales = torch.empty(ss, dtype=sd, device=x.device)
    _quant_outputs(lib, rows, n, fmt, group, codes, scales, x.device)
    _check(lib.hadq_rotate_quant_rpbh(x.data_ptr(), _dtype_code(x.dtype), rows, n, block, pp, sp, FMTS[fmt], group,
                                      codes.data_ptr(), scales.data_ptr(), _stream_handle(stream)))
    return codes, scales


def hadq_rotate_quant_codebook(x: torch.Tensor, bits: int, thresholds: torch.Tensor, block: int = 0,
                               perm: torch.Tensor | None = None, signs: torch.Tensor | None = None,
                               codes: torch.Tensor | None = None, norms: torch.Tensor | None = None, stream=None):
    """Per-token norm + nearest-centroid codes of the (RPBH or plain) rotation;
    ``thresholds``: float64 device tensor of 2^bits - 1 decision boundaries
    (e.g. from hadq_codebook(n, bits)).  Returns (codes uint8, norms fp32)."""
    lib = load_library()
    rows, n = _rows_n(x)
    _on_device("x", x, x.device)
    pp = sp = None
    if perm is not None or signs is not None:
        pp, sp = _rpbh_ptrs(perm, signs, x.device, n)
    if thresholds.dtype != torch.float64:
        raise HadqError(HADQ_ERR_INVALID_ARG, "thresholds must be float64")
    _on_device("thresholds", thresholds, x.device)
    _holds("thresholds", thresholds, ((1 << bits) - 1) * 8)
    if codes is None:
        codes = torch.empty((rows, n * bits // 8), dtype=torch.uint8, device=x.device)
    if norms is None:
        norms = torch.empty((rows,), dtype=torch.float32, device=x.device)
    for name, t, nb in (("codes", codes, rows * n * bits // 8), ("norms", norms, rows * 4)):
        _on_device(name, t, x.device)
        _holds(name, t, nb)
    _check(lib.hadq_rotate_quant_codebook(x.data_ptr(), _dtype_code(x.dtype), rows, n, block, pp, sp, int(bits),
                                          thresholds.data_ptr(), codes.data_ptr(), norms.data_ptr(),
                                          _stream_handle(stream)))
    return codes, norms


# ------------------------------------------------- int8 linear and int4 cache

def _invalid(message: str) -> HadqError:
    return HadqError(HADQ_ERR_INVALID_ARG, message)


def _takes(name: str, t: torch.Tensor, index: int, dtype: torch.dtype, shape, contiguous: bool = True) -> int:
    """Address of a tensor that must lie on CUDA device ``index`` (-1: none, refused) and have this dtype and shape."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0:
        if not contiguous or t.is_contiguous():
            return t.data_ptr()
    if not t.is_cuda:
        raise _invalid(f"{name} must be a CUDA tensor (got {t.device})")
    if t.get_device() != index:
        raise _invalid(f"{name} is on {t.device}, the first tensor is not")
    if t.dtype != dtype:
        raise _invalid(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != tuple(shape):
        raise _invalid(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    raise _invalid(f"{name} must be contiguous")


def _call(fn, index: int, stream, *args) -> None:
    """fn(*args, stream) with device ``index`` current: on the stream given, or
    on that device's current stream.  Outputs come from that device's
    allocator, so a stream given explicitly is the caller's to order with their
    use, as elsewhere."""
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream_handle(stream)
    if index == torch._C._cuda_getDevice():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status != HADQ_OK:
        _check(status)


def hadq_rmsnorm_quant(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: torch.Tensor | None = None,
                       residual_out: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                       scales: torch.Tensor | None = None, stream=None):
    """RMSNorm(x + residual) * weight as int8 codes with a scale per token (see
    include/hadq.h).  Returns (codes, scales, residual_out); the last is
    x + residual, or None without a residual.  residual_out may be x or residual."""
    lib = _lib or load_library()
    dev, dtype, shape = x.get_device(), x.dtype, x.shape
    xp = _takes("x", x, dev, dtype, shape)
    lead, n = shape[:-1], shape[-1] if shape else 1
    rows = x.numel() // n if n else 0
    wp = _takes("weight", weight, dev, dtype, (n,))
    rp = op = None
    if residual is not None:
        rp = _takes("residual", residual, dev, dtype, shape)
        if residual_out is None:
            residual_out = torch.empty_like(x)
            op = residual_out.data_ptr()
        else:
            op = _takes("residual_out", residual_out, dev, dtype, shape)
    elif residual_out is not None:
        raise _invalid("residual_out needs a residual")
    if codes is None:
        codes = torch.empty_like(x, dtype=torch.int8)
        cp = codes.data_ptr()
    else:
        cp = _takes("codes", codes, dev, torch.int8, shape)
    if scales is None:
        scales = x.new_empty(lead, dtype=torch.float32)
        sp = scales.data_ptr()
    else:
        sp = _takes("scales", scales, dev, torch.float32, lead)
    _call(lib.hadq_rmsnorm_quant, dev, stream, xp, _dtype_code(dtype), rows, n, rp, wp, eps, op, cp, sp)
    return codes, scales, residual_out


def hadq_matmul_int8(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                     bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """(a . w^T) * a_scales[:, None] * w_scales + bias of int8 codes a [..., k]
    and weights w [cols, k] (see include/hadq.h)."""
    lib = _lib or load_library()
    dev, shape = a.get_device(), a.shape
    ap = _takes("a", a, dev, torch.int8, shape)
    lead, k = shape[:-1], shape[-1] if shape else 1
    rows = a.numel() // k if k else 0
    asp = _takes("a_scales", a_scales, dev, torch.float32, lead)
    cols = w.shape[0] if w.dim() else 0
    wp = _takes("w", w, dev, torch.int8, (cols, k))
    wsp = _takes("w_scales", w_scales, dev, torch.float32, (cols,))
    bp = None if bias is None else _takes("bias", bias, dev, torch.float32, (cols,))
    if out is None:
        out = a.new_empty((*lead, cols), dtype=out_dtype)
        op = out.data_ptr()
    else:
        out_dtype = out.dtype
        op = _takes("out", out, dev, out_dtype, (*lead, cols))
    _call(lib.hadq_matmul_int8, dev, stream, ap, asp, rows, wp, wsp, cols, k, bp, op, _dtype_code(out_dtype))
    return out


def _kv4_cache(dev, k_codes, k_scales, v_codes, v_scales):
    """Addresses and (num_pages, kv_heads, page_size, head_dim, group) of a cache's four tensors."""
    if k_codes.dim() != 4 or k_scales.dim() != 4:
        raise _invalid("k_codes and k_scales must be [num_pages, kv_heads, page_size, ...]")
    pages, heads, size, half = k_codes.shape
    groups = k_scales.shape[3]
    if groups == 0 or (2 * half) % groups:
        raise _invalid(f"{groups} scales for {2 * half} elements")
    cs, ss = k_codes.shape, (pages, heads, size, groups)
    ptrs = (_takes("k_codes", k_codes, dev, torch.uint8, cs), _takes("k_scales", k_scales, dev, torch.float16, ss),
            _takes("v_codes", v_codes, dev, torch.uint8, cs), _takes("v_scales", v_scales, dev, torch.float16, ss))
    return ptrs, pages, heads, size, 2 * half, 2 * half // groups


def _token_rows(name: str, x: torch.Tensor, tail) -> int:
    """Elements between the tokens of x [..., heads, head_dim]: heads and their
    elements dense, tokens (all leading dimensions) evenly spaced."""
    width, stride = tail[0] * tail[1], x.stride()
    if stride[-1] != 1 or stride[-2] != tail[1]:
        raise _invalid(f"{name}: the last two dimensions must be dense")
    shape = x.shape
    if len(shape) == 3:
        return stride[0] if shape[0] > 1 else width
    spacing, step = None, 1
    for d in range(len(shape) - 3, -1, -1):
        if shape[d] > 1:
            if spacing is None:
                spacing = stride[d]
            elif stride[d] != spacing * step:
                raise _invalid(f"{name}: tokens must be evenly spaced")
        if spacing is not None:
            step *= shape[d]
    return width if spacing is None else spacing


def hadq_kv4_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_codes: torch.Tensor,
                    k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor, block: int = 0,
                    stream=None) -> None:
    """Rotate (block 0; 1: do not) and quantize the tokens' K, quantize their V,
    and store both at ``slots`` of the paged int4 cache (see include/hadq.h).
    k, v: [tokens, kv_heads, head_dim], tokens at any even spacing; slots: int64,
    negative for tokens that are not stored."""
    lib = _lib or load_library()
    dev, dtype = k.get_device(), k.dtype
    ptrs, pages, heads, size, d, group = _kv4_cache(dev, k_codes, k_scales, v_codes, v_scales)
    tokens = k.shape[0] if k.dim() else 0
    kp = _takes("k", k, dev, dtype, (tokens, heads, d), contiguous=False)
    vp = _takes("v", v, dev, dtype, (tokens, heads, d), contiguous=False)
    ks, vs = _token_rows("k", k, (heads, d)), _token_rows("v", v, (heads, d))
    sp = _takes("slots", slots, dev, torch.int64, (tokens,))
    _call(lib.hadq_kv4_append, dev, stream, kp, ks, vp, vs, _dtype_code(dtype), tokens, heads, d, block, group, sp, pages,
          size, *ptrs)


@functools.lru_cache(maxsize=1024)
def _kv4_workspace(*sizes: int) -> int:
    """Bytes for these sizes, -1 where the call refuses them."""
    return int(load_library().hadq_kv4_attention_workspace(*sizes))


def hadq_kv4_attention_workspace(batch: int, q_len: int, heads: int, kv_heads: int, head_dim: int,
                                 max_positions: int) -> int:
    """Bytes of hadq_kv4_attention's workspace (see include/hadq.h)."""
    n = int(load_library().hadq_kv4_attention_workspace(batch, q_len, heads, kv_heads, head_dim, max_positions))
    if n < 0:
        raise _invalid(load_library().hadq_last_error().decode())
    return n


def hadq_kv4_attention(q: torch.Tensor, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor,
                       v_scales: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
                       scale: float | None = None, block: int = 0, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of each sequence's newest tokens q [batch, q_len, heads, head_dim]
    (or [batch, heads, head_dim]) over the paged int4 cache (see include/hadq.h).
    scale: 1 / sqrt(head_dim) when None.  Without ``workspace`` one is allocated, of
    ``stream``."""
    lib = _lib or load_library()
    dev, dtype, shape = q.get_device(), q.dtype, q.shape
    ptrs, pages, kv_heads, size, d, group = _kv4_cache(dev, k_codes, k_scales, v_codes, v_scales)
    if len(shape) not in (3, 4):
        raise _invalid("q must be [batch, q_len, heads, head_dim] or [batch, heads, head_dim]")
    batch, heads = shape[0], shape[-2]
    q_len = shape[1] if len(shape) == 4 else 1
    qp = _takes("q", q, dev, dtype, (*shape[:-1], d), contiguous=False)
    qs = _token_rows("q", q, (heads, d))
    max_pages = page_table.shape[1] if page_table.dim() == 2 else 0
    tp = _takes("page_table", page_table, dev, torch.int32, (batch, max_pages))
    lp = _takes("lengths", lengths, dev, torch.int32, (batch,))
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        op = out.data_ptr()
    else:
        op = _takes("out", out, dev, dtype, shape)
    nbytes, ws = 0, None
    if workspace is None:
        need = _kv4_workspace(batch, q_len, heads, kv_heads, d, max_pages * size)
        if need > 0 and stream is None:
            workspace = q.new_empty(need, dtype=torch.uint8)
        elif need > 0:                         # of the stream that uses it: nobody else holds it until then
            with torch.cuda.stream(torch.cuda.ExternalStream(_stream_handle(stream), dev)):
                workspace = q.new_empty(need, dtype=torch.uint8)
    if workspace is not None:
        _takes("workspace", workspace, dev, workspace.dtype, workspace.shape)
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call(lib.hadq_kv4_attention, dev, stream, qp, qs, _dtype_code(dtype), batch, q_len, heads, kv_heads, d, block, group,
          *ptrs, pages, size, tp, max_pages, lp, d ** -0.5 if scale is None else scale, op, ws, nbytes)
    return out
