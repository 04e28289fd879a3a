"""Python binding of libdf11 (DFloat11-style lossless BF16 compression on MI355X).

Argument marshalling only: every step of compression runs in the library's
C++ host code and every step of decompression in its HIP kernels.  PyTorch is
used for device memory and streams (``tensor.data_ptr()``,
``torch.cuda.current_stream().cuda_stream``).  The functions keep the C names:
``df11_build_codebook``, ``df11_encode_size``, ``df11_encode``,
``df11_decompress_block``, ``df11_decompress_tensor``.

The library must be built (``entropy_decoding_amd.build.build_library()``);
importing this module without it raises ImportError.  There is no fallback.
"""

from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdf11.so")

DF11_MAX_CODE_LEN = 32
DF11_MAX_LUTS = 64
DF11_STREAM_PAD = 16
DF11_MULTI_BITS = 10
DF11_COUNT_BITS = 12

DF11_OK = 0
DF11_E_INVALID = 1
DF11_E_LUT_BUDGET = 2
DF11_E_SYMBOL = 3
DF11_E_CAPACITY = 4
DF11_E_HIP = 5
DF11_E_CORRUPT = 6

DEFAULT_TILE_WINDOWS = 64
DEFAULT_WINDOW_BYTES = 8


class Df11Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} ({status})")
        self.status = status


_u8p = ctypes.POINTER(ctypes.c_uint8)
_u16p = ctypes.POINTER(ctypes.c_uint16)
_u32p = ctypes.POINTER(ctypes.c_uint32)
_u64p = ctypes.POINTER(ctypes.c_uint64)


class df11_codebook(ctypes.Structure):
    _fields_ = [
        ("code_len", ctypes.c_uint8 * 256),
        ("code", ctypes.c_uint32 * 256),
        ("n_luts", ctypes.c_uint32),
        ("max_len", ctypes.c_uint32),
        ("multi", ctypes.c_uint32 * (1 << DF11_MULTI_BITS)),
        ("count", ctypes.c_uint16 * (1 << DF11_COUNT_BITS)),
        ("lut", (ctypes.c_uint16 * 256) * DF11_MAX_LUTS),
    ]


class df11_sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in (
        "n_weights", "total_bits", "n_tiles", "n_windows", "stream_bytes", "sm_bytes",
        "bop_entries")]


class df11_host_stream(ctypes.Structure):
    _fields_ = [
        ("stream", _u8p),
        ("sm", _u8p),
        ("gaps", _u8p),
        ("block_out_pos", _u32p),
        ("tensor_offsets", _u64p),
        ("tensor_tiles", _u64p),
        ("stream_capacity", ctypes.c_uint64),
        ("sm_capacity", ctypes.c_uint64),
        ("gaps_capacity", ctypes.c_uint64),
        ("bop_capacity", ctypes.c_uint64),
        ("n_tensors", ctypes.c_uint32),
        ("tile_windows", ctypes.c_uint32),
        ("window_bytes", ctypes.c_uint32),
        ("max_tile_symbols", ctypes.c_uint32),
        ("n_weights", ctypes.c_uint64),
        ("total_bits", ctypes.c_uint64),
        ("n_tiles", ctypes.c_uint64),
        ("format", ctypes.c_uint32),
    ]


class df11_device_stream(ctypes.Structure):
    _fields_ = [
        ("stream", ctypes.c_void_p),
        ("sm", ctypes.c_void_p),
        ("gaps", ctypes.c_void_p),
        ("block_out_pos", ctypes.c_void_p),
        ("tables", ctypes.c_void_p),
        ("tensor_offsets", _u64p),
        ("tensor_tiles", _u64p),
        ("n_weights", ctypes.c_uint64),
        ("total_bits", ctypes.c_uint64),
        ("n_tiles", ctypes.c_uint64),
        ("n_luts", ctypes.c_uint32),
        ("tile_windows", ctypes.c_uint32),
        ("window_bytes", ctypes.c_uint32),
        ("max_tile_symbols", ctypes.c_uint32),
        ("n_tensors", ctypes.c_uint32),
        ("format", ctypes.c_uint32),
    ]


class df11_gemv_tensor(ctypes.Structure):
    _fields_ = [
        ("w_offset", ctypes.c_uint64),
        ("x_offset", ctypes.c_uint64),
        ("y_offset", ctypes.c_uint64),
        ("rows", ctypes.c_uint32),
        ("cols", ctypes.c_uint32),
    ]


class df11_device_encode(ctypes.Structure):
    _fields_ = [
        ("stream", ctypes.c_void_p),
        ("sm", ctypes.c_void_p),
        ("gaps", ctypes.c_void_p),
        ("block_out_pos", ctypes.c_void_p),
        ("d_max_tile_symbols", ctypes.c_void_p),
        ("scratch", ctypes.c_void_p),
        ("scratch_bytes", ctypes.c_uint64),
    ]


class df11_adamw_tensor(ctypes.Structure):
    _fields_ = [
        ("w", ctypes.c_void_p),
        ("master", ctypes.c_void_p),
        ("g", ctypes.c_void_p),
        ("m", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("m_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("counts", ctypes.c_void_p),
        ("numel", ctypes.c_uint64),
        ("lr_scale", ctypes.c_double),
        ("weight_decay", ctypes.c_double),
    ]


class df11_adamw_config(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_double),
        ("beta1", ctypes.c_double),
        ("beta2", ctypes.c_double),
        ("eps", ctypes.c_double),
        ("step", ctypes.c_uint64),
        ("w_type", ctypes.c_uint32),
        ("g_type", ctypes.c_uint32),
        ("state_bits", ctypes.c_uint32),
        ("reserved", ctypes.c_uint32),
        ("d_lr", ctypes.c_void_p),
        ("d_step", ctypes.c_void_p),
        ("d_grad_factor", ctypes.c_void_p),
    ]


class df11_int8_rows(ctypes.Structure):
    _fields_ = [
        ("src", ctypes.c_void_p),
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("src_stride", ctypes.c_uint64),
        ("code_stride", ctypes.c_uint64),
        ("rows", ctypes.c_uint32),
        ("cols", ctypes.c_uint32),
    ]


class df11_int8_tensor(ctypes.Structure):
    _fields_ = [
        ("w", ctypes.c_void_p),
        ("w_scale", ctypes.c_void_p),
        ("x", ctypes.c_void_p),
        ("x_scale", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("w_stride", ctypes.c_uint64),
        ("x_stride", ctypes.c_uint64),
        ("y_stride", ctypes.c_uint64),
        ("rows", ctypes.c_uint32),
        ("cols", ctypes.c_uint32),
    ]


class df11_embedding_lookup(ctypes.Structure):
    _fields_ = [
        ("table", ctypes.c_void_p),
        ("tokens", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("table_stride", ctypes.c_uint64),
        ("out_stride", ctypes.c_uint64),
        ("rows", ctypes.c_uint64),
        ("n", ctypes.c_uint64),
        ("cols", ctypes.c_uint32),
        ("table_type", ctypes.c_uint32),
        ("out_type", ctypes.c_uint32),
        ("token_bits", ctypes.c_uint32),
        ("scale", ctypes.c_float),
    ]


class df11_embedding_grad(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_void_p),
        ("dy", ctypes.c_void_p),
        ("dw", ctypes.c_void_p),
        ("dy_stride", ctypes.c_uint64),
        ("dw_stride", ctypes.c_uint64),
        ("rows", ctypes.c_uint64),
        ("n", ctypes.c_uint64),
        ("padding", ctypes.c_int64),
        ("cols", ctypes.c_uint32),
        ("dy_type", ctypes.c_uint32),
        ("dw_type", ctypes.c_uint32),
        ("token_bits", ctypes.c_uint32),
        ("accumulate", ctypes.c_uint32),
        ("scale", ctypes.c_float),
    ]


class df11_vocab_piece(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("targets", ctypes.c_void_p),
        ("w", ctypes.c_void_p),
        ("x_stride", ctypes.c_uint64),
        ("w_stride", ctypes.c_uint64),
        ("ignored", ctypes.c_int64),
        ("n", ctypes.c_uint32),
        ("cols", ctypes.c_uint32),
        ("vocab", ctypes.c_uint32),
        ("first", ctypes.c_uint32),
        ("rows", ctypes.c_uint32),
        ("target_bits", ctypes.c_uint32),
        ("begin", ctypes.c_uint32),
        ("end", ctypes.c_uint32),
    ]


class df11_vocab_sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in ("n", "cols", "rows", "dx", "two_terms")]


class df11_vocab_grad(ctypes.Structure):
    _fields_ = [
        ("lse", ctypes.c_void_p),
        ("losses", ctypes.c_void_p),
        ("loss_grad", ctypes.c_void_p),
        ("lse_grad", ctypes.c_void_p),
        ("dx", ctypes.c_void_p),
        ("dw", ctypes.c_void_p),
        ("dx_stride", ctypes.c_uint64),
        ("dw_stride", ctypes.c_uint64),
        ("loss_grads", ctypes.c_uint32),
        ("lse_grads", ctypes.c_uint32),
        ("dx_type", ctypes.c_uint32),
        ("dw_type", ctypes.c_uint32),
        ("accumulate", ctypes.c_uint32),
        ("loss_grad_all", ctypes.c_float),
    ]


DF11_INT8_MAX_TENSORS = 16
DF11_INT8_MAX_COLS = 131071
DF11_INT8_MAX_STRIDE = 1 << 22
DF11_PIPELINE_MAX_SLOTS = 4
DF11_ADAMW_BLOCK = 256
DF11_EMBEDDING_MAX_TOKENS = 1 << 24
DF11_EMBEDDING_MAX_ROWS = 1 << 24
DF11_EMBEDDING_MAX_COLS = 1 << 20
DF11_VOCAB_MAX_TOKENS = 1 << 20
DF11_VOCAB_MAX_ROWS = 1 << 24
DF11_VOCAB_MAX_COLS = 1 << 20
DF11_VOCAB_MAX_STRIDE = 1 << 21
# df11_type, by the names of torch's types
TYPES = {"float32": 0, "bfloat16": 1, "float16": 2}
# df11_format; the names are what the binding's ``fmt`` arguments accept
FORMATS = {"bf16": 0, "fp8_e4m3": 1, "fp8_e5m2": 2}
DF11_GEMV_MAX_TENSORS = 16


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run python entropy_decoding_amd/build.py")
    # PyTorch ships its own libamdhip64 (soname libamdhip64.so.7).  Loading torch
    # first lets the dynamic loader satisfy libdf11's dependency with that same
    # runtime; loading libdf11 first would bring in a second HIP runtime, whose
    # streams and launches are invisible to torch's.
    import torch  # noqa: F401

    L = ctypes.CDLL(LIB_PATH)
    tens = ctypes.POINTER(ctypes.c_void_p)
    L.df11_build_codebook.argtypes = [tens, _u64p, ctypes.c_uint32, ctypes.POINTER(df11_codebook)]
    L.df11_build_codebook_fmt.argtypes = [ctypes.c_uint32, tens, _u64p, ctypes.c_uint32,
                                          ctypes.POINTER(df11_codebook)]
    L.df11_encode_size_fmt.argtypes = [ctypes.c_uint32, ctypes.POINTER(df11_codebook), tens, _u64p,
                                       ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32,
                                       ctypes.POINTER(df11_sizes)]
    L.df11_encode_fmt.argtypes = [ctypes.c_uint32, ctypes.POINTER(df11_codebook), tens, _u64p,
                                  ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32,
                                  ctypes.POINTER(df11_host_stream)]
    L.df11_encode_size.argtypes = [ctypes.POINTER(df11_codebook), tens, _u64p, ctypes.c_uint32,
                                   ctypes.c_uint32, ctypes.c_uint32, ctypes.POINTER(df11_sizes)]
    L.df11_encode.argtypes = [ctypes.POINTER(df11_codebook), tens, _u64p, ctypes.c_uint32,
                              ctypes.c_uint32, ctypes.c_uint32, ctypes.POINTER(df11_host_stream)]
    L.df11_decompress_block.argtypes = [ctypes.POINTER(df11_device_stream), ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p]
    L.df11_decompress_tensor.argtypes = [ctypes.POINTER(df11_device_stream), ctypes.c_uint32,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    L.df11_window_counts.argtypes = [ctypes.POINTER(df11_device_stream), ctypes.c_void_p,
                                     ctypes.c_void_p]
    L.df11_status_string.argtypes = [ctypes.c_int]
    L.df11_status_string.restype = ctypes.c_char_p
    vp = ctypes.c_void_p
    L.df11_pipeline_create.argtypes = [vp, ctypes.c_uint32, ctypes.POINTER(vp)]
    L.df11_pipeline_destroy.argtypes = [vp]
    L.df11_pipeline_decompress.argtypes = [vp, ctypes.c_uint32, ctypes.POINTER(df11_device_stream),
                                           vp, vp]
    L.df11_pipeline_acquire.argtypes = [vp, ctypes.c_uint32, vp]
    L.df11_pipeline_release.argtypes = [vp, ctypes.c_uint32, vp]
    L.df11_pipeline_set_decode_share.argtypes = [vp, ctypes.c_uint32]
    L.df11_gemv_bf16.argtypes = [vp, ctypes.POINTER(df11_gemv_tensor), ctypes.c_uint32, vp, vp, vp]
    L.df11_build_codebook_from_counts.argtypes = [_u64p, ctypes.POINTER(df11_codebook)]
    L.df11_decompress_gemv_scratch_bytes.argtypes = [ctypes.POINTER(df11_device_stream)]
    L.df11_decompress_gemv_scratch_bytes.restype = ctypes.c_uint64
    L.df11_decompress_gemv.argtypes = [ctypes.POINTER(df11_device_stream),
                                       ctypes.POINTER(df11_gemv_tensor), ctypes.c_uint32, vp, vp,
                                       vp, ctypes.c_uint64, vp, vp]
    L.df11_decompress_gemv_noalloc.argtypes = [ctypes.POINTER(df11_device_stream),
                                               ctypes.POINTER(df11_gemv_tensor), ctypes.c_uint32,
                                               vp, vp, vp, vp]
    L.df11_gemm_order.argtypes = [_u16p, ctypes.c_uint32, ctypes.c_uint32, _u16p]
    L.df11_decompress_gemm_scratch_bytes.argtypes = [ctypes.POINTER(df11_gemv_tensor),
                                                     ctypes.c_uint32, ctypes.c_uint32]
    L.df11_decompress_gemm_scratch_bytes.restype = ctypes.c_uint64
    L.df11_decompress_gemm.argtypes = [ctypes.POINTER(df11_device_stream),
                                       ctypes.POINTER(df11_gemv_tensor), ctypes.c_uint32,
                                       ctypes.c_uint32, vp, vp, vp, ctypes.c_uint64, vp, vp]
    L.df11_encode_size_from_counts.argtypes = [ctypes.c_uint32, ctypes.POINTER(df11_codebook),
                                               _u64p, ctypes.c_uint64, ctypes.c_uint32,
                                               ctypes.c_uint32, ctypes.POINTER(df11_sizes)]
    L.df11_histogram_device.argtypes = [ctypes.c_uint32, vp, ctypes.c_uint64, vp, vp]
    L.df11_tensor_ranges_from_counts.argtypes = [ctypes.c_uint32, ctypes.POINTER(df11_codebook),
                                                 _u64p, _u32p, ctypes.c_uint32, ctypes.c_uint32,
                                                 ctypes.c_uint32, _u64p, _u64p]
    L.df11_encode_device_scratch_bytes.argtypes = [ctypes.c_uint64]
    L.df11_encode_device_scratch_bytes.restype = ctypes.c_uint64
    L.df11_encode_device.argtypes = [ctypes.c_uint32, ctypes.POINTER(df11_codebook), vp,
                                     ctypes.c_uint64, ctypes.c_uint32, ctypes.c_uint32,
                                     ctypes.POINTER(df11_sizes), ctypes.POINTER(df11_device_encode),
                                     vp]
    at = ctypes.POINTER(df11_adamw_tensor)
    L.df11_adamw_step.argtypes = [ctypes.POINTER(df11_adamw_config), at, ctypes.c_uint32, vp]
    L.df11_adamw_step_counted.argtypes = [ctypes.POINTER(df11_adamw_config), at, ctypes.c_uint32, vp, vp]
    L.df11_adamw_values.argtypes = [at, ctypes.c_uint32, ctypes.c_uint32, ctypes.POINTER(vp),
                                    ctypes.POINTER(vp), vp]
    L.df11_grad_norm_scratch_bytes.argtypes = [at, ctypes.c_uint32]
    L.df11_grad_norm_scratch_bytes.restype = ctypes.c_uint64
    L.df11_grad_norm.argtypes = [ctypes.c_uint32, at, ctypes.c_uint32, ctypes.c_double, vp, vp,
                                 ctypes.c_uint64, vp]
    L.df11_quantize_int8.argtypes = [ctypes.c_uint32, ctypes.POINTER(df11_int8_rows),
                                     ctypes.c_uint32, vp]
    L.df11_gemm_int8.argtypes = [ctypes.c_uint32, ctypes.POINTER(df11_int8_tensor),
                                 ctypes.c_uint32, ctypes.c_uint32, vp]
    L.df11_linear_int8_scratch_bytes.argtypes = [ctypes.POINTER(df11_int8_tensor), ctypes.c_uint32,
                                                 ctypes.c_uint32]
    L.df11_linear_int8_scratch_bytes.restype = ctypes.c_uint64
    L.df11_linear_int8.argtypes = [ctypes.c_uint32, ctypes.c_uint32,
                                   ctypes.POINTER(df11_int8_tensor), ctypes.c_uint32,
                                   ctypes.c_uint32, vp, ctypes.c_uint64, vp]
    L.df11_embedding.argtypes = [ctypes.POINTER(df11_embedding_lookup), vp]
    L.df11_embedding_gradient_scratch_bytes.argtypes = [ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint32]
    L.df11_embedding_gradient_scratch_bytes.restype = ctypes.c_uint64
    L.df11_embedding_gradient.argtypes = [ctypes.POINTER(df11_embedding_grad), vp, ctypes.c_uint64, vp]
    vs = ctypes.POINTER(df11_vocab_sizes)
    for f in (L.df11_vocab_loss_scratch_bytes, L.df11_vocab_loss_gradient_scratch_bytes):
        f.argtypes, f.restype = [vs], ctypes.c_uint64
    L.df11_vocab_loss.argtypes = [ctypes.POINTER(df11_vocab_piece), vp, vp, vs, vp, ctypes.c_uint64, vp]
    L.df11_vocab_loss_gradient.argtypes = [ctypes.POINTER(df11_vocab_piece),
                                           ctypes.POINTER(df11_vocab_grad), vs, vp, ctypes.c_uint64, vp]
    for f in (L.df11_build_codebook, L.df11_encode_size, L.df11_encode,
              L.df11_quantize_int8, L.df11_gemm_int8, L.df11_linear_int8, L.df11_adamw_step,
              L.df11_adamw_step_counted, L.df11_adamw_values, L.df11_grad_norm,
              L.df11_embedding, L.df11_embedding_gradient, L.df11_vocab_loss,
              L.df11_vocab_loss_gradient,
              L.df11_build_codebook_fmt, L.df11_encode_size_fmt, L.df11_encode_fmt,
              L.df11_decompress_block, L.df11_decompress_tensor, L.df11_pipeline_create,
              L.df11_pipeline_destroy, L.df11_pipeline_decompress, L.df11_pipeline_acquire,
              L.df11_pipeline_release, L.df11_pipeline_set_decode_share, L.df11_gemv_bf16,
              L.df11_build_codebook_from_counts,
              L.df11_encode_size_from_counts, L.df11_histogram_device, L.df11_encode_device,
              L.df11_decompress_gemv, L.df11_gemm_order, L.df11_decompress_gemm,
              L.df11_window_counts, L.df11_tensor_ranges_from_counts,
              L.df11_decompress_gemv_noalloc):
        f.restype = ctypes.c_int
    return L


LIB = _load()


def status_string(status: int) -> str:
    return LIB.df11_status_string(int(status)).decode()


def _check(fn: str, rc: int):
    if rc != DF11_OK:
        raise Df11Error(fn, rc)


def _format(fmt: str) -> int:
    if fmt not in FORMATS:
        raise ValueError(f"fmt must be one of {sorted(FORMATS)}")
    return FORMATS[fmt]


def _tensor_args(tensors, fmt: str = "bf16"):
    if isinstance(tensors, np.ndarray):
        tensors = [tensors]
    want = np.uint16 if fmt == "bf16" else np.uint8
    arrs = []
    for t in tensors:
        a = np.asarray(t)
        if a.dtype != want:
            raise TypeError(f"{fmt} tensors must be {np.dtype(want).name} bit patterns")
        arrs.append(np.ascontiguousarray(a).reshape(-1))
    n = len(arrs)
    ptrs = (ctypes.c_void_p * max(n, 1))(*[a.ctypes.data for a in arrs])
    numel = (ctypes.c_uint64 * max(n, 1))(*[a.size for a in arrs])
    return arrs, ptrs, numel, n


# ---------------------------------------------------------------- host calls


def df11_build_codebook(tensors, fmt: str = "bf16") -> df11_codebook:
    """Histogram + Huffman (+ package-merge at 32 bits) + canonical codes + LUTs.
    BF16 tensors are uint16 arrays (df11_build_codebook); FP8 ones uint8
    arrays (df11_build_codebook_fmt)."""
    arrs, ptrs, numel, n = _tensor_args(tensors, fmt)
    cb = df11_codebook()
    if fmt == "bf16":
        _check("df11_build_codebook", LIB.df11_build_codebook(ptrs, numel, n, ctypes.byref(cb)))
    else:
        _check("df11_build_codebook_fmt",
               LIB.df11_build_codebook_fmt(_format(fmt), ptrs, numel, n, ctypes.byref(cb)))
    return cb


def df11_encode_size(cb: df11_codebook, tensors, tile_windows: int = DEFAULT_TILE_WINDOWS,
                     window_bytes: int = DEFAULT_WINDOW_BYTES, fmt: str = "bf16") -> df11_sizes:
    arrs, ptrs, numel, n = _tensor_args(tensors, fmt)
    sz = df11_sizes()
    if fmt == "bf16":
        _check("df11_encode_size", LIB.df11_encode_size(ctypes.byref(cb), ptrs, numel, n,
                                                        tile_windows, window_bytes,
                                                        ctypes.byref(sz)))
    else:
        _check("df11_encode_size_fmt",
               LIB.df11_encode_size_fmt(_format(fmt), ctypes.byref(cb), ptrs, numel, n,
                                        tile_windows, window_bytes, ctypes.byref(sz)))
    return sz


@dataclass
class HostStream:
    """A compressed unit in host memory (numpy arrays owned by this object)."""

    stream: np.ndarray
    sm: np.ndarray
    gaps: np.ndarray
    block_out_pos: np.ndarray
    tensor_offsets: np.ndarray
    tensor_tiles: np.ndarray
    tile_windows: int
    window_bytes: int
    max_tile_symbols: int
    n_weights: int
    total_bits: int
    n_tiles: int
    format: int = 0

    @property
    def n_tensors(self) -> int:
        return self.tensor_offsets.size - 1

    def compressed_bytes(self, cb: df11_codebook | None = None) -> dict:
        """Bytes of every array a decompression reads (payload and auxiliary)."""
        d = {
            "stream": (self.total_bits + 7) // 8,
            "sm": self.n_weights if self.format == 0 else (self.n_weights + 1) // 2,
            "gaps": self.gaps.size,
            "block_out_pos": 4 * self.block_out_pos.size,
        }
        if cb is not None:
            d["tables"] = table_bytes(cb)
        return d


def df11_encode(cb: df11_codebook, tensors, tile_windows: int = DEFAULT_TILE_WINDOWS,
                window_bytes: int = DEFAULT_WINDOW_BYTES, fmt: str = "bf16") -> HostStream:
    arrs, ptrs, numel, n = _tensor_args(tensors, fmt)
    sz = df11_encode_size(cb, arrs, tile_windows, window_bytes, fmt)
    stream = np.empty(sz.stream_bytes, dtype=np.uint8)
    sm = np.empty(sz.sm_bytes, dtype=np.uint8)
    gaps = np.empty(max(1, sz.n_windows), dtype=np.uint8)
    bop = np.empty(sz.bop_entries, dtype=np.uint32)
    offs = np.empty(n + 1, dtype=np.uint64)
    tiles = np.empty(max(1, 2 * n), dtype=np.uint64)
    hs = df11_host_stream()
    hs.stream = stream.ctypes.data_as(_u8p)
    hs.sm = sm.ctypes.data_as(_u8p)
    hs.gaps = gaps.ctypes.data_as(_u8p)
    hs.block_out_pos = bop.ctypes.data_as(_u32p)
    hs.tensor_offsets = offs.ctypes.data_as(_u64p)
    hs.tensor_tiles = tiles.ctypes.data_as(_u64p)
    hs.stream_capacity = stream.size
    hs.sm_capacity = sm.size
    hs.gaps_capacity = sz.n_windows
    hs.bop_capacity = bop.size
    hs.n_tensors = n
    if fmt == "bf16":
        _check("df11_encode", LIB.df11_encode(ctypes.byref(cb), ptrs, numel, n, tile_windows,
                                              window_bytes, ctypes.byref(hs)))
    else:
        _check("df11_encode_fmt", LIB.df11_encode_fmt(_format(fmt), ctypes.byref(cb), ptrs, numel,
                                                      n, tile_windows, window_bytes,
                                                      ctypes.byref(hs)))
    return HostStream(stream, sm, gaps[: sz.n_windows], bop, offs, tiles[: 2 * n],
                      hs.tile_windows, hs.window_bytes, hs.max_tile_symbols, hs.n_weights,
                      hs.total_bits, hs.n_tiles, hs.format)


# ---------------------------------------------------------------- device side


class DeviceStream:
    """A compressed unit resident in device memory (torch uint8/int32 tensors).

    Holds the ctypes descriptor passed to df11_decompress_*; the host-side
    tensor metadata (offsets, tile ranges) stays in numpy arrays it owns.
    Built from a HostStream (uploaded) or, by encode_on_device, from arrays
    written on the device.
    """

    def __init__(self, hs: HostStream, cb: df11_codebook, device="cuda", arrays=None):
        import torch

        def up(a):
            t = torch.from_numpy(np.ascontiguousarray(a).view(np.uint8).reshape(-1))
            return t.to(device)

        self.host = hs
        if arrays is None:
            self.stream = up(hs.stream)
            self.sm = up(hs.sm)
            self.gaps = up(hs.gaps if hs.gaps.size else np.zeros(1, np.uint8))
            self.block_out_pos = up(hs.block_out_pos)
        else:
            self.stream, self.sm, self.gaps, self.block_out_pos = arrays
        self.tables = up(table_image(cb))
        self.tensor_offsets = np.ascontiguousarray(hs.tensor_offsets, dtype=np.uint64)
        self.tensor_tiles = np.ascontiguousarray(
            hs.tensor_tiles if hs.tensor_tiles.size else np.zeros(2, np.uint64), dtype=np.uint64)
        d = df11_device_stream()
        d.stream = self.stream.data_ptr()
        d.sm = self.sm.data_ptr()
        d.gaps = self.gaps.data_ptr()
        d.block_out_pos = self.block_out_pos.data_ptr()
        d.tables = self.tables.data_ptr()
        d.tensor_offsets = self.tensor_offsets.ctypes.data_as(_u64p)
        d.tensor_tiles = self.tensor_tiles.ctypes.data_as(_u64p)
        d.n_weights = hs.n_weights
        d.total_bits = hs.total_bits
        d.n_tiles = hs.n_tiles
        d.n_luts = cb.n_luts
        d.tile_windows = hs.tile_windows
        d.window_bytes = hs.window_bytes
        d.max_tile_symbols = hs.max_tile_symbols
        d.n_tensors = hs.n_tensors
        d.format = hs.format
        self.desc = d

    @property
    def n_weights(self) -> int:
        return int(self.desc.n_weights)

    def device_bytes(self) -> int:
        return sum(t.numel() for t in (self.stream, self.sm, self.gaps, self.block_out_pos,
                                       self.tables))


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check_out(ds: DeviceStream, out, n: int) -> None:
    size = 2 if ds.desc.format == 0 else 1
    if out.numel() < n or out.element_size() != size or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous device tensor of {n} {8 * size}-bit elements")


def df11_decompress_block(ds: DeviceStream, out, status=None, stream=None) -> None:
    """One launch decompressing the whole unit into ``out`` (a device tensor of
    n_weights elements: 16-bit (torch.bfloat16, torch.int16) for BF16 units,
    8-bit (torch.uint8, torch.float8_*) for FP8 units)."""
    _check_out(ds, out, ds.n_weights)
    sp = ctypes.c_void_p(status.data_ptr()) if status is not None else ctypes.c_void_p(0)
    _check("df11_decompress_block",
           LIB.df11_decompress_block(ctypes.byref(ds.desc), ctypes.c_void_p(out.data_ptr()), sp,
                                     _stream_handle(stream)))


def df11_decompress_tensor(ds: DeviceStream, k: int, out, status=None, stream=None) -> None:
    """Decompress tensor k of the unit into ``out`` (its numel 16-bit elements)."""
    n = 0
    if 0 <= k < ds.tensor_offsets.size - 1:
        n = int(ds.tensor_offsets[k + 1] - ds.tensor_offsets[k])
    _check_out(ds, out, n)
    sp = ctypes.c_void_p(status.data_ptr()) if status is not None else ctypes.c_void_p(0)
    _check("df11_decompress_tensor",
           LIB.df11_decompress_tensor(ctypes.byref(ds.desc), int(k),
                                      ctypes.c_void_p(out.data_ptr()), sp,
                                      _stream_handle(stream)))


def df11_window_counts(ds: DeviceStream, counts, stream=None) -> None:
    """Phase 1 of the decode on its own: ``counts`` (a device int32 tensor of
    n_tiles * tile_windows elements) receives each stream window's number of
    code starts."""
    n = int(ds.desc.n_tiles) * int(ds.desc.tile_windows)
    if counts.numel() != n or counts.element_size() != 4 or not counts.is_contiguous():
        raise Df11Error(f"df11_window_counts: counts must be {n} contiguous 4-byte elements")
    _check("df11_window_counts",
           LIB.df11_window_counts(ctypes.byref(ds.desc), ctypes.c_void_p(counts.data_ptr()),
                                  _stream_handle(stream)))


# ---------------------------------------------------------------- block pipeline


class Pipeline:
    """df11_pipeline_*: a ring of n_slots output buffers decompressed on
    ``decode_stream`` and read by consumer streams, ordered by events."""

    def __init__(self, decode_stream, n_slots: int = 2):
        self._p = ctypes.c_void_p(0)
        self.decode_stream = decode_stream
        _check("df11_pipeline_create",
               LIB.df11_pipeline_create(_stream_handle(decode_stream), int(n_slots),
                                        ctypes.byref(self._p)))

    def decompress(self, slot: int, ds: DeviceStream, out, status=None) -> None:
        _check_out(ds, out, ds.n_weights)
        sp = ctypes.c_void_p(status.data_ptr()) if status is not None else ctypes.c_void_p(0)
        _check("df11_pipeline_decompress",
               LIB.df11_pipeline_decompress(self._p, int(slot), ctypes.byref(ds.desc),
                                            ctypes.c_void_p(out.data_ptr()), sp))

    def set_decode_share(self, workgroups_per_cu: int) -> None:
        """Cap the decode at this many workgroups per compute unit (0: full grid)."""
        _check("df11_pipeline_set_decode_share",
               LIB.df11_pipeline_set_decode_share(self._p, int(workgroups_per_cu)))

    def acquire(self, slot: int, consumer_stream) -> None:
        _check("df11_pipeline_acquire",
               LIB.df11_pipeline_acquire(self._p, int(slot), _stream_handle(consumer_stream)))

    def release(self, slot: int, consumer_stream) -> None:
        _check("df11_pipeline_release",
               LIB.df11_pipeline_release(self._p, int(slot), _stream_handle(consumer_stream)))

    def close(self) -> None:
        if self._p:
            _check("df11_pipeline_destroy", LIB.df11_pipeline_destroy(self._p))
            self._p = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gemv_layout(shapes):
    """df11_gemv_tensor descriptors for row-major matrices stored back to back
    (one decompressed unit), with x and y slices also back to back."""
    descs, w, x, y = [], 0, 0, 0
    for rows, cols in shapes:
        descs.append((w, x, y, rows, cols))
        w += rows * cols
        x += cols
        y += rows
    arr = (df11_gemv_tensor * max(len(descs), 1))()
    for i, (wo, xo, yo, r, c) in enumerate(descs):
        arr[i].w_offset, arr[i].x_offset, arr[i].y_offset, arr[i].rows, arr[i].cols = wo, xo, yo, r, c
    return arr, len(descs), x, y


def df11_gemv_bf16(w, layout, x, y, stream=None) -> None:
    """y = W x per tensor of ``layout`` (from gemv_layout) over the 16-bit
    device tensor ``w``; x and y are float32 device tensors."""
    arr, n, nx, ny = layout
    if w.element_size() != 2 or x.dtype.itemsize != 4 or y.dtype.itemsize != 4:
        raise ValueError("w must be 16-bit, x and y float32")
    if x.numel() < nx or y.numel() < ny:
        raise ValueError("x or y too small for the layout")
    _check("df11_gemv_bf16",
           LIB.df11_gemv_bf16(ctypes.c_void_p(w.data_ptr()), arr, n, ctypes.c_void_p(x.data_ptr()),
                              ctypes.c_void_p(y.data_ptr()), _stream_handle(stream)))


def df11_gemm_order(w, rows: int, cols: int) -> np.ndarray:
    """The host permutation df11_decompress_gemm expects (see include/df11.h):
    16-row blocks of 32-column sub-blocks, each in the matrix cores' lane
    order (four 8-column quarters of 16 rows of 8 weights)."""
    src = np.ascontiguousarray(np.asarray(w).reshape(-1)).view(np.uint16)
    if src.size != rows * cols:
        raise ValueError("w must hold rows * cols weights")
    out = np.empty(rows * cols, dtype=np.uint16)
    _check("df11_gemm_order", LIB.df11_gemm_order(src.ctypes.data_as(_u16p), rows, cols,
                                                  out.ctypes.data_as(_u16p)))
    return out


def gemm_layout(shapes, n_tokens: int):
    """df11_gemv_tensor descriptors for df11_decompress_gemm: matrices back to
    back in the unit, and for each a token-major x slice (n_tokens x cols,
    BF16) and y slice (n_tokens x rows, float32), also back to back."""
    descs, w, x, y = [], 0, 0, 0
    for rows, cols in shapes:
        descs.append((w, x, y, rows, cols))
        w += rows * cols
        x += n_tokens * cols
        y += n_tokens * rows
    arr = (df11_gemv_tensor * max(len(descs), 1))()
    for i, (wo, xo, yo, r, c) in enumerate(descs):
        arr[i].w_offset, arr[i].x_offset, arr[i].y_offset, arr[i].rows, arr[i].cols = wo, xo, yo, r, c
    return arr, len(descs), x, y


def df11_decompress_gemm_scratch_bytes(layout, n_tokens: int) -> int:
    arr, n, _, _ = layout
    return int(LIB.df11_decompress_gemm_scratch_bytes(arr, n, n_tokens))


def df11_decompress_gemm(ds: DeviceStream, layout, n_tokens: int, x, y, scratch=None,
                         status=None, stream=None) -> None:
    """y = W x for n_tokens tokens per matrix of ``layout`` (from gemm_layout)
    on the matrix cores, straight from the compressed unit ``ds`` (encoded
    from df11_gemm_order weights).  x: 16-bit device tensor (BF16 bits), y:
    float32 device tensor; ``scratch``: a device uint8 tensor of
    df11_decompress_gemm_scratch_bytes bytes, allocated here when not given."""
    import torch

    arr, n, nx, ny = layout
    if x.element_size() != 2 or y.dtype.itemsize != 4 or x.numel() < nx or y.numel() < ny:
        raise ValueError("x must be a 16-bit and y a float32 device tensor covering the layout")
    need = df11_decompress_gemm_scratch_bytes(layout, n_tokens)
    if scratch is None:
        scratch = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    sp = ctypes.c_void_p(status.data_ptr()) if status is not None else ctypes.c_void_p(0)
    _check("df11_decompress_gemm",
           LIB.df11_decompress_gemm(ctypes.byref(ds.desc), arr, n, n_tokens,
                                    ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(y.data_ptr()),
                                    ctypes.c_void_p(scratch.data_ptr()), scratch.numel(), sp,
                                    _stream_handle(stream)))


# ---------------------------------------------------------------- device encoder


def df11_histogram_device(w, fmt: str = "bf16", stream=None, counts=None):
    """Exponent histogram of the device tensor ``w`` (uint64[256] on its device;
    written into ``counts``, a 256-element 8-byte device tensor, when given)."""
    import torch

    if counts is None:
        counts = torch.empty(256, dtype=torch.int64, device=w.device)
    elif counts.numel() != 256 or counts.element_size() != 8 or not counts.is_contiguous():
        raise ValueError("counts must be 256 contiguous 8-byte elements")
    _check("df11_histogram_device",
           LIB.df11_histogram_device(_format(fmt), ctypes.c_void_p(w.data_ptr()), w.numel(),
                                     ctypes.c_void_p(counts.data_ptr()), _stream_handle(stream)))
    return counts


def df11_build_codebook_from_counts(counts) -> df11_codebook:
    c = np.ascontiguousarray(np.asarray(counts), dtype=np.uint64)
    cb = df11_codebook()
    _check("df11_build_codebook_from_counts",
           LIB.df11_build_codebook_from_counts(c.ctypes.data_as(_u64p), ctypes.byref(cb)))
    return cb


def df11_tensor_ranges_from_counts(cb: df11_codebook, counts, last_weights, fmt: str = "bf16",
                                   tile_windows: int = DEFAULT_TILE_WINDOWS,
                                   window_bytes: int = DEFAULT_WINDOW_BYTES):
    """(tensor_offsets uint64[n+1], tensor_tiles uint64[2n]) from per-tensor
    histograms ``counts`` (n x 256) and the tensors' last weights (n bit patterns)."""
    c = np.ascontiguousarray(np.asarray(counts), dtype=np.uint64).reshape(-1, 256)
    n = c.shape[0]
    last = np.ascontiguousarray(np.asarray(last_weights), dtype=np.uint32).reshape(-1)
    if last.size != n:
        raise ValueError("one last weight per tensor")
    offs = np.zeros(n + 1, dtype=np.uint64)
    tiles = np.zeros(max(2 * n, 1), dtype=np.uint64)
    _check("df11_tensor_ranges_from_counts",
           LIB.df11_tensor_ranges_from_counts(_format(fmt), ctypes.byref(cb), c.ctypes.data_as(_u64p),
                                              last.ctypes.data_as(_u32p), n, tile_windows,
                                              window_bytes, offs.ctypes.data_as(_u64p),
                                              tiles.ctypes.data_as(_u64p)))
    return offs, tiles[: 2 * n]


def encode_on_device(tensors, fmt: str = "bf16", tile_windows: int = DEFAULT_TILE_WINDOWS,
                     window_bytes: int = DEFAULT_WINDOW_BYTES, stream=None):
    """Compress device tensors (16-bit for BF16, 8-bit for FP8) into a
    DeviceStream without moving the weights to the host: per-tensor device
    histograms, the codebook built on the host from them, then
    df11_encode_device on the concatenated unit.  Every allocation, copy and
    launch is ordered on ``stream`` (a torch stream or a raw hipStream_t; the
    current stream when None), and the call returns once that stream has
    finished the encoding.  Returns (DeviceStream, codebook)."""
    import torch

    if stream is None:
        st = torch.cuda.current_stream()
    elif isinstance(stream, torch.cuda.Stream):
        st = stream
    else:
        st = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)))
    size = 2 if fmt == "bf16" else 1
    for t in tensors:
        if t.element_size() != size:
            raise TypeError(f"{fmt} tensors must have {8 * size}-bit elements")
    cur = torch.cuda.current_stream()
    with torch.cuda.stream(st):
        if st != cur:
            st.wait_stream(cur)  # the work that wrote the tensors comes first
        flat = [t.reshape(-1).view(torch.int16 if size == 2 else torch.uint8).contiguous()
                for t in tensors]
        # the histogram and the encoder read 16 bytes at a time
        flat = [t.clone() if t.data_ptr() % 16 else t for t in flat]
        unit = torch.cat(flat) if len(flat) != 1 else flat[0]
        n = unit.numel()
        dev = unit.device
        per = torch.zeros((max(len(flat), 1), 256), dtype=torch.int64, device=dev)
        lasts = torch.zeros(max(len(flat), 1), dtype=torch.int32, device=dev)
        for k, t in enumerate(flat):
            if t.numel():
                df11_histogram_device(t, fmt, st, per[k])
                lasts[k] = t[-1].to(torch.int32)
        per_h = per.cpu().numpy().view(np.uint64)[: len(flat)]  # waits for st
        lasts_h = lasts.cpu().numpy().view(np.uint32)[: len(flat)] & (0xFFFF if size == 2 else 0xFF)
        counts = per_h.sum(axis=0, dtype=np.uint64) if len(flat) else np.zeros(256, np.uint64)
        cb = df11_build_codebook_from_counts(counts)
        sz = df11_sizes()
        _check("df11_encode_size_from_counts",
               LIB.df11_encode_size_from_counts(_format(fmt), ctypes.byref(cb),
                                                counts.ctypes.data_as(_u64p), n, tile_windows,
                                                window_bytes, ctypes.byref(sz)))
        offs, tiles = df11_tensor_ranges_from_counts(cb, per_h, lasts_h, fmt, tile_windows,
                                                     window_bytes)
        stm = torch.empty(sz.stream_bytes, dtype=torch.uint8, device=dev)
        sm = torch.empty(sz.sm_bytes, dtype=torch.uint8, device=dev)
        gaps = torch.empty(max(16, sz.n_windows), dtype=torch.uint8, device=dev)
        bop = torch.empty(sz.bop_entries, dtype=torch.int32, device=dev)
        mx = torch.empty(4, dtype=torch.int32, device=dev)
        nbytes = int(LIB.df11_encode_device_scratch_bytes(n))
        scratch = torch.empty(nbytes + 256, dtype=torch.uint8, device=dev)
        sp = scratch.data_ptr()
        out = df11_device_encode(stm.data_ptr(), sm.data_ptr(), gaps.data_ptr(), bop.data_ptr(),
                                 mx.data_ptr(), (sp + 255) // 256 * 256, nbytes)
        _check("df11_encode_device",
               LIB.df11_encode_device(_format(fmt), ctypes.byref(cb),
                                      ctypes.c_void_p(unit.data_ptr()), n, tile_windows,
                                      window_bytes, ctypes.byref(sz), ctypes.byref(out),
                                      _stream_handle(st)))
        max_tile = int(mx.cpu()[0])  # waits for st: the arrays are complete
    hs = HostStream(np.zeros(0, np.uint8), np.zeros(0, np.uint8), np.zeros(sz.n_windows, np.uint8),
                    np.zeros(sz.bop_entries, np.uint32), offs, tiles, tile_windows, window_bytes,
                    max_tile, n, int(sz.total_bits), int(sz.n_tiles), _format(fmt))
    ds = DeviceStream(hs, cb, dev, arrays=(stm, sm, gaps, bop))
    return ds, cb


def df11_decompress_gemv(ds: DeviceStream, layout, x, y, scratch=None, status=None,
                         stream=None) -> None:
    """y = W x per matrix of ``layout`` (from gemv_layout, matching the unit's
    tensors) computed straight from the compressed unit ``ds``.  ``scratch``: a
    device uint8 tensor of df11_decompress_gemv_scratch_bytes bytes, allocated
    here when not given."""
    import torch

    arr, n, nx, ny = layout
    if x.dtype.itemsize != 4 or y.dtype.itemsize != 4 or x.numel() < nx or y.numel() < ny:
        raise ValueError("x and y must be float32 device tensors covering the layout")
    need = int(LIB.df11_decompress_gemv_scratch_bytes(ctypes.byref(ds.desc)))
    if scratch is None:
        scratch = torch.empty(need, dtype=torch.uint8, device=x.device)
    sp = ctypes.c_void_p(status.data_ptr()) if status is not None else ctypes.c_void_p(0)
    _check("df11_decompress_gemv",
           LIB.df11_decompress_gemv(ctypes.byref(ds.desc), arr, n, ctypes.c_void_p(x.data_ptr()),
                                    ctypes.c_void_p(y.data_ptr()),
                                    ctypes.c_void_p(scratch.data_ptr()), scratch.numel(), sp,
                                    _stream_handle(stream)))


DF11_GEMV_NOALLOC_MAX_TILES = 786432


def df11_decompress_gemv_noalloc(ds: DeviceStream, layout, x, y, status=None,
                                 stream=None) -> None:
    """df11_decompress_gemv on the library's static per-GPU workspace (no
    allocation anywhere in the call; units of at most
    DF11_GEMV_NOALLOC_MAX_TILES tiles; calls on one GPU must not overlap)."""
    arr, n, nx, ny = layout
    if x.dtype.itemsize != 4 or y.dtype.itemsize != 4 or x.numel() < nx or y.numel() < ny:
        raise ValueError("x and y must be float32 device tensors covering the layout")
    sp = ctypes.c_void_p(status.data_ptr()) if status is not None else ctypes.c_void_p(0)
    _check("df11_decompress_gemv_noalloc",
           LIB.df11_decompress_gemv_noalloc(ctypes.byref(ds.desc), arr, n,
                                            ctypes.c_void_p(x.data_ptr()),
                                            ctypes.c_void_p(y.data_ptr()), sp,
                                            _stream_handle(stream)))


# ---------------------------------------------------------------- products in 8-bit integers


def _matrices(tensors, what):
    """Checks 2-D device tensors of one type whose rows are contiguous."""
    tensors = list(tensors)
    if not 1 <= len(tensors) <= DF11_INT8_MAX_TENSORS:
        raise ValueError(f"1 to {DF11_INT8_MAX_TENSORS} {what}")
    first = tensors[0]
    for t in tensors:
        if t.dim() != 2 or not t.is_cuda or (t.size(1) > 1 and t.stride(1) != 1) or t.stride(0) < 0:
            raise ValueError(f"{what} must be 2-D device tensors with contiguous rows")
        if t.dtype != first.dtype or t.device != first.device:
            raise TypeError(f"{what} must be of one type, on one device")
    return tensors


def _quantize(tensors, st):
    """(code tensor, scale tensor) of each matrix, launched on the handle st."""
    import torch

    rows = (df11_int8_rows * len(tensors))()
    out = []
    for a, t in zip(rows, tensors):
        r, c = t.shape
        stride = (c + 127) // 128 * 128  # rows on cache lines
        codes = torch.empty((r, stride), dtype=torch.int8, device=t.device)[:, :(c + 15) // 16 * 16]
        scales = torch.empty(r, dtype=torch.float32, device=t.device)
        a.src, a.codes, a.scales = t.data_ptr(), codes.data_ptr(), scales.data_ptr()
        a.src_stride, a.code_stride, a.rows, a.cols = t.stride(0), stride, r, c
        out.append((codes, scales))
    _check("df11_quantize_int8", LIB.df11_quantize_int8(_type(tensors[0].dtype), rows, len(rows), st))
    return out


def quantize_int8(tensors, stream=None):
    """df11_quantize_int8 of up to DF11_INT8_MAX_TENSORS matrices (BF16, F16 or
    float32 device tensors, contiguous rows): a list of (codes, scales), the
    codes int8 [rows, cols rounded up to 16] with zeros behind the columns, the
    rows 128-byte aligned; memory of the stream, where one is named."""
    tensors = _matrices(tensors, "matrices")
    guard, st = _on(tensors[0].device, stream)
    with guard:
        out = _quantize(tensors, st)
    _lend(tensors[0].device, stream, tensors)
    return out


class _Lender:
    """What calls use for longer than one of them: the first call on each stream
    lends it ``_memory``, which stays lent until it is freed.  ``_lent``: the
    handles of the streams that have it."""

    def _lend(self, stream, st):
        import torch

        _lend(self.device, torch.cuda.current_stream(self.device) if stream is None else stream,
              self._memory)
        self._lent.add(st)


class Int8Linear(_Lender):
    """The matrices of a block as 8-bit integers with a scale for each output
    channel, multiplied with activations that are quantised token by token
    (df11_linear_int8: two launches a call, one for a single token).

    ``codes``: int8 device tensors [rows, at least cols rounded up to 16];
    ``scales``: float32 [rows]; ``shapes``: (rows, cols) of each matrix.  Codes
    whose rows start on cache lines (quantize_int8's do) are kept as they are,
    and so are their scales: later calls read what they hold then.  Others are
    copied here with their scales, on the current stream, to rows that do: what
    happens to the given ones later is not seen.
    """

    def __init__(self, codes, scales, shapes):
        import torch

        codes = _matrices(codes, "codes")
        self.scales, self.shapes = list(scales), [(int(r), int(c)) for r, c in shapes]
        self.device = codes[0].device
        if not len(codes) == len(self.scales) == len(self.shapes):
            raise ValueError("one codes tensor, scales tensor and shape per matrix")
        self._t = (df11_int8_tensor * len(codes))()
        self._bytes = {}  # scratch for a number of tokens
        # what the calls read, codes and scales in turn: its memory, whatever the
        # tensors are given later
        self._memory = []
        self._lent = set()
        for k, (a, q, s, (r, c)) in enumerate(zip(self._t, codes, self.scales, self.shapes)):
            if q.dtype != torch.int8 or q.size(0) != r or q.size(1) < c:
                raise ValueError("codes must be int8 of the shape's rows and at least its columns")
            if s.dtype != torch.float32 or s.numel() != r or not s.is_contiguous() or s.device != self.device:
                raise ValueError("scales must be float32, one per row")
            # the product reads whole groups of 16 columns
            whole = (c + 15) // 16 * 16
            if q.size(1) < whole:
                raise ValueError("codes must reach to the next multiple of 16 columns")
            if q.data_ptr() % 128 or (r > 1 and (q.stride(0) % 128 or q.stride(0) < whole)):
                lines = torch.empty((r, (c + 127) // 128 * 128), dtype=torch.int8, device=self.device)
                q = lines[:, :whole].copy_(q[:, :whole])
                s = self.scales[k] = s.clone()
            self._memory += q.detach(), s.detach()
            a.w, a.w_scale, a.rows, a.cols = q.data_ptr(), s.data_ptr(), r, c
            a.w_stride = q.stride(0) if r > 1 else whole
            a.y_stride = r  # of outputs that a call makes

    @classmethod
    def from_tensors(cls, tensors, stream=None):
        """Quantises weight matrices (BF16, F16 or float32, [rows, cols])."""
        tensors = _matrices(tensors, "matrices")
        guard, st = _on(tensors[0].device, stream)
        with guard:
            held = _quantize(tensors, st)
        _lend(tensors[0].device, stream, tensors)
        return cls._made(held, [tuple(t.shape) for t in tensors], st)

    @classmethod
    def _made(cls, held, shapes, st):
        """A layer of codes and scales that were made on the stream st."""
        layer = cls([q for q, _ in held], [s for _, s in held], shapes)
        layer._lent.add(st)
        return layer

    @classmethod
    def from_unit(cls, ds: DeviceStream, shapes, status=None, stream=None):
        """Decompresses a BF16 unit and quantises its matrices, whose ``shapes``
        follow one another in it."""
        import torch

        shapes = [(int(r), int(c)) for r, c in shapes]
        if not 1 <= len(shapes) <= DF11_INT8_MAX_TENSORS:
            raise ValueError(f"1 to {DF11_INT8_MAX_TENSORS} matrices")
        if sum(r * c for r, c in shapes) != ds.n_weights or ds.desc.format != 0:
            raise ValueError("the shapes must tile a BF16 unit")
        guard, st = _on(ds.stream.device, stream)
        with guard:
            unit = torch.empty(ds.n_weights, dtype=torch.bfloat16, device=ds.stream.device)
            df11_decompress_block(ds, unit, status, st)
            parts = unit.split([r * c for r, c in shapes])
            held = _quantize(_matrices([p.view(s) for p, s in zip(parts, shapes)], "matrices"), st)
        _lend(ds.stream.device, stream, [ds.stream, ds.sm, ds.gaps, ds.block_out_pos, ds.tables] +
              ([] if status is None else [status]))
        return cls._made(held, shapes, st)

    def __call__(self, xs, out_dtype=None, out=None, stream=None):
        """y = x W^T of every matrix: a list of [n_tokens, rows] tensors of
        ``out_dtype`` (BF16 by default, F16 or float32), or written into the
        tensors ``out``.  ``xs``: one [n_tokens, cols] tensor (BF16, F16 or
        float32) per matrix; a tensor given for several is quantised once.  The
        rounding to codes has no derivative: activations that require a
        gradient are refused (detach them, or call under torch.no_grad())."""
        import torch

        if len(xs) != len(self.shapes):
            raise ValueError("one activation tensor per matrix")
        first = xs[0]
        if first.dim() != 2 or first.device != self.device:
            raise ValueError(f"activations must be 2-D tensors on {self.device}")
        n_tokens, kind = first.size(0), first.dtype
        if out is not None:
            out = _matrices(out, "outputs")
            if out[0].device != self.device or [tuple(y.shape) for y in out] != [
                    (n_tokens, r) for r, _ in self.shapes] or out_dtype not in (None, out[0].dtype):
                raise ValueError("outputs must be [n_tokens, rows] of their matrix")
            out_dtype = out[0].dtype
        elif out_dtype is None:
            out_dtype = torch.bfloat16
        x_type, y_type = _type(kind), _type(out_dtype)
        n = len(self.shapes)
        t = type(self._t).from_buffer_copy(self._t)
        last = None
        for a, x, (_, c) in zip(t, xs, self.shapes):
            if x is not last:
                if x.shape != (n_tokens, c) or x.dtype != kind or x.device != self.device:
                    raise ValueError("activations must be [n_tokens, cols] of their matrix, of one "
                                     f"type, on {self.device}")
                if x.requires_grad and torch.is_grad_enabled():
                    raise RuntimeError("an int8 product gives its activations no gradient: detach them")
                strides = x.stride()
                if (strides[1] != 1 and c > 1) or strides[0] < 0:
                    raise ValueError("activations must have contiguous rows")
                last, p, stride = x, x.data_ptr(), strides[0]
            elif c != last.size(1):
                raise ValueError("activations must be [n_tokens, cols] of their matrix")
            a.x, a.x_stride = p, stride
        guard, st = _on(self.device, stream)
        with guard:
            if out is None:
                dev = self.device
                out = [torch.empty(n_tokens, r, dtype=out_dtype, device=dev) for r, _ in self.shapes]
                for a, y in zip(t, out):
                    a.y = y.data_ptr()
            else:
                for a, y in zip(t, out):
                    a.y = y.data_ptr()
                    a.y_stride = y.stride(0) if n_tokens > 1 else y.size(1)
            need = self._bytes.get(n_tokens)
            if need is None:
                need = self._bytes[n_tokens] = int(
                    LIB.df11_linear_int8_scratch_bytes(self._t, n, n_tokens))
            scratch = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
            _check("df11_linear_int8",
                   LIB.df11_linear_int8(x_type, y_type, t, n, n_tokens,
                                        scratch.data_ptr() if need else None, need, st))
        if st not in self._lent:
            self._lend(stream, st)
        if stream is not None:
            _lend(self.device, stream, [*xs, *out])
        return out


# ---------------------------------------------------------------- optimiser step


_TYPE_OF = {}  # torch's types, filled when first seen


def _type(dtype) -> int:
    kind = _TYPE_OF.get(dtype)
    if kind is None:
        name = str(dtype).replace("torch.", "")
        if name not in TYPES:
            raise TypeError(f"no operator for {dtype}")
        kind = _TYPE_OF[dtype] = TYPES[name]
    return kind


def _same(tensors, what, dtype=None, sizes=None, device=None):
    """Checks a list of contiguous device tensors of one type; returns them."""
    tensors = list(tensors)
    if sizes is not None and [t.numel() for t in tensors] != sizes:
        raise ValueError(f"{what} must have {sizes[:8]} elements, one tensor each")
    if not tensors:
        return tensors
    kind = tensors[0].dtype if dtype is None else dtype
    where = tensors[0].device if device is None else device
    if where.type != "cuda":
        raise ValueError(f"{what} must be device tensors")
    for t in tensors:
        if t.dtype != kind:
            raise TypeError(f"{what} must be of one type" if dtype is None else f"{what} must be {dtype}")
        if t.device != where or not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous tensors on {where}")
    return tensors


class _AsIs:
    """No guard: device and stream are current already."""

    def __enter__(self):
        return self

    def __exit__(self, *_):
        return False


_AS_IS = _AsIs()


def _stream_of(device, stream):
    """A stream object, or a stream's handle, as torch's stream."""
    import torch

    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)


def _lend(device, stream, tensors):
    """Keeps the memory of tensors that a call on ``stream`` uses from another
    use before that call is done, when they are freed earlier on their own stream."""
    if stream is not None:
        stream = _stream_of(device, stream)
        for t in tensors:
            t.record_stream(stream)


def _on(device, stream):
    """(a guard that makes ``stream``, or the device's current stream, and the
    device current; the stream's handle)."""
    import torch

    if stream is None:
        guard = _AS_IS if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)
        return guard, torch._C._cuda_getCurrentRawStream(device.index)
    stream = _stream_of(device, stream)
    if stream.device != device:
        raise ValueError(f"the stream is not on {device}")
    return torch.cuda.stream(stream), stream.cuda_stream


class AdamW(_Lender):
    """df11_adamw_step over a list of device tensors (BF16 or float32 weights,
    e.g. a unit's, at any offset of a larger buffer), with what the step keeps.

    Weights, masters and states must not overlap: a weight that layers share is
    given once.  ``grads``: one tensor per weight, all BF16 or all float32, apart
    from what a step writes.  ``masters``:
    float32 copies of BF16 weights that carry the update.  ``state_bits``: 32
    (float32 states) or 8 (codes of blocks of DF11_ADAMW_BLOCK elements, a
    quarter of the memory).  ``state``: lists "m" and "v" (and "m_scale",
    "v_scale" for 8 bits) to go on from instead of zeros; they are updated in
    place.  ``counts``: keep each tensor's exponent histogram of the new BF16
    weights in ``self.counts`` (one row of 256 per tensor).
    ``weight_decay`` and ``lr_scale``: one number, or one per tensor.  ``step``:
    steps already made.  ``device_step``: keep the step's number on the device
    (``self.d_step``) and advance it there, so that a captured step counts on
    when it is replayed; without it a captured step replays the number it was
    captured with.  Steps that a gradient factor skips are not counted.  Steps
    work on the memory that the tensors have when they are given: one that gets
    other memory later (``t.data = ...``) is not followed there.  Used from one
    host thread at a time.
    """

    def __init__(self, weights, grads, masters=None, state_bits: int = 32, state=None,
                 counts: bool = False, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay=0.01, lr_scale=1.0, step: int = 0, device_step: bool = False):
        import torch

        self.weights = _same(weights, "weights")
        if not self.weights:
            raise ValueError("no weights")
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        if int(step) < 0:
            raise ValueError("step must be at least 0")
        self.device = dev = self.weights[0].device
        sizes = self._sizes = [t.numel() for t in self.weights]
        n = len(sizes)
        blocks = [-(-s // DF11_ADAMW_BLOCK) for s in sizes]
        self.masters = None if masters is None else _same(masters, "masters", torch.float32, sizes, dev)
        self.state_bits = state_bits
        kinds = ({"m": torch.float32, "v": torch.float32} if state_bits == 32 else
                 {"m": torch.int8, "v": torch.uint8, "m_scale": torch.float32,
                  "v_scale": torch.float32})
        if state is None:
            state = {k: [torch.zeros(c, dtype=d, device=dev)
                         for c in (blocks if k.endswith("scale") else sizes)]
                     for k, d in kinds.items()}
        elif set(state) != set(kinds):
            raise ValueError(f"state must hold {sorted(kinds)}")
        self.state = {k: _same(state[k], k, d, blocks if k.endswith("scale") else sizes, dev)
                      for k, d in kinds.items()}
        # what two tensors share would be updated twice, in any order
        spans = []
        for part in (self.weights, self.masters or [], *self.state.values()):
            spans += [(t.data_ptr(), t.data_ptr() + t.numel() * part[0].element_size())
                      for t in part if t.numel()]
        spans.sort()
        if any(lo < end for (_, end), (lo, _) in zip(spans, spans[1:])):
            raise ValueError("weights, masters or states overlap: give a shared tensor once")
        self.counts = (torch.zeros((n, 256), dtype=torch.int64, device=dev) if counts else None)
        self.lr, self._calls = float(lr), int(step)
        # the step's number, or how many of the calls were skipped (once factors are in use)
        self.d_step = (torch.full((1,), int(step), dtype=torch.int64, device=dev)
                       if device_step else None)
        self._skipped = None if device_step else torch.zeros(1, dtype=torch.int64, device=dev)
        self._factors = False
        # the memory of all that steps write, whatever the tensors are given later:
        # one tensor of each storage
        parts = sum(self.state.values(), self.weights + (self.masters or []))
        parts += [t for t in (self.counts, self.d_step, self._skipped) if t is not None]
        self._memory = [t.detach() for t in
                        {t.untyped_storage().data_ptr(): t for t in parts}.values()]
        self._lent = set()
        each = lambda x: [float(v) for v in x] if np.ndim(x) else [float(x)] * n  # noqa: E731
        decays, scales = each(weight_decay), each(lr_scale)
        if len(decays) != n or len(scales) != n:
            raise ValueError("one weight_decay and one lr_scale per tensor")
        self._t = (df11_adamw_tensor * n)()
        for k, a in enumerate(self._t):
            a.w = self.weights[k].data_ptr()
            a.master = self.masters[k].data_ptr() if self.masters else None
            for name, parts in self.state.items():
                setattr(a, name, parts[k].data_ptr())
            a.counts = self.counts[k].data_ptr() if counts else None
            a.numel, a.lr_scale, a.weight_decay = sizes[k], scales[k], decays[k]
        self._c = df11_adamw_config(self.lr, betas[0], betas[1], eps, 0,
                                    self._kind(self.weights, "weights"), 0, state_bits, 0)
        self._c_ref = ctypes.byref(self._c)
        # what a step changes that graphs may have saved; views count with their base
        bases = [t if t._base is None else t._base for t in self.weights + (self.masters or [])]
        self._changed = list({id(t): t for t in bases}.values())
        self._norm_bytes = int(LIB.df11_grad_norm_scratch_bytes(self._t, n))
        self.set_grads(grads)

    def set_grads(self, grads) -> None:
        """The gradients that later steps read."""
        grads = _same(grads, "grads", None, self._sizes, self.device)
        kind = self._kind(grads, "gradients")  # refused before anything is replaced
        self.grads, self._c.g_type = grads, kind
        self._grad_memory = [g.untyped_storage() for g in grads]
        for a, g in zip(self._t, grads):
            a.g = g.data_ptr()

    @staticmethod
    def _kind(tensors, what) -> int:
        kind = _type(tensors[0].dtype)
        if kind > TYPES["bfloat16"]:
            raise Df11Error(f"AdamW of {what} in {tensors[0].dtype}", DF11_E_INVALID)
        return kind

    def grad_norm(self, max_norm: float, stream=None):
        """A float32 device tensor [norm, clip factor] of all gradients together."""
        guard, st = _on(self.device, stream)
        with guard:
            out = self._norm(max_norm, st)
        _lend(self.device, stream, self.grads)
        return out

    def _norm(self, max_norm, st):
        import torch

        # memory of the stream that uses it: its reuse is ordered there
        out = torch.empty(2, dtype=torch.float32, device=self.device)
        scratch = torch.empty(self._norm_bytes, dtype=torch.uint8, device=self.device)
        _check("df11_grad_norm",
               LIB.df11_grad_norm(self._c.g_type, self._t, len(self._t), float(max_norm),
                                  out.data_ptr(), scratch.data_ptr(), self._norm_bytes, st))
        return out

    def step(self, lr=None, max_norm=None, grad_factor=None, stream=None):
        """One step.  ``lr``: this step's learning rate (a number, or a float32
        device tensor that the kernel reads).  ``max_norm``: clip the
        gradients' norm; returns grad_norm's tensor then.  ``grad_factor``: a
        float32 device tensor of one element to multiply the gradients with;
        a factor that is not finite (that of a norm that is not, too) leaves
        everything as it was, the step's number among it."""
        import torch

        if max_norm is not None and grad_factor is not None:
            raise ValueError("max_norm or grad_factor")
        c = self._c
        by_tensor = hasattr(lr, "data_ptr")
        if by_tensor or grad_factor is not None:
            for x, what in ((grad_factor, "grad_factor"), (lr if by_tensor else None, "lr")):
                if x is not None and (_type(x.dtype) != 0 or x.numel() != 1 or x.device != self.device):
                    raise ValueError(f"{what} must be one float32 on {self.device}")
        c.lr = self.lr if lr is None or by_tensor else float(lr)
        c.d_lr = lr.data_ptr() if by_tensor else None
        c.step = self._calls + 1
        guard, st = _on(self.device, stream)
        norm = count = None
        with guard:
            if max_norm is not None:
                norm = self._norm(max_norm, st)
                factor = norm.data_ptr() + 4
            else:
                factor = None if grad_factor is None else grad_factor.data_ptr()
            c.d_grad_factor = factor
            if self.d_step is not None:
                self.d_step += 1
                c.d_step = self.d_step.data_ptr()
                count = c.d_step if factor else None
            elif (factor or self._factors) and not torch._C._cuda_isCurrentStreamCapturing():
                self._factors, count = True, self._skipped.data_ptr()
            rc = (LIB.df11_adamw_step(self._c_ref, self._t, len(self._t), st) if count is None else
                  LIB.df11_adamw_step_counted(self._c_ref, self._t, len(self._t), count, st))
            if rc != DF11_OK:
                if self.d_step is not None:
                    self.d_step -= 1  # no step was made
                _check("df11_adamw_step", rc)
        torch._C._increment_version(self._changed)
        if st not in self._lent:
            self._lend(stream, st)
        if stream is not None:
            _lend(self.device, stream, self.grads + [x for x in (grad_factor, lr if by_tensor else None)
                                                     if x is not None])
        self._calls += 1
        return norm

    @property
    def steps(self) -> int:
        """Steps made.  Waits for the GPU where only it knows whether some were
        skipped, or replayed (device_step)."""
        import torch

        if self.d_step is None and not self._factors:
            return self._calls
        torch.cuda.synchronize(self.device)
        return int(self.d_step) if self.d_step is not None else self._calls - int(self._skipped)

    @steps.setter
    def steps(self, made: int) -> None:
        self._calls = int(made)
        (self._skipped.zero_() if self.d_step is None else self.d_step.fill_(self._calls))

    def state_values(self, m_out=None, v_out=None, stream=None):
        """(m, v) as lists of float32 tensors, or written into the given lists
        of float32 or BF16 tensors: what 8-bit states stand for."""
        import torch

        if self.state_bits == 32:
            raise ValueError("32-bit states are their own values")
        sizes = self._sizes
        guard, st = _on(self.device, stream)
        with guard:
            if m_out is None and v_out is None:
                # memory of the stream that writes it: its last use there is over by then
                m_out, v_out = ([torch.empty(s, dtype=torch.float32, device=self.device) for s in sizes]
                                for _ in range(2))
            lists = []
            for out, what in ((m_out, "m_out"), (v_out, "v_out")):
                kind = (m_out if m_out is not None else v_out)[0].dtype
                if out is not None:
                    out = _same(out, what, kind, sizes, self.device)
                lists.append(None if out is None
                             else (ctypes.c_void_p * len(out))(*[t.data_ptr() for t in out]))
            _check("df11_adamw_values",
                   LIB.df11_adamw_values(self._t, len(self._t), _type(kind), lists[0], lists[1], st))
        if stream is not None:
            _lend(self.device, stream, [*(m_out or []), *(v_out or [])])
        if st not in self._lent:
            self._lend(stream, st)
        return m_out, v_out

    def compressed_sizes(self) -> df11_sizes:
        """What the weights of the last step would take as one compressed unit
        (payload bits, arrays), from ``counts``: whether, and into how much
        memory, to encode them.  Waits for the step, whatever its stream."""
        import torch

        if self.counts is not None:
            torch.cuda.synchronize(self.device)
            counts = self.counts.sum(0).cpu().numpy().view(np.uint64)
        if self.counts is None or not counts.any():  # every step counts every weight
            raise ValueError("counts are kept by steps of AdamW(counts=True)")
        cb, sz = df11_build_codebook_from_counts(counts), df11_sizes()
        _check("df11_encode_size_from_counts",
               LIB.df11_encode_size_from_counts(_format("bf16"), ctypes.byref(cb),
                                                counts.ctypes.data_as(_u64p), int(counts.sum()),
                                                DEFAULT_TILE_WINDOWS, DEFAULT_WINDOW_BYTES,
                                                ctypes.byref(sz)))
        return sz

    def compress(self, stream=None):
        """The BF16 weights as one compressed unit: encode_on_device's
        (DeviceStream, codebook).  Waits for the steps before it, whatever their
        stream: the codebook must be that of the weights that are encoded."""
        import torch

        torch.cuda.synchronize(self.device)
        with torch.cuda.device(self.device):  # the encoder works on the current device's streams
            return encode_on_device(self.weights, stream=stream)


# ---------------------------------------------------------------- embedding and output head


def _rows_apart(t, what, device=None):
    """Checks a 2-D device tensor whose rows are contiguous; returns its row stride."""
    if t.dim() != 2 or not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{what} must be a 2-D device tensor" + ("" if device is None else f" on {device}"))
    if (t.size(1) > 1 and t.stride(1) != 1) or t.stride(0) < 0:
        raise ValueError(f"{what} must have contiguous rows")
    return t.stride(0) if t.size(0) > 1 else t.size(1)


def _flat(t, n, what, device, stream):
    """[*, cols] as [n, cols]; where no one stride reaches all rows (a batch without
    each sequence's last token), a copy, made on the call's stream."""
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{what} must be a device tensor on {device}")
    if t.size(-1) > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must have contiguous rows")
    with _on(device, stream)[0]:
        return t.reshape(n, t.size(-1))


def _output(t, what, shape, dtype, device):
    """Checks a given output: rows that lie apart, of the shape and type; returns its row stride."""
    stride = _rows_apart(t, what, device)
    if tuple(t.shape) != tuple(shape) or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{what} must be {list(shape)}" + (f" of {dtype}" if dtype is not None else ""))
    if stride < t.size(1):
        raise ValueError(f"{what} must have rows of their own")
    return stride


def _token_bits(tokens, device) -> int:
    bits = _TOKEN_BITS.get(tokens.dtype)
    if bits is None:
        bits = {"torch.int32": 32, "torch.int64": 64}.get(str(tokens.dtype))
        if bits is None:
            raise TypeError("tokens must be int32 or int64")
        _TOKEN_BITS[tokens.dtype] = bits
    if tokens.device != device:
        raise ValueError(f"tokens must be on {device}")
    return bits


def _check_padding(padding_idx, rows):
    if padding_idx is not None and not 0 <= padding_idx < rows:
        raise ValueError("padding_idx must be a row of the table")


_TOKEN_BITS = {}  # by torch's types, filled when first seen


class Embedding(_Lender):
    """Rows of a table [rows, cols] (BF16, F16 or float32, contiguous rows), looked
    up by token and multiplied with ``scale`` (df11_embedding: one launch).  The
    table is used in place: a step of AdamW on it is seen by later calls."""

    def __init__(self, table, scale: float = 1.0, padding_idx: int | None = None):
        stride = _rows_apart(table, "the table")
        _check_padding(padding_idx, table.size(0))
        self.table, self.scale, self.padding_idx = table, float(scale), padding_idx
        self.device, self._memory, self._lent = table.device, [table.detach()], set()
        self._a = df11_embedding_lookup(table=table.data_ptr(), table_stride=stride, rows=table.size(0),
                                        cols=table.size(1), table_type=_type(table.dtype), scale=scale)

    def __call__(self, tokens, out_dtype=None, out=None, stream=None):
        """The tokens' rows: [*tokens.shape, cols] of ``out_dtype`` (the table's by
        default), or written into ``out`` [number of tokens, cols].  ``tokens``:
        int32 or int64; one outside the table gives a row of NaN.  The call
        records no graph: a table that requires a gradient is refused (call
        under torch.no_grad(), and ``gradient`` makes the table's)."""
        import torch

        if self.table.requires_grad and torch.is_grad_enabled():
            raise RuntimeError("a lookup records no gradient for its table: call it under torch.no_grad()")
        a = df11_embedding_lookup.from_buffer_copy(self._a)
        a.token_bits, a.n = _token_bits(tokens, self.device), tokens.numel()
        if out is not None:
            a.out_stride = _output(out, "out", (a.n, a.cols), out_dtype, self.device)
            out_dtype = out.dtype
        elif out_dtype is None:
            out_dtype = self.table.dtype
        a.out_type = _type(out_dtype)
        guard, st = _on(self.device, stream)
        with guard:
            given, tokens, made = tokens, tokens.contiguous(), out is None
            if made:
                out, a.out_stride = torch.empty(*tokens.shape, a.cols, dtype=out_dtype, device=self.device), a.cols
            a.tokens, a.out = tokens.data_ptr(), out.data_ptr()
            _check("df11_embedding", LIB.df11_embedding(a, st))
        if not made:
            torch._C._increment_version([out])
        if st not in self._lent:
            self._lend(stream, st)
        if stream is not None:
            _lend(self.device, stream, [given, out])
        return out

    def gradient(self, tokens, dy, out=None, dtype=None, accumulate: bool = False, stream=None):
        """The table's gradient of a call with these tokens whose output's gradient
        is ``dy``: embedding_gradient with the table's rows, scale and padding, of the
        table's type by default."""
        if dtype is None and out is None:
            dtype = self.table.dtype
        return embedding_gradient(tokens, dy, self.table.size(0), dtype, out, accumulate, self.scale,
                                  self.padding_idx, stream)


def embedding_gradient(tokens, dy, rows: int, dtype=None, out=None, accumulate: bool = False,
                       scale: float = 1.0, padding_idx: int | None = None, stream=None):
    """df11_embedding_gradient: the gradient [rows, cols] of a table whose lookup of
    ``tokens`` (int32 or int64, any shape) has the output gradient ``dy``
    [*tokens.shape, cols] or [number of tokens, cols] (BF16, F16 or float32), as
    a new tensor of ``dtype`` (dy's by default), or written into ``out``, or with
    ``accumulate`` added to it.  dy's rows are contiguous; those that no one stride
    reaches (``dy[:, 1:]`` of several sequences) are copied first.  Tokens equal to
    ``padding_idx``, and tokens outside the table, add nothing.  Deterministic."""
    import torch

    device, used = dy.device, [tokens, dy]
    if dy.dim() != 2:
        if dy.dim() < 1 or dy.shape[:-1] != tokens.shape:
            raise ValueError("dy must be [number of tokens, cols]")
        dy = _flat(dy, tokens.numel(), "dy", device, stream)
    _check_padding(padding_idx, rows)
    g = df11_embedding_grad(dy_stride=_rows_apart(dy, "dy", device), rows=rows, n=tokens.numel(),
                            padding=-1 if padding_idx is None else padding_idx, cols=dy.size(1),
                            dy_type=_type(dy.dtype), token_bits=_token_bits(tokens, device),
                            accumulate=bool(accumulate), scale=scale)
    if dy.size(0) != g.n or rows < 0:
        raise ValueError("dy must be [number of tokens, cols]")
    if out is not None:
        g.dw_stride = _output(out, "out", (rows, g.cols), dtype, device)
    elif accumulate:
        raise ValueError("accumulate adds to out")
    guard, st = _on(device, stream)
    with guard:
        tokens, made = tokens.contiguous(), out is None
        if made:
            out, g.dw_stride = torch.empty(rows, g.cols, dtype=dtype or dy.dtype, device=device), g.cols
        g.dw_type = _type(out.dtype)
        need = LIB.df11_embedding_gradient_scratch_bytes(g.n, rows, g.cols)
        scratch = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        g.tokens, g.dy, g.dw = tokens.data_ptr(), dy.data_ptr(), out.data_ptr()
        _check("df11_embedding_gradient",
               LIB.df11_embedding_gradient(g, scratch.data_ptr() if need else None, need, st))
    if not made:
        torch._C._increment_version([out])
    if stream is not None:
        _lend(device, stream, used + [out])
    return out


@functools.cache
def _undifferentiable():
    """f(why, outputs): the outputs as of a function whose derivative is the error
    ``why``.  It is one of a leaf of its own: outputs that hold the nodes of a program's
    leaves must not live while a backward pass of those is captured."""
    import torch

    leaf = torch.zeros((), requires_grad=True)

    class Undifferentiable(torch.autograd.Function):
        @staticmethod
        def forward(ctx, why, outputs, *_):
            ctx.why = why
            return tuple(outputs)

        @staticmethod
        def backward(ctx, *_):
            raise RuntimeError(ctx.why)

    return lambda why, outputs: Undifferentiable.apply(why, outputs, leaf)


class VocabLoss(_Lender):
    """Softmax cross entropy of hidden states under an output head, without keeping
    the logits (df11_vocab_loss), and its gradients (df11_vocab_loss_gradient).

    ``pieces``: BF16 device tensors [rows, cols] that hold consecutive rows of the
    head (one tensor for a whole one), cols and row strides multiples of 8, on 16
    bytes.  They are used in place: a step of AdamW on them is seen by later calls.
    """

    def __init__(self, pieces):
        import torch

        pieces = list(pieces)
        if not pieces:
            raise ValueError("no pieces")
        strides = [_rows_apart(w, "pieces", pieces[0].device) for w in pieces]
        for w in pieces:
            if w.dtype != torch.bfloat16 or w.size(1) != pieces[0].size(1):
                raise ValueError("pieces must be bfloat16 with equal columns")
        self._hold([tuple(w.shape) for w in pieces], pieces[0].device, [w.detach() for w in pieces])
        self.pieces = pieces
        self._held = [(w.data_ptr(), stride) for w, stride in zip(pieces, strides)]

    @classmethod
    def from_unit(cls, ds: DeviceStream, shapes):
        """A head that stays compressed: a BF16 unit whose tensors are its pieces, of
        ``shapes``.  Every call decompresses one at a time into memory of the
        largest one's size, a gradient's call too."""
        shapes = [(int(r), int(c)) for r, c in shapes]
        if ds.desc.format != 0 or ds.desc.n_tensors != len(shapes) or not shapes:
            raise ValueError("one shape for each tensor of a BF16 unit")
        ends = np.cumsum([0] + [r * c for r, c in shapes])
        if any(int(ds.desc.tensor_offsets[k]) != e for k, e in enumerate(ends)):
            raise ValueError("the shapes must be those of the unit's tensors")
        head = cls.__new__(cls)
        head._hold(shapes, ds.stream.device, [ds.stream, ds.sm, ds.gaps, ds.block_out_pos, ds.tables])
        head.unit, head.pieces = ds, None
        return head

    def _hold(self, shapes, device, memory):
        self.shapes, self.device, self._memory, self._lent = shapes, device, memory, set()
        self.vocab, self.cols = sum(r for r, _ in shapes), shapes[0][1]
        if any(c != self.cols for _, c in shapes):
            raise ValueError("pieces must have equal columns")
        self._first = np.cumsum([0] + [r for r, _ in shapes]).tolist()
        self._rows = max(r for r, _ in shapes)
        self._p = df11_vocab_piece(cols=self.cols, vocab=self.vocab, rows=self._rows, begin=1, end=1)
        self._bytes = {}  # scratch for a number of tokens

    def _each(self, p, status, st):
        """Sets p to each piece in turn, decompressed where it has to be."""
        if self.pieces is not None and len(self.shapes) == 1:  # p is this one already
            p.w, p.w_stride = self._held[0]
            return 0,
        return self._in_turn(p, status, st)

    def _in_turn(self, p, status, st):
        import torch

        slot = None
        if self.pieces is None:
            slot = torch.empty(self._rows * self.cols, dtype=torch.bfloat16, device=self.device)
        last = len(self.shapes) - 1
        for k, (rows, cols) in enumerate(self.shapes):
            p.first, p.rows, p.begin, p.end = self._first[k], rows, k == 0, k == last
            if slot is None:
                p.w, p.w_stride = self._held[k]
            else:
                df11_decompress_tensor(self.unit, k, slot[:rows * cols], status, st)
                p.w, p.w_stride = slot.data_ptr(), cols
            yield k

    def _piece(self, x, targets, ignore_index, stream):
        """x as [n, cols], and what all pieces of a call share."""
        import torch

        if x.dtype != torch.bfloat16:
            raise TypeError("hidden states must be bfloat16")
        if x.dim() != 2:
            if x.dim() < 1 or x.shape[:-1] != targets.shape:
                raise ValueError("hidden states must be [*targets.shape, cols]")
            x = _flat(x, targets.numel(), "hidden states", self.device, stream)
        stride = _rows_apart(x, "hidden states", self.device)
        if x.shape != (targets.numel(), self.cols):
            raise ValueError("hidden states must be [number of targets, cols]")
        at = x.data_ptr()
        if at % 16 or stride % 8 or not self.cols <= stride <= DF11_VOCAB_MAX_STRIDE:
            with _on(self.device, stream)[0]:
                x = x.clone(memory_format=torch.contiguous_format)
            at, stride = x.data_ptr(), self.cols
        p = df11_vocab_piece.from_buffer_copy(self._p)
        p.x, p.x_stride, p.n, p.ignored = at, stride, x.size(0), ignore_index
        p.target_bits = _token_bits(targets, self.device)
        return x, p

    def __call__(self, x, targets, ignore_index: int = -100, status=None, stream=None):
        """(losses, lse), float32 like ``targets`` (int32 or int64): the cross entropy
        of each token, and the logarithm of its sum of exponentials.  ``x``: BF16
        hidden states [*targets.shape, cols] or [number of targets, cols], contiguous
        rows; those that no one stride reaches (``x[:, :-1]`` of several sequences), or
        that lie otherwise than df11_vocab_loss takes them (``x[:, -1]`` of long ones),
        are copied first.  A target
        of ``ignore_index`` has loss 0, another one outside the vocabulary NaN.
        ``status``: for a compressed head, as in df11_decompress_tensor.  The call
        records no graph: hidden states that require a gradient are refused (detach
        them; ``gradient`` makes it), and under pieces that require one the outputs
        refuse to be differentiated (outside torch.no_grad())."""
        import torch

        if x.requires_grad and torch.is_grad_enabled():
            raise RuntimeError("a loss records no gradient for its hidden states: detach them")
        used, (x, p) = [x, targets], self._piece(x, targets, ignore_index, stream)
        guard, st = _on(self.device, stream)
        with guard:
            targets = targets.contiguous()
            p.targets = targets.data_ptr()
            losses = torch.empty(targets.shape, dtype=torch.float32, device=self.device)
            lse = torch.empty_like(losses)
            held = self._bytes.get(p.n)
            if held is None:
                sizes = df11_vocab_sizes(p.n, p.cols, self._rows, 0, 0)
                held = self._bytes[p.n] = sizes, LIB.df11_vocab_loss_scratch_bytes(sizes)
            sizes, need = held
            scratch = torch.empty(need, dtype=torch.uint8, device=self.device)
            given_to = losses.data_ptr(), lse.data_ptr(), sizes, scratch.data_ptr(), need, st
            for _ in self._each(p, status, st):
                _check("df11_vocab_loss", LIB.df11_vocab_loss(p, *given_to))
        if stream is not None or st not in self._lent:
            self._used(stream, st, used + [losses, lse] + ([] if status is None else [status]))
        if self.pieces is not None and torch.is_grad_enabled() and any(w.requires_grad for w in self.pieces):
            return _undifferentiable()("a loss records no gradient for its head: `gradient` makes it; detach the "
                                       "losses, or call under torch.no_grad()", [losses, lse])
        return losses, lse

    def _used(self, stream, st, tensors):
        if st not in self._lent:
            self._lend(stream, st)
        if stream is not None:
            _lend(self.device, stream, tensors)

    def gradient(self, x, targets, lse, loss_grad=1.0, lse_grad=None, ignore_index: int = -100,
                 dx_dtype=None, dw_dtype=None, dx=None, dws=None, accumulate: bool = False,
                 needs_dx: bool = True, needs_dw: bool = True, losses=None, status=None, stream=None):
        """(dx, dws) of a call with these arguments that returned ``lse``: the hidden
        states' gradient [n, cols] and a list of the pieces' gradients, BF16 or
        float32 (``dx_dtype``, ``dw_dtype``: BF16 by default; float32 takes up to three
        times that product's work), as new tensors or written into ``dx`` and ``dws``, with
        ``accumulate`` added to dws.  ``loss_grad``: the gradient that the losses
        have, a number or a float32 device tensor of one or of n elements;
        ``lse_grad``: that of lse, such a tensor or None.  ``losses``: the call's; with
        them the gradient keeps its digits where a target is nearly certain.  Ignored
        tokens have no gradient and add none.  Without ``needs_dx`` or ``needs_dw`` that
        one is None."""
        import torch

        used, (x, p) = [x, targets, lse], self._piece(x, targets, ignore_index, stream)
        n, cols, g = p.n, p.cols, df11_vocab_grad()
        g.accumulate = bool(accumulate)
        g.lse = self._per_token("lse", lse, (n,))
        if losses is not None:
            g.losses = self._per_token("losses", losses, (n,))
            used.append(losses)
        if hasattr(loss_grad, "data_ptr"):
            g.loss_grad, g.loss_grads = self._per_token("loss_grad", loss_grad, (1, n)), loss_grad.numel()
            used.append(loss_grad)
        else:
            g.loss_grad_all = loss_grad
        if lse_grad is not None:
            g.lse_grad, g.lse_grads = self._per_token("lse_grad", lse_grad, (1, n)), lse_grad.numel()
            used.append(lse_grad)
        given = []  # outputs
        if dx is not None:
            _output(dx, "dx", (n, cols), dx_dtype, self.device)
            dx_dtype = dx.dtype
            given.append(dx)
        if dws is not None:
            dws = list(dws)
            if len(dws) != len(self.shapes):
                raise ValueError("dws must be a tensor for each piece")
            dw_dtype = dw_dtype or dws[0].dtype
            for t, shape in zip(dws, self.shapes):
                _output(t, "dws", shape, dw_dtype, self.device)
            given += dws
        if (accumulate and dws is None) or (dx is not None and not needs_dx) or (dws is not None and not needs_dw):
            raise ValueError("accumulate adds to dws; outputs are given for gradients that are needed")
        dx_dtype, dw_dtype = dx_dtype or torch.bfloat16, dw_dtype or torch.bfloat16
        for kind in (dx_dtype, dw_dtype):
            if kind is not torch.bfloat16 and kind is not torch.float32:
                raise TypeError("gradients are bfloat16 or float32")
        two = (needs_dx and dx_dtype is torch.float32) or (needs_dw and dw_dtype is torch.float32)
        guard, st = _on(self.device, stream)
        with guard:
            at = targets.contiguous()
            p.targets = at.data_ptr()
            if needs_dx:
                if dx is None:
                    dx = torch.empty(n, cols, dtype=dx_dtype, device=self.device)
                g.dx, g.dx_stride, g.dx_type = dx.data_ptr(), dx.stride(0) if n > 1 else cols, _type(dx_dtype)
            if needs_dw:
                if dws is None:
                    dws = [torch.empty(shape, dtype=dw_dtype, device=self.device) for shape in self.shapes]
                g.dw_type = _type(dw_dtype)
            held = self._bytes.get((n, needs_dx, two))
            if held is None:
                sizes = df11_vocab_sizes(n, cols, self._rows, bool(needs_dx), two)
                held = self._bytes[n, needs_dx, two] = sizes, LIB.df11_vocab_loss_gradient_scratch_bytes(sizes)
            sizes, need = held
            scratch = torch.empty(need, dtype=torch.uint8, device=self.device)
            for k in self._each(p, status, st):
                if needs_dw:
                    dw = dws[k]
                    g.dw, g.dw_stride = dw.data_ptr(), dw.stride(0) if p.rows > 1 else cols
                _check("df11_vocab_loss_gradient",
                       LIB.df11_vocab_loss_gradient(p, g, sizes, scratch.data_ptr(), need, st))
        if given:
            torch._C._increment_version(given)
        if stream is not None or st not in self._lent:
            self._used(stream, st, used + ([dx] if needs_dx else []) + (dws if needs_dw else []) +
                       ([] if status is None else [status]))
        return dx if needs_dx else None, dws if needs_dw else None

    def _per_token(self, name, value, counts):
        """The address of a float32 tensor of one of these numbers of elements."""
        import torch

        if (value.dtype is not torch.float32 or value.device != self.device or not value.is_contiguous()
                or value.numel() not in counts):
            raise ValueError(f"{name} must be contiguous float32 on {self.device}, one for each token")
        return value.data_ptr()


def table_bytes(cb: df11_codebook) -> int:
    """df11_table_bytes(): multi-symbol, count and n_luts hierarchical tables."""
    return ctypes.sizeof(cb.multi) + ctypes.sizeof(cb.count) + 512 * int(cb.n_luts)


def table_image(cb: df11_codebook) -> np.ndarray:
    """The device copy of the codebook's tables (bytes from cb.multi onward)."""
    start = df11_codebook.multi.offset
    raw = ctypes.string_at(ctypes.addressof(cb) + start, table_bytes(cb))
    return np.frombuffer(raw, dtype=np.uint8).copy()


def codebook_arrays(cb: df11_codebook):
    """(code_len uint8[256], code uint32[256]) views of a codebook."""
    return (np.ctypeslib.as_array(cb.code_len).copy(), np.ctypeslib.as_array(cb.code).copy())
