"""Thin ctypes binding of libtrace_fp4.so (C ABI in include/trace_fp4.h).

Argument marshalling only: every step of the path runs in the library's
CUDA kernels.  Tensors must be CUDA tensors; bf16 data is passed by pointer
as raw 16-bit words.  Calls are asynchronous on the given stream (default:
torch's current stream).  If the library is missing or fails to load, the
first call raises -- there is no fallback of any kind.  The expert operators
make their usual call through csrc/binding.cpp, one native step; where that
module is missing they warn and make it from here, to the same kernels.

Method: rcap.io post "TRACE: Rollout-Guided Quantization-Aware Training for
FP4" -- rollout capture of the compact cache (1 mantissa bit + scales), the
guided QAT fake-quant forward and its straight-through backward.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import functools
import importlib.util
import os
import threading
import warnings

import torch

from . import _build

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtrace_fp4.so")
_lock = threading.Lock()
_lib = None

TRACE_OK = 0
TRACE_ERR_TIMEOUT = 6


class TraceError(RuntimeError):
    pass


def library() -> ctypes.CDLL:
    """Load libtrace_fp4.so (raises if it is missing: build it with
    ``python -c 'import __graft_entry__ as g; g.build()'``)."""
    global _lib
    lib = _lib
    if lib is not None:  # loaded: no lock on the per-call path
        return lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise TraceError(f"{LIB_PATH} is missing: the CUDA library has not been built")
        lib = ctypes.CDLL(LIB_PATH)
        P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        lib.trace_strerror.argtypes = [ctypes.c_int]
        lib.trace_strerror.restype = ctypes.c_char_p
        lib.trace_abi_version.argtypes = []
        lib.trace_abi_version.restype = ctypes.c_int
        lib.trace_capture_workspace_bytes.argtypes = [i64, i64, i32]
        lib.trace_capture_workspace_bytes.restype = sz
        lib.trace_capture.argtypes = [P, i64, i64, i32, P, P, P, P, P, P, sz, P]
        lib.trace_capture.restype = ctypes.c_int
        lib.trace_guided_fq_fwd.argtypes = [P, i64, i64, i32, P, P, P, P, P, P, P]
        lib.trace_guided_fq_fwd.restype = ctypes.c_int
        lib.trace_fq_bwd.argtypes = [P, P, i64, P, P]
        lib.trace_fq_bwd.restype = ctypes.c_int
        lib.trace_rtn_fq_fwd.argtypes = [P, i64, i64, i32, P, P, P, P, P, P]
        lib.trace_rtn_fq_fwd.restype = ctypes.c_int
        lib.trace_copy_bf16.argtypes = [P, P, i64, P]
        lib.trace_copy_bf16.restype = ctypes.c_int
        lib.trace_copy_bf16_staged.argtypes = [P, P, i64, P, P]
        lib.trace_copy_bf16_staged.restype = ctypes.c_int
        lib.trace_full_guided_fq_fwd.argtypes = [P, i64, i64, i32, P, P, P, P, P, P, P]
        lib.trace_full_guided_fq_fwd.restype = ctypes.c_int
        lib.trace_capture_static_ws.argtypes = [P, i64, i64, i32, P, P, P, P, P, P]
        lib.trace_capture_static_ws.restype = ctypes.c_int
        lib.trace_mismatch_histogram.argtypes = [P, i64, i64, i32, P, P, P, P, P, P]
        lib.trace_mismatch_histogram.restype = ctypes.c_int
        lib.trace_mx_mismatch_histogram.argtypes = [P, i64, i64, P, P, P, P]
        lib.trace_mx_mismatch_histogram.restype = ctypes.c_int
        lib.trace_cache_record_bytes.argtypes = [i64, i64, i32, P, P, P]
        lib.trace_cache_record_bytes.restype = sz
        lib.trace_mx_capture.argtypes = [P, i64, i64, P, P, P, P]
        lib.trace_mx_capture.restype = ctypes.c_int
        lib.trace_mx_guided_fq_fwd.argtypes = [P, i64, i64, P, P, P, P, P]
        lib.trace_mx_guided_fq_fwd.restype = ctypes.c_int
        lib.trace_mx_full_guided_fq_fwd.argtypes = [P, i64, i64, P, P, P, P, P]
        lib.trace_mx_full_guided_fq_fwd.restype = ctypes.c_int
        lib.trace_mx_rtn_fq_fwd.argtypes = [P, i64, i64, P, P, P, P]
        lib.trace_mx_rtn_fq_fwd.restype = ctypes.c_int
        lib.trace_scale_bytes.argtypes = [i64, i64, i32, i32]
        lib.trace_scale_bytes.restype = sz
        lib.trace_capture_ex.argtypes = [P, i64, i64, i32, P, P, P, P, P, P, sz, i32, P]
        lib.trace_capture_ex.restype = ctypes.c_int
        lib.trace_fq_fwd_ex.argtypes = [i32, P, i64, i64, i32, P, P, P, P, P, P, P, i32, P]
        lib.trace_fq_fwd_ex.restype = ctypes.c_int
        lib.trace_mx_capture_ex.argtypes = [P, i64, i64, P, P, P, i32, P]
        lib.trace_mx_capture_ex.restype = ctypes.c_int
        lib.trace_mx_fq_fwd_ex.argtypes = [i32, P, i64, i64, P, P, P, P, P, i32, P]
        lib.trace_mx_fq_fwd_ex.restype = ctypes.c_int
        lib.trace_capture_amax.argtypes = [P, i64, i64, i32, P, P, P]
        lib.trace_capture_amax.restype = ctypes.c_int
        lib.trace_mx8_capture.argtypes = [P, i64, i64, P, P, P, P]
        lib.trace_mx8_capture.restype = ctypes.c_int
        lib.trace_mx8_guided_fq_fwd.argtypes = [P, i64, i64, P, P, P, P, P]
        lib.trace_mx8_guided_fq_fwd.restype = ctypes.c_int
        lib.trace_mx8_full_guided_fq_fwd.argtypes = [P, i64, i64, P, P, P, P, P]
        lib.trace_mx8_full_guided_fq_fwd.restype = ctypes.c_int
        lib.trace_mx8_rtn_fq_fwd.argtypes = [P, i64, i64, P, P, P, P]
        lib.trace_mx8_rtn_fq_fwd.restype = ctypes.c_int
        lib.trace_validate_offsets.argtypes = [P, i32, i64, P, P]
        lib.trace_validate_offsets.restype = ctypes.c_int
        lib.trace_selftest_e4m3_sweep.argtypes = [ctypes.c_uint32, ctypes.c_uint32, P, P]
        lib.trace_selftest_e4m3_sweep.restype = ctypes.c_int
        lib.trace_mx8_capture_ex.argtypes = [P, i64, i64, P, P, P, i32, P]
        lib.trace_mx8_capture_ex.restype = ctypes.c_int
        lib.trace_mx8_fq_fwd_ex.argtypes = [i32, P, i64, i64, P, P, P, P, P, i32, P]
        lib.trace_mx8_fq_fwd_ex.restype = ctypes.c_int
        lib.trace_capture_amax_accumulate.argtypes = [P, i64, i64, i32, P, P, P]
        lib.trace_capture_amax_accumulate.restype = ctypes.c_int
        lib.trace_capture_with_amax.argtypes = [P, i64, i64, i32, P, P, P, P, P, P, i32, P]
        lib.trace_capture_with_amax.restype = ctypes.c_int
        lib.trace_moe_sort_workspace_bytes.argtypes = [i64, i64, i32]
        lib.trace_moe_sort_workspace_bytes.restype = sz
        lib.trace_moe_sort.argtypes = [P, i32, i64, i64, i32, P, P, P, P, sz, P]
        lib.trace_moe_sort.restype = ctypes.c_int
        lib.trace_moe_dispatch.argtypes = [P, i64, i64, i64, P, P, P, P]
        lib.trace_moe_dispatch.restype = ctypes.c_int
        lib.trace_moe_combine.argtypes = [P, i64, i64, i64, P, P, P, P]
        lib.trace_moe_combine.restype = ctypes.c_int
        lib.trace_moe_combine_bwd.argtypes = [P, P, i64, i64, i64, P, P, P, P, P, P]
        lib.trace_moe_combine_bwd.restype = ctypes.c_int
        lib.trace_fp4_matmul.argtypes = [P, P, P, i64, i64, i32, P, i32, P, P, P, i64, i32, i32,
                                         P, P]
        lib.trace_fp4_matmul.restype = ctypes.c_int
        lib.trace_mx_matmul.argtypes = [P, P, i64, i64, i32, P, i32, P, P, i64, i32, i32, P, P]
        lib.trace_mx_matmul.restype = ctypes.c_int
        lib.trace_fp4_matmul_ws.argtypes = [P, P, P, i64, i64, i32, P, i32, P, P, P, i64, i32, i32,
                                            P, P, sz, P]
        lib.trace_fp4_matmul_ws.restype = ctypes.c_int
        lib.trace_mx_matmul_ws.argtypes = [P, P, i64, i64, i32, P, i32, P, P, i64, i32, i32, P, P,
                                           sz, P]
        lib.trace_mx_matmul_ws.restype = ctypes.c_int
        for f in (lib.trace_fp4_matmul_workspace_bytes, lib.trace_mx_matmul_workspace_bytes):
            f.argtypes = [i64, i64, i32, i32, i64, i32, i32]
            f.restype = sz
        lib.trace_matmul_status.argtypes = [P]
        lib.trace_matmul_status.restype = ctypes.c_int
        lib.trace_capture_status.argtypes = [P, P]
        lib.trace_capture_status.restype = ctypes.c_int
        _lib = lib
        return lib


def _check(status: int, what: str) -> None:
    if status != TRACE_OK:
        msg = library().trace_strerror(status).decode()
        raise TraceError(f"{what}: status {status} ({msg})")


def _p(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise TraceError("tensors passed to libtrace_fp4 must be CUDA tensors")
    if not t.is_contiguous():
        raise TraceError("tensors passed to libtrace_fp4 must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if type(stream) is int:
        return stream
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


DEBUG = os.environ.get("TRACE_DEBUG", "0") not in ("", "0")


def validate_offsets(offsets: torch.Tensor, rows: int, stream=None) -> int:
    """0 when the device offsets are valid for `rows` rows, else 1 + the
    first offending index (synchronises the stream)."""
    flag = torch.empty(1, dtype=torch.int32, device=offsets.device)
    _check(library().trace_validate_offsets(_p(offsets), int(offsets.numel()) - 1, rows, _p(flag),
                                            _stream(stream)), "trace_validate_offsets")
    return int(flag.item())


def _groups(offsets: torch.Tensor | None, rows: int | None = None) -> int:
    if offsets is None:
        return 1
    if offsets.dtype != torch.int64:
        raise TraceError("group offsets must be int64")
    if DEBUG and rows is not None:   # TRACE_DEBUG=1: check the device offsets first
        bad = validate_offsets(offsets, rows)
        if bad:
            raise TraceError(f"group offsets invalid at entry {bad - 1}")
    return int(offsets.numel()) - 1


# ---------------------------------------------------------------------------
# Raw C-ABI calls, same names and argument order as include/trace_fp4.h
# ---------------------------------------------------------------------------

def trace_capture_workspace_bytes(rows: int, cols: int, num_groups: int) -> int:
    return int(library().trace_capture_workspace_bytes(rows, cols, num_groups))


def trace_cache_record_bytes(rows: int, cols: int, num_groups: int) -> tuple[int, int, int, int]:
    """(record bytes, mbits offset, scales offset, gscale offset); record
    bytes is 0 for an invalid shape."""
    om, os_, og = ctypes.c_size_t(0), ctypes.c_size_t(0), ctypes.c_size_t(0)
    nb = library().trace_cache_record_bytes(rows, cols, num_groups, ctypes.byref(om),
                                            ctypes.byref(os_), ctypes.byref(og))
    return int(nb), om.value, os_.value, og.value


def trace_capture(x, rows, cols, num_groups, offsets, codes, mbits, scales, gscale,
                  workspace, workspace_bytes, stream=None) -> None:
    _check(library().trace_capture(_p(x), rows, cols, num_groups, _p(offsets), _p(codes),
                                   _p(mbits), _p(scales), _p(gscale), _p(workspace),
                                   workspace_bytes, _stream(stream)), "trace_capture")


def trace_guided_fq_fwd(x_train, rows, cols, num_groups, offsets, mbits, scales, gscale,
                        out, ste_mask, stream=None) -> None:
    _check(library().trace_guided_fq_fwd(_p(x_train), rows, cols, num_groups, _p(offsets),
                                         _p(mbits), _p(scales), _p(gscale), _p(out),
                                         _p(ste_mask), _stream(stream)), "trace_guided_fq_fwd")


def trace_full_guided_fq_fwd(x_train, rows, cols, num_groups, offsets, codes, scales, gscale,
                             out, ste_mask, stream=None) -> None:
    _check(library().trace_full_guided_fq_fwd(_p(x_train), rows, cols, num_groups, _p(offsets),
                                              _p(codes), _p(scales), _p(gscale), _p(out),
                                              _p(ste_mask), _stream(stream)),
           "trace_full_guided_fq_fwd")


def trace_fq_bwd(grad_out, ste_mask, numel, grad_in, stream=None) -> None:
    _check(library().trace_fq_bwd(_p(grad_out), _p(ste_mask), numel, _p(grad_in),
                                  _stream(stream)), "trace_fq_bwd")


def trace_rtn_fq_fwd(x, rows, cols, num_groups, offsets, scales, gscale, out, ste_mask,
                     stream=None) -> None:
    _check(library().trace_rtn_fq_fwd(_p(x), rows, cols, num_groups, _p(offsets), _p(scales),
                                      _p(gscale), _p(out), _p(ste_mask), _stream(stream)),
           "trace_rtn_fq_fwd")


def trace_capture_static_ws(x, rows, cols, num_groups, offsets, codes, mbits, scales, gscale,
                            stream=None) -> None:
    """trace_capture for callers that cannot supply a workspace: the library
    keeps the scratch in a fixed per-GPU array (at most
    TRACE_STATIC_MAX_GROUPS groups; calls must not overlap on the GPU)."""
    _check(library().trace_capture_static_ws(_p(x), rows, cols, num_groups, _p(offsets),
                                             _p(codes), _p(mbits), _p(scales), _p(gscale),
                                             _stream(stream)), "trace_capture_static_ws")


TRACE_STATIC_MAX_GROUPS = 4096


def trace_mismatch_histogram(x_train, rows, cols, num_groups, offsets, codes, scales, gscale,
                             hist, stream=None) -> None:
    _check(library().trace_mismatch_histogram(_p(x_train), rows, cols, num_groups, _p(offsets),
                                              _p(codes), _p(scales), _p(gscale), _p(hist),
                                              _stream(stream)), "trace_mismatch_histogram")


def trace_selftest_e4m3_sweep(first_bits: int, count: int, out, stream=None) -> None:
    _check(library().trace_selftest_e4m3_sweep(first_bits, count, _p(out), _stream(stream)),
           "trace_selftest_e4m3_sweep")


def trace_copy_bf16(src, dst, numel, stream=None) -> None:
    _check(library().trace_copy_bf16(_p(src), _p(dst), numel, _stream(stream)), "trace_copy_bf16")


def trace_copy_bf16_staged(src, dst, numel, err, stream=None) -> None:
    _check(library().trace_copy_bf16_staged(_p(src), _p(dst), numel, _p(err), _stream(stream)),
           "trace_copy_bf16_staged")


# ---------------------------------------------------------------------------
# Convenience wrappers that allocate their outputs (still no arithmetic here)
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class Capture:
    """What one capture site records: the rollout's full FP4 codes (for its
    own FP4 GEMM) and the compact cache (mbits + scales + gscale)."""
    codes: torch.Tensor    # uint8 [N/2]
    mbits: torch.Tensor    # int32 words [N/32] (bit patterns; uint32 ABI)
    scales: torch.Tensor   # uint8 [rows, cols/16] E4M3
    gscale: torch.Tensor   # float32 [G]
    offsets: torch.Tensor | None = None

    def cache_nbytes(self) -> int:
        """Bytes of the compact cache (mantissa bits + block and global scales)."""
        return self.mbits.numel() * 4 + self.scales.numel() + self.gscale.numel() * 4


def _bf16_2d(x: torch.Tensor) -> tuple[int, int]:
    if x.dtype != torch.bfloat16:
        raise TraceError("activations must be bf16")
    if x.dim() != 2:
        raise TraceError("activations must be 2-D [rows, cols]")
    return int(x.shape[0]), int(x.shape[1])


def alloc_capture(rows: int, cols: int, num_groups: int = 1, device="cuda",
                  offsets: torch.Tensor | None = None) -> tuple[Capture, torch.Tensor]:
    """Allocate capture outputs and the workspace (torch device memory)."""
    n = rows * cols
    cap = Capture(codes=torch.empty(n // 2, dtype=torch.uint8, device=device),
                  mbits=torch.empty(n // 32, dtype=torch.int32, device=device),
                  scales=torch.empty(rows, cols // 16, dtype=torch.uint8, device=device),
                  gscale=torch.empty(num_groups, dtype=torch.float32, device=device),
                  offsets=offsets)
    # zeros before its first use; every capture leaves it zeroed again
    ws = torch.zeros(max(trace_capture_workspace_bytes(rows, cols, num_groups), 256),
                     dtype=torch.uint8, device=device)
    return cap, ws


def capture(x: torch.Tensor, offsets: torch.Tensor | None = None, out: Capture | None = None,
            workspace: torch.Tensor | None = None, stream=None) -> Capture:
    """Rollout capture of one site (x bf16 [rows, cols]; offsets int64 [G+1])."""
    rows, cols = _bf16_2d(x)
    G = _groups(offsets, rows)
    if out is None or workspace is None:
        out, workspace = alloc_capture(rows, cols, G, x.device, offsets)
    trace_capture(x, rows, cols, G, offsets, out.codes, out.mbits, out.scales, out.gscale,
                  workspace, workspace.numel(), stream)
    return out


def capture_status(workspace: torch.Tensor, stream=None) -> bool:
    """True when no capture that used `workspace` has given up waiting at
    its grid barrier since the last check (trace_capture_status: waits for
    the stream, reads and clears the workspace's error word)."""
    st = library().trace_capture_status(_p(workspace), _stream(stream))
    if st == TRACE_ERR_TIMEOUT:
        return False
    _check(st, "trace_capture_status")
    return True

def guided_fq_fwd(x_train: torch.Tensor, cache: Capture, out: torch.Tensor | None = None,
                  mask: torch.Tensor | None = None, stream=None):
    """Guided fake-quant forward with a rollout cache.  Returns (out, mask)."""
    rows, cols = _bf16_2d(x_train)
    out = torch.empty_like(x_train) if out is None else out
    mask = torch.empty(rows * cols // 32, dtype=torch.int32, device=x_train.device) if mask is None else mask
    trace_guided_fq_fwd(x_train, rows, cols, _groups(cache.offsets), cache.offsets, cache.mbits,
                        cache.scales, cache.gscale, out, mask, stream)
    return out, mask


def full_guided_fq_fwd(x_train: torch.Tensor, cache: Capture, out: torch.Tensor | None = None,
                       mask: torch.Tensor | None = None, stream=None):
    """Full-information guided forward (the cache keeps the rollout's whole
    codes).  Returns (out, mask)."""
    rows, cols = _bf16_2d(x_train)
    out = torch.empty_like(x_train) if out is None else out
    mask = torch.empty(rows * cols // 32, dtype=torch.int32, device=x_train.device) if mask is None else mask
    trace_full_guided_fq_fwd(x_train, rows, cols, _groups(cache.offsets), cache.offsets, cache.codes,
                             cache.scales, cache.gscale, out, mask, stream)
    return out, mask


def rtn_fq_fwd(x: torch.Tensor, scales: torch.Tensor, gscale: torch.Tensor,
               offsets: torch.Tensor | None = None, out: torch.Tensor | None = None,
               mask: torch.Tensor | None = None, stream=None):
    """Round-to-nearest fake-quant with given scales.  Returns (out, mask)."""
    rows, cols = _bf16_2d(x)
    out = torch.empty_like(x) if out is None else out
    mask = torch.empty(rows * cols // 32, dtype=torch.int32, device=x.device) if mask is None else mask
    trace_rtn_fq_fwd(x, rows, cols, _groups(offsets), offsets, scales, gscale, out, mask, stream)
    return out, mask


def fq_bwd(grad_out: torch.Tensor, mask: torch.Tensor, out: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """Masked straight-through backward."""
    if grad_out.dtype != torch.bfloat16:
        raise TraceError("gradients must be bf16")
    out = torch.empty_like(grad_out) if out is None else out
    trace_fq_bwd(grad_out, mask, grad_out.numel(), out, stream)
    return out


def trace_mx_capture(x, rows, cols, codes, mbits, scales, stream=None) -> None:
    _check(library().trace_mx_capture(_p(x), rows, cols, _p(codes), _p(mbits), _p(scales),
                                      _stream(stream)), "trace_mx_capture")


def trace_mx_guided_fq_fwd(x_train, rows, cols, mbits, scales, out, ste_mask, stream=None) -> None:
    _check(library().trace_mx_guided_fq_fwd(_p(x_train), rows, cols, _p(mbits), _p(scales),
                                            _p(out), _p(ste_mask), _stream(stream)),
           "trace_mx_guided_fq_fwd")


def trace_mx_full_guided_fq_fwd(x_train, rows, cols, codes, scales, out, ste_mask,
                                stream=None) -> None:
    _check(library().trace_mx_full_guided_fq_fwd(_p(x_train), rows, cols, _p(codes), _p(scales),
                                                 _p(out), _p(ste_mask), _stream(stream)),
           "trace_mx_full_guided_fq_fwd")


def trace_mx_rtn_fq_fwd(x, rows, cols, scales, out, ste_mask, stream=None) -> None:
    _check(library().trace_mx_rtn_fq_fwd(_p(x), rows, cols, _p(scales), _p(out), _p(ste_mask),
                                         _stream(stream)), "trace_mx_rtn_fq_fwd")


@dataclasses.dataclass
class MxCapture:
    """One MXFP4 capture site: full codes plus the compact cache (mantissa
    bits + E8M0 block scales, 1.25 bits per element)."""
    codes: torch.Tensor    # uint8 [N/2]
    mbits: torch.Tensor    # int32 words [N/32]
    scales: torch.Tensor   # uint8 [rows, cols/32] E8M0

    def cache_nbytes(self) -> int:
        return self.mbits.numel() * 4 + self.scales.numel()


def mx_capture(x: torch.Tensor, out: MxCapture | None = None, stream=None) -> MxCapture:
    """MXFP4 rollout capture of one site (x bf16 [rows, cols])."""
    rows, cols = _bf16_2d(x)
    n = rows * cols
    if out is None:
        out = MxCapture(codes=torch.empty(n // 2, dtype=torch.uint8, device=x.device),
                        mbits=torch.empty(n // 32, dtype=torch.int32, device=x.device),
                        scales=torch.empty(rows, cols // 32, dtype=torch.uint8, device=x.device))
    trace_mx_capture(x, rows, cols, out.codes, out.mbits, out.scales, stream)
    return out


def _fq_outputs(x, out, mask):
    rows, cols = _bf16_2d(x)
    out = torch.empty_like(x) if out is None else out
    mask = torch.empty(rows * cols // 32, dtype=torch.int32, device=x.device) if mask is None else mask
    return rows, cols, out, mask


def mx_guided_fq_fwd(x_train: torch.Tensor, cache: MxCapture, out=None, mask=None, stream=None):
    """MXFP4 1-bit guided forward.  Returns (out, mask)."""
    rows, cols, out, mask = _fq_outputs(x_train, out, mask)
    trace_mx_guided_fq_fwd(x_train, rows, cols, cache.mbits, cache.scales, out, mask, stream)
    return out, mask


def mx_full_guided_fq_fwd(x_train: torch.Tensor, cache: MxCapture, out=None, mask=None,
                          stream=None):
    """MXFP4 full-information guided forward.  Returns (out, mask)."""
    rows, cols, out, mask = _fq_outputs(x_train, out, mask)
    trace_mx_full_guided_fq_fwd(x_train, rows, cols, cache.codes, cache.scales, out, mask, stream)
    return out, mask


def mx_rtn_fq_fwd(x: torch.Tensor, scales: torch.Tensor, out=None, mask=None, stream=None):
    """MXFP4 round-to-nearest fake-quant with given E8M0 scales."""
    rows, cols, out, mask = _fq_outputs(x, out, mask)
    trace_mx_rtn_fq_fwd(x, rows, cols, scales, out, mask, stream)
    return out, mask


def trace_mx8_capture(x, rows, cols, codes, mbits, scales, stream=None) -> None:
    _check(library().trace_mx8_capture(_p(x), rows, cols, _p(codes), _p(mbits), _p(scales),
                                       _stream(stream)), "trace_mx8_capture")


def trace_mx8_guided_fq_fwd(x_train, rows, cols, mbits, scales, out, ste_mask, stream=None) -> None:
    _check(library().trace_mx8_guided_fq_fwd(_p(x_train), rows, cols, _p(mbits), _p(scales),
                                             _p(out), _p(ste_mask), _stream(stream)),
           "trace_mx8_guided_fq_fwd")


def trace_mx8_full_guided_fq_fwd(x_train, rows, cols, codes, scales, out, ste_mask,
                                 stream=None) -> None:
    _check(library().trace_mx8_full_guided_fq_fwd(_p(x_train), rows, cols, _p(codes), _p(scales),
                                                  _p(out), _p(ste_mask), _stream(stream)),
           "trace_mx8_full_guided_fq_fwd")


def trace_mx8_rtn_fq_fwd(x, rows, cols, scales, out, ste_mask, stream=None) -> None:
    _check(library().trace_mx8_rtn_fq_fwd(_p(x), rows, cols, _p(scales), _p(out), _p(ste_mask),
                                          _stream(stream)), "trace_mx8_rtn_fq_fwd")


def mx8_capture(x: torch.Tensor, out: MxCapture | None = None, stream=None) -> MxCapture:
    """W4A8 rollout capture (E4M3 activations, MX scales): codes are one
    byte per element."""
    rows, cols = _bf16_2d(x)
    n = rows * cols
    if out is None:
        out = MxCapture(codes=torch.empty(n, dtype=torch.uint8, device=x.device),
                        mbits=torch.empty(n // 32, dtype=torch.int32, device=x.device),
                        scales=torch.empty(rows, cols // 32, dtype=torch.uint8, device=x.device))
    trace_mx8_capture(x, rows, cols, out.codes, out.mbits, out.scales, stream)
    return out


def mx8_guided_fq_fwd(x_train: torch.Tensor, cache: MxCapture, out=None, mask=None, stream=None):
    rows, cols, out, mask = _fq_outputs(x_train, out, mask)
    trace_mx8_guided_fq_fwd(x_train, rows, cols, cache.mbits, cache.scales, out, mask, stream)
    return out, mask


def mx8_full_guided_fq_fwd(x_train: torch.Tensor, cache: MxCapture, out=None, mask=None,
                           stream=None):
    rows, cols, out, mask = _fq_outputs(x_train, out, mask)
    trace_mx8_full_guided_fq_fwd(x_train, rows, cols, cache.codes, cache.scales, out, mask, stream)
    return out, mask


def mx8_rtn_fq_fwd(x: torch.Tensor, scales: torch.Tensor, out=None, mask=None, stream=None):
    rows, cols, out, mask = _fq_outputs(x, out, mask)
    trace_mx8_rtn_fq_fwd(x, rows, cols, scales, out, mask, stream)
    return out, mask


# scale layouts and rounding rules of the _ex calls
TRACE_SCALES_ROW_MAJOR, TRACE_SCALES_TILED_128x4 = 0, 1
TRACE_RULE_RTN, TRACE_RULE_GUIDED, TRACE_RULE_FULL = 0, 1, 2


def trace_scale_bytes(rows: int, cols: int, block_size: int, scale_layout: int) -> int:
    return int(library().trace_scale_bytes(rows, cols, block_size, scale_layout))


def trace_capture_ex(x, rows, cols, num_groups, offsets, codes, mbits, scales, gscale, workspace,
                     workspace_bytes, scale_layout, stream=None) -> None:
    _check(library().trace_capture_ex(_p(x), rows, cols, num_groups, _p(offsets), _p(codes),
                                      _p(mbits), _p(scales), _p(gscale), _p(workspace),
                                      workspace_bytes, scale_layout, _stream(stream)),
           "trace_capture_ex")


def trace_fq_fwd_ex(rule, x_train, rows, cols, num_groups, offsets, mbits, codes, scales, gscale,
                    out, ste_mask, scale_layout, stream=None) -> None:
    _check(library().trace_fq_fwd_ex(rule, _p(x_train), rows, cols, num_groups, _p(offsets),
                                     _p(mbits), _p(codes), _p(scales), _p(gscale), _p(out),
                                     _p(ste_mask), scale_layout, _stream(stream)), "trace_fq_fwd_ex")


def trace_mx_capture_ex(x, rows, cols, codes, mbits, scales, scale_layout, stream=None) -> None:
    _check(library().trace_mx_capture_ex(_p(x), rows, cols, _p(codes), _p(mbits), _p(scales),
                                         scale_layout, _stream(stream)), "trace_mx_capture_ex")


def trace_mx_fq_fwd_ex(rule, x_train, rows, cols, mbits, codes, scales, out, ste_mask,
                       scale_layout, stream=None) -> None:
    _check(library().trace_mx_fq_fwd_ex(rule, _p(x_train), rows, cols, _p(mbits), _p(codes),
                                        _p(scales), _p(out), _p(ste_mask), scale_layout,
                                        _stream(stream)), "trace_mx_fq_fwd_ex")


def capture_tiled(x: torch.Tensor, offsets: torch.Tensor | None = None, stream=None) -> Capture:
    """NVFP4 capture with the scales in the 128 x 4 tiled layout of a
    block-scaled FP4 GEMM (Capture.scales is then a flat uint8 tensor of
    trace_scale_bytes(...) bytes, padding zeroed)."""
    rows, cols = _bf16_2d(x)
    G = _groups(offsets)
    cap, ws = alloc_capture(rows, cols, G, x.device, offsets)
    cap.scales = torch.zeros(trace_scale_bytes(rows, cols, 16, TRACE_SCALES_TILED_128x4),
                             dtype=torch.uint8, device=x.device)
    trace_capture_ex(x, rows, cols, G, offsets, cap.codes, cap.mbits, cap.scales, cap.gscale, ws,
                     ws.numel(), TRACE_SCALES_TILED_128x4, stream)
    return cap


def fq_fwd_tiled(rule: int, x_train: torch.Tensor, cache: Capture, out=None, mask=None,
                 stream=None):
    """NVFP4 forward (rule TRACE_RULE_*) reading tiled scales.  Returns (out, mask)."""
    rows, cols, out, mask = _fq_outputs(x_train, out, mask)
    trace_fq_fwd_ex(rule, x_train, rows, cols, _groups(cache.offsets), cache.offsets, cache.mbits,
                    cache.codes, cache.scales, cache.gscale, out, mask, TRACE_SCALES_TILED_128x4,
                    stream)
    return out, mask


def mx_capture_tiled(x: torch.Tensor, stream=None) -> MxCapture:
    """MXFP4 capture with the E8M0 scales in the 128 x 4 tiled layout."""
    rows, cols = _bf16_2d(x)
    n = rows * cols
    cap = MxCapture(codes=torch.empty(n // 2, dtype=torch.uint8, device=x.device),
                    mbits=torch.empty(n // 32, dtype=torch.int32, device=x.device),
                    scales=torch.zeros(trace_scale_bytes(rows, cols, 32, TRACE_SCALES_TILED_128x4),
                                       dtype=torch.uint8, device=x.device))
    trace_mx_capture_ex(x, rows, cols, cap.codes, cap.mbits, cap.scales, TRACE_SCALES_TILED_128x4,
                        stream)
    return cap


def mx_fq_fwd_tiled(rule: int, x_train: torch.Tensor, cache: MxCapture, out=None, mask=None,
                    stream=None):
    """MXFP4 forward (rule TRACE_RULE_*) reading tiled scales."""
    rows, cols, out, mask = _fq_outputs(x_train, out, mask)
    trace_mx_fq_fwd_ex(rule, x_train, rows, cols, cache.mbits, cache.codes, cache.scales, out,
                       mask, TRACE_SCALES_TILED_128x4, stream)
    return out, mask


def trace_capture_amax(x, rows, cols, num_groups, offsets, amax, stream=None) -> None:
    _check(library().trace_capture_amax(_p(x), rows, cols, num_groups, _p(offsets), _p(amax),
                                        _stream(stream)), "trace_capture_amax")


def trace_capture_amax_accumulate(x, rows, cols, num_groups, offsets, amax, stream=None) -> None:
    _check(library().trace_capture_amax_accumulate(_p(x), rows, cols, num_groups, _p(offsets),
                                                   _p(amax), _stream(stream)),
           "trace_capture_amax_accumulate")


def trace_capture_with_amax(x, rows, cols, num_groups, offsets, amax, codes, mbits, scales,
                            gscale, scale_layout=0, stream=None) -> None:
    _check(library().trace_capture_with_amax(_p(x), rows, cols, num_groups, _p(offsets), _p(amax),
                                             _p(codes), _p(mbits), _p(scales), _p(gscale),
                                             scale_layout, _stream(stream)),
           "trace_capture_with_amax")


def capture_sharded(x: torch.Tensor, offsets: torch.Tensor | None = None, group=None,
                    stream=None) -> Capture:
    """Capture of this rank's row shard of a tensor whose rows are spread
    over the ranks of `group` (torch.distributed; None = no reduction): the
    per-group amax is all-reduced (MAX) between the two passes, so every
    rank ends with the global scales of the whole tensor.  The one
    collective moves 4 bytes per group."""
    rows, cols = _bf16_2d(x)
    G = _groups(offsets)
    cap, _ = alloc_capture(rows, cols, G, x.device, offsets)
    amax = torch.empty(G, dtype=torch.int32, device=x.device)
    trace_capture_amax(x, rows, cols, G, offsets, amax, stream)
    if group is not None:
        import torch.distributed as dist
        s = torch.cuda.current_stream(x.device) if stream is None else stream
        with torch.cuda.stream(s):
            dist.all_reduce(amax, op=dist.ReduceOp.MAX, group=group)
    trace_capture_with_amax(x, rows, cols, G, offsets, amax, cap.codes, cap.mbits, cap.scales,
                            cap.gscale, TRACE_SCALES_ROW_MAJOR, stream)
    return cap


def mx8_capture_tiled(x: torch.Tensor, stream=None) -> MxCapture:
    """W4A8 capture with the E8M0 scales in the 128 x 4 tiled layout."""
    rows, cols = _bf16_2d(x)
    n = rows * cols
    cap = MxCapture(codes=torch.empty(n, dtype=torch.uint8, device=x.device),
                    mbits=torch.empty(n // 32, dtype=torch.int32, device=x.device),
                    scales=torch.zeros(trace_scale_bytes(rows, cols, 32, TRACE_SCALES_TILED_128x4),
                                       dtype=torch.uint8, device=x.device))
    _check(library().trace_mx8_capture_ex(_p(x), rows, cols, _p(cap.codes), _p(cap.mbits),
                                          _p(cap.scales), TRACE_SCALES_TILED_128x4,
                                          _stream(stream)), "trace_mx8_capture_ex")
    return cap


def mx8_fq_fwd_tiled(rule: int, x_train: torch.Tensor, cache: MxCapture, out=None, mask=None,
                     stream=None):
    """W4A8 forward (rule TRACE_RULE_*) reading tiled scales."""
    rows, cols, out, mask = _fq_outputs(x_train, out, mask)
    _check(library().trace_mx8_fq_fwd_ex(rule, _p(x_train), rows, cols, _p(cache.mbits),
                                         _p(cache.codes), _p(cache.scales), _p(out), _p(mask),
                                         TRACE_SCALES_TILED_128x4, _stream(stream)),
           "trace_mx8_fq_fwd_ex")
    return out, mask


MISMATCH_RULES = ("rtn", "guided_1bit", "full_guided")
MISMATCH_BINS = 15


def mismatch_histogram(x_train: torch.Tensor, cache: Capture, hist: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """Add the ladder-distance counts of x_train against the rollout cache
    into hist (int64 [3, 15], the uint64 counts' bits; zeros if None).  Row k
    is the rule MISMATCH_RULES[k]; column d counts the elements d codewords
    from the rollout's code."""
    rows, cols = _bf16_2d(x_train)
    if hist is None:
        hist = torch.zeros(len(MISMATCH_RULES), MISMATCH_BINS, dtype=torch.int64,
                           device=x_train.device)
    trace_mismatch_histogram(x_train, rows, cols, _groups(cache.offsets), cache.offsets,
                             cache.codes, cache.scales, cache.gscale, hist, stream)
    return hist


_FORWARDS = {
    ("nvfp4", "guided"): lambda x, c: guided_fq_fwd(x, c),
    ("nvfp4", "full"): lambda x, c: full_guided_fq_fwd(x, c),
    ("nvfp4", "rtn"): lambda x, c: rtn_fq_fwd(x, c.scales, c.gscale, c.offsets),
    ("mxfp4", "guided"): lambda x, c: mx_guided_fq_fwd(x, c),
    ("mxfp4", "full"): lambda x, c: mx_full_guided_fq_fwd(x, c),
    ("mxfp4", "rtn"): lambda x, c: mx_rtn_fq_fwd(x, c.scales),
    ("w4a8", "guided"): lambda x, c: mx8_guided_fq_fwd(x, c),
    ("w4a8", "full"): lambda x, c: mx8_full_guided_fq_fwd(x, c),
    ("w4a8", "rtn"): lambda x, c: mx8_rtn_fq_fwd(x, c.scales),
}


def mx_mismatch_histogram(x_train: torch.Tensor, cache: MxCapture,
                          hist: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """mismatch_histogram for the MXFP4 variant (E8M0 scales)."""
    rows, cols = _bf16_2d(x_train)
    if hist is None:
        hist = torch.zeros(len(MISMATCH_RULES), MISMATCH_BINS, dtype=torch.int64,
                           device=x_train.device)
    _check(library().trace_mx_mismatch_histogram(_p(x_train), rows, cols, _p(cache.codes),
                                                 _p(cache.scales), _p(hist), _stream(stream)),
           "trace_mx_mismatch_histogram")
    return hist


class TraceFakeQuant(torch.autograd.Function):
    """Autograd wrapper: forward = the fake-quant forward of `fmt` ("nvfp4",
    "mxfp4", "w4a8") with `rule` ("guided": the 1-bit cache, "full": the
    whole rollout codes, "rtn": round to nearest with the rollout's scales)
    against a rollout capture of that format; backward = the masked
    straight-through estimator.  Both run in the library."""

    @staticmethod
    def forward(ctx, x_train, cache, fmt="nvfp4", rule="guided"):
        fwd = _FORWARDS.get((fmt, rule))
        if fwd is None:
            raise TraceError(f"unknown format / rule {fmt!r} / {rule!r}")
        out, mask = fwd(x_train, cache)
        ctx.save_for_backward(mask)
        return out

    @staticmethod
    def backward(ctx, grad):
        (mask,) = ctx.saved_tensors
        return fq_bwd(grad.contiguous(), mask), None, None, None


def trace_fake_quant(x_train: torch.Tensor, cache, fmt: str = "nvfp4", rule: str = "guided"):
    """Differentiable fake-quant of x_train guided by a rollout capture."""
    return TraceFakeQuant.apply(x_train, cache, fmt, rule)


class GuidedFakeQuant(torch.autograd.Function):
    """NVFP4 1-bit guided forward with the masked straight-through backward
    (the common case of TraceFakeQuant)."""

    @staticmethod
    def forward(ctx, x_train, cache: Capture):
        out, mask = guided_fq_fwd(x_train, cache)
        ctx.save_for_backward(mask)
        return out

    @staticmethod
    def backward(ctx, grad):
        (mask,) = ctx.saved_tensors
        return fq_bwd(grad.contiguous(), mask), None


# ---------------------------------------------------------------------------
# FP4 experts: the routing sort, tokens into expert order and back, and the
# product of captured operands
# ---------------------------------------------------------------------------

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


_bind = None


def binding():
    """The module that makes the usual call of an expert operator in one native
    step (csrc/binding.cpp); each of its functions returns None for any other
    call.  Raises if it has not been built for this torch and Python."""
    global _bind
    if _bind is None or _bind is _NoBinding:
        lib = library()
        with _lock:
            path = _build.binding_path()
            if not os.path.exists(path):
                raise TraceError(f"{path} is missing: it has not been built for this torch")
            name = f"{__package__}._binding"
            spec = importlib.util.spec_from_file_location(name, path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.setup(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                lib.trace_moe_sort, lib.trace_moe_sort_workspace_bytes, lib.trace_moe_dispatch,
                lib.trace_moe_combine, lib.trace_moe_combine_bwd, lib.trace_fp4_matmul,
                lib.trace_mx_matmul, lib.trace_fp4_matmul_workspace_bytes, lib.trace_mx_matmul_workspace_bytes)))
            _bind = module
    return _bind


class _NoBinding:
    """Answers None to every call, as the module does to an unusual one: without
    it ops.py goes its own way to the same kernels, which takes the host longer."""

    @staticmethod
    def matmul(*args):
        return None

    sort = dispatch = combine = matmul


def _native():
    """The module, or, with a warning, what stands in for it on a machine where it
    has not been built (no g++ or Python headers) or does not load."""
    global _bind
    try:
        return binding()
    except (TraceError, ImportError, OSError) as e:
        library()  # without the library there is no other way
        warnings.warn(f"expert operators take longer to call: {e}", RuntimeWarning, stacklevel=3)
        _bind = _NoBinding
        return _bind


class _On:
    """Work on the tensors' own device and on `stream` (default: that
    device's current stream), so that outputs are allocated there too; gives
    the stream's handle.  Nothing is switched in the common case, where the
    device is current and the stream is its own."""
    __slots__ = ("index", "stream", "undo")

    def __init__(self, stream, *tensors):
        index = tensors[0].get_device()
        for t in tensors:
            if t is not None and t.get_device() != index:
                raise TraceError(f"tensors on different devices: {tensors[0].device} and {t.device}")
        if index < 0:
            raise TraceError("tensors passed to libtrace_fp4 must be CUDA tensors")
        self.index, self.stream, self.undo = index, stream, None

    def __enter__(self) -> int:
        stream, index = self.stream, self.index
        if stream is None and index == _current_device():
            return _raw_stream(index)
        self.undo = contextlib.ExitStack()
        self.undo.enter_context(torch.cuda.device(index))
        if stream is None:
            return _raw_stream(index)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=index)
        self.undo.enter_context(torch.cuda.stream(stream))
        return stream.cuda_stream

    def __exit__(self, *exc):
        if self.undo is not None:
            self.undo.close()
        return False


def _ptrs(*tensors):
    """Addresses for the library (0: none); the devices are checked by _On."""
    for t in tensors:
        if t is not None and not t.is_contiguous():
            raise TraceError("tensors passed to libtrace_fp4 must be contiguous")
    return [0 if t is None else t.data_ptr() for t in tensors]


def _written(*outputs) -> None:
    """Tells autograd of what the library has written into the caller's own
    tensors: a backward pass that still needs what they held is then refused."""
    for t in outputs:
        if not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _want(t: torch.Tensor, what: str, dtype, shape=None) -> None:
    if t.dtype is not dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TraceError(f"{what}: unexpected dtype {t.dtype}")
    if shape is not None and t.shape != shape:
        raise TraceError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")


@functools.lru_cache(maxsize=256)
def trace_moe_sort_workspace_bytes(tokens: int, k: int, num_experts: int) -> int:
    return int(library().trace_moe_sort_workspace_bytes(tokens, k, num_experts))


@dataclasses.dataclass
class MoeRoute:
    """Where a batch's slots (token, choice) go: what moe_sort writes.
    `offsets` groups the rows for capture: one group per expert and a last
    one of the dropped slots (zero rows after dispatch)."""
    offsets: torch.Tensor  # int64 [experts + 2]
    rows: torch.Tensor     # int32 [tokens, k]: the slot's row, -1 if dropped
    slots: torch.Tensor    # int32 [tokens * k]: the row's slot, -1 in the last group


def moe_sort(expert_ids: torch.Tensor, num_experts: int, out: MoeRoute | None = None,
             workspace: torch.Tensor | None = None, stream=None) -> MoeRoute:
    """Stable sort of the slots of expert_ids (int32 / int64 [tokens, k]) by
    expert; ids outside [0, num_experts) drop their slot."""
    if out is None and workspace is None and stream is None:
        got = (_bind or _native()).sort(expert_ids, num_experts)
        if got is not None:
            return MoeRoute(*got)
    if expert_ids.dim() != 2 or expert_ids.shape[1] < 1:
        raise TraceError("expert ids must be [tokens, k]")
    _want(expert_ids, "expert ids", (torch.int32, torch.int64))
    tokens, k = expert_ids.shape
    lib = library()
    nbytes = trace_moe_sort_workspace_bytes(tokens, k, num_experts)
    if nbytes == 0:
        raise TraceError(f"moe_sort: {num_experts} experts for [{tokens}, {k}] ids")
    with _On(stream, expert_ids, workspace) as s:
        given = out is not None
        if not given:
            new = lambda *shape: expert_ids.new_empty(shape, dtype=torch.int32)  # noqa: E731
            out = MoeRoute(expert_ids.new_empty(num_experts + 2, dtype=torch.int64), new(tokens, k),
                           new(tokens * k))
        else:
            _want(out.offsets, "offsets", torch.int64, (num_experts + 2,))
            _want(out.rows, "rows", torch.int32, (tokens, k))
            _want(out.slots, "slots", torch.int32, (tokens * k,))
            _On(None, expert_ids, out.offsets, out.rows, out.slots)
        if workspace is None:
            workspace = expert_ids.new_empty(nbytes, dtype=torch.uint8)
        ids, offsets, rows, slots, ws = _ptrs(expert_ids, out.offsets, out.rows, out.slots, workspace)
        st = lib.trace_moe_sort(ids, expert_ids.element_size(), tokens, k, num_experts, offsets, rows,
                                slots, ws, workspace.numel() * workspace.element_size(), s)
        _check(st, "trace_moe_sort")
        if given:
            _written(out.offsets, out.rows, out.slots)
    return out


def _route_of(route: MoeRoute) -> tuple[int, int]:
    rows = route.rows
    if rows.dim() != 2 or rows.dtype is not torch.int32:
        raise TraceError("route rows must be int32 [tokens, k]")
    tokens, k = rows.shape
    _want(route.slots, "route slots", torch.int32, (tokens * k,))
    return tokens, k


def moe_dispatch_fwd(x: torch.Tensor, route: MoeRoute, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Tokens into expert order, bf16 [tokens, cols] -> [tokens * k, cols];
    rows of the dropped group are zero."""
    rows, cols = _bf16_2d(x)
    tokens, k = _route_of(route)
    if rows != tokens:
        raise TraceError(f"{rows} tokens, and a route of {tokens}")
    with _On(stream, x, route.rows, route.slots, out) as s:
        given = out is not None
        if given:
            _want(out, "out", torch.bfloat16, (tokens * k, cols))
        else:
            out = x.new_empty((tokens * k, cols))
        px, rows, slots, po = _ptrs(x, route.rows, route.slots, out)
        _check(library().trace_moe_dispatch(px, tokens, k, cols, rows, slots, po, s),
               "trace_moe_dispatch")
        if given:
            _written(out)
    return out


def moe_dispatch_bwd(grad: torch.Tensor, route: MoeRoute, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Gradient of moe_dispatch_fwd: each token's rows summed in fp32."""
    return moe_combine_fwd(grad, route, None, out, stream)


def moe_combine_fwd(y: torch.Tensor, route: MoeRoute, weights: torch.Tensor | None,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Back to token order with the routing weights (float [tokens, k]; None:
    all ones), bf16 [tokens * k, cols] -> [tokens, cols]."""
    _, cols = _bf16_2d(y)
    tokens, k = _route_of(route)
    _want(y, "expert rows", torch.bfloat16, (tokens * k, cols))
    if weights is not None:
        _want(weights, "weights", torch.float32, (tokens, k))
    with _On(stream, y, route.rows, weights, out) as s:
        given = out is not None
        if given:
            _want(out, "out", torch.bfloat16, (tokens, cols))
        else:
            out = y.new_empty((tokens, cols))
        py, rows, w, po = _ptrs(y, route.rows, weights, out)
        _check(library().trace_moe_combine(py, tokens, k, cols, rows, w, po, s),
               "trace_moe_combine")
        if given:
            _written(out)
    return out


def moe_combine_bwd(grad: torch.Tensor, y: torch.Tensor, route: MoeRoute, weights: torch.Tensor,
                    stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradients of moe_combine_fwd: (grad_y, grad_weights)."""
    _, cols = _bf16_2d(y)
    tokens, k = _route_of(route)
    _want(y, "expert rows", torch.bfloat16, (tokens * k, cols))
    _want(grad, "gradient", torch.bfloat16, (tokens, cols))
    _want(weights, "weights", torch.float32, (tokens, k))
    with _On(stream, grad, y, route.rows, route.slots, weights) as s:
        grad_y = torch.empty_like(y)
        grad_w = torch.empty_like(weights)
        pg, py, rows, slots, w, gy, gw = _ptrs(grad, y, route.rows, route.slots, weights, grad_y,
                                               grad_w)
        _check(library().trace_moe_combine_bwd(pg, py, tokens, k, cols, rows, slots, w, gy, gw, s),
               "trace_moe_combine_bwd")
    return grad_y, grad_w


def _upstream(grad: torch.Tensor) -> torch.Tensor:
    """A gradient as the kernels read it: contiguous, and moved if it is a part
    of a larger one that starts at an odd address."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 32 == 0 else grad.clone()


class MoeDispatch(torch.autograd.Function):
    """Autograd wrapper of the dispatch; both directions run in the library."""

    @staticmethod
    def forward(ctx, x, route: MoeRoute):
        ctx.save_for_backward(route.offsets, route.rows, route.slots)
        return moe_dispatch_fwd(x, route)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        return moe_dispatch_bwd(_upstream(grad), MoeRoute(*ctx.saved_tensors)), None


class MoeCombine(torch.autograd.Function):
    """Autograd wrapper of the combine (gradients to the rows and the weights)."""

    @staticmethod
    def forward(ctx, y, route: MoeRoute, weights):
        ctx.save_for_backward(y, weights, route.offsets, route.rows, route.slots)
        return moe_combine_fwd(y, route, weights)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        y, weights, *route = ctx.saved_tensors
        grad_y, grad_w = moe_combine_bwd(_upstream(grad), y, MoeRoute(*route), weights)
        return grad_y, None, grad_w


def moe_dispatch(x: torch.Tensor, route: MoeRoute) -> torch.Tensor:
    """Differentiable dispatch of tokens into expert order (for
    capture(y, route.offsets) and the grouped product).  Tensors that carry a
    tangent of forward-mode differentiation are refused, here and in moe_combine."""
    y = (_bind or _native()).dispatch(x, route.rows, route.slots)
    if y is not None:
        return y
    return MoeDispatch.apply(x, route)


def moe_combine(y: torch.Tensor, route: MoeRoute, weights: torch.Tensor) -> torch.Tensor:
    """Differentiable return to token order, weighted by the router."""
    out = (_bind or _native()).combine(y, route.rows, route.slots, weights)
    if out is not None:
        return out
    if weights is None:
        raise TraceError("moe_combine needs weights (moe_combine_fwd takes None for all ones)")
    return MoeCombine.apply(y, route, weights)


def _matmul_operand(cap, cols: int, bs: int, what: str) -> tuple[int, int]:
    """(rows, scale layout) of a captured FP4 operand: row-major scales are
    2-D, tiled ones flat."""
    codes, scales = cap.codes, cap.scales
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise TraceError(f"{what}: codes and scales must be uint8")
    rows, odd = divmod(codes.numel() * 2, cols)
    if odd:
        raise TraceError(f"{what}: {codes.numel()} bytes of codes are no rows of {cols}")
    c = cols // bs
    if scales.dim() == 2:
        layout, want = TRACE_SCALES_ROW_MAJOR, (rows, c)
    else:
        layout, want = TRACE_SCALES_TILED_128x4, (-(-rows // 128) * -(-c // 4) * 512,)
    if scales.shape != want:
        raise TraceError(f"{what}: scales of {tuple(scales.shape)} for [{rows}, {cols}], "
                         f"expected {want}")
    return rows, layout


@functools.lru_cache(maxsize=256)
def trace_matmul_workspace_bytes(mx: bool, rows: int, cols: int, num_groups: int,
                                 a_scale_layout: int, n: int, num_matrices: int,
                                 w_scale_layout: int) -> int:
    lib = library()
    f = lib.trace_mx_matmul_workspace_bytes if mx else lib.trace_fp4_matmul_workspace_bytes
    return int(f(rows, cols, num_groups, a_scale_layout, n, num_matrices, w_scale_layout))


def _matmul(a, w, cols, offsets, matrices, out, workspace, stream, bs):
    if cols is None:
        s = next((c.scales for c in (a, w) if c.scales.dim() == 2), None)
        if s is None:
            raise TraceError("cols is needed when both scales are tiled")
        cols = s.shape[1] * bs
    if cols <= 0 or cols % 32:
        raise TraceError(f"cols must be a multiple of 32: {cols}")
    if out is None and workspace is None and stream is None and not (DEBUG and offsets is not None):
        got = (_bind or _native()).matmul(bs, cols, matrices, offsets, a.codes, a.scales,
                                          a.gscale if bs == 16 else None, w.codes, w.scales,
                                          w.gscale if bs == 16 else None)
        if got is not None:
            return got
    rows, la = _matmul_operand(a, cols, bs, "a")
    wrows, lw = _matmul_operand(w, cols, bs, "w")
    groups = _groups(offsets, rows)
    if matrices < 1 or wrows % matrices or wrows == 0:
        raise TraceError(f"w: {wrows} rows are no {matrices} matrices")
    n = wrows // matrices
    ga, gw = (a.gscale, w.gscale) if bs == 16 else (None, None)
    with _On(stream, a.codes, a.scales, w.codes, w.scales, offsets, ga, gw, out, workspace) as s:
        given = out is not None
        if given:
            _want(out, "out", torch.bfloat16, (rows, n))
        else:
            out = a.codes.new_empty((rows, n), dtype=torch.bfloat16)
        if workspace is None:
            nbytes = trace_matmul_workspace_bytes(bs == 32, rows, cols, groups, la, n, matrices, lw)
            workspace = a.codes.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
        else:
            nbytes = workspace.numel() * workspace.element_size()
        ac, asc, wc, wsc, po, pf, pws = _ptrs(a.codes, a.scales, w.codes, w.scales, out, offsets,
                                              workspace)
        if bs == 16:
            _want(ga, "a global scales", torch.float32, (groups,))
            _want(gw, "w global scales", torch.float32, (matrices,))
            pa, pw = _ptrs(ga, gw)
            st = library().trace_fp4_matmul_ws(ac, asc, pa, rows, cols, groups, pf, la, wc, wsc, pw,
                                               n, matrices, lw, po, pws, nbytes, s)
        else:
            st = library().trace_mx_matmul_ws(ac, asc, rows, cols, groups, pf, la, wc, wsc, n,
                                              matrices, lw, po, pws, nbytes, s)
        _check(st, "trace_fp4_matmul" if bs == 16 else "trace_mx_matmul")
        if given:
            _written(out)
    return out


def fp4_matmul(a: Capture, w: Capture, cols: int | None = None, out: torch.Tensor | None = None,
               stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Product of two NVFP4 captures, bf16 [rows, n]: a of [rows, cols], w of
    one matrix [n, cols], or of one per expert stacked by rows (w.gscale has
    one entry per matrix, a.offsets groups the rows).  Rows of a's groups
    behind w's matrices (dropped slots) become zero; rows outside a.offsets
    are left as they were in `out` (undefined if None).  cols is needed when
    both scales are tiled.  Large products copy scales that are not tiled
    into `workspace` (trace_matmul_workspace_bytes; allocated if None).  Has
    no gradient: codes are the rollout's; the
    training side differentiates through trace_fake_quant."""
    if not isinstance(a, Capture) or not isinstance(w, Capture):
        raise TraceError("fp4_matmul takes two NVFP4 captures")
    return _matmul(a, w, cols, a.offsets, w.gscale.numel(), out, workspace, stream, 16)


def mx_matmul(a: MxCapture, w: MxCapture, cols: int | None = None,
              offsets: torch.Tensor | None = None, groups: int = 1,
              out: torch.Tensor | None = None, stream=None,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Product of two MXFP4 captures, bf16 [rows, n]; grouped when `offsets`
    (int64 row bounds of a) and `groups` (matrices stacked in w) are given."""
    if not isinstance(a, MxCapture) or not isinstance(w, MxCapture):
        raise TraceError("mx_matmul takes two MXFP4 captures")
    return _matmul(a, w, cols, offsets, groups, out, workspace, stream, 32)


def matmul_status(stream=None) -> bool:
    """True when no product on the current device has given up a wait since
    this thread last asked about this stream (trace_matmul_status: waits for
    the stream)."""
    st = library().trace_matmul_status(_stream(stream))
    if st == TRACE_ERR_TIMEOUT:
        return False
    _check(st, "trace_matmul_status")
    return True
