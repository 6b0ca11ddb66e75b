"""Thin ctypes binding of libunweight.so (include/unweight.h).

Argument marshalling only: every step of the codec and the GEMMs runs in the
library's HIP kernels.  torch tensors are accepted for device buffers and
their ``data_ptr()`` is passed through; streams default to torch's current
stream.  Importing this module fails loudly when the library is missing.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libunweight.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: run __graft_entry__.build() (hipcc for gfx950) first")

_lib = ctypes.CDLL(LIB_PATH)

UW_OK = 0
UW_ERR_UNSUPPORTED = -2
STATUS = {0: "ok", -1: "invalid", -2: "unsupported", -3: "nomem", -4: "device", -5: "corrupt",
          -6: "state", -7: "workspace"}
PIPE_FULL, PIPE_EXPONENT, PIPE_PALETTE_TRANSCODE, PIPE_PALETTE_DIRECT = 0, 1, 2, 3
PIPE_AUTO = 15
PIPELINES = {"full": 0, "exponent": 1, "transcode": 2, "direct": 3, "auto": 15}
LAYOUT_NK, LAYOUT_KN = 0, 1


class UwError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status})")
        self.status = status


class uw_compress_opts(ctypes.Structure):
    _fields_ = [("seg_groups", ctypes.c_uint32), ("flags", ctypes.c_uint32)]


class uw_kernel_cfg(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("split_k", ctypes.c_int32), ("decode_cus", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class uw_info(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_uint32), ("seg_groups", ctypes.c_uint32),
                ("rows", ctypes.c_uint64), ("cols", ctypes.c_uint64), ("n", ctypes.c_uint64),
                ("k", ctypes.c_uint64), ("numel", ctypes.c_uint64), ("groups", ctypes.c_uint64),
                ("segments", ctypes.c_uint64), ("palette_size", ctypes.c_uint32), ("n_coded", ctypes.c_uint32),
                ("palette", ctypes.c_uint8 * 16), ("code_len", ctypes.c_uint8 * 16),
                ("code", ctypes.c_uint16 * 16), ("hist", ctypes.c_uint64 * 256),
                ("coded_count", ctypes.c_uint64 * 16), ("verbatim_groups", ctypes.c_uint64),
                ("stream_words", ctypes.c_uint64), ("code_bits", ctypes.c_uint64),
                ("compressed_bytes", ctypes.c_uint64), ("export_bytes", ctypes.c_uint64),
                ("bits_per_weight", ctypes.c_double), ("has_stream", ctypes.c_int32),
                ("has_palette_idx", ctypes.c_int32), ("element_bits", ctypes.c_int32)]


class uw_tune_entry(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("projection", ctypes.c_int32), ("pipeline", ctypes.c_int32),
                ("variant", ctypes.c_int32), ("split_k", ctypes.c_int32), ("decode_cus", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("residency", ctypes.c_int32), ("group", ctypes.c_int32),
                ("n", ctypes.c_uint64), ("k", ctypes.c_uint64), ("sequence_us", ctypes.c_double)]


ALLOC_FN = ctypes.CFUNCTYPE(ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p)
FREE_FN = ctypes.CFUNCTYPE(None, ctypes.c_void_p, ctypes.c_void_p)


class uw_allocator(ctypes.Structure):
    _fields_ = [("alloc", ALLOC_FN), ("free", FREE_FN), ("ctx", ctypes.c_void_p)]


class uw_gemm_plan(ctypes.Structure):
    _fields_ = [("pipeline", ctypes.c_int32), ("variant", ctypes.c_int32), ("fmt", ctypes.c_int32),
                ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("waves", ctypes.c_int32),
                ("k_slices", ctypes.c_int32), ("reserved", ctypes.c_int32), ("kernel", ctypes.c_char * 64)]


class uw_job(ctypes.Structure):
    _fields_ = [("m", ctypes.c_void_p), ("pipeline", ctypes.c_int32), ("cfg", uw_kernel_cfg),
                ("x_dev", ctypes.c_void_p), ("y_dev", ctypes.c_void_p), ("batch", ctypes.c_int64)]


_vp, _i64, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
_SIGS = {
    "uw_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "uw_version": (ctypes.c_uint32, []),
    "uw_compress": (ctypes.c_int, [_vp, _i64, _i64, ctypes.c_int, ctypes.POINTER(uw_compress_opts), _vp,
                                   ctypes.POINTER(_vp)]),
    "uw_compress_fp8": (ctypes.c_int, [_vp, _i64, _i64, ctypes.c_int, ctypes.POINTER(uw_compress_opts), _vp,
                                   ctypes.POINTER(_vp)]),
    "uw_get_info": (ctypes.c_int, [_vp, ctypes.POINTER(uw_info)]),
    "uw_export": (ctypes.c_int, [_vp, _vp, _sz, ctypes.POINTER(_sz)]),
    "uw_import": (ctypes.c_int, [_vp, _sz, _vp, ctypes.POINTER(_vp)]),
    "uw_free": (None, [_vp]),
    "uw_decode_full": (ctypes.c_int, [_vp, _vp, _vp]),
    "uw_decode_fp8": (ctypes.c_int, [_vp, _vp, _vp]),
    "uw_decode_exponent": (ctypes.c_int, [_vp, _vp, _vp]),
    "uw_transcode_palette": (ctypes.c_int, [_vp, _vp, _vp]),
    "uw_drop_stream": (ctypes.c_int, [_vp, _vp]),
    "uw_workspace_size": (ctypes.c_int, [_vp, ctypes.c_int, _i64, ctypes.POINTER(_sz)]),
    "uw_matmul_reconstruct": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _i64, _vp, _vp, _sz,
                                             ctypes.POINTER(uw_kernel_cfg), _vp]),
    "uw_matmul_stage": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _vp, _i64, _vp, _vp, _sz,
                                       ctypes.POINTER(uw_kernel_cfg), _vp]),
    "uw_matmul_reconstruct_grouped": (ctypes.c_int, [ctypes.POINTER(_vp), ctypes.c_int, ctypes.c_int, _vp, _i64,
                                                     _vp, _vp, _sz, ctypes.POINTER(uw_kernel_cfg), _vp]),
    "uw_gemm_bf16": (ctypes.c_int, [_vp, _i64, _i64, ctypes.c_int, _vp, _i64, _vp,
                                    ctypes.POINTER(uw_kernel_cfg), _vp]),
    "uw_variant_count": (ctypes.c_int32, []),
    "uw_sequence_workspace_size": (ctypes.c_int, [ctypes.POINTER(uw_job), ctypes.c_int, ctypes.POINTER(_sz)]),
    "uw_run_sequence": (ctypes.c_int, [ctypes.POINTER(uw_job), ctypes.c_int, ctypes.c_int32, _vp, _sz, _vp]),
    "uw_sync_status": (ctypes.c_int, [_vp, _vp]),
    "uw_autotune": (ctypes.c_int, [ctypes.POINTER(_vp), ctypes.POINTER(ctypes.c_int32), ctypes.c_int, ctypes.c_int,
                                   ctypes.POINTER(ctypes.c_int64), ctypes.c_int, ctypes.c_int, ctypes.c_char_p,
                                   ctypes.POINTER(uw_tune_entry), _vp]),
    "uw_autotune_grouped": (ctypes.c_int, [ctypes.POINTER(_vp), ctypes.c_int, ctypes.c_int,
                                           ctypes.POINTER(ctypes.c_int64), ctypes.c_int, ctypes.c_char_p,
                                           ctypes.POINTER(uw_tune_entry), _vp]),
    "uw_drop_palette": (ctypes.c_int, [_vp, _vp]),
    "uw_workspace_size_cfg": (ctypes.c_int, [_vp, ctypes.c_int, _i64, ctypes.POINTER(uw_kernel_cfg),
                                             ctypes.POINTER(_sz)]),
    "uw_workspace_size_grouped": (ctypes.c_int, [ctypes.POINTER(_vp), ctypes.c_int, ctypes.c_int, _i64,
                                                 ctypes.POINTER(uw_kernel_cfg), ctypes.POINTER(_sz)]),
    "uw_matmul_stage_static": (ctypes.c_int, [_vp, ctypes.c_int, _vp, _vp, _i64, _vp,
                                              ctypes.POINTER(uw_kernel_cfg), _vp]),
    "uw_plan_gemm": (ctypes.c_int, [_vp, ctypes.c_int, _i64, ctypes.POINTER(uw_kernel_cfg),
                                    ctypes.POINTER(uw_gemm_plan)]),
    "uw_yardstick": (ctypes.c_int, [ctypes.c_int, _vp, _vp, _sz, _i64, _vp, ctypes.POINTER(ctypes.c_double)]),
    "uw_set_allocator": (ctypes.c_int, [ctypes.POINTER(uw_allocator)]),
    "uw_release_resources": (ctypes.c_int, []),
    "uw_set_kernel_events": (ctypes.c_int, [_vp, _vp]),
    "uw_set_tuning": (ctypes.c_int, [ctypes.POINTER(uw_tune_entry), ctypes.c_int]),
    "uw_load_tuning": (ctypes.c_int, [ctypes.c_char_p]),
    "uw_clear_tuning": (ctypes.c_int, []),
    "uw_lookup_tuning": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_uint64, ctypes.c_int32, ctypes.c_int32, _i64,
                                        ctypes.POINTER(uw_tune_entry)]),
    "uw_lookup_tuning_grouped": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_uint64, ctypes.c_int32, ctypes.c_int32,
                                                ctypes.c_int32, _i64, ctypes.POINTER(uw_tune_entry)]),
    "uw_quantize_mx4": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp]),
    "uw_dequantize_mx4": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _i64, _vp]),
    "uw_workspace_size_mx4": (ctypes.c_int, [_i64, _i64, _i64, ctypes.c_int, ctypes.POINTER(_sz)]),
    "uw_matmul_mx4": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _i64, _vp, ctypes.c_int, _vp, _sz, _vp]),
    "uw_quantize_fp8": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, ctypes.c_int32, _vp, _vp, _vp]),
    "uw_dequantize_fp8": (ctypes.c_int, [_vp, _vp, _i64, _i64, ctypes.c_int32, _vp, _i64, _vp]),
    "uw_workspace_size_fp8": (ctypes.c_int, [_i64, _i64, _i64, ctypes.c_int, ctypes.POINTER(_sz)]),
    "uw_matmul_fp8": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _i64, _vp, ctypes.c_int, _vp, _sz, _vp]),
    "uw_experts_fp8": (ctypes.c_int, [_vp, _vp, ctypes.c_int32, _i64, _i64, _i64, _i64, ctypes.POINTER(_vp)]),
    "uw_workspace_size_route": (ctypes.c_int, [_i64, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(_sz)]),
    "uw_route_experts": (ctypes.c_int, [_vp, ctypes.c_int, _i64, ctypes.c_int32, _i64, _vp, ctypes.c_int32,
                                        ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "uw_plan_experts": (ctypes.c_int, [_vp, _i64, ctypes.c_int32, ctypes.c_int32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "uw_experts_bf16": (ctypes.c_int, [_vp, ctypes.c_int32, _i64, _i64, _i64, ctypes.POINTER(_vp)]),
    "uw_experts_mx4": (ctypes.c_int, [_vp, _vp, ctypes.c_int32, _i64, _i64, _i64, _i64, ctypes.POINTER(_vp)]),
    "uw_experts_uwf1": (ctypes.c_int, [ctypes.POINTER(_vp), ctypes.c_int32, _vp, ctypes.POINTER(_vp)]),
    "uw_free_experts": (None, [_vp]),
    "uw_matmul_experts": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp]),
    "uw_matmul_experts_gated": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp]),
    "uw_workspace_size_expert_mlp": (ctypes.c_int, [_vp, _vp, _i64, ctypes.c_int32, ctypes.POINTER(_sz)]),
    "uw_expert_mlp": (ctypes.c_int, [_vp, _vp, _vp, _i64, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                     _vp]),
    "uw_workspace_size_expert_layer": (ctypes.c_int, [_vp, _vp, _i64, ctypes.c_int32, ctypes.POINTER(_sz)]),
    "uw_expert_layer": (ctypes.c_int, [_vp, _vp, _vp, _vp, ctypes.c_int, _i64, _i64, _vp, ctypes.c_int32, ctypes.c_int,
                                       _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)


def _check(st: int, what: str) -> None:
    if st != UW_OK:
        raise UwError(st, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        return t.data_ptr()
    return int(t)


# torch's current stream as a raw handle: a tenth of the time of building a
# Stream object, which small calls notice
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)   # once torch's GPU state is there


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(_device())
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _cfg(cfg) -> ctypes.POINTER(uw_kernel_cfg) | None:
    if cfg is None:
        return None
    if isinstance(cfg, dict):
        c = uw_kernel_cfg(cfg.get("variant", 0), cfg.get("split_k", 0), cfg.get("decode_cus", 0), 0)
    else:
        c = cfg
    return ctypes.pointer(c)


def version() -> int:
    return _lib.uw_version()


def variant_count() -> int:
    return _lib.uw_variant_count()


class Matrix:
    """Owns one uw_matrix handle."""

    def __init__(self, handle: int):
        self.handle = ctypes.c_void_p(handle)

    def info(self) -> uw_info:
        inf = uw_info()
        _check(_lib.uw_get_info(self.handle, ctypes.byref(inf)), "uw_get_info")
        return inf

    def free(self) -> None:
        if self.handle and self.handle.value:
            _lib.uw_free(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def uw_compress(w_dev: torch.Tensor, n: int, k: int, layout: int = LAYOUT_NK, seg_groups: int = 4,
                stream=None) -> Matrix:
    opts = uw_compress_opts(seg_groups, 0)
    h = ctypes.c_void_p()
    _check(_lib.uw_compress(_ptr(w_dev), n, k, layout, ctypes.byref(opts), _stream(stream), ctypes.byref(h)),
           "uw_compress")
    return Matrix(h.value)


def uw_get_info(m: Matrix) -> uw_info:
    return m.info()


def uw_export(m: Matrix) -> bytes:
    n = ctypes.c_size_t()
    _check(_lib.uw_export(m.handle, None, 0, ctypes.byref(n)), "uw_export(size)")
    buf = np.zeros(n.value, dtype=np.uint8)
    _check(_lib.uw_export(m.handle, buf.ctypes.data, n.value, ctypes.byref(n)), "uw_export")
    return buf.tobytes()


def uw_import(blob: bytes, stream=None) -> Matrix:
    arr = np.frombuffer(blob, dtype=np.uint8)
    h = ctypes.c_void_p()
    _check(_lib.uw_import(arr.ctypes.data, len(blob), _stream(stream), ctypes.byref(h)), "uw_import")
    return Matrix(h.value)


def uw_import_status(blob: bytes) -> int:
    """Status of uw_import without keeping the handle (validation tests)."""
    arr = np.frombuffer(blob, dtype=np.uint8)
    h = ctypes.c_void_p()
    st = _lib.uw_import(arr.ctypes.data if len(blob) else None, len(blob), None, ctypes.byref(h))
    if h.value:
        _lib.uw_free(h)
    return st


def uw_free(m: Matrix) -> None:
    m.free()


def uw_compress_fp8(w_dev: torch.Tensor, n: int, k: int, layout: int = LAYOUT_NK, seg_groups: int = 4,
                    stream=None) -> Matrix:
    """FP8 E4M3 weights given as a uint8 device tensor of the stored shape."""
    opts = uw_compress_opts(seg_groups, 0)
    h = ctypes.c_void_p()
    _check(_lib.uw_compress_fp8(_ptr(w_dev), n, k, layout, ctypes.byref(opts), _stream(stream), ctypes.byref(h)),
           "uw_compress_fp8")
    return Matrix(h.value)


def uw_decode_fp8(m: Matrix, out: torch.Tensor, stream=None) -> None:
    _check(_lib.uw_decode_fp8(m.handle, _ptr(out), _stream(stream)), "uw_decode_fp8")


def uw_decode_full(m: Matrix, out: torch.Tensor, stream=None) -> None:
    _check(_lib.uw_decode_full(m.handle, _ptr(out), _stream(stream)), "uw_decode_full")


def uw_decode_exponent(m: Matrix, out: torch.Tensor, stream=None) -> None:
    _check(_lib.uw_decode_exponent(m.handle, _ptr(out), _stream(stream)), "uw_decode_exponent")


def uw_transcode_palette(m: Matrix, out: torch.Tensor | None, stream=None) -> None:
    _check(_lib.uw_transcode_palette(m.handle, _ptr(out), _stream(stream)), "uw_transcode_palette")


def uw_drop_stream(m: Matrix, stream=None) -> None:
    _check(_lib.uw_drop_stream(m.handle, _stream(stream)), "uw_drop_stream")


def uw_workspace_size(m: Matrix, pipeline: int, batch: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.uw_workspace_size(m.handle, pipeline, batch, ctypes.byref(n)), "uw_workspace_size")
    return n.value


def uw_workspace_size_cfg(m: Matrix, pipeline: int, batch: int, cfg=None) -> int:
    n = ctypes.c_size_t()
    _check(_lib.uw_workspace_size_cfg(m.handle, pipeline, batch, _cfg(cfg), ctypes.byref(n)),
           "uw_workspace_size_cfg")
    return n.value


def uw_workspace_size_grouped(ms, pipeline: int, batch: int, cfg=None) -> int:
    arr = (ctypes.c_void_p * len(ms))(*[m.handle.value for m in ms])
    n = ctypes.c_size_t()
    _check(_lib.uw_workspace_size_grouped(arr, len(ms), pipeline, batch, _cfg(cfg), ctypes.byref(n)),
           "uw_workspace_size_grouped")
    return n.value


def uw_matmul_reconstruct(m: Matrix, pipeline: int, x: torch.Tensor, y: torch.Tensor, ws: torch.Tensor | None,
                          cfg=None, stream=None) -> None:
    batch = x.shape[0]
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check(_lib.uw_matmul_reconstruct(m.handle, pipeline, _ptr(x), batch, _ptr(y), _ptr(ws), nbytes, _cfg(cfg),
                                      _stream(stream)), "uw_matmul_reconstruct")


def uw_matmul_stage(m: Matrix, pipeline: int, prep: torch.Tensor | None, x: torch.Tensor, y: torch.Tensor,
                    ws: torch.Tensor | None, cfg=None, stream=None) -> None:
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check(_lib.uw_matmul_stage(m.handle, pipeline, _ptr(prep), _ptr(x), x.shape[0], _ptr(y), _ptr(ws), nbytes,
                                _cfg(cfg), _stream(stream)), "uw_matmul_stage")


STATIC_SCRATCH_BYTES = 64 << 20


def uw_matmul_stage_static(m: Matrix, pipeline: int, prep: torch.Tensor | None, x: torch.Tensor, y: torch.Tensor,
                           cfg=None, stream=None) -> None:
    _check(_lib.uw_matmul_stage_static(m.handle, pipeline, _ptr(prep), _ptr(x), x.shape[0], _ptr(y), _cfg(cfg),
                                       _stream(stream)), "uw_matmul_stage_static")


def uw_matmul_reconstruct_grouped(ms, pipeline: int, x: torch.Tensor, y: torch.Tensor, ws: torch.Tensor | None,
                                  cfg=None, stream=None) -> None:
    arr = (ctypes.c_void_p * len(ms))(*[m.handle.value for m in ms])
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check(_lib.uw_matmul_reconstruct_grouped(arr, len(ms), pipeline, _ptr(x), x.shape[0], _ptr(y), _ptr(ws),
                                              nbytes, _cfg(cfg), _stream(stream)), "uw_matmul_reconstruct_grouped")


def uw_gemm_bf16(w: torch.Tensor, n: int, k: int, layout: int, x: torch.Tensor, y: torch.Tensor, cfg=None,
                 stream=None) -> None:
    _check(_lib.uw_gemm_bf16(_ptr(w), n, k, layout, _ptr(x), x.shape[0], _ptr(y), _cfg(cfg), _stream(stream)),
           "uw_gemm_bf16")


@dataclass
class Job:
    m: Matrix
    pipeline: int
    x: torch.Tensor
    y: torch.Tensor
    cfg: dict | None = None


def _jobs(jobs) -> ctypes.Array:
    arr = (uw_job * len(jobs))()
    for i, j in enumerate(jobs):
        c = j.cfg or {}
        arr[i] = uw_job(j.m.handle.value, j.pipeline,
                        uw_kernel_cfg(c.get("variant", 0), c.get("split_k", 0), c.get("decode_cus", 0), 0),
                        _ptr(j.x), _ptr(j.y), j.x.shape[0])
    return arr


def uw_sequence_workspace_size(jobs) -> int:
    n = ctypes.c_size_t()
    _check(_lib.uw_sequence_workspace_size(_jobs(jobs), len(jobs), ctypes.byref(n)), "uw_sequence_workspace_size")
    return n.value


def uw_run_sequence(jobs, decode_cus: int, ws: torch.Tensor | None, stream=None, _arr=None) -> None:
    arr = _arr if _arr is not None else _jobs(jobs)
    nbytes = ws.numel() * ws.element_size() if ws is not None else 0
    _check(_lib.uw_run_sequence(arr, len(jobs), decode_cus, _ptr(ws), nbytes, _stream(stream)),
           "uw_run_sequence")


def uw_drop_palette(m: Matrix, stream=None) -> None:
    _check(_lib.uw_drop_palette(m.handle, _stream(stream)), "uw_drop_palette")


def uw_autotune(ms, proj, batches, max_passes: int = 3, json_path: str | None = None, stream=None):
    """Returns a list of dicts, one per (batch, projection)."""
    nproj = max(proj) + 1
    arr = (ctypes.c_void_p * len(ms))(*[m.handle.value for m in ms])
    pj = (ctypes.c_int32 * len(proj))(*proj)
    bs = (ctypes.c_int64 * len(batches))(*batches)
    out = (uw_tune_entry * (len(batches) * nproj))()
    _check(_lib.uw_autotune(arr, pj, len(ms), nproj, bs, len(batches), max_passes,
                            json_path.encode() if json_path else None, out, _stream(stream)), "uw_autotune")
    return [_entry_dict(e) for e in out]


def uw_autotune_grouped(groups, batches, json_path: str | None = None, stream=None):
    """groups: a list of equal-shaped groups (lists of Matrix), e.g. the gate
    and up matrices of successive layers.  Returns one dict per batch."""
    size = len(groups[0])
    flat = [m for g in groups for m in g]
    if any(len(g) != size for g in groups):
        raise ValueError("uw_autotune_grouped: groups of different sizes")
    arr = (ctypes.c_void_p * len(flat))(*[m.handle.value for m in flat])
    bs = (ctypes.c_int64 * len(batches))(*batches)
    out = (uw_tune_entry * len(batches))()
    _check(_lib.uw_autotune_grouped(arr, size, len(groups), bs, len(batches),
                                    json_path.encode() if json_path else None, out, _stream(stream)),
           "uw_autotune_grouped")
    return [_entry_dict(e) for e in out]


def uw_plan_gemm(m: Matrix, pipeline: int, batch: int, cfg=None) -> dict:
    pl = uw_gemm_plan()
    _check(_lib.uw_plan_gemm(m.handle, pipeline, batch, _cfg(cfg), ctypes.byref(pl)), "uw_plan_gemm")
    d = {f: getattr(pl, f) for f, _ in uw_gemm_plan._fields_ if f != "reserved"}
    d["kernel"] = pl.kernel.decode()
    return d


YARDSTICK_SINK_BYTES = 4 << 20


def uw_yardstick(kind: int, src, dst, nbytes: int = 0, iters: int = 0, stream=None) -> float:
    """kind 0 copy, 1 read, 2 MFMA loop; returns the work (bytes or flops)."""
    w = ctypes.c_double()
    _check(_lib.uw_yardstick(kind, _ptr(src), _ptr(dst), nbytes, iters, _stream(stream), ctypes.byref(w)),
           "uw_yardstick")
    return w.value


def uw_sync_status(m: Matrix, stream=None) -> int:
    return _lib.uw_sync_status(m.handle, _stream(stream))


_TUNE_FIELDS = [f for f, _ in uw_tune_entry._fields_ if f != "reserved"]


def _entry_dict(e: uw_tune_entry) -> dict:
    return {f: getattr(e, f) for f in _TUNE_FIELDS}


def uw_set_tuning(entries) -> None:
    """entries: dicts with the uw_tune_entry fields (as uw_autotune returns)."""
    arr = (uw_tune_entry * max(1, len(entries)))()
    for i, d in enumerate(entries):
        for f in _TUNE_FIELDS:
            if f in d:
                setattr(arr[i], f, d[f])
    _check(_lib.uw_set_tuning(arr, len(entries)), "uw_set_tuning")


def uw_load_tuning(json_path: str) -> None:
    _check(_lib.uw_load_tuning(json_path.encode()), "uw_load_tuning")


def uw_clear_tuning() -> None:
    _check(_lib.uw_clear_tuning(), "uw_clear_tuning")


def uw_lookup_tuning(n: int, k: int, layout: int, residency: int, batch: int) -> dict | None:
    e = uw_tune_entry()
    st = _lib.uw_lookup_tuning(n, k, layout, residency, batch, ctypes.byref(e))
    if st == -6:
        return None
    _check(st, "uw_lookup_tuning")
    return _entry_dict(e)


def uw_lookup_tuning_grouped(n: int, k: int, layout: int, residency: int, group: int, batch: int) -> dict | None:
    e = uw_tune_entry()
    st = _lib.uw_lookup_tuning_grouped(n, k, layout, residency, group, batch, ctypes.byref(e))
    if st == -6:
        return None
    _check(st, "uw_lookup_tuning_grouped")
    return _entry_dict(e)


def uw_set_kernel_events(before, after) -> None:
    """before, after: torch.cuda.Event objects already recorded once (so that
    they exist), or None for both to clear."""
    b = ctypes.c_void_p(before.cuda_event) if before is not None else None
    a = ctypes.c_void_p(after.cuda_event) if after is not None else None
    _check(_lib.uw_set_kernel_events(b, a), "uw_set_kernel_events")


def uw_release_resources() -> None:
    _check(_lib.uw_release_resources(), "uw_release_resources")


# The hooks given to uw_set_allocator must outlive every handle made under
# them; the binding keeps the last ones alive for the life of the process.
_ALLOCATORS: list = []


def uw_set_allocator(alloc=None, free=None, ctx: int | None = None) -> None:
    """alloc(bytes) -> device pointer (int, 0 for failure); free(ptr).  Both
    None restores hipMalloc / hipFree."""
    if alloc is None and free is None:
        _check(_lib.uw_set_allocator(None), "uw_set_allocator")
        return
    a = uw_allocator(ALLOC_FN(lambda n, c: alloc(n) or None), FREE_FN(lambda p, c: free(p)), ctx)
    _ALLOCATORS.append(a)
    _check(_lib.uw_set_allocator(ctypes.byref(a)), "uw_set_allocator")


class TorchAllocator:
    """Device memory from torch's caching allocator for uw_set_allocator:
    each block is a uint8 tensor kept alive until the library frees it."""

    def __init__(self, device="cuda:0"):
        self.device = device
        self.live: dict[int, torch.Tensor] = {}
        self.allocs = 0
        self.frees = 0

    def alloc(self, nbytes: int) -> int:
        t = torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)
        p = (t.data_ptr() + 255) // 256 * 256
        self.live[p] = t
        self.allocs += 1
        return p

    def free(self, p: int) -> None:
        self.live.pop(p, None)
        self.frees += 1


# ---- MXFP4 -----------------------------------------------------------------
# The calls below check what a pointer cannot carry -- element type, shape,
# contiguity, device -- and raise ValueError before the library sees them.

ACT_BF16, ACT_MX4, ACT_FP8 = 0, 1, 2
SCORE = {"softmax": 0, "softmax_topk": 1, "sigmoid": 2, "sigmoid_biased": 4}
_TYPES = {torch.float32: 0, torch.bfloat16: 1}


def _want(t: torch.Tensor, what: str, dtype, shape, dev: int) -> int:
    """Pointer of a contiguous tensor of this type (and shape, unless None) on the current device `dev`."""
    if t.dtype is not dtype:
        raise ValueError(f"{what}: {dtype} expected, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if t.get_device() != dev:
        _on_device(t, what, dev)
    return t.data_ptr()


def _current() -> int:
    """The current device; without one every tensor is refused as being elsewhere."""
    if torch.cuda.is_initialized():
        return _device()
    return torch.cuda.current_device() if torch.cuda.is_available() else -2


def _on_device(t: torch.Tensor, what: str, dev: int) -> None:
    if t.get_device() != dev:
        raise ValueError(f"{what}: must be on the current device, is on {t.device}")


def _rows2d(t: torch.Tensor, what: str, dev: int) -> int:
    """Row stride in elements of a 2-D tensor whose rows are contiguous."""
    if t.get_device() != dev:
        _on_device(t, what, dev)
    shape = t.shape
    if len(shape) == 2:
        if t.is_contiguous():
            return shape[1]
        ld, step = t.stride()
        if shape[1] <= 1 or step == 1:
            return ld if shape[0] > 1 else shape[1]
    raise ValueError(f"{what}: two dimensions with contiguous rows expected")


def _ws(ws: torch.Tensor | None, dev: int) -> tuple[int | None, int]:
    if ws is None:
        return None, 0
    if not ws.is_contiguous():
        raise ValueError("ws: must be contiguous")
    _on_device(ws, "ws", dev)
    return ws.data_ptr(), ws.numel() * ws.element_size()


def mx4_scale_stride(cols: int) -> int:
    """Bytes of scales per row (UW_MX4_SCALE_STRIDE)."""
    return (cols + 127) // 128 * 4


def uw_quantize_mx4(src: torch.Tensor, elem: torch.Tensor, scale: torch.Tensor, stream=None) -> None:
    """src [rows][cols] BF16 or FP32 (rows may be strided) -> elem [rows][cols/2], scale [rows][mx4_scale_stride]."""
    if src.dtype not in _TYPES:
        raise ValueError(f"src: float32 or bfloat16 expected, got {src.dtype}")
    dev = _current()
    ld = _rows2d(src, "src", dev)
    rows, cols = src.shape
    pe = _want(elem, "elem", torch.uint8, (rows, cols // 2), dev)
    ps = _want(scale, "scale", torch.uint8, (rows, mx4_scale_stride(cols)), dev)
    _check(_lib.uw_quantize_mx4(src.data_ptr(), _TYPES[src.dtype], rows, cols, ld, pe, ps, _stream(stream)),
           "uw_quantize_mx4")


def uw_dequantize_mx4(elem: torch.Tensor, scale: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """The values of uw_quantize_mx4's arrays into out [rows][cols] BF16 (rows may be strided)."""
    if out.dtype is not torch.bfloat16:
        raise ValueError(f"out: bfloat16 expected, got {out.dtype}")
    dev = _current()
    ld = _rows2d(out, "out", dev)
    rows, cols = out.shape
    pe = _want(elem, "elem", torch.uint8, (rows, cols // 2), dev)
    ps = _want(scale, "scale", torch.uint8, (rows, mx4_scale_stride(cols)), dev)
    _check(_lib.uw_dequantize_mx4(pe, ps, rows, cols, out.data_ptr(), ld, _stream(stream)), "uw_dequantize_mx4")


def uw_workspace_size_mx4(n: int, k: int, batch: int, act: int = ACT_BF16) -> int:
    b = ctypes.c_size_t()
    _check(_lib.uw_workspace_size_mx4(n, k, batch, act, ctypes.byref(b)), "uw_workspace_size_mx4")
    return b.value


def uw_matmul_mx4(elem: torch.Tensor, scale: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                  ws: torch.Tensor | None = None, act: int = ACT_BF16, stream=None) -> None:
    """y [batch][n] FP32 = x [batch][k] BF16 times the MXFP4 matrix (elem [n][k/2], scale [n][stride])."""
    if x.dim() != 2 or elem.dim() != 2:
        raise ValueError("x and elem: two dimensions expected")
    dev = _current()
    (batch, k), n = x.shape, elem.shape[0]
    pe = _want(elem, "elem", torch.uint8, (n, k // 2), dev)
    ps = _want(scale, "scale", torch.uint8, (n, mx4_scale_stride(k)), dev)
    px = _want(x, "x", torch.bfloat16, None, dev)
    py = _want(y, "y", torch.float32, (batch, n), dev)
    pw, nb = _ws(ws, dev)
    _check(_lib.uw_matmul_mx4(pe, ps, n, k, px, batch, py, act, pw, nb, _stream(stream)), "uw_matmul_mx4")


# ---- FP8 -----------------------------------------------------------------------

_E4M3 = (torch.float8_e4m3fn, torch.uint8)   # elements: as E4M3, or as bytes


def fp8_scale_shape(rows: int, cols: int, block_rows: int = 1) -> tuple[int, int]:
    """Shape of the scales of a [rows][cols] array in blocks of block_rows x 128."""
    return (rows + block_rows - 1) // block_rows, (cols + 127) // 128


def _want_fp8(t: torch.Tensor, what: str, shape, dev: int) -> int:
    return _want(t, what, torch.uint8 if t.dtype is torch.uint8 else torch.float8_e4m3fn, shape, dev)


def _block_rows(block_rows: int) -> None:
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows: 1 or 128 expected, got {block_rows}")


def uw_quantize_fp8(src: torch.Tensor, elem: torch.Tensor, scale: torch.Tensor, block_rows: int = 1,
                    stream=None) -> None:
    """src [rows][cols] BF16 or FP32 (rows may be strided) -> elem [rows][cols] float8_e4m3fn (or uint8), scale
    [fp8_scale_shape(rows, cols, block_rows)] FP32."""
    if src.dtype not in _TYPES:
        raise ValueError(f"src: float32 or bfloat16 expected, got {src.dtype}")
    _block_rows(block_rows)
    dev = _current()
    ld = _rows2d(src, "src", dev)
    rows, cols = src.shape
    pe = _want_fp8(elem, "elem", (rows, cols), dev)
    ps = _want(scale, "scale", torch.float32, fp8_scale_shape(rows, cols, block_rows), dev)
    _check(_lib.uw_quantize_fp8(src.data_ptr(), _TYPES[src.dtype], rows, cols, ld, block_rows, pe, ps,
                                _stream(stream)), "uw_quantize_fp8")


def uw_dequantize_fp8(elem: torch.Tensor, scale: torch.Tensor, out: torch.Tensor, block_rows: int = 1,
                      stream=None) -> None:
    """The values of uw_quantize_fp8's arrays into out [rows][cols] BF16 (rows may be strided)."""
    if out.dtype is not torch.bfloat16:
        raise ValueError(f"out: bfloat16 expected, got {out.dtype}")
    _block_rows(block_rows)
    dev = _current()
    ld = _rows2d(out, "out", dev)
    rows, cols = out.shape
    pe = _want_fp8(elem, "elem", (rows, cols), dev)
    ps = _want(scale, "scale", torch.float32, fp8_scale_shape(rows, cols, block_rows), dev)
    _check(_lib.uw_dequantize_fp8(pe, ps, rows, cols, block_rows, out.data_ptr(), ld, _stream(stream)),
           "uw_dequantize_fp8")


def uw_workspace_size_fp8(n: int, k: int, batch: int, act: int = ACT_BF16) -> int:
    b = ctypes.c_size_t()
    _check(_lib.uw_workspace_size_fp8(n, k, batch, act, ctypes.byref(b)), "uw_workspace_size_fp8")
    return b.value


def uw_matmul_fp8(elem: torch.Tensor, scale: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                  ws: torch.Tensor | None = None, act: int = ACT_BF16, stream=None) -> None:
    """y [batch][n] FP32 = x [batch][k] BF16 times the FP8 matrix (elem [n][k], scale [fp8_scale_shape(n, k, 128)])."""
    if x.dim() != 2 or elem.dim() != 2:
        raise ValueError("x and elem: two dimensions expected")
    dev = _current()
    (batch, k), n = x.shape, elem.shape[0]
    pe = _want_fp8(elem, "elem", (n, k), dev)
    ps = _want(scale, "scale", torch.float32, fp8_scale_shape(n, k, 128), dev)
    px = _want(x, "x", torch.bfloat16, None, dev)
    py = _want(y, "y", torch.float32, (batch, n), dev)
    pw, nb = _ws(ws, dev)
    _check(_lib.uw_matmul_fp8(pe, ps, n, k, px, batch, py, act, pw, nb, _stream(stream)), "uw_matmul_fp8")


# ---- mixture of experts ------------------------------------------------------

class Routing:
    """The buffers of a router's choice and of the plan that sorts its pairs by expert (see unweight.h).

    ids, weights, slots [tokens][topk], offsets [experts + 1], rows [tokens * topk]; read-only attributes
    (their contents may be written), so that a call need not ask each tensor for its pointer again.
    """

    def __init__(self, tokens: int, experts: int, topk: int, device="cuda"):
        n = ctypes.c_size_t()
        _check(_lib.uw_workspace_size_route(tokens, experts, topk, ctypes.byref(n)), "uw_workspace_size_route")
        self._shape = tokens, experts, topk
        pair = lambda dtype: torch.empty(tokens, topk, dtype=dtype, device=device)  # noqa: E731
        self._t = (pair(torch.int32), pair(torch.float32),
                   torch.empty(experts + 1, dtype=torch.int32, device=device),
                   torch.zeros(tokens * topk, dtype=torch.int32, device=device), pair(torch.int32))
        self._ws = torch.empty(n.value, dtype=torch.uint8, device=device) if n.value else None
        self._ptrs = tuple(_vp(t.data_ptr()) for t in self._t)
        self._ws_args = (_vp(self._ws.data_ptr()), n.value) if n.value else (None, 0)
        self._dev = self._t[2].get_device()

    tokens = property(lambda self: self._shape[0])
    experts = property(lambda self: self._shape[1])
    topk = property(lambda self: self._shape[2])
    ids = property(lambda self: self._t[0])
    weights = property(lambda self: self._t[1])
    offsets = property(lambda self: self._t[2])
    rows = property(lambda self: self._t[3])
    slots = property(lambda self: self._t[4])

    def _check_device(self, dev: int) -> None:
        if self._dev != dev:
            raise ValueError(f"routing: must be on the current device, is on {self._t[2].device}")


def _router(logits: torch.Tensor, bias: torch.Tensor | None, scoring: str, tokens: int, experts: int, dev: int):
    """Type, scoring, row stride and bias pointer of a router's scores."""
    kind = _TYPES.get(logits.dtype)
    if kind is None:
        raise ValueError(f"logits: float32 or bfloat16 expected, got {logits.dtype}")
    score = SCORE.get(scoring)
    if score is None:
        raise ValueError(f"scoring: one of {sorted(SCORE)} expected, got {scoring!r}")
    ld = _rows2d(logits, "logits", dev)
    if logits.shape != (tokens, experts):
        raise ValueError(f"logits: shape {(tokens, experts)} expected, got {tuple(logits.shape)}")
    return kind, score, ld, _want(bias, "bias", torch.float32, (experts,), dev) if bias is not None else None


def uw_route_experts(logits: torch.Tensor, routing: Routing, scoring: str = "softmax_topk",
                     bias: torch.Tensor | None = None, stream=None) -> None:
    """logits [tokens][experts] FP32 or BF16 (rows may be strided) -> routing's ids, weights and plan.

    bias [experts] FP32 is added to the logits for the choice, with "sigmoid_biased" to their sigmoids; the
    weights are without it.
    """
    tokens, experts, topk = routing._shape
    dev = _current()
    kind, score, ld, pb = _router(logits, bias, scoring, tokens, experts, dev)
    routing._check_device(dev)
    _check(_lib.uw_route_experts(logits.data_ptr(), kind, tokens, experts, ld, pb, topk, score, *routing._ptrs,
                                 *routing._ws_args, _stream(stream)), "uw_route_experts")


def uw_plan_experts(ids: torch.Tensor, routing: Routing, stream=None) -> None:
    """The plan for choices made elsewhere: ids [tokens][topk] int32, outside 0..experts-1 = none."""
    tokens, experts, topk = routing._shape
    dev = _current()
    pi = _want(ids, "ids", torch.int32, (tokens, topk), dev)
    routing._check_device(dev)
    _check(_lib.uw_plan_experts(pi, tokens, experts, topk, *routing._ptrs[2:], *routing._ws_args, _stream(stream)),
           "uw_plan_experts")


class Experts:
    """Owns one uw_experts handle and keeps the weights it names alive."""

    def __init__(self, handle: int, count: int, n: int, k: int, keep):
        self.handle = ctypes.c_void_p(handle)
        self.count, self.n, self.k, self.keep = count, n, k, keep

    def free(self) -> None:
        if self.handle and self.handle.value:
            _lib.uw_free_experts(self.handle)
            self.handle = ctypes.c_void_p(None)
        self.keep = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def uw_experts_bf16(w: torch.Tensor, count: int, n: int, k: int, stride: int = 0) -> Experts:
    """w: BF16, expert e's [n][k] at element e * stride (0: n * k); w may be a view into a larger array, whose
    rows are k long and adjacent (see _stack)."""
    if w.dtype is not torch.bfloat16:
        raise ValueError(f"w: bfloat16 expected, got {w.dtype}")
    _on_device(w, "w", _current())
    h = ctypes.c_void_p()
    _check(_lib.uw_experts_bf16(w.data_ptr(), count, n, k, stride, ctypes.byref(h)), "uw_experts_bf16")
    try:
        _stack(w, "w", count, n, k, stride)
        _holds(w, 2 * (((stride or n * k) * (count - 1)) + n * k), "w")
    except ValueError:
        _lib.uw_free_experts(h)
        raise
    return Experts(h.value, count, n, k, w)


def _stack(t: torch.Tensor, what: str, count: int, n: int, cols: int, stride: int) -> None:
    """t's own shape and strides agree with `count` matrices [n][cols], `stride` elements apart (0: n * cols).

    In one dimension t is contiguous.  In two or more its rows are the matrices' rows, adjacent.  A stack that
    is not contiguous as a whole, like [:, 0] of [experts][2][n][cols], is walked along its first dimension, so
    stride has to be a multiple of that dimension's; without a stride a stack is [experts][n][cols] or holds
    nothing but the matrices.
    """
    if t.dim() < 2:
        ok = t.is_contiguous()
    else:
        shape, total = t.shape, count * n * cols
        ok = shape[-1] == cols and t.stride(-1) == 1 and (shape[-2] <= 1 or t.stride(-2) == cols)
        if t.dim() > 2 and t.is_contiguous():
            ok &= stride != 0 or t.numel() == total or (t.dim() == 3 and shape[1] == n and t.numel() > total)
        elif t.dim() > 2:
            ok &= shape[-2] >= n
            if count > 1:
                m, rest = divmod(stride or n * cols, t.stride(0)) if t.stride(0) else (0, 1)
                ok &= rest == 0 and (count - 1) * m < shape[0]
    if not ok:
        raise ValueError(f"{what}: {count} matrices [{n}][{cols}], {stride or n * cols} elements apart, are not a tensor "
                         f"of shape {tuple(t.shape)} and strides {t.stride()}")


def _holds(t: torch.Tensor, nbytes: int, what: str) -> None:
    """t's storage holds nbytes from t's first element on."""
    have = t.untyped_storage().nbytes() - t.storage_offset() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{what}: {nbytes} bytes expected, {have} there")


def uw_experts_mx4(elem: torch.Tensor, scale: torch.Tensor, count: int, n: int, k: int, elem_stride: int = 0,
                   scale_stride: int = 0) -> Experts:
    """elem, scale: uint8, expert e's [n][k/2] and [n][mx4_scale_stride(k)] at byte e * their stride (0: contiguous);
    views as for uw_experts_bf16."""
    for t, what in ((elem, "elem"), (scale, "scale")):
        if t.dtype is not torch.uint8:
            raise ValueError(f"{what}: uint8 expected, got {t.dtype}")
        _on_device(t, what, _current())
    h = ctypes.c_void_p()
    _check(_lib.uw_experts_mx4(elem.data_ptr(), scale.data_ptr(), count, n, k, elem_stride, scale_stride,
                               ctypes.byref(h)), "uw_experts_mx4")
    eb, sb = n * (k // 2), n * mx4_scale_stride(k)
    try:
        _stack(elem, "elem", count, n, k // 2, elem_stride)
        _stack(scale, "scale", count, n, mx4_scale_stride(k), scale_stride)
        _holds(elem, (elem_stride or eb) * (count - 1) + eb, "elem")
        _holds(scale, (scale_stride or sb) * (count - 1) + sb, "scale")
    except ValueError:
        _lib.uw_free_experts(h)
        raise
    return Experts(h.value, count, n, k, (elem, scale))


def uw_experts_fp8(elem: torch.Tensor, scale: torch.Tensor, count: int, n: int, k: int, elem_stride: int = 0,
                   scale_stride: int = 0) -> Experts:
    """elem: float8_e4m3fn (or uint8), expert e's [n][k] at element e * elem_stride; scale: FP32, expert e's
    [fp8_scale_shape(n, k, 128)] at element e * scale_stride (0: contiguous); views as for uw_experts_bf16."""
    if elem.dtype not in _E4M3:
        raise ValueError(f"elem: {_E4M3[0]} or {_E4M3[1]} expected, got {elem.dtype}")
    if scale.dtype is not torch.float32:
        raise ValueError(f"scale: {torch.float32} expected, got {scale.dtype}")
    for t, what in ((elem, "elem"), (scale, "scale")):
        _on_device(t, what, _current())
    h = ctypes.c_void_p()
    _check(_lib.uw_experts_fp8(elem.data_ptr(), scale.data_ptr(), count, n, k, elem_stride, scale_stride,
                               ctypes.byref(h)), "uw_experts_fp8")
    sr, sc = fp8_scale_shape(n, k, 128)
    try:
        _stack(elem, "elem", count, n, k, elem_stride)
        _stack(scale, "scale", count, sr, sc, scale_stride)
        _holds(elem, (elem_stride or n * k) * (count - 1) + n * k, "elem")
        _holds(scale, 4 * ((scale_stride or sr * sc) * (count - 1) + sr * sc), "scale")
    except ValueError:
        _lib.uw_free_experts(h)
        raise
    return Experts(h.value, count, n, k, (elem, scale))


def uw_experts_uwf1(ms, stream=None) -> Experts:
    """ms: compressed matrices of one shape with resident palette indices, one per expert."""
    arr = (ctypes.c_void_p * len(ms))(*[m.handle.value for m in ms])
    h = ctypes.c_void_p()
    _check(_lib.uw_experts_uwf1(arr, len(ms), _stream(stream), ctypes.byref(h)), "uw_experts_uwf1")
    i = ms[0].info()
    return Experts(h.value, len(ms), i.n, i.k, list(ms))


def uw_free_experts(w: Experts) -> None:
    w.free()


def _ragged(w: Experts, offsets: torch.Tensor, rows, x: torch.Tensor, y: torch.Tensor, dtype):
    if x.dim() != 2 or x.shape[1] != w.k:
        raise ValueError(f"x: shape [rows, {w.k}] expected, got {tuple(x.shape)}")
    if y.dim() != 2 or y.shape[1] != w.n:
        raise ValueError(f"output: shape [slots, {w.n}] expected, got {tuple(y.shape)}")
    slots, dev = y.shape[0], _current()
    po = _want(offsets, "offsets", torch.int32, (w.count + 1,), dev)
    pr = _want(rows, "rows", torch.int32, (slots,), dev) if rows is not None else None
    return po, pr, slots, _want(x, "x", torch.bfloat16, None, dev), x.shape[0], _want(y, "output", dtype, None, dev)


def uw_matmul_experts(w: Experts, offsets: torch.Tensor, rows: torch.Tensor | None, x: torch.Tensor,
                      y: torch.Tensor, stream=None) -> None:
    """y [slots][n] FP32, x [x_rows][k] BF16; rows [slots] int32 or None (slot s multiplies row s)."""
    _check(_lib.uw_matmul_experts(w.handle, *_ragged(w, offsets, rows, x, y, torch.float32), _stream(stream)),
           "uw_matmul_experts")


def uw_matmul_experts_gated(gate: Experts, up: Experts, offsets: torch.Tensor, rows: torch.Tensor | None,
                            x: torch.Tensor, h: torch.Tensor, stream=None) -> None:
    """h [slots][n] BF16 = silu(x . gate^T) * (x . up^T)."""
    _check(_lib.uw_matmul_experts_gated(gate.handle, up.handle, *_ragged(gate, offsets, rows, x, h, torch.bfloat16),
                                        _stream(stream)), "uw_matmul_experts_gated")


def uw_workspace_size_expert_mlp(gate: Experts, down: Experts, tokens: int, topk: int) -> int:
    b = ctypes.c_size_t()
    _check(_lib.uw_workspace_size_expert_mlp(gate.handle, down.handle, tokens, topk, ctypes.byref(b)),
           "uw_workspace_size_expert_mlp")
    return b.value


def uw_expert_mlp(gate: Experts, up: Experts, down: Experts, routing: Routing, x: torch.Tensor, out: torch.Tensor,
                  ws: torch.Tensor, stream=None) -> None:
    """out [tokens][k] BF16: the layer's MLP on a routing made by uw_route_experts (or a plan and weights)."""
    tokens, experts, topk = routing._shape
    if experts != gate.count:
        raise ValueError(f"routing: {gate.count} experts expected, got {experts}")
    dev = _current()
    px = _want(x, "x", torch.bfloat16, (tokens, gate.k), dev)
    po = _want(out, "out", torch.bfloat16, (tokens, gate.k), dev)
    routing._check_device(dev)
    _, weights, offsets, rows, slots = routing._ptrs
    _check(_lib.uw_expert_mlp(gate.handle, up.handle, down.handle, tokens, topk, offsets, rows, slots, weights, px, po,
                              *_ws(ws, dev), _stream(stream)), "uw_expert_mlp")


def uw_workspace_size_expert_layer(gate: Experts, down: Experts, tokens: int, topk: int) -> int:
    b = ctypes.c_size_t()
    _check(_lib.uw_workspace_size_expert_layer(gate.handle, down.handle, tokens, topk, ctypes.byref(b)),
           "uw_workspace_size_expert_layer")
    return b.value


def uw_expert_layer(gate: Experts, up: Experts, down: Experts, logits: torch.Tensor, routing: Routing, x: torch.Tensor,
                    out: torch.Tensor, ws: torch.Tensor, scoring: str = "softmax_topk",
                    bias: torch.Tensor | None = None, stream=None) -> None:
    """uw_route_experts into routing and uw_expert_mlp on it: out [tokens][k] BF16, logits [tokens][experts]."""
    tokens, experts, topk = routing._shape
    if experts != gate.count:
        raise ValueError(f"routing: {gate.count} experts expected, got {experts}")
    dev = _current()
    kind, score, ld, pb = _router(logits, bias, scoring, tokens, experts, dev)
    px = _want(x, "x", torch.bfloat16, (tokens, gate.k), dev)
    po = _want(out, "out", torch.bfloat16, (tokens, gate.k), dev)
    routing._check_device(dev)
    _check(_lib.uw_expert_layer(gate.handle, up.handle, down.handle, logits.data_ptr(), kind, tokens, ld, pb, topk, score,
                                *routing._ptrs, px, po, *_ws(ws, dev), _stream(stream)), "uw_expert_layer")
