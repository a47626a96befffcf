"""Python binding of libmla (absorbed MLA decode over a latent KV cache, GB300).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch provides device memory and the current stream.  There is no
fallback: if ``_build/libmla.so`` is missing the first call raises.

Functions mirror the C ABI in ``include/mla.h``:
    cache_append, workspace_size, decode, decode_sparse, workspace_status
and over a paged cache:
    paged_append, paged_workspace_size, paged_decode, paged_weights, paged_evict,
    paged_append_rotary, paged_read, paged_decode_window
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import threading

import torch

from . import layout  # noqa: F401  (byte/flop accounting)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmla.so")

MLA_KV_BF16 = 0
MLA_KV_FP8_E4M3_B128 = 1
MLA_KV_FP8_E4M3_B128_POW2 = 2
DEV_END_POS_CLAMPED = 0x1
DEV_APPEND_SKIPPED = 0x2
DEV_PIPELINE_TIMEOUT = 0x4
DEV_BAD_PAGE = 0x8

STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_OUT_OF_RANGE",
          3: "MLA_ERR_UNSUPPORTED", 4: "MLA_ERR_WORKSPACE", 5: "MLA_ERR_CUDA"}


class MLAError(RuntimeError):
    def __init__(self, code: int, what: str, detail: str = ""):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}" + (f" ({detail})" if detail else ""))


class _CCache(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("max_batch", ctypes.c_int32),
                ("max_seq_len", ctypes.c_int32), ("kv", ctypes.c_void_p),
                ("kv_scale", ctypes.c_void_p), ("pe", ctypes.c_void_p)]


class _CRotary(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("gain", ctypes.c_float), ("halves", ctypes.c_int32)]


class _CPagedCache(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("kv", ctypes.c_void_p),
                ("kv_scale", ctypes.c_void_p), ("pe", ctypes.c_void_p), ("weight", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmla.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: run `python -m mla_latent_kv_07_gb300.build`")
            L = ctypes.CDLL(LIB_PATH)
            P, I32, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
            L.mla_cache_append.argtypes = [P, P, P, P, I32, P]
            L.mla_cache_append.restype = I32
            L.mla_workspace_size.argtypes = [I32, I32, I32, I32]
            L.mla_workspace_size.restype = SZ
            L.mla_decode.argtypes = [P, P, P, P, I32, I32, I32, F, P, P, P, SZ, P]
            L.mla_decode.restype = I32
            L.mla_decode_append.argtypes = [P, P, P, P, P, P, I32, I32, I32, F, P, P, P, SZ, P]
            L.mla_decode_append.restype = I32
            L.mla_topk_select.argtypes = [P, P, I32, I32, I32, P, P]
            L.mla_topk_select.restype = I32
            L.mla_selftest_decode_timeout.argtypes = [P, P, P, P, I32, I32, I32, F, P, P, P, SZ, P]
            L.mla_selftest_decode_timeout.restype = I32
            L.mla_decode_mtp.argtypes = [P, P, P, P, I32, I32, I32, I32, F, P, P, P, SZ, P]
            L.mla_decode_mtp.restype = I32
            L.mla_decode_sparse.argtypes = [P, P, P, P, I32, I32, I32, F, P, I32, P, P, P, P, P,
                                            P, P, SZ, P]
            L.mla_decode_sparse.restype = I32
            L.mla_workspace_status.argtypes = [P, P, P]
            L.mla_workspace_status.restype = I32
            L.mla_status_string.argtypes = [I32]
            L.mla_status_string.restype = ctypes.c_char_p
            L.mla_last_error.restype = ctypes.c_char_p
            L.mla_decode_noalloc.argtypes = [P, P, P, P, I32, I32, I32, F, P, P, P]
            L.mla_decode_noalloc.restype = I32
            L.mla_absorb_q.argtypes = [P, P, I32, I32, P, P, P]
            L.mla_absorb_q.restype = I32
            L.mla_project_out.argtypes = [P, P, I32, I32, P, P, P]
            L.mla_project_out.restype = I32
            L.mla_read_ceiling.argtypes = [P, SZ, P, P]
            L.mla_read_ceiling.restype = I32
            L.mla_trace_begin.argtypes = [I32]
            L.mla_trace_begin.restype = I32
            L.mla_trace_end.argtypes = [P, P, P]
            L.mla_trace_end.restype = I32
            L.mla_paged_append.argtypes = [P, P, I32, P, P, P, I32, I32, P, P]
            L.mla_paged_append.restype = I32
            L.mla_paged_workspace_size.argtypes = [I32, I32]
            L.mla_paged_workspace_size.restype = SZ
            L.mla_paged_decode.argtypes = [P, P, I32, P, P, P, I32, I32, I32, F, P, P, P, P, P, SZ, P]
            L.mla_paged_decode.restype = I32
            L.mla_paged_weights.argtypes = [P, P, I32, P, P, P, P, I32, I32, I32, F, P, P]
            L.mla_paged_weights.restype = I32
            L.mla_selftest_paged_decode_timeout.argtypes = [P, P, I32, P, P, P, I32, I32, I32, F, P, P, P, SZ, P]
            L.mla_selftest_paged_decode_timeout.restype = I32
            L.mla_selftest_paged_weights_timeout.argtypes = [P, P, I32, P, P, P, P, I32, I32, I32, F, P, P]
            L.mla_selftest_paged_weights_timeout.restype = I32
            L.mla_paged_evict.argtypes = [P, P, I32, P, I32, I32, I32, I32, I32, P, I32, P, P, P, P]
            L.mla_paged_evict.restype = I32
            I64 = ctypes.c_int64
            L.mla_rotary_turns.argtypes = [P, I32, P]
            L.mla_rotary_turns.restype = I32
            L.mla_paged_append_rotary.argtypes = [P, P, I32, P, I64, I64, P, I32, F, P, P, P, I32, I32, P, I64, I64, I64,
                                                  I32, P, P, P, P]
            L.mla_paged_append_rotary.restype = I32
            L.mla_paged_read.argtypes = [P, P, I32, P, P, I32, I32, P, I64, P, I64, P, P]
            L.mla_paged_read.restype = I32
            L.mla_paged_window_workspace_size.argtypes = [I32, I32, I32]
            L.mla_paged_window_workspace_size.restype = SZ
            L.mla_paged_decode_window.argtypes = [P, P, I32, P, P, P, I32, I32, I32, I32, F, I32, I32, P, P, P, SZ, P]
            L.mla_paged_decode_window.restype = I32
            L.mla_selftest_paged_window_timeout.argtypes = L.mla_paged_decode_window.argtypes
            L.mla_selftest_paged_window_timeout.restype = I32
            _lib = L
    return _lib


_host = None


def native():
    """The host extension (csrc/native.cpp), bound to the loaded libmla (raises if
    it was not built)."""
    global _host
    if _host is None:
        L = lib()
        path = os.path.join(os.path.dirname(LIB_PATH), "_mla_native.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: run `python -m mla_latent_kv_07_gb300.build`")
        spec = importlib.util.spec_from_loader("_mla_native", importlib.machinery.ExtensionFileLoader("_mla_native", path))
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        if str(torch.__version__) != m.torch_version:   # (it uses torch's C++ classes as they were then)
            raise RuntimeError(f"{path} was built against torch {m.torch_version}, this is {torch.__version__}: "
                               "run `python -m mla_latent_kv_07_gb300.build`")
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.mla_paged_append_rotary, L.mla_paged_read, L.mla_paged_decode_window, L.mla_paged_window_workspace_size)))
        _host = m
    return _host


def _check(code: int, what: str):
    if code != 0:
        raise MLAError(code, what, lib().mla_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, shape, name):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: want contiguous cuda {dtype} {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


class Cache:
    """Caller-owned latent cache: kv [Bmax, S, 512] (bf16 or e4m3 bytes),
    kv_scale fp32 [Bmax, S, 4] (FP8 formats only), pe bf16 [Bmax, S, 64].
    fmt: MLA_KV_BF16, MLA_KV_FP8_E4M3_B128, or MLA_KV_FP8_E4M3_B128_POW2
    (FP8 whose appends round every block scale up to a power of two)."""

    def __init__(self, max_batch: int, max_seq_len: int, fmt: int = MLA_KV_BF16,
                 device="cuda", kv=None, kv_scale=None, pe=None):
        self.fmt, self.max_batch, self.max_seq_len = fmt, max_batch, max_seq_len
        shape = (max_batch, max_seq_len)
        if kv is None:
            kv = torch.zeros(shape + (512,), dtype=torch.bfloat16 if fmt == 0 else torch.uint8,
                             device=device)
        if fmt != MLA_KV_BF16 and kv_scale is None:
            kv_scale = torch.zeros(shape + (4,), dtype=torch.float32, device=device)
        if pe is None:
            pe = torch.zeros(shape + (64,), dtype=torch.bfloat16, device=device)
        _need(kv, torch.bfloat16 if fmt == 0 else torch.uint8, shape + (512,), "kv")
        _need(pe, torch.bfloat16, shape + (64,), "pe")
        if fmt != MLA_KV_BF16:
            _need(kv_scale, torch.float32, shape + (4,), "kv_scale")
        self.kv, self.kv_scale, self.pe = kv, kv_scale, pe
        self._c = _CCache(fmt, max_batch, max_seq_len, kv.data_ptr(),
                          kv_scale.data_ptr() if kv_scale is not None else None, pe.data_ptr())

    @property
    def ref(self):
        return ctypes.byref(self._c)


def cache_append(cache: Cache, kv_new, pe_new, start_pos, stream=None) -> None:
    """Write kv_new[b] / pe_new[b] (bf16 [B,512] / [B,64]) at row start_pos[b]."""
    B = kv_new.shape[0]
    _need(kv_new, torch.bfloat16, (B, 512), "kv_new")
    _need(pe_new, torch.bfloat16, (B, 64), "pe_new")
    pos = (ctypes.c_int32 * B)(*[int(x) for x in start_pos])
    _check(lib().mla_cache_append(cache.ref, _ptr(kv_new), _ptr(pe_new), pos, B,
                                  _stream(stream)), "mla_cache_append")


def workspace_size(B: int, H: int, max_end_pos: int, topk: int = 0) -> int:
    n = lib().mla_workspace_size(B, H, max_end_pos, topk)
    if n == 0:
        raise MLAError(3, "mla_workspace_size")
    return int(n)


def alloc_workspace(B: int, H: int, max_end_pos: int, topk: int = 0, device="cuda"):
    return torch.empty(workspace_size(B, H, max_end_pos, topk), dtype=torch.uint8, device=device)


def _outputs(B, H, device, out, lse, want_lse):
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=device)
    if lse is None and want_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=device)
    return out, lse


def decode(cache: Cache, q_latent, q_pe, end_pos, max_end_pos: int, softmax_scale: float,
           out=None, lse=None, workspace=None, want_lse: bool = True, stream=None):
    """Absorbed decode; returns (out bf16 [B,H,512], lse fp32 [B,H] or None)."""
    B, H, _ = q_latent.shape
    _need(q_latent, torch.bfloat16, (B, H, 512), "q_latent")
    _need(q_pe, torch.bfloat16, (B, H, 64), "q_pe")
    _need(end_pos, torch.int32, (B,), "end_pos")
    out, lse = _outputs(B, H, q_latent.device, out, lse, want_lse)
    if workspace is None:
        workspace = alloc_workspace(B, H, max_end_pos, 0, q_latent.device)
    _check(lib().mla_decode(cache.ref, _ptr(q_latent), _ptr(q_pe), _ptr(end_pos), int(max_end_pos),
                            B, H, float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                            workspace.numel(), _stream(stream)), "mla_decode")
    return out, lse


def decode_append(cache: Cache, kv_new, pe_new, q_latent, q_pe, end_pos, max_end_pos: int,
                  softmax_scale: float, out=None, lse=None, workspace=None, want_lse: bool = True,
                  stream=None):
    """Append row end_pos[b]-1 of every sequence (kv_new bf16 [B,512], pe_new
    bf16 [B,64]) and decode over it, in one call (see mla_decode_append);
    returns (out, lse) as decode."""
    B, H, _ = q_latent.shape
    _need(kv_new, torch.bfloat16, (B, 512), "kv_new")
    _need(pe_new, torch.bfloat16, (B, 64), "pe_new")
    _need(q_latent, torch.bfloat16, (B, H, 512), "q_latent")
    _need(q_pe, torch.bfloat16, (B, H, 64), "q_pe")
    _need(end_pos, torch.int32, (B,), "end_pos")
    out, lse = _outputs(B, H, q_latent.device, out, lse, want_lse)
    if workspace is None:
        workspace = alloc_workspace(B, H, max_end_pos, 0, q_latent.device)
    _check(lib().mla_decode_append(cache.ref, _ptr(kv_new), _ptr(pe_new), _ptr(q_latent), _ptr(q_pe),
                                   _ptr(end_pos), int(max_end_pos), B, H, float(softmax_scale), _ptr(out),
                                   _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)),
           "mla_decode_append")
    return out, lse


def topk_select(scores, end_pos, K: int, out=None, stream=None):
    """Top-k positions per sequence from fp32 scores [B, max_end_pos]:
    int32 [B, K], increasing, -1 padded (the index lists decode_sparse takes)."""
    B, S = scores.shape
    if scores.dtype != torch.float32 or not scores.is_contiguous() or not scores.is_cuda:
        raise ValueError(f"scores: want contiguous cuda float32 [B, S], got {scores.dtype} on {scores.device}")
    _need(end_pos, torch.int32, (B,), "end_pos")
    if out is None:
        out = torch.empty((B, K), dtype=torch.int32, device=scores.device)
    _need(out, torch.int32, (B, K), "out")
    _check(lib().mla_topk_select(_ptr(scores), _ptr(end_pos), B, S, int(K), _ptr(out), _stream(stream)),
           "mla_topk_select")
    return out


def selftest_decode_timeout(cache: Cache, q_latent, q_pe, end_pos, max_end_pos: int,
                            softmax_scale: float, workspace, stream=None) -> int:
    """mla_decode with the first unit's first tile withheld and short waits:
    returns the workspace status word (MLA_DEV_PIPELINE_TIMEOUT expected)."""
    B, H, _ = q_latent.shape
    _need(q_latent, torch.bfloat16, (B, H, 512), "q_latent")
    _need(q_pe, torch.bfloat16, (B, H, 64), "q_pe")
    _need(end_pos, torch.int32, (B,), "end_pos")
    out, lse = _outputs(B, H, q_latent.device, None, None, True)
    _check(lib().mla_selftest_decode_timeout(cache.ref, _ptr(q_latent), _ptr(q_pe), _ptr(end_pos),
                                             int(max_end_pos), B, H, float(softmax_scale), _ptr(out),
                                             _ptr(lse), _ptr(workspace), workspace.numel(),
                                             _stream(stream)), "mla_selftest_decode_timeout")
    return workspace_status(workspace, stream)


def decode_mtp(cache: Cache, q_latent, q_pe, end_pos, max_end_pos: int, softmax_scale: float,
               out=None, lse=None, workspace=None, want_lse: bool = True, stream=None):
    """Multi-token decode of s new tokens per sequence (token j of sequence b
    attends to positions 0 .. end_pos[b]-s+j); q_latent [B,s,H,512], q_pe
    [B,s,H,64].  Returns (out bf16 [B,s,H,512], lse fp32 [B,s,H] or None)."""
    B, s, H, _ = q_latent.shape
    _need(q_latent, torch.bfloat16, (B, s, H, 512), "q_latent")
    _need(q_pe, torch.bfloat16, (B, s, H, 64), "q_pe")
    _need(end_pos, torch.int32, (B,), "end_pos")
    out, lse = _outputs(B * s, H, q_latent.device, None if out is None else out.view(B * s, H, 512),
                        None if lse is None else lse.view(B * s, H), want_lse)
    if workspace is None:
        workspace = alloc_workspace(B * s, H, max_end_pos, 0, q_latent.device)
    _check(lib().mla_decode_mtp(cache.ref, _ptr(q_latent), _ptr(q_pe), _ptr(end_pos),
                                int(max_end_pos), B, s, H, float(softmax_scale), _ptr(out), _ptr(lse),
                                _ptr(workspace), workspace.numel(), _stream(stream)), "mla_decode_mtp")
    return out.view(B, s, H, 512), None if lse is None else lse.view(B, s, H)


def decode_noalloc(cache: Cache, q_latent, q_pe, end_pos, max_end_pos: int, softmax_scale: float,
                   out=None, lse=None, want_lse: bool = True, stream=None):
    """Dense decode through mla_decode_noalloc: no workspace is passed; the
    library uses its own static device scratch (for callers that cannot
    allocate).  Returns (out, lse)."""
    B, H, _ = q_latent.shape
    _need(q_latent, torch.bfloat16, (B, H, 512), "q_latent")
    _need(q_pe, torch.bfloat16, (B, H, 64), "q_pe")
    _need(end_pos, torch.int32, (B,), "end_pos")
    out, lse = _outputs(B, H, q_latent.device, out, lse, want_lse)
    _check(lib().mla_decode_noalloc(cache.ref, _ptr(q_latent), _ptr(q_pe), _ptr(end_pos),
                                    int(max_end_pos), B, H, float(softmax_scale), _ptr(out),
                                    _ptr(lse), _stream(stream)), "mla_decode_noalloc")
    return out, lse


def decode_sparse(cache: Cache, q_latent, q_pe, end_pos, max_end_pos: int, softmax_scale: float,
                  topk, kv_new=None, pe_new=None, out=None, lse=None, gidx=None, gcount=None,
                  workspace=None, want_lse: bool = True, stream=None):
    """Top-k sparse decode (optionally appending kv_new/pe_new at end_pos-1 first).
    Returns (out, lse)."""
    B, H, _ = q_latent.shape
    K = topk.shape[1]
    _need(q_latent, torch.bfloat16, (B, H, 512), "q_latent")
    _need(q_pe, torch.bfloat16, (B, H, 64), "q_pe")
    _need(end_pos, torch.int32, (B,), "end_pos")
    _need(topk, torch.int32, (B, K), "topk")
    if kv_new is not None:
        _need(kv_new, torch.bfloat16, (B, 512), "kv_new")
        _need(pe_new, torch.bfloat16, (B, 64), "pe_new")
    out, lse = _outputs(B, H, q_latent.device, out, lse, want_lse)
    if workspace is None:
        workspace = alloc_workspace(B, H, max_end_pos, K, q_latent.device)
    _check(lib().mla_decode_sparse(cache.ref, _ptr(q_latent), _ptr(q_pe), _ptr(end_pos),
                                   int(max_end_pos), B, H, float(softmax_scale), _ptr(topk), K,
                                   _ptr(kv_new), _ptr(pe_new), _ptr(out), _ptr(lse), _ptr(gidx),
                                   _ptr(gcount), _ptr(workspace), workspace.numel(),
                                   _stream(stream)), "mla_decode_sparse")
    return out, lse


def workspace_status(workspace, stream=None) -> int:
    flags = ctypes.c_uint32(0)
    _check(lib().mla_workspace_status(_ptr(workspace), ctypes.byref(flags), _stream(stream)),
           "mla_workspace_status")
    return int(flags.value)


def absorb_q(q_nope, wkv_b, out=None, status=None, stream=None):
    """q_latent [B,H,512] bf16 = q_nope [B,H,128] . W_UK (rows 0..127 of each
    head of wkv_b [H,256,512] bf16)."""
    B, H, _ = q_nope.shape
    _need(q_nope, torch.bfloat16, (B, H, 128), "q_nope")
    _need(wkv_b, torch.bfloat16, (H, 256, 512), "wkv_b")
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q_nope.device)
    _need(out, torch.bfloat16, (B, H, 512), "out")
    _check(lib().mla_absorb_q(_ptr(q_nope), _ptr(wkv_b), B, H, _ptr(out), _ptr(status), _stream(stream)),
           "mla_absorb_q")
    return out


def project_out(x, wkv_b, out=None, status=None, stream=None):
    """o [B,H,128] bf16 = W_UV . x for x [B,H,512] bf16 (W_UV: rows 128..255
    of each head of wkv_b)."""
    B, H, _ = x.shape
    _need(x, torch.bfloat16, (B, H, 512), "x")
    _need(wkv_b, torch.bfloat16, (H, 256, 512), "wkv_b")
    if out is None:
        out = torch.empty((B, H, 128), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, (B, H, 128), "out")
    _check(lib().mla_project_out(_ptr(x), _ptr(wkv_b), B, H, _ptr(out), _ptr(status), _stream(stream)),
           "mla_project_out")
    return out


def read_ceiling(buf: torch.Tensor, sink: torch.Tensor, stream=None) -> None:
    """Stream all bytes of the contiguous CUDA tensor `buf` (a measurement of
    the achievable HBM read rate); XOR-folds them into the int32 `sink`."""
    if not (buf.is_cuda and buf.is_contiguous()):
        raise ValueError("buf must be a contiguous CUDA tensor")
    if sink.dtype != torch.int32 or not sink.is_cuda or sink.numel() < 1:
        raise ValueError("sink must be a CUDA int32 tensor")
    nbytes = buf.numel() * buf.element_size()
    _check(lib().mla_read_ceiling(buf.data_ptr(), nbytes, sink.data_ptr(), _stream(stream)),
           "mla_read_ceiling")


# ------------------------------------------------------------ paged cache

class PagedCache:
    """Caller-owned pool of pages: kv [num_pages, page_size, 512] (bf16 or e4m3
    bytes), kv_scale fp32 [num_pages, page_size, 4] (FP8 formats only), pe bf16
    [num_pages, page_size, 64], weight fp32 [num_pages, page_size] (the
    attention weight each row has received; needed by paged_weights and
    paged_evict; made unless ``weight=False`` says the pool has none).  page_size: a multiple of 16.
    The tensors may be replaced by assignment (``pool.weight = ...``; None: no weights).
    Position t of sequence b is row t % page_size of page table[b, t // page_size]."""

    def __init__(self, num_pages: int, page_size: int, fmt: int = MLA_KV_BF16, device="cuda",
                 kv=None, kv_scale=None, pe=None, weight=None):
        shape = (num_pages, page_size)
        if kv is None:
            kv = torch.zeros(shape + (512,), dtype=torch.bfloat16 if fmt == 0 else torch.uint8,
                             device=device)
        if fmt != MLA_KV_BF16 and kv_scale is None:
            kv_scale = torch.zeros(shape + (4,), dtype=torch.float32, device=device)
        if pe is None:
            pe = torch.zeros(shape + (64,), dtype=torch.bfloat16, device=device)
        if weight is None:
            weight = torch.zeros(shape, dtype=torch.float32, device=device)
        self._c = _CPagedCache(fmt, num_pages, page_size)
        self.ref, self._addr = ctypes.byref(self._c), ctypes.addressof(self._c)
        self.device, self._dev = kv.device, kv.get_device()
        self._t = {}
        self.kv, self.pe = kv, pe
        self.kv_scale = kv_scale if fmt != MLA_KV_BF16 else None
        self.weight = None if weight is False else weight

    fmt = property(lambda self: self._c.fmt)
    num_pages = property(lambda self: self._c.num_pages)
    page_size = property(lambda self: self._c.page_size)

    def _member(name):
        """A tensor of the pool; assigning another one checks it, and later
        calls use it (captured graphs keep the tensor they were captured with)."""
        def put(self, t):
            fp8 = self.fmt != MLA_KV_BF16
            dtype, width = {"kv": (torch.uint8 if fp8 else torch.bfloat16, (512,)), "pe": (torch.bfloat16, (64,)),
                            "kv_scale": (torch.float32, (4,)), "weight": (torch.float32, ())}[name]
            if t is None and (name == "weight" or (name == "kv_scale" and not fp8)):
                setattr(self._c, name, None)
            else:
                if name == "kv_scale" and not fp8:
                    raise ValueError("kv_scale: a bf16 pool has none")
                if t is None:
                    raise ValueError(f"{name}: the pool needs one")
                _need(t, dtype, (self.num_pages, self.page_size) + width, name)
                if t.device != self.device:
                    raise ValueError(f"{name}: on {t.device}, the pool on {self.device}")
                setattr(self._c, name, t.data_ptr())
            self._t[name] = t
        return property(lambda self: self._t[name], put)

    kv, kv_scale, pe, weight = _member("kv"), _member("kv_scale"), _member("pe"), _member("weight")
    del _member


# A serving loop makes these calls for every layer of every step, so their
# checks are written out: an attribute of a tensor costs about 0.1 us, the
# stream object of torch.cuda.current_stream() 2.8 us.
_raw_stream = torch._C._cuda_getCurrentRawStream
_bf16, _i32, _f32 = torch.bfloat16, torch.int32, torch.float32


def _off(t, dtype, shape, dev):
    return t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev


def _refuse(name, t, dtype, shape, dev):
    raise ValueError(f"{name}: want contiguous {dtype} {tuple(shape)} on cuda:{dev}, got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _new(shape, dtype, cache, stream):
    """A tensor for a call on `stream` (None: the current one), from that
    stream's memory: what other streams still do with a block they gave back
    does not reach it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=cache.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=cache.device)


def _int32(v, fn, name):
    """v for an int32 argument (which would keep the low 32 bits of a larger number)."""
    v = int(v)
    if not -0x80000000 <= v <= 0x7FFFFFFF:
        raise MLAError(2, fn, name)
    return v


def _paged_call(cache, fn, args, stream):
    """fn(pool, *args, stream) on the pool's device."""
    dev = cache._dev
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            code = fn(cache.ref, *args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    else:
        code = fn(cache.ref, *args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if code != 0:
        _check(code, fn.__name__)


def _table_width(name, t, B, dev):
    if t.dim() != 2:
        raise ValueError(f"{name}: want [{B}, max_pages], got {tuple(t.shape)}")
    n = t.shape[1]
    if _off(t, _i32, (B, n), dev):
        _refuse(name, t, _i32, (B, n), dev)
    return n


def paged_append(cache: PagedCache, table, kv_new, pe_new, end_pos, status=None, stream=None) -> None:
    """Write new row j of sequence b (kv_new bf16 [B, s, 512], pe_new bf16
    [B, s, 64]) at position end_pos[b] - s + j; its weight becomes 0.  status:
    None or an int32 [1] the DEV_* bits are ORed into (here and below)."""
    dev = cache._dev
    B, s = kv_new.shape[:2]
    if _off(kv_new, _bf16, (B, s, 512), dev):
        _refuse("kv_new", kv_new, _bf16, (B, s, 512), dev)
    if _off(pe_new, _bf16, (B, s, 64), dev):
        _refuse("pe_new", pe_new, _bf16, (B, s, 64), dev)
    if _off(end_pos, _i32, (B,), dev):
        _refuse("end_pos", end_pos, _i32, (B,), dev)
    if status is not None and _off(status, _i32, (1,), dev):
        _refuse("status", status, _i32, (1,), dev)
    n = _table_width("table", table, B, dev)
    _paged_call(cache, lib().mla_paged_append,
                (table.data_ptr(), n, kv_new.data_ptr(), pe_new.data_ptr(), end_pos.data_ptr(), B, s,
                 None if status is None else status.data_ptr()), stream)


def paged_workspace_size(B: int, H: int) -> int:
    n = lib().mla_paged_workspace_size(B, H)
    if n == 0:
        raise MLAError(3, "mla_paged_workspace_size")
    return int(n)


def alloc_paged_workspace(B: int, H: int, device="cuda"):
    return torch.empty(paged_workspace_size(B, H), dtype=torch.uint8, device=device)


def paged_decode(cache: PagedCache, table, q_latent, q_pe, end_pos, max_end_pos: int,
                 softmax_scale: float, kv_new=None, pe_new=None, out=None, lse=None, workspace=None,
                 want_lse: bool = True, stream=None):
    """Absorbed decode over a paged cache (table int32 [B, max_pages]), writing
    row end_pos[b] - 1 of every sequence first if kv_new (bf16 [B, 512]) and
    pe_new (bf16 [B, 64]) are given; returns (out bf16 [B, H, 512], lse fp32
    [B, H] or None).  Tensors that the call makes (outputs, workspace) belong to
    the stream it runs on."""
    dev, max_end_pos = cache._dev, _int32(max_end_pos, "mla_paged_decode", "max_end_pos")
    B, H = q_latent.shape[:2]
    if _off(q_latent, _bf16, (B, H, 512), dev):
        _refuse("q_latent", q_latent, _bf16, (B, H, 512), dev)
    if _off(q_pe, _bf16, (B, H, 64), dev):
        _refuse("q_pe", q_pe, _bf16, (B, H, 64), dev)
    if _off(end_pos, _i32, (B,), dev):
        _refuse("end_pos", end_pos, _i32, (B,), dev)
    n = _table_width("table", table, B, dev)
    new_kv = new_pe = None
    if kv_new is not None or pe_new is not None:
        if kv_new is None or pe_new is None:
            raise ValueError("kv_new and pe_new: both or neither")
        if _off(kv_new, _bf16, (B, 512), dev):
            _refuse("kv_new", kv_new, _bf16, (B, 512), dev)
        if _off(pe_new, _bf16, (B, 64), dev):
            _refuse("pe_new", pe_new, _bf16, (B, 64), dev)
        new_kv, new_pe = kv_new.data_ptr(), pe_new.data_ptr()
    if out is None:
        out = _new((B, H, 512), _bf16, cache, stream)
    elif _off(out, _bf16, (B, H, 512), dev):
        _refuse("out", out, _bf16, (B, H, 512), dev)
    if lse is None:
        if want_lse:
            lse = _new((B, H), _f32, cache, stream)
    elif _off(lse, _f32, (B, H), dev):
        _refuse("lse", lse, _f32, (B, H), dev)
    if workspace is None:
        workspace = _new((paged_workspace_size(B, H),), torch.uint8, cache, stream)
    nbytes = workspace.numel()
    if _off(workspace, torch.uint8, (nbytes,), dev):
        _refuse("workspace", workspace, torch.uint8, (nbytes,), dev)
    _paged_call(cache, lib().mla_paged_decode,
                (table.data_ptr(), n, q_latent.data_ptr(), q_pe.data_ptr(), end_pos.data_ptr(), max_end_pos,
                 B, H, float(softmax_scale), new_kv, new_pe, out.data_ptr(), None if lse is None else lse.data_ptr(),
                 workspace.data_ptr(), nbytes), stream)
    return out, lse


def paged_weights(cache: PagedCache, table, q_latent, q_pe, lse, end_pos, max_end_pos: int,
                  softmax_scale: float, status=None, stream=None) -> None:
    """cache.weight of every row of the sequences += the attention weight that
    the step gave it, summed over heads; lse fp32 [B, H] as paged_decode
    returned it for the same queries."""
    dev, max_end_pos = cache._dev, _int32(max_end_pos, "mla_paged_weights", "max_end_pos")
    B, H = q_latent.shape[:2]
    if _off(q_latent, _bf16, (B, H, 512), dev):
        _refuse("q_latent", q_latent, _bf16, (B, H, 512), dev)
    if _off(q_pe, _bf16, (B, H, 64), dev):
        _refuse("q_pe", q_pe, _bf16, (B, H, 64), dev)
    if _off(lse, _f32, (B, H), dev):
        _refuse("lse", lse, _f32, (B, H), dev)
    if _off(end_pos, _i32, (B,), dev):
        _refuse("end_pos", end_pos, _i32, (B,), dev)
    if status is not None and _off(status, _i32, (1,), dev):
        _refuse("status", status, _i32, (1,), dev)
    n = _table_width("table", table, B, dev)
    _paged_call(cache, lib().mla_paged_weights,
                (table.data_ptr(), n, q_latent.data_ptr(), q_pe.data_ptr(), lse.data_ptr(), end_pos.data_ptr(),
                 max_end_pos, B, H, float(softmax_scale), None if status is None else status.data_ptr()), stream)


def selftest_paged_decode_timeout(cache: PagedCache, table, q_latent, q_pe, end_pos, max_end_pos: int,
                                  softmax_scale: float, workspace, stream=None) -> int:
    """mla_paged_decode with a part of the first tile withheld and short waits:
    returns the workspace status word (MLA_DEV_PIPELINE_TIMEOUT expected)."""
    B, H, _ = q_latent.shape
    _need(q_latent, torch.bfloat16, (B, H, 512), "q_latent")
    _need(q_pe, torch.bfloat16, (B, H, 64), "q_pe")
    _need(end_pos, torch.int32, (B,), "end_pos")
    n = _table_width("table", table, B, cache._dev)
    out, lse = _new((B, H, 512), _bf16, cache, stream), _new((B, H), _f32, cache, stream)
    _paged_call(cache, lib().mla_selftest_paged_decode_timeout,
                (table.data_ptr(), n, q_latent.data_ptr(), q_pe.data_ptr(), end_pos.data_ptr(), int(max_end_pos), B, H,
                 float(softmax_scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel()), stream)
    return workspace_status(workspace, stream)


def selftest_paged_weights_timeout(cache: PagedCache, table, q_latent, q_pe, lse, end_pos, max_end_pos: int,
                                   softmax_scale: float, status, stream=None) -> None:
    """mla_paged_weights likewise; ORs MLA_DEV_PIPELINE_TIMEOUT into status (int32 [1])."""
    B, H, _ = q_latent.shape
    _need(q_latent, torch.bfloat16, (B, H, 512), "q_latent")
    _need(q_pe, torch.bfloat16, (B, H, 64), "q_pe")
    _need(lse, torch.float32, (B, H), "lse")
    _need(end_pos, torch.int32, (B,), "end_pos")
    _need(status, torch.int32, (1,), "status")
    n = _table_width("table", table, B, cache._dev)
    _paged_call(cache, lib().mla_selftest_paged_weights_timeout,
                (table.data_ptr(), n, q_latent.data_ptr(), q_pe.data_ptr(), lse.data_ptr(), end_pos.data_ptr(),
                 int(max_end_pos), B, H, float(softmax_scale), status.data_ptr()), stream)


def paged_evict(cache: PagedCache, table, end_pos, max_end_pos: int, keep: int, new_table,
                sinks: int = 0, recent: int = 0, kept=None, new_end_pos=None, status=None, stream=None):
    """Copy the `keep` rows of most accumulated weight of every sequence (the
    first `sinks` and last `recent` always among them) into the pages of
    new_table (int32 [B, new_max_pages]), in order of position.  Returns (kept
    int32 [B, keep]: their positions, then -1; new_end_pos int32 [B], which
    may be end_pos: its lengths are then replaced).  The new lengths count rows;
    the rotary position of a sequence's next token goes on from its own count."""
    dev, max_end_pos = cache._dev, _int32(max_end_pos, "mla_paged_evict", "max_end_pos")
    B, keep = end_pos.shape[0], _int32(keep, "mla_paged_evict", "keep")
    sinks, recent = _int32(sinks, "mla_paged_evict", "sinks"), _int32(recent, "mla_paged_evict", "recent")
    if keep < 1:
        raise MLAError(1, "mla_paged_evict", "keep")
    if _off(end_pos, _i32, (B,), dev):
        _refuse("end_pos", end_pos, _i32, (B,), dev)
    n, m = _table_width("table", table, B, dev), _table_width("new_table", new_table, B, dev)
    if kept is None:
        kept = _new((B, keep), _i32, cache, stream)
    elif _off(kept, _i32, (B, keep), dev):
        _refuse("kept", kept, _i32, (B, keep), dev)
    if new_end_pos is None:
        new_end_pos = _new((B,), _i32, cache, stream)
    elif _off(new_end_pos, _i32, (B,), dev):
        _refuse("new_end_pos", new_end_pos, _i32, (B,), dev)
    if status is not None and _off(status, _i32, (1,), dev):
        _refuse("status", status, _i32, (1,), dev)
    _paged_call(cache, lib().mla_paged_evict,
                (table.data_ptr(), n, end_pos.data_ptr(), max_end_pos, B, keep, sinks, recent,
                 new_table.data_ptr(), m, kept.data_ptr(), new_end_pos.data_ptr(),
                 None if status is None else status.data_ptr()), stream)
    return kept, new_end_pos


def rotary_frequencies(base: float = 10000.0, factor: float = 1.0, original_len: int = 4096,
                       beta_fast: float = 32.0, beta_slow: float = 1.0) -> list:
    """The 32 frequencies (radians a position) of the rotary columns: base^(-i/32),
    and with a YaRN factor above 1 (DeepSeek-V3.2-Exp . KV cache: rope_factor 40,
    beta_fast 32, beta_slow 1) divided by it where a column turns less than
    beta_slow times in original_len positions, kept where it turns more than
    beta_fast times, and in between by a linear ramp over the columns."""
    f = [base ** (-i / 32) for i in range(32)]
    if factor == 1.0:
        return f
    # the column that turns n times in original_len positions
    col = [32 * math.log(original_len / (n * 2 * math.pi)) / math.log(base) for n in (beta_fast, beta_slow)]
    low, high = max(math.floor(col[0]), 0), min(math.ceil(col[1]), 63)
    ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(32)]
    return [x / factor * r + x * (1.0 - r) for x, r in zip(f, ramp)]


class Rotary:
    """The position rotation of 64 rotary columns: `frequencies`, 32 numbers in
    radians a position (see rotary_frequencies); pairs of columns are 2 i and
    2 i + 1, or with interleaved=False i and i + 32; gain: a factor on the
    rotated columns."""

    def __init__(self, frequencies, interleaved: bool = True, gain: float = 1.0, device="cuda"):
        freq = [float(x) for x in frequencies]
        if len(freq) != 32:
            raise ValueError(f"frequencies: want 32, got {len(freq)}")
        turns = torch.empty(32, dtype=torch.int64)
        _check(lib().mla_rotary_turns((ctypes.c_double * 32)(*freq), 32, turns.data_ptr()), "mla_rotary_turns")
        if not math.isfinite(gain):
            raise ValueError("gain: want a finite number")
        self.frequencies, self.interleaved, self.gain = freq, bool(interleaved), float(gain)
        self.turns = turns.to(device)
        self._dev = self.turns.get_device()
        self._c = _CRotary(self.turns.data_ptr(), self.gain, 0 if interleaved else 1)
        self.ref, self._addr = ctypes.byref(self._c), ctypes.addressof(self._c)


# The calls below go through the host extension where the call is the plain case
# (a pool on the current device, the current stream, tensors as they should be):
# it answers with the outputs, or with the library's status.  Anything else (None)
# takes the way written out after it, which says what is wrong with a tensor.
# Issue of a call, on the host of a GB300, that way and through the extension:
# paged_append_rotary 17.6 and 5.6 us, paged_read 13.4 and 5.1,
# paged_decode_window 17.9 and 7.8.

def _off_rows(t, dtype, shape, dev):
    """Whether t is not [..., columns] of that shape with its columns side by side."""
    return t.dtype is not dtype or t.shape != shape or t.stride(-1) != 1 or t.get_device() != dev


def paged_append_rotary(cache: PagedCache, table, kv_a, norm_weight, eps: float, rotary: Rotary, pos, end_pos,
                        q=None, q_nope=None, q_pe=None, status=None, stream=None):
    """The cache write from the projections' outputs, in one pass: kv_a bf16
    [B, s, 576] (latent and rotary key; any strides of sequences and tokens that
    are multiples of 8), whose latent is normalised (RMS, norm_weight [512] fp32
    or bf16) and whose key is rotated to position pos[b, j] (int32 [B, s]), goes
    to row end_pos[b] - s + j of sequence b as in paged_append.  With q bf16
    [B, s, H, 192] (such strides too) returns (q_nope bf16 [B, s, H, 128], q_pe
    bf16 [B, s, H, 64]): its content part, and its rotary part rotated; without,
    (None, None)."""
    if stream is None and type(cache) is PagedCache:
        r = (_host or native()).append_rotary(cache._addr, cache._dev, pos, table, kv_a, norm_weight, eps, rotary._addr, rotary._dev,
                                              end_pos, q, q_nope, q_pe, status)
        if r is not None:
            return r if type(r) is tuple else _check(r, "mla_paged_append_rotary")
    dev = cache._dev
    B, s = pos.shape
    if _off_rows(kv_a, _bf16, (B, s, 576), dev):
        _refuse("kv_a", kv_a, _bf16, (B, s, 576), dev)
    f32 = norm_weight.dtype is _f32
    if _off(norm_weight, _f32 if f32 else _bf16, (512,), dev):
        _refuse("norm_weight", norm_weight, _bf16, (512,), dev)
    if _off(pos, _i32, (B, s), dev):
        _refuse("pos", pos, _i32, (B, s), dev)
    if _off(end_pos, _i32, (B,), dev):
        _refuse("end_pos", end_pos, _i32, (B,), dev)
    if status is not None and _off(status, _i32, (1,), dev):
        _refuse("status", status, _i32, (1,), dev)
    if rotary._dev != dev:
        raise ValueError(f"rotary: on {rotary.turns.device}, the pool on {cache.device}")
    n = _table_width("table", table, B, dev)
    sb, ss, _ = kv_a.stride()
    H, qs, at_q, at_nope, at_pe = 0, (0, 0, 0), None, None, None
    if q is not None:
        H = q.shape[2] if q.dim() == 4 else 0
        if _off_rows(q, _bf16, (B, s, H, 192), dev):
            _refuse("q", q, _bf16, (B, s, H, 192), dev)
        if q_nope is None:
            q_nope = _new((B, s, H, 128), _bf16, cache, stream)
        elif _off(q_nope, _bf16, (B, s, H, 128), dev):
            _refuse("q_nope", q_nope, _bf16, (B, s, H, 128), dev)
        if q_pe is None:
            q_pe = _new((B, s, H, 64), _bf16, cache, stream)
        elif _off(q_pe, _bf16, (B, s, H, 64), dev):
            _refuse("q_pe", q_pe, _bf16, (B, s, H, 64), dev)
        qs, at_q, at_nope, at_pe = q.stride(), q.data_ptr(), q_nope.data_ptr(), q_pe.data_ptr()
    elif q_nope is not None or q_pe is not None:
        raise ValueError("q_nope and q_pe: only with q")
    _paged_call(cache, lib().mla_paged_append_rotary,
                (table.data_ptr(), n, kv_a.data_ptr(), sb, ss, norm_weight.data_ptr(), f32, eps, rotary.ref, pos.data_ptr(),
                 end_pos.data_ptr(), B, s, at_q, qs[0], qs[1], qs[2], H, at_nope, at_pe,
                 None if status is None else status.data_ptr()), stream)
    return q_nope, q_pe


def paged_read(cache: PagedCache, table, offsets, total: int, first=None, kv=None, pe=None, status=None, stream=None):
    """Cached rows back as bf16, packed one sequence behind another: row n with
    offsets[b] <= n < offsets[b + 1] (int32 [B + 1]) is position first[b] + n -
    offsets[b] of sequence b (first int32 [B]; None: 0).  Returns (kv bf16
    [total, 512], pe bf16 [total, 64]), which may be given, with any row strides
    that are multiples of 8; rows outside offsets[0] .. offsets[B] - 1 are left as
    they were."""
    if stream is None and type(cache) is PagedCache:
        r = (_host or native()).read(cache._addr, cache._dev, offsets, table, total, first, kv, pe, status)
        if r is not None:
            return r if type(r) is tuple else _check(r, "mla_paged_read")
    dev, total = cache._dev, _int32(total, "mla_paged_read", "total")
    B = offsets.numel() - 1
    if total < 0 or B < 1:
        raise MLAError(1, "mla_paged_read", "total" if total < 0 else "offsets")
    if _off(offsets, _i32, (B + 1,), dev):
        _refuse("offsets", offsets, _i32, (B + 1,), dev)
    if first is not None and _off(first, _i32, (B,), dev):
        _refuse("first", first, _i32, (B,), dev)
    if status is not None and _off(status, _i32, (1,), dev):
        _refuse("status", status, _i32, (1,), dev)
    n = _table_width("table", table, B, dev)
    if kv is None:
        kv = _new((total, 512), _bf16, cache, stream)
    elif _off_rows(kv, _bf16, (total, 512), dev):
        _refuse("kv", kv, _bf16, (total, 512), dev)
    if pe is None:
        pe = _new((total, 64), _bf16, cache, stream)
    elif _off_rows(pe, _bf16, (total, 64), dev):
        _refuse("pe", pe, _bf16, (total, 64), dev)
    _paged_call(cache, lib().mla_paged_read,
                (table.data_ptr(), n, offsets.data_ptr(), None if first is None else first.data_ptr(), B, total,
                 kv.data_ptr(), kv.stride(0), pe.data_ptr(), pe.stride(0), None if status is None else status.data_ptr()), stream)
    return kv, pe


def paged_window_workspace_size(B: int, s: int, H: int) -> int:
    n = lib().mla_paged_window_workspace_size(B, s, H)
    if n == 0:
        raise MLAError(3, "mla_paged_window_workspace_size")
    return int(n)


def alloc_paged_window_workspace(B: int, s: int, H: int, device="cuda"):
    return torch.empty(paged_window_workspace_size(B, s, H), dtype=torch.uint8, device=device)


def paged_decode_window(cache: PagedCache, table, q_latent, q_pe, end_pos, max_end_pos: int, softmax_scale: float,
                        window: int, sinks: int = 0, out=None, lse=None, workspace=None, want_lse: bool = True,
                        stream=None):
    """Absorbed decode of s tokens of every sequence (q_latent bf16 [B, s, H, 512],
    q_pe bf16 [B, s, H, 64]; their rows are in the cache already) in which token j,
    at position t = end_pos[b] - s + j, sees positions p <= t with p < sinks or
    p > t - window; returns (out bf16 [B, s, H, 512], lse fp32 [B, s, H] or None)."""
    if stream is None and type(cache) is PagedCache:
        r = (_host or native()).decode_window(cache._addr, cache._dev, q_latent, table, q_pe, end_pos, max_end_pos, softmax_scale,
                                              window, sinks, out, lse, want_lse, workspace)
        if r is not None:
            return r if type(r) is tuple else _check(r, "mla_paged_decode_window")
    dev, max_end_pos = cache._dev, _int32(max_end_pos, "mla_paged_decode_window", "max_end_pos")
    window, sinks = _int32(window, "mla_paged_decode_window", "window"), _int32(sinks, "mla_paged_decode_window", "sinks")
    B, s, H = q_latent.shape[:3]
    if _off(q_latent, _bf16, (B, s, H, 512), dev):
        _refuse("q_latent", q_latent, _bf16, (B, s, H, 512), dev)
    if _off(q_pe, _bf16, (B, s, H, 64), dev):
        _refuse("q_pe", q_pe, _bf16, (B, s, H, 64), dev)
    if _off(end_pos, _i32, (B,), dev):
        _refuse("end_pos", end_pos, _i32, (B,), dev)
    n = _table_width("table", table, B, dev)
    if out is None:
        out = _new((B, s, H, 512), _bf16, cache, stream)
    elif _off(out, _bf16, (B, s, H, 512), dev):
        _refuse("out", out, _bf16, (B, s, H, 512), dev)
    if lse is None:
        if want_lse:
            lse = _new((B, s, H), _f32, cache, stream)
    elif _off(lse, _f32, (B, s, H), dev):
        _refuse("lse", lse, _f32, (B, s, H), dev)
    if workspace is None:
        workspace = _new((paged_window_workspace_size(B, s, H),), torch.uint8, cache, stream)
    nbytes = workspace.numel()
    if _off(workspace, torch.uint8, (nbytes,), dev):
        _refuse("workspace", workspace, torch.uint8, (nbytes,), dev)
    _paged_call(cache, lib().mla_paged_decode_window,
                (table.data_ptr(), n, q_latent.data_ptr(), q_pe.data_ptr(), end_pos.data_ptr(), max_end_pos, B, s, H,
                 float(softmax_scale), window, sinks, out.data_ptr(), None if lse is None else lse.data_ptr(),
                 workspace.data_ptr(), nbytes), stream)
    return out, lse


def selftest_paged_window_timeout(cache: PagedCache, table, q_latent, q_pe, end_pos, max_end_pos: int, softmax_scale: float,
                                  window: int, sinks: int, workspace, stream=None) -> int:
    """mla_paged_decode_window with a part of the first tile withheld and short waits:
    returns the workspace status word (MLA_DEV_PIPELINE_TIMEOUT expected)."""
    B, s, H, _ = q_latent.shape
    _need(q_latent, torch.bfloat16, (B, s, H, 512), "q_latent")
    _need(q_pe, torch.bfloat16, (B, s, H, 64), "q_pe")
    _need(end_pos, torch.int32, (B,), "end_pos")
    n = _table_width("table", table, B, cache._dev)
    out, lse = _new((B, s, H, 512), _bf16, cache, stream), _new((B, s, H), _f32, cache, stream)
    _paged_call(cache, lib().mla_selftest_paged_window_timeout,
                (table.data_ptr(), n, q_latent.data_ptr(), q_pe.data_ptr(), end_pos.data_ptr(), int(max_end_pos), B, s, H,
                 float(softmax_scale), int(window), int(sinks), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                 workspace.numel()), stream)
    return workspace_status(workspace, stream)


def trace_begin(max_records: int) -> None:
    """Start timing the main decode kernel of every call on this thread."""
    _check(lib().mla_trace_begin(int(max_records)), "mla_trace_begin")


def trace_end():
    """Stop tracing; returns (summed main-kernel ms, timed launches, kernel launches)."""
    ms = ctypes.c_float(0)
    n = ctypes.c_int32(0)
    k = ctypes.c_int32(0)
    _check(lib().mla_trace_end(ctypes.byref(ms), ctypes.byref(n), ctypes.byref(k)), "mla_trace_end")
    return float(ms.value), int(n.value), int(k.value)
