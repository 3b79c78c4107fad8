"""Python binding of libfa.so (include/fa.h), argument marshalling only.

The functions with the C names (``fa_fwd``, ``fa_bwd``, ...) take torch CUDA
tensors that the caller allocated and pass their device pointers, sizes and the
current CUDA stream straight to the C ABI; every step of the computation runs
in the library's kernels.  ``forward`` / ``backward`` are conveniences that
allocate the outputs with torch and then call those.

There is no fallback: if libfa.so is missing or cannot be loaded, importing
this module raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "fa.h")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_CUDA = 3
FA_ERR_TIMEOUT = 4
FA_ERR_WORKSPACE = 5
FA_ERR_TOO_LARGE = 6


class FAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where} failed: {status_string(code)} ({code})")


FA_CACHE_BF16 = 0
FA_CACHE_FP4 = 1


class PagedCache(ctypes.Structure):
    """fa_paged_cache of include/fa.h."""
    _fields_ = [("pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("format", ctypes.c_int), ("B", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("d", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -m exact_attention_98_gb300.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.fa_fwd_workspace_bytes.restype = sz
    lib.fa_set_exp2_poly_share.argtypes = [i]
    lib.fa_set_exp2_poly_share.restype = i
    lib.fa_get_exp2_poly_share.argtypes = []
    lib.fa_get_exp2_poly_share.restype = i
    lib.fa_fwd_2cta.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_fwd_2cta.restype = i
    lib.fa_fwd_splitkv_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.fa_fwd_splitkv_workspace_bytes.restype = sz
    lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp, sz, vp]
    lib.fa_fwd_splitkv.restype = i
    lib.fa_fwd_fp8_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_fwd_fp8_workspace_bytes.restype = sz
    lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp, sz, vp]
    lib.fa_fwd_fp8.restype = i
    lib.fa_bwd_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_bwd_workspace_bytes.restype = sz
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
    lib.fa_bwd.restype = i
    lib.fa_last_device_status.argtypes = [vp]
    lib.fa_last_device_status.restype = i
    lib.fa_last_device_site.argtypes = []
    lib.fa_last_device_site.restype = i
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_exp2_poly_eval.argtypes = [vp, vp, ctypes.c_longlong, vp]
    lib.fa_exp2_poly_eval.restype = i
    lib.fa_debug_bounded_wait.argtypes = [ctypes.c_ulonglong, vp]
    lib.fa_debug_bounded_wait.restype = i
    lib.fa_bwd_2cta.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
    lib.fa_bwd_2cta.restype = i
    lib.fa_bwd_deterministic_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_bwd_deterministic_workspace_bytes.restype = sz
    lib.fa_bwd_deterministic.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp,
                                         sz, vp]
    lib.fa_bwd_deterministic.restype = i
    lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_bwd_noalloc.restype = i
    lib.fa_timing_enable.argtypes = [i]
    lib.fa_timing_enable.restype = i
    lib.fa_timing_last_ms.argtypes = [i, ctypes.POINTER(ctypes.c_float)]
    lib.fa_timing_last_ms.restype = i
    lib.fa_fwd_window.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_window.restype = i
    lib.fa_bwd_window_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.fa_bwd_window_workspace_bytes.restype = sz
    lib.fa_bwd_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, sz, vp]
    lib.fa_bwd_window.restype = i
    ll = ctypes.c_longlong
    cache = ctypes.POINTER(PagedCache)
    lib.fa_paged_block_bytes.argtypes = [i, i, i]
    lib.fa_paged_block_bytes.restype = sz
    lib.fa_paged_append.argtypes = [cache, vp, ll, ll, vp, ll, ll, vp, i, vp, ll, ll, vp, i, vp, i, i,
                                    i, vp]
    lib.fa_paged_append.restype = i
    lib.fa_paged_read.argtypes = [cache, vp, i, vp, vp, vp]
    lib.fa_paged_read.restype = i
    lib.fa_fwd_paged_workspace_bytes.argtypes = [i]
    lib.fa_fwd_paged_workspace_bytes.restype = sz
    lib.fa_fwd_paged.argtypes = [cache, vp, ll, ll, vp, vp, vp, i, i, i, f, i, i, vp, sz, vp]
    lib.fa_fwd_paged.restype = i
    lib.fa_launch_count.argtypes = []
    lib.fa_launch_count.restype = ctypes.c_ulonglong
    return lib


lib = _load()


def declared_functions() -> list[str]:
    """Names of the functions include/fa.h declares."""
    text = open(HEADER_PATH).read()
    return sorted(set(re.findall(r"^[ \t]*(?:const[ \t]+)?(?:\w+[ \t]+)*\w+[ \t]*\*?[ \t]*(fa_\w+)\s*\(",
                                 text, re.M)))


def status_string(code: int) -> str:
    return lib.fa_status_string(int(code)).decode()


def _check(code: int, where: str):
    if code != FA_OK:
        raise FAError(code, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    """The cudaStream_t of `stream`, or of the current stream of the current
    device (looked up without building a torch.cuda.Stream, which takes 3 us)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _shape(q):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d]")
    return tuple(q.shape)


def _check_tensor(t, name, dtype, shape, device=None):
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and (t.is_cuda if device is None else t.get_device() == device.index)):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_attention(q, names_and_tensors, lse):
    """Shape, dtype, device and layout checks shared by the forward and
    backward calls; every operand lives on q's device."""
    B, H, N, d = _shape(q)
    if q.is_cuda and q.device.index != torch.cuda.current_device():
        raise ValueError(f"q is on {q.device}; the library launches on the current device "
                         f"cuda:{torch.cuda.current_device()}")
    for name, t in names_and_tensors:
        _check_tensor(t, name, torch.bfloat16, (B, H, N, d), q.device)
    _check_tensor(lse, "lse", torch.float32, (B, H, N), q.device)
    return B, H, N, d


def _workspace(ws, device):
    """(pointer, bytes) of a caller workspace: None, or a contiguous CUDA
    tensor on the operands' device (the library checks size and alignment)."""
    if ws is None:
        return None, 0
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.device != device:
        raise ValueError(f"workspace must be a CUDA tensor on {device}")
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return _ptr(ws), ws.numel() * ws.element_size()


# --- the C entry points --------------------------------------------------------


def fa_fwd(q, k, v, o, lse, scale: float, causal: bool, workspace=None, stream=None) -> None:
    """workspace: None, or a CUDA tensor of at least fa_fwd_workspace_bytes()
    bytes that lets the call split its last partial round of work."""
    B, H, N, d = _check_attention(q, (("q", q), ("k", k), ("v", v), ("o", o)), lse)
    ws_ptr, ws_bytes = _workspace(workspace, q.device)
    _check(lib.fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale),
                      int(bool(causal)), ws_ptr, ws_bytes, _stream(stream)), "fa_fwd")


def fa_fwd_workspace_bytes(B: int, H: int, N: int, d: int, causal: bool) -> int:
    return int(lib.fa_fwd_workspace_bytes(B, H, N, d, int(bool(causal))))


def fa_set_exp2_poly_share(per_octet: int) -> None:
    _check(lib.fa_set_exp2_poly_share(int(per_octet)), "fa_set_exp2_poly_share")


def fa_get_exp2_poly_share() -> int:
    return int(lib.fa_get_exp2_poly_share())


def fa_fwd_2cta(q, k, v, o, lse, scale: float, causal: bool, stream=None) -> None:
    """fa_fwd computed by CTA pairs sharing each M = 256 product (d = 128)."""
    B, H, N, d = _check_attention(q, (("q", q), ("k", k), ("v", v), ("o", o)), lse)
    _check(lib.fa_fwd_2cta(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale),
                           int(bool(causal)), _stream(stream)), "fa_fwd_2cta")


def fa_fwd_splitkv_workspace_bytes(B: int, H: int, N: int, d: int, num_splits: int) -> int:
    return int(lib.fa_fwd_splitkv_workspace_bytes(B, H, N, d, num_splits))


def fa_fwd_splitkv(q, k, v, o, lse, scale: float, causal: bool, num_splits: int, workspace,
                   stream=None) -> None:
    B, H, N, d = _check_attention(q, (("q", q), ("k", k), ("v", v), ("o", o)), lse)
    ws_ptr, ws_bytes = _workspace(workspace, q.device)
    _check(lib.fa_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                              float(scale), int(bool(causal)), int(num_splits), ws_ptr,
                              ws_bytes, _stream(stream)), "fa_fwd_splitkv")


def fa_fwd_fp8_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib.fa_fwd_fp8_workspace_bytes(B, H, N, d))


def fa_fwd_fp8(q, k, v, o, lse, scale: float, causal: bool, rotate: bool, workspace,
               stream=None) -> None:
    B, H, N, d = _check_attention(q, (("q", q), ("k", k), ("v", v), ("o", o)), lse)
    ws_ptr, ws_bytes = _workspace(workspace, q.device)
    _check(lib.fa_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale),
                          int(bool(causal)), int(bool(rotate)), ws_ptr, ws_bytes,
                          _stream(stream)), "fa_fwd_fp8")


def forward_fp8(q, k, v, causal: bool = False, scale: float | None = None, rotate: bool = True,
                stream=None):
    """FP8 forward (fa_fwd_fp8); returns (o, lse) freshly allocated."""
    B, H, N, d = _shape(q)
    scale = default_scale(d) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    ws = torch.empty(max(fa_fwd_fp8_workspace_bytes(B, H, N, d), 1), dtype=torch.uint8,
                     device=q.device)
    fa_fwd_fp8(q, k, v, o, lse, scale, causal, rotate, ws, stream)
    return o, lse


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib.fa_bwd_workspace_bytes(B, H, N, d))


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, scale: float, causal: bool, workspace,
           stream=None) -> None:
    B, H, N, d = _check_attention(q, (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout),
                                      ("dq", dq), ("dk", dk), ("dv", dv)), lse)
    ws_ptr, ws_bytes = _workspace(workspace, q.device)
    _check(lib.fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                      _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                      ws_ptr, ws_bytes, _stream(stream)), "fa_bwd")


def fa_bwd_2cta(q, k, v, o, lse, dout, dq, dk, dv, scale: float, causal: bool, workspace,
                stream=None) -> None:
    """fa_bwd computed by CTA pairs sharing each product (d = 128); same
    workspace as fa_bwd."""
    B, H, N, d = _check_attention(q, (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout),
                                      ("dq", dq), ("dk", dk), ("dv", dv)), lse)
    ws_ptr, ws_bytes = _workspace(workspace, q.device)
    _check(lib.fa_bwd_2cta(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                           _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                           ws_ptr, ws_bytes, _stream(stream)), "fa_bwd_2cta")


def fa_bwd_deterministic_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib.fa_bwd_deterministic_workspace_bytes(B, H, N, d))


def fa_bwd_deterministic(q, k, v, o, lse, dout, dq, dk, dv, scale: float, causal: bool,
                         workspace, stream=None) -> None:
    """fa_bwd with run-to-run bit-identical results (no dQ atomics)."""
    B, H, N, d = _check_attention(q, (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout),
                                      ("dq", dq), ("dk", dk), ("dv", dv)), lse)
    ws_ptr, ws_bytes = _workspace(workspace, q.device)
    _check(lib.fa_bwd_deterministic(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                    _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                    int(bool(causal)), ws_ptr, ws_bytes,
                                    _stream(stream)), "fa_bwd_deterministic")


def fa_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, scale: float, causal: bool,
                   stream=None) -> None:
    """fa_bwd with the library's fixed scratch array instead of a caller
    workspace: for callers that cannot allocate device memory."""
    B, H, N, d = _check_attention(q, (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout),
                                      ("dq", dq), ("dk", dk), ("dv", dv)), lse)
    _check(lib.fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                              _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                              _stream(stream)), "fa_bwd_noalloc")


def _check_window(q, q_like, k, kv_like, lse):
    """As _check_attention, with the key heads' tensors [B, Hkv, N, d]."""
    B, H, N, d = _check_attention(q, q_like, lse)
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("expected k [B, Hkv, N, d]")
    Hkv = int(k.shape[1])
    for name, t in kv_like:
        _check_tensor(t, name, torch.bfloat16, (B, Hkv, N, d), q.device)
    return B, H, Hkv, N, d


def fa_fwd_window(q, k, v, o, lse, scale: float, window: int, sinks: int, stream=None) -> None:
    B, H, Hkv, N, d = _check_window(q, (("q", q), ("o", o)), k, (("k", k), ("v", v)), lse)
    _check(lib.fa_fwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, N, d,
                             float(scale), int(window), int(sinks), _stream(stream)), "fa_fwd_window")


def fa_bwd_window_workspace_bytes(B: int, H: int, Hkv: int, N: int, d: int, window: int,
                                  sinks: int) -> int:
    return int(lib.fa_bwd_window_workspace_bytes(B, H, Hkv, N, d, window, sinks))


def fa_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, scale: float, window: int, sinks: int, workspace,
                  stream=None) -> None:
    B, H, Hkv, N, d = _check_window(q, (("q", q), ("o", o), ("dout", dout), ("dq", dq)), k,
                                    (("k", k), ("v", v), ("dk", dk), ("dv", dv)), lse)
    ws_ptr, ws_bytes = _workspace(workspace, q.device)
    _check(lib.fa_bwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                             _ptr(dk), _ptr(dv), B, H, Hkv, N, d, float(scale), int(window), int(sinks),
                             ws_ptr, ws_bytes, _stream(stream)), "fa_bwd_window")


def fa_paged_block_bytes(format: int, page_size: int, d: int) -> int:
    return int(lib.fa_paged_block_bytes(int(format), int(page_size), int(d)))


def _paged_cache(pages, page_table, seq_lens, d, k_scale, v_scale):
    """The cache's descriptor from its tensors (see paged_append); the
    tensors have to outlive the call that takes it."""
    if not isinstance(pages, torch.Tensor) or not pages.is_cuda:
        raise ValueError("pages must be a CUDA tensor")
    dev = pages.device
    if dev.index != torch._C._cuda_getDevice():
        raise ValueError(f"pages is on {dev}; the library launches on the current device "
                         f"cuda:{torch.cuda.current_device()}")
    if not pages.is_contiguous():
        raise ValueError("pages must be contiguous")
    shape = pages.shape
    if pages.dtype == torch.bfloat16:
        if len(shape) != 5 or shape[2] != 2 or shape[4] != d:
            raise ValueError(f"bf16 pages are [num_pages, Hkv, 2, page_size, {d}], got {tuple(shape)}")
        fmt, page_size = FA_CACHE_BF16, shape[3]
    elif pages.dtype == torch.uint8:
        row = d // 2 + d // 16
        if len(shape) != 4 or shape[2] != 2 or row == 0 or shape[3] % row != 0:
            raise ValueError(f"4-bit pages are uint8 [num_pages, Hkv, 2, page_size * {row}], got "
                             f"{tuple(shape)}")
        fmt, page_size = FA_CACHE_FP4, shape[3] // row
    else:
        raise ValueError(f"pages must be torch.bfloat16 or torch.uint8 (4 bits), got {pages.dtype}")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, max_pages = page_table.shape
    _check_tensor(page_table, "page_table", torch.int32, (B, max_pages), dev)
    _check_tensor(seq_lens, "seq_lens", torch.int32, (B,), dev)
    if k_scale is not None:
        _check_tensor(k_scale, "k_scale", torch.float32, (shape[1],), dev)
    if v_scale is not None:
        _check_tensor(v_scale, "v_scale", torch.float32, (shape[1],), dev)
    return PagedCache(pages.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), _ptr(k_scale),
                      _ptr(v_scale), fmt, B, shape[1], d, shape[0], page_size, max_pages)


def _rows(t, name, heads, d, device, rows=None):
    """(rows, row stride, head stride) of a bf16 [rows, heads, d] tensor whose
    rows of d values are contiguous."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device.index:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != d or (heads is not None and shape[1] != heads) or (
            rows is not None and shape[0] != rows):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected "
                         f"[{'rows' if rows is None else rows}, {'H' if heads is None else heads}, {d}]")
    row, head, one = t.stride()
    if one != 1 and t.numel():
        raise ValueError(f"{name}'s rows of {d} values must be contiguous")
    return shape[0], row, head


def fa_paged_append(cache: PagedCache, k, k_row, k_head, v, v_row, v_head, cu_new, rows, q, q_row,
                    q_head, q_out, H, rope, rope_len, rot, interleaved, stream=None) -> None:
    _check(lib.fa_paged_append(ctypes.byref(cache), _ptr(k), k_row, k_head, _ptr(v), v_row, v_head,
                               _ptr(cu_new), rows, _ptr(q), q_row, q_head, _ptr(q_out), H, _ptr(rope),
                               rope_len, rot, int(bool(interleaved)), _stream(stream)),
           "fa_paged_append")


def fa_paged_read(cache: PagedCache, cu_new, rows, k, v, stream=None) -> None:
    _check(lib.fa_paged_read(ctypes.byref(cache), _ptr(cu_new), rows, _ptr(k), _ptr(v),
                             _stream(stream)), "fa_paged_read")


def fa_fwd_paged_workspace_bytes(d: int) -> int:
    return lib.fa_fwd_paged_workspace_bytes(d)


@functools.lru_cache(maxsize=None)
def _paged_workspace_bytes(device: int, d: int) -> int:
    return max(fa_fwd_paged_workspace_bytes(d), 1)


def fa_fwd_paged(cache: PagedCache, q, q_row, q_head, o, lse, cu_new, rows, max_new, H, scale, window,
                 sinks, workspace, stream=None) -> None:
    ws_ptr, ws_bytes = _workspace(workspace, q.device)
    _check(lib.fa_fwd_paged(ctypes.byref(cache), _ptr(q), q_row, q_head, _ptr(o), _ptr(lse),
                            _ptr(cu_new), rows, max_new, H, float(scale), window, sinks, ws_ptr,
                            ws_bytes, _stream(stream)), "fa_fwd_paged")


def fa_last_device_status(stream=None) -> int:
    return int(lib.fa_last_device_status(_stream(stream)))


def fa_last_device_site() -> int:
    return int(lib.fa_last_device_site())


def fa_status_string(code: int) -> str:
    return status_string(code)


def fa_exp2_poly_eval(x, y, stream=None) -> None:
    _check_tensor(x, "x", torch.float32, x.shape)
    _check_tensor(y, "y", torch.float32, x.shape)
    _check(lib.fa_exp2_poly_eval(_ptr(x), _ptr(y), x.numel(), _stream(stream)),
           "fa_exp2_poly_eval")


def fa_debug_bounded_wait(limit_ns: int, stream=None) -> None:
    _check(lib.fa_debug_bounded_wait(int(limit_ns), _stream(stream)), "fa_debug_bounded_wait")


KERNEL_FWD = 0
KERNEL_BWD_MAIN = 1


def fa_timing_enable(enable: bool) -> None:
    _check(lib.fa_timing_enable(int(bool(enable))), "fa_timing_enable")


def fa_timing_last_ms(kernel: int) -> float:
    ms = ctypes.c_float(0.0)
    _check(lib.fa_timing_last_ms(int(kernel), ctypes.byref(ms)), "fa_timing_last_ms")
    return float(ms.value)


def fa_launch_count() -> int:
    return int(lib.fa_launch_count())


# --- conveniences ----------------------------------------------------------------


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


def forward(q, k, v, causal: bool = False, scale: float | None = None, stream=None,
            num_splits: int = 1, two_cta: bool = False):
    """Returns (o, lse) freshly allocated on q's device.  num_splits > 1:
    split-KV forward (fa_fwd_splitkv) with a freshly allocated workspace;
    two_cta: the CTA-pair forward (fa_fwd_2cta)."""
    B, H, N, d = _shape(q)
    scale = default_scale(d) if scale is None else scale
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if two_cta:
        if num_splits != 1:
            raise ValueError("the CTA-pair forward has no key-range split")
        fa_fwd_2cta(q, k, v, o, lse, scale, causal, stream)
    elif num_splits == 1:
        fa_fwd(q, k, v, o, lse, scale, causal, fwd_workspace_for(q, causal), stream)
    else:
        n = fa_fwd_splitkv_workspace_bytes(B, H, N, d, num_splits)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)
        fa_fwd_splitkv(q, k, v, o, lse, scale, causal, num_splits, ws, stream)
    return o, lse


def fwd_workspace_for(q, causal: bool):
    """fa_fwd's optional workspace for q's shape on the current device (None
    when the call would not use one)."""
    B, H, N, d = _shape(q)
    n = fa_fwd_workspace_bytes(B, H, N, d, causal)
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n > 0 else None


def workspace_for(q, deterministic: bool = False):
    B, H, N, d = _shape(q)
    n = (fa_bwd_deterministic_workspace_bytes if deterministic else fa_bwd_workspace_bytes)(
        B, H, N, d)
    # torch's caching allocator hands out 512-byte aligned blocks
    return torch.empty(max(n, 1), dtype=torch.uint8, device=q.device)


def backward(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None,
             workspace=None, stream=None, deterministic: bool = False, two_cta: bool = False):
    """Returns (dq, dk, dv) freshly allocated on q's device.  deterministic:
    fa_bwd_deterministic (bit-identical from run to run) instead of fa_bwd;
    two_cta: the CTA-pair backward (fa_bwd_2cta)."""
    B, H, N, d = _shape(q)
    scale = default_scale(d) if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    if deterministic and two_cta:
        raise ValueError("the CTA-pair backward adds dQ with atomics")
    if workspace is None:
        workspace = workspace_for(q, deterministic)
    run = fa_bwd_deterministic if deterministic else fa_bwd_2cta if two_cta else fa_bwd
    run(q, k, v, o, lse, dout, dq, dk, dv, scale, causal, workspace, stream)
    return dq, dk, dv


def _empty(stream, device, *shapes_and_types):
    """Uninitialised tensors whose memory belongs to the stream that uses them."""
    empty = torch.empty
    if stream is not None:
        with torch.cuda.stream(stream):
            return [empty(s, dtype=t, device=device) for s, t in shapes_and_types]
    return [empty(s, dtype=t, device=device) for s, t in shapes_and_types]


def window_forward(q, k, v, window: int, sinks: int = 0, scale: float | None = None, stream=None):
    """Causal attention of q [B, H, N, d] over k, v [B, Hkv, N, d] through a
    sliding window (the `window` keys up to each query, itself included) and
    the first `sinks` keys; query head h reads key head h / (H / Hkv).  Returns
    (o, lse)."""
    B, H, N, d = _shape(q)
    o, lse = _empty(stream, q.device, (q.shape, torch.bfloat16), ((B, H, N), torch.float32))
    fa_fwd_window(q, k, v, o, lse, default_scale(d) if scale is None else scale, window, sinks, stream)
    return o, lse


def window_backward(q, k, v, o, lse, dout, window: int, sinks: int = 0, scale: float | None = None,
                    workspace=None, stream=None):
    """Gradients (dq, dk, dv) of window_forward; dk and dv [B, Hkv, N, d] are
    summed over the query heads that share a key head."""
    B, H, N, d = _shape(q)
    dq, dk, dv = _empty(stream, q.device, (q.shape, torch.bfloat16), (k.shape, torch.bfloat16),
                        (v.shape, torch.bfloat16))
    if workspace is None:
        n = fa_bwd_window_workspace_bytes(B, H, k.shape[1], N, d, window, sinks) if k.dim() == 4 else 0
        workspace, = _empty(stream, q.device, (max(n, 1), torch.uint8))
    fa_bwd_window(q, k, v, o, lse, dout, dq, dk, dv, default_scale(d) if scale is None else scale, window,
                  sinks, workspace, stream)
    return dq, dk, dv


# --- the paged key/value cache -----------------------------------------------------


def paged_pages(num_pages: int, heads: int, page_size: int, d: int, format: str = "bf16", device="cuda"):
    """A cache's pages, zeroed: bf16 [num_pages, heads, 2, page_size, d], or for
    format "fp4" uint8 [num_pages, heads, 2, page_size * (d/2 + d/16)]."""
    if format not in ("bf16", "fp4"):
        raise ValueError(f"format must be 'bf16' or 'fp4', got {format!r}")
    if fa_paged_block_bytes(FA_CACHE_FP4 if format == "fp4" else FA_CACHE_BF16, page_size, d) == 0:
        raise ValueError("a cache has page_size 16, 32, 64 or 128 and d 64 or 128")
    if format == "fp4":
        return torch.zeros((num_pages, heads, 2, page_size * (d // 2 + d // 16)), dtype=torch.uint8,
                           device=device)
    return torch.zeros((num_pages, heads, 2, page_size, d), dtype=torch.bfloat16, device=device)


def rope_table(length: int, rot: int, base: float = 10000.0, device="cuda"):
    """fp32 [length, rot]: cos, then sin of position * base^(-2 i / rot), the
    angles taken in 64 bits."""
    rate = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    angle = torch.arange(length, dtype=torch.float64)[:, None] * rate
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def paged_append(k, v, pages, page_table, seq_lens, cu_new, q=None, rope=None, interleaved: bool = False,
                 k_scale=None, v_scale=None, stream=None):
    """Appends K and V rows [rows, Hkv, d] (any row and head strides that are
    multiples of 8) to the cache `pages` (see paged_pages), K rotated by its
    position with the table `rope` [length, rot] (see rope_table; None: no
    rotation).  The rows cu_new[b] .. cu_new[b+1]-1 are sequence b's last ones,
    seq_lens [B] counts them, page_table is [B, max_pages] (all int32).
    k_scale, v_scale: a 4-bit cache's factors [Hkv] (None: 1).  With q [rows,
    H, d] returns it rotated, [rows, H, d] contiguous; padding rows of the
    result are not written."""
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("expected k [rows, Hkv, d]")
    d = k.shape[2]
    cache = _paged_cache(pages, page_table, seq_lens, d, k_scale, v_scale)
    dev = pages.device
    rows, k_row, k_head = _rows(k, "k", cache.Hkv, d, dev)
    _, v_row, v_head = _rows(v, "v", cache.Hkv, d, dev, rows)
    _check_tensor(cu_new, "cu_new", torch.int32, (cache.B + 1,), dev)
    H = q_row = q_head = rope_len = rot = 0
    q_out = None
    if q is not None:
        _, q_row, q_head = _rows(q, "q", None, d, dev, rows)
        H = q.shape[1]
        q_out, = _empty(stream, dev, ((rows, H, d), torch.bfloat16))
        if H == 0:
            q = None
    if rope is not None:
        if not isinstance(rope, torch.Tensor) or rope.dim() != 2:
            raise ValueError("rope must be [length, rot]")
        rope_len, rot = rope.shape
        _check_tensor(rope, "rope", torch.float32, (rope_len, rot), dev)
    fa_paged_append(cache, k, k_row, k_head, v, v_row, v_head, cu_new, rows, q, q_row, q_head,
                    None if q is None else q_out, H, rope, rope_len, rot, interleaved, stream)
    return q_out


def paged_read(pages, page_table, seq_lens, cu_new, rows: int, d: int, k_scale=None, v_scale=None,
               stream=None):
    """The last rows of each sequence (cu_new as in paged_append) out of the
    cache: (k, v), each bf16 [rows, Hkv, d]; padding rows are not written."""
    cache = _paged_cache(pages, page_table, seq_lens, d, k_scale, v_scale)
    _check_tensor(cu_new, "cu_new", torch.int32, (cache.B + 1,), pages.device)
    k, v = _empty(stream, pages.device, *[((rows, cache.Hkv, d), torch.bfloat16)] * 2)
    fa_paged_read(cache, cu_new, rows, k, v, stream)
    return k, v


def paged_forward(q, pages, page_table, seq_lens, cu_new, max_new: int = 1, window: int = 0,
                  sinks: int = 0, scale: float | None = None, k_scale=None, v_scale=None, workspace=None,
                  stream=None):
    """Attention of each sequence's last rows over its cached positions: q
    [rows, H, d] (H a multiple of the cache's heads; strides as paged_append)
    -> (o [rows, H, d], lse [rows, H]).  max_new: rows of a sequence at most;
    window: positions that a row sees, itself included (0: all before it);
    sinks: first positions that it sees besides."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("expected q [rows, H, d]")
    H, d = q.shape[1:]
    cache = _paged_cache(pages, page_table, seq_lens, d, k_scale, v_scale)
    dev = pages.device
    rows, q_row, q_head = _rows(q, "q", H, d, dev)
    _check_tensor(cu_new, "cu_new", torch.int32, (cache.B + 1,), dev)
    o, lse = _empty(stream, dev, ((rows, H, d), torch.bfloat16), ((rows, H), torch.float32))
    if workspace is None:
        workspace, = _empty(stream, dev, (_paged_workspace_bytes(dev.index, d), torch.uint8))
    fa_fwd_paged(cache, q, q_row, q_head, o, lse, cu_new, rows, max_new, H,
                 default_scale(d) if scale is None else scale, window, sinks, workspace, stream)
    return o, lse
