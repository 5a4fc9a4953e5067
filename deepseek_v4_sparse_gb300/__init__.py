"""Python binding of libds4x.so — the GB300 lightning-indexer path.

Thin argument marshalling over the C ABI declared in include/ds4x.h: torch tensors
(device memory) are passed as raw pointers together with the current CUDA stream; every
step of the computation runs in the library's CUDA kernels. There is no fallback: if
libds4x.so has not been built (``python -c "import __graft_entry__ as g; g.build()"``)
every call raises.

Entry points (same names as the C ABI, without the ``ds4x_`` prefix):
  indexer_score, topk, sparse_attn, index_and_attend, workspace_bytes, decode,
  decode_workspace_bytes, topk_workspace_bytes, topk_static_scratch, device_status,
  selftest_bounded_wait, last_launch_count; the paged 4-bit cache: page_plan, kv4_append,
  kv4_read, kv4_attn, kv4_attn_workspace_bytes
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libds4x.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE, ERR_TIMEOUT = 0, -1, -2, -3, -4, -5
F16, BF16 = 0, 1
MAX_KTOP = 1024
MAX_WINDOW = 1024
MAX_RATIO = 65536
MAX_REQ = 4096
MAX_PAGE_ROWS = 65536
KV4_CODE_BYTES, KV4_SCALE_BYTES = 256, 16  # of one 512-dim row of the 4-bit cache
EXPORTS = (
    "ds4x_indexer_score", "ds4x_topk", "ds4x_topk_workspace_bytes", "ds4x_sparse_attn",
    "ds4x_index_and_attend", "ds4x_workspace_bytes", "ds4x_status_string",
    "ds4x_last_launch_count", "ds4x_device_status", "ds4x_selftest_bounded_wait",
    "ds4x_topk_static_scratch", "ds4x_decode", "ds4x_decode_workspace_bytes",
    "ds4x_index_and_attend_host", "ds4x_index_and_attend_host_bytes",
    "ds4x_local_pooled_attn", "ds4x_index_and_attend_local", "ds4x_workspace_bytes_local",
    "ds4x_index_and_attend_local_host", "ds4x_index_and_attend_local_host_bytes", "ds4x_compress",
    "ds4x_decode_local", "ds4x_decode_local_workspace_bytes",
    "ds4x_page_plan", "ds4x_kv4_append", "ds4x_kv4_read", "ds4x_kv4_attn", "ds4x_kv4_attn_workspace_bytes",
)

_lock = threading.Lock()
_lib = None


class Ds4xError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libds4x.so (once) and declare the C signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"libds4x.so is not built ({path}); run deepseek_v4_sparse_gb300.build.build()")
        lib = ctypes.CDLL(path)
        P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        lib.ds4x_indexer_score.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, P, i64, P]
        lib.ds4x_topk.argtypes = [P, i64, P, i32, i32, i32, i32, P, P, P, sz, P]
        lib.ds4x_topk_workspace_bytes.argtypes = [i32, i32, i32]
        lib.ds4x_topk_workspace_bytes.restype = sz
        lib.ds4x_sparse_attn.argtypes = [P, P, ctypes.c_int, P, i32, i32, i32, i32, i32, f32, P, P, P]
        lib.ds4x_index_and_attend.argtypes = [P, P, P, P, P, P, ctypes.c_int, i32, i32, i32, i32, i32,
                                              i32, i32, i32, f32, P, P, P, P, sz, P]
        lib.ds4x_workspace_bytes.argtypes = [i32, i32, i32]
        lib.ds4x_workspace_bytes.restype = sz
        lib.ds4x_index_and_attend_host.argtypes = [P, P, P, P, P, P, ctypes.c_int, i32, i32, i32, i32, i32,
                                                   i32, i32, i32, f32, P, P, P, i32, P, sz, P]
        lib.ds4x_index_and_attend_host_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32]
        lib.ds4x_index_and_attend_host_bytes.restype = sz
        lib.ds4x_local_pooled_attn.argtypes = [P, P, P, ctypes.c_int, P, P, i32, i32, i32, i32, i32, i32, i32,
                                               i32, f32, P, P, P]
        lib.ds4x_index_and_attend_local.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, i32, i32, i32, i32, i32,
                                                    i32, i32, i32, i32, i32, i32, f32, P, P, P, P, sz, P]
        lib.ds4x_workspace_bytes_local.argtypes = [i32, i32, i32, i32]
        lib.ds4x_workspace_bytes_local.restype = sz
        lib.ds4x_index_and_attend_local_host.argtypes = [P, P, P, P, P, P, P, ctypes.c_int, i32, i32, i32, i32,
                                                         i32, i32, i32, i32, i32, i32, i32, f32, P, P, P, i32, P,
                                                         sz, P]
        lib.ds4x_index_and_attend_local_host_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, i32]
        lib.ds4x_index_and_attend_local_host_bytes.restype = sz
        lib.ds4x_compress.argtypes = [P, P, P, ctypes.c_int, i32, i32, i32, P, P, i32, P, P, P, P]
        lib.ds4x_decode.argtypes = [P, P, P, P, P, ctypes.c_int, i32, i32, P, P, i32, i32, i32, i32, i32, i32, i32,
                                    i32, i32, f32, P, P, P, P, P, sz, ctypes.POINTER(i32), P]
        lib.ds4x_decode_local.argtypes = [P, P, P, P, P, ctypes.c_int, i32, i32, P, P, i32, i32, i32, i32, i32, i32,
                                          i32, i32, i32, f32, P, i32, P, i32, P, P, P, P, P, sz, ctypes.POINTER(i32), P]
        lib.ds4x_decode_local_workspace_bytes.argtypes = [i32, i32, i32]
        lib.ds4x_decode_local_workspace_bytes.restype = sz
        lib.ds4x_decode_workspace_bytes.argtypes = [i32, i32]
        lib.ds4x_decode_workspace_bytes.restype = sz
        lib.ds4x_status_string.argtypes = [ctypes.c_int]
        lib.ds4x_status_string.restype = ctypes.c_char_p
        lib.ds4x_last_launch_count.argtypes = []
        lib.ds4x_device_status.argtypes = [P, ctypes.c_int]
        lib.ds4x_selftest_bounded_wait.argtypes = [i64, P]
        lib.ds4x_page_plan.argtypes = [P, P, P, P, P, i32, P, i32, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, P]
        lib.ds4x_kv4_append.argtypes = [P, ctypes.c_int, P, i32, i32, P, P, i32, P]
        lib.ds4x_kv4_read.argtypes = [P, P, i32, P, i32, i32, P, ctypes.c_int, P]
        lib.ds4x_kv4_attn.argtypes = [P, ctypes.c_int, P, P, i32, P, P, i32, i32, i32, P, P, i32, P, P, i32, i32, i32,
                                      i32, f32, P, P, P, sz, P]
        lib.ds4x_kv4_attn_workspace_bytes.argtypes = [i32, i32]
        lib.ds4x_kv4_attn_workspace_bytes.restype = sz
        for f in ("ds4x_page_plan", "ds4x_kv4_append", "ds4x_kv4_read", "ds4x_kv4_attn", "ds4x_indexer_score", "ds4x_topk", "ds4x_sparse_attn", "ds4x_index_and_attend", "ds4x_decode",
                  "ds4x_index_and_attend_host", "ds4x_local_pooled_attn", "ds4x_index_and_attend_local",
                  "ds4x_index_and_attend_local_host", "ds4x_compress", "ds4x_decode_local",
                  "ds4x_last_launch_count", "ds4x_device_status", "ds4x_selftest_bounded_wait"):
            getattr(lib, f).restype = ctypes.c_int
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().ds4x_status_string(status).decode()


def _check(fn: str, rc: int):
    if rc != OK:
        raise Ds4xError(fn, rc)


# ---------------------------------------------------------------------------- torch helpers
def _torch():
    import torch
    return torch


def _ptr(t):
    if t is None:
        return None
    torch = _torch()
    if isinstance(t, torch.Tensor):
        if not t.is_cuda:
            raise ValueError("tensors passed to libds4x must live on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors passed to libds4x must be contiguous")
        return ctypes.c_void_p(t.data_ptr())
    return ctypes.c_void_p(int(t))


def _stream(stream):
    if stream is None:
        torch = _torch()
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if hasattr(stream, "cuda_stream"):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


# Buffers of host-entry calls whose work may still be running: the copies read and write host memory
# asynchronously, and PyTorch recycles a freed page-locked block (or a device block of another
# stream) without knowing about copies it did not issue, so each call's tensors stay referenced
# until an event recorded after it on its stream has completed.
_inflight = []


def _keep_until_done(stream, tensors):
    torch = _torch()
    if stream is None:
        s = torch.cuda.current_stream()
    elif isinstance(stream, torch.cuda.Stream):
        s = stream
    else:
        s = torch.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))
    ev = torch.cuda.Event()
    ev.record(s)
    _inflight[:] = [(e, t) for (e, t) in _inflight if not e.query()]
    _inflight.append((ev, tuple(x for x in tensors if x is not None)))


def _kv_dtype(t) -> int:
    torch = _torch()
    if t.dtype == torch.float16:
        return F16
    if t.dtype == torch.bfloat16:
        return BF16
    raise ValueError(f"kv / q_attn must be float16 or bfloat16, got {t.dtype}")


def _need(t, dtype, name):
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _need_positions(positions, T: int):
    """positions must be int32 with at least one entry per token (the kernels read T of them)."""
    _need(positions, _torch().int32, "positions")
    if positions.numel() < T:
        raise ValueError(f"positions holds {positions.numel()} entries for {T} tokens")


# ------------------------------------------------------------------------------ entry points
def workspace_bytes(T: int, S: int, k_top: int) -> int:
    return int(load().ds4x_workspace_bytes(T, S, k_top))


def topk_workspace_bytes(T: int, S: int, k_top: int) -> int:
    return int(load().ds4x_topk_workspace_bytes(T, S, k_top))


def last_launch_count() -> int:
    return int(load().ds4x_last_launch_count())


def indexer_score(q, w, k, positions, ratio: int, scores=None, S: int | None = None, stream=None):
    """scores[t, s] = sum_h w[t,h] relu(q[t,h,:] . k[s,:]) for visible s, -inf for masked.
    q [T,H,D] fp16, w [T,H] fp16, k [>=S, D] fp16, positions [T] int32 (CUDA tensors)."""
    torch = _torch()
    _need(q, torch.float16, "q"); _need(w, torch.float16, "w"); _need(k, torch.float16, "k")
    T, H, D = q.shape
    _need_positions(positions, T)
    S = k.shape[0] if S is None else S
    if scores is None:
        scores = torch.empty((T, S), dtype=torch.float32, device=q.device)
    _need(scores, torch.float32, "scores")
    rc = load().ds4x_indexer_score(_ptr(q), _ptr(w), _ptr(k), _ptr(positions), T, H, D, S, ratio,
                                   _ptr(scores), scores.shape[1] if scores.dim() == 2 else S,
                                   _stream(stream))
    _check("ds4x_indexer_score", rc)
    return scores


def topk(scores, positions, S: int, ratio: int, k_top: int = 512, indices=None, counts=None,
         workspace=None, stream=None):
    """Exact per-token top-k of the visible scores, ascending row order, -1 padded."""
    torch = _torch()
    _need(scores, torch.float32, "scores")
    T, ld = scores.shape
    _need_positions(positions, T)
    dev = scores.device
    if indices is None:
        indices = torch.empty((T, k_top), dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty((T,), dtype=torch.int32, device=dev)
    need = topk_workspace_bytes(T, S, k_top)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ds4x_topk(_ptr(scores), ld, _ptr(positions), T, S, ratio, k_top, _ptr(indices),
                          _ptr(counts), _ptr(workspace), wbytes, _stream(stream))
    _check("ds4x_topk", rc)
    return indices, counts


def sparse_attn(q_attn, kv, indices, S: int | None = None, scale: float | None = None, out=None,
                lse=None, want_lse: bool = True, stream=None):
    """64-head MQA over the selected rows. q_attn [T,64,512], kv [>=S,512] (fp16 or bf16)."""
    torch = _torch()
    dt = _kv_dtype(q_attn)
    if kv.dtype != q_attn.dtype:
        raise ValueError("kv and q_attn must have the same dtype")
    T, Hq, Dkv = q_attn.shape
    S = kv.shape[0] if S is None else S
    k_top = indices.shape[1]
    scale = 1.0 / math.sqrt(Dkv) if scale is None else scale
    if out is None:
        out = torch.empty_like(q_attn)
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q_attn.device)
    rc = load().ds4x_sparse_attn(_ptr(q_attn), _ptr(kv), dt, _ptr(indices), T, Hq, Dkv, S, k_top,
                                 scale, _ptr(out), _ptr(lse), _stream(stream))
    _check("ds4x_sparse_attn", rc)
    return out, lse


def index_and_attend(q, w, k, positions, q_attn, kv, ratio: int, k_top: int = 512, S: int | None = None,
                     scale: float | None = None, indices=None, out=None, lse=None, workspace=None,
                     want_lse: bool = True, stream=None):
    """The whole path: score -> top-k -> sparse MQA. Returns (indices, out, lse)."""
    torch = _torch()
    dt = _kv_dtype(q_attn)
    T, H, D = q.shape
    _, Hq, Dkv = q_attn.shape
    S = k.shape[0] if S is None else S
    scale = 1.0 / math.sqrt(Dkv) if scale is None else scale
    dev = q.device
    if indices is None:
        indices = torch.empty((T, k_top), dtype=torch.int32, device=dev)
    if out is None:
        out = torch.empty_like(q_attn)
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    need = workspace_bytes(T, S, k_top)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ds4x_index_and_attend(_ptr(q), _ptr(w), _ptr(k), _ptr(positions), _ptr(q_attn), _ptr(kv),
                                      dt, T, H, D, S, ratio, k_top, Hq, Dkv, scale, _ptr(indices),
                                      _ptr(out), _ptr(lse), _ptr(workspace), wbytes, _stream(stream))
    _check("ds4x_index_and_attend", rc)
    return indices, out, lse


def _host_ptr(t):
    """A contiguous CPU tensor's host address (page-locked memory lets the copies overlap)."""
    if t is None:
        return None
    if t.is_cuda or not t.is_contiguous():
        raise ValueError("host tensors passed to ds4x_index_and_attend_host must be contiguous CPU tensors")
    return ctypes.c_void_p(t.data_ptr())


def index_and_attend_host_bytes(T: int, H: int, D: int, S: int, k_top: int, Hq: int, Dkv: int,
                                n_chunks: int = 0) -> int:
    return int(load().ds4x_index_and_attend_host_bytes(T, H, D, S, k_top, Hq, Dkv, n_chunks))


def index_and_attend_host(q, w, k, positions, q_attn, kv, ratio: int, k_top: int = 512, S: int | None = None,
                          scale: float | None = None, n_chunks: int = 0, indices=None, out=None, lse=None,
                          device_buffer=None, want_lse: bool = True, device=None, stream=None):
    """The whole path on host (CPU) tensors: copies in, computes, copies out, overlapped by sub-chunks
    of tokens.  Outputs are page-locked CPU tensors, valid once `stream` is synchronised.  The copies
    run after the call returns: every tensor passed or created here stays referenced until the
    call's work on `stream` is done.  Returns (indices, out, lse)."""
    torch = _torch()
    dt = _kv_dtype(q_attn)
    T, H, D = q.shape
    _, Hq, Dkv = q_attn.shape
    S = k.shape[0] if S is None else S
    scale = 1.0 / math.sqrt(Dkv) if scale is None else scale
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if indices is None:
        indices = torch.empty((T, k_top), dtype=torch.int32).pin_memory()
    if out is None:
        out = torch.empty(q_attn.shape, dtype=q_attn.dtype).pin_memory()
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32).pin_memory()
    need = index_and_attend_host_bytes(T, H, D, S, k_top, Hq, Dkv, n_chunks)
    if device_buffer is None:
        device_buffer = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
    dbytes = device_buffer.numel() * device_buffer.element_size()
    rc = load().ds4x_index_and_attend_host(
        _host_ptr(q), _host_ptr(w), _host_ptr(k), _host_ptr(positions), _host_ptr(q_attn), _host_ptr(kv), dt, T,
        H, D, S, ratio, k_top, Hq, Dkv, scale, _host_ptr(indices), _host_ptr(out), _host_ptr(lse), n_chunks,
        _ptr(device_buffer), dbytes, _stream(stream))
    _check("ds4x_index_and_attend_host", rc)
    _keep_until_done(stream, (q, w, k, positions, q_attn, kv, indices, out, lse, device_buffer))
    return indices, out, lse


# ------------------------------------------------------------------ local-plus-pooled attention
def _rows(t):
    return 0 if t is None else int(t.shape[0])


def workspace_bytes_local(T: int, S: int, k_top: int, window: int) -> int:
    return int(load().ds4x_workspace_bytes_local(T, S, k_top, window))


def local_pooled_attn(q_attn, kv, kv_local, indices, positions, local_pos0: int, window: int,
                      S: int | None = None, scale: float | None = None, out=None, lse=None,
                      want_lse: bool = True, stream=None):
    """One softmax over the selected pooled rows of kv and the raw window rows of kv_local
    [L, 512] (row r = position local_pos0 + r). Returns (out, lse)."""
    torch = _torch()
    dt = _kv_dtype(q_attn)
    if kv.dtype != q_attn.dtype or (kv_local is not None and kv_local.dtype != q_attn.dtype):
        raise ValueError("kv, kv_local and q_attn must have the same dtype")
    T, Hq, Dkv = q_attn.shape
    S = kv.shape[0] if S is None else S
    k_top = indices.shape[1]
    scale = 1.0 / math.sqrt(Dkv) if scale is None else scale
    if out is None:
        out = torch.empty_like(q_attn)
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q_attn.device)
    rc = load().ds4x_local_pooled_attn(_ptr(q_attn), _ptr(kv), _ptr(kv_local), dt, _ptr(indices), _ptr(positions),
                                       T, Hq, Dkv, S, k_top, local_pos0, _rows(kv_local), window, scale, _ptr(out),
                                       _ptr(lse), _stream(stream))
    _check("ds4x_local_pooled_attn", rc)
    return out, lse


def index_and_attend_local(q, w, k, positions, q_attn, kv, kv_local, ratio: int, local_pos0: int, window: int,
                           k_top: int = 512, S: int | None = None, scale: float | None = None, indices=None,
                           out=None, lse=None, workspace=None, want_lse: bool = True, stream=None):
    """The whole path with local-plus-pooled attention. Returns (indices, out, lse)."""
    torch = _torch()
    dt = _kv_dtype(q_attn)
    T, H, D = q.shape
    _, Hq, Dkv = q_attn.shape
    S = k.shape[0] if S is None else S
    scale = 1.0 / math.sqrt(Dkv) if scale is None else scale
    dev = q.device
    if indices is None:
        indices = torch.empty((T, k_top), dtype=torch.int32, device=dev)
    if out is None:
        out = torch.empty_like(q_attn)
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    need = workspace_bytes_local(T, S, k_top, window)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().ds4x_index_and_attend_local(_ptr(q), _ptr(w), _ptr(k), _ptr(positions), _ptr(q_attn), _ptr(kv),
                                            _ptr(kv_local), dt, T, H, D, S, ratio, k_top, Hq, Dkv, local_pos0,
                                            _rows(kv_local), window, scale, _ptr(indices), _ptr(out), _ptr(lse),
                                            _ptr(workspace), wbytes, _stream(stream))
    _check("ds4x_index_and_attend_local", rc)
    return indices, out, lse


def index_and_attend_local_host_bytes(T: int, H: int, D: int, S: int, k_top: int, Hq: int, Dkv: int, L: int,
                                      window: int, n_chunks: int = 0) -> int:
    return int(load().ds4x_index_and_attend_local_host_bytes(T, H, D, S, k_top, Hq, Dkv, L, window, n_chunks))


def index_and_attend_local_host(q, w, k, positions, q_attn, kv, kv_local, ratio: int, local_pos0: int,
                                window: int, k_top: int = 512, S: int | None = None, scale: float | None = None,
                                n_chunks: int = 0, indices=None, out=None, lse=None, device_buffer=None,
                                want_lse: bool = True, device=None, stream=None):
    """index_and_attend_host with the raw window (kv_local a CPU tensor too)."""
    torch = _torch()
    dt = _kv_dtype(q_attn)
    T, H, D = q.shape
    _, Hq, Dkv = q_attn.shape
    S = k.shape[0] if S is None else S
    L = _rows(kv_local)
    scale = 1.0 / math.sqrt(Dkv) if scale is None else scale
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if indices is None:
        indices = torch.empty((T, k_top), dtype=torch.int32).pin_memory()
    if out is None:
        out = torch.empty(q_attn.shape, dtype=q_attn.dtype).pin_memory()
    if lse is None and want_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32).pin_memory()
    need = index_and_attend_local_host_bytes(T, H, D, S, k_top, Hq, Dkv, L, window, n_chunks)
    if device_buffer is None:
        device_buffer = torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
    dbytes = device_buffer.numel() * device_buffer.element_size()
    rc = load().ds4x_index_and_attend_local_host(
        _host_ptr(q), _host_ptr(w), _host_ptr(k), _host_ptr(positions), _host_ptr(q_attn), _host_ptr(kv),
        _host_ptr(kv_local), dt, T, H, D, S, ratio, k_top, Hq, Dkv, local_pos0, L, window, scale,
        _host_ptr(indices), _host_ptr(out), _host_ptr(lse), n_chunks, _ptr(device_buffer), dbytes, _stream(stream))
    _check("ds4x_index_and_attend_local_host", rc)
    _keep_until_done(stream, (q, w, k, positions, q_attn, kv, kv_local, indices, out, lse, device_buffer))
    return indices, out, lse


# ------------------------------------------------------------------------------- compressor
def compress(x, g, bias, ratio: int, frontier_x=None, frontier_g=None, rows=None, frontier_x_out=None,
             frontier_g_out=None, stream=None):
    """One gated-pooled row per `ratio` positions of the sequence frontier + (x, g).
    x, g [T, D] and the frontier [f, D] (f < ratio) fp16 or bf16; bias [ratio, D] fp32.
    Returns (rows [(f+T)//ratio, D], new frontier x, new frontier g [(f+T)%ratio, D])."""
    torch = _torch()
    dt = _kv_dtype(x)
    T, D = x.shape
    f = 0 if frontier_x is None else int(frontier_x.shape[0])
    n_out, rem = (f + T) // ratio, (f + T) % ratio
    if rows is None:
        rows = torch.empty((n_out, D), dtype=x.dtype, device=x.device)
    if frontier_x_out is None:
        frontier_x_out = torch.empty((rem, D), dtype=x.dtype, device=x.device)
    if frontier_g_out is None:
        frontier_g_out = torch.empty((rem, D), dtype=x.dtype, device=x.device)
    rc = load().ds4x_compress(_ptr(x), _ptr(g), _ptr(bias), dt, T, D, ratio, _ptr(frontier_x), _ptr(frontier_g), f,
                              _ptr(rows) if n_out else None, _ptr(frontier_x_out) if rem else None,
                              _ptr(frontier_g_out) if rem else None, _stream(stream))
    _check("ds4x_compress", rc)
    return rows, frontier_x_out, frontier_g_out


def decode_workspace_bytes(capacity: int, k_top: int = 512) -> int:
    return int(load().ds4x_decode_workspace_bytes(capacity, k_top))


def decode(q, w, q_attn, k, kv, S0: int, pos0: int, ratio: int, k_new=None, kv_new=None, k_top: int = 512,
           scale: float | None = None, positions=None, indices=None, out=None, lse=None, workspace=None,
           want_lse: bool = True, stream=None):
    """n_steps = q.shape[0] decode steps at positions pos0, pos0+1, ...; rows of k_new / kv_new are
    appended to k / kv (capacity = k.shape[0]) as the positions complete them.
    Returns (indices, out, lse, positions, S_final)."""
    torch = _torch()
    dt = _kv_dtype(kv)
    n_steps, H, D = q.shape
    _, Hq, Dkv = q_attn.shape
    capacity = k.shape[0]
    if kv.shape[0] != capacity:
        raise ValueError("k and kv must have the same capacity")
    n_new = 0 if k_new is None else k_new.shape[0]
    scale = 1.0 / math.sqrt(Dkv) if scale is None else scale
    dev = q.device
    if positions is None:
        positions = torch.empty((n_steps,), dtype=torch.int32, device=dev)
    if indices is None:
        indices = torch.empty((n_steps, k_top), dtype=torch.int32, device=dev)
    if out is None:
        out = torch.empty_like(q_attn)
    if lse is None and want_lse:
        lse = torch.empty((n_steps, Hq), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty((max(decode_workspace_bytes(capacity, k_top), 16),), dtype=torch.uint8, device=dev)
    s_final = ctypes.c_int32(0)
    rc = load().ds4x_decode(_ptr(q), _ptr(w), _ptr(q_attn), _ptr(k), _ptr(kv), dt, capacity, S0, _ptr(k_new),
                            _ptr(kv_new), n_new, pos0, n_steps, H, D, ratio, k_top, Hq, Dkv, scale, _ptr(positions),
                            _ptr(indices), _ptr(out), _ptr(lse), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), ctypes.byref(s_final), _stream(stream))
    _check("ds4x_decode", rc)
    return indices, out, lse, positions, int(s_final.value)


def decode_local_workspace_bytes(capacity: int, k_top: int = 512, window: int = 128) -> int:
    return int(load().ds4x_decode_local_workspace_bytes(capacity, k_top, window))


def decode_local(q, w, q_attn, k, kv, S0: int, pos0: int, ratio: int, kv_raw, kv_raw_new, window: int,
                 k_new=None, kv_new=None, k_top: int = 512, scale: float | None = None, positions=None,
                 indices=None, out=None, lse=None, workspace=None, want_lse: bool = True, stream=None):
    """decode() with local-plus-pooled attention: kv_raw [raw_capacity, 512] holds the raw row of
    each position (rows below pos0 are the window's history), kv_raw_new [n_steps, 512] the steps'
    own raw rows, written at rows pos0.. by the call. Returns (indices, out, lse, positions, S_final)."""
    torch = _torch()
    dt = _kv_dtype(kv)
    n_steps, H, D = q.shape
    _, Hq, Dkv = q_attn.shape
    capacity = k.shape[0]
    if kv.shape[0] != capacity:
        raise ValueError("k and kv must have the same capacity")
    if kv_raw.dtype != kv.dtype or kv_raw_new.dtype != kv.dtype:
        raise ValueError("kv_raw and kv_raw_new must have kv's dtype")
    n_new = 0 if k_new is None else k_new.shape[0]
    scale = 1.0 / math.sqrt(Dkv) if scale is None else scale
    dev = q.device
    if positions is None:
        positions = torch.empty((n_steps,), dtype=torch.int32, device=dev)
    if indices is None:
        indices = torch.empty((n_steps, k_top), dtype=torch.int32, device=dev)
    if out is None:
        out = torch.empty_like(q_attn)
    if lse is None and want_lse:
        lse = torch.empty((n_steps, Hq), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty((max(decode_local_workspace_bytes(capacity, k_top, window), 16),), dtype=torch.uint8,
                                device=dev)
    s_final = ctypes.c_int32(0)
    rc = load().ds4x_decode_local(_ptr(q), _ptr(w), _ptr(q_attn), _ptr(k), _ptr(kv), dt, capacity, S0, _ptr(k_new),
                                  _ptr(kv_new), n_new, pos0, n_steps, H, D, ratio, k_top, Hq, Dkv, scale, _ptr(kv_raw),
                                  kv_raw.shape[0], _ptr(kv_raw_new), window, _ptr(positions), _ptr(indices),
                                  _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  ctypes.byref(s_final), _stream(stream))
    _check("ds4x_decode_local", rc)
    return indices, out, lse, positions, int(s_final.value)


# ----------------------------------------------------------------------- paged 4-bit cache
# A decode step calls these with a few microseconds of GPU work each, so the checks are written to cost
# little: a tensor that passes is looked at once, and the current stream is asked for by its address.
def _addr(name, t, dtype, dev):
    """The address of a contiguous tensor of `dtype` on CUDA device number `dev`."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _refuse(name, t, dtype, dev)
    return t.data_ptr()


def _refuse(name, t, dtype, dev):
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device, got {t.device}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def _addr_n(name, t, dtype, dev, n):
    """_addr of a tensor of at least n elements."""
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, {n} are needed")
    return _addr(name, t, dtype, dev)


def _elsewhere(dev, stream):
    """None when a call may run as it is: `dev` is current and no stream was given.  Otherwise the contexts
    to run it in, so that what it allocates belongs to the device and stream that its kernels run on."""
    torch = _torch()
    if dev < 0:
        raise ValueError("tensors passed to libds4x must live on a CUDA device")
    if stream is None:
        return None if torch._C._cuda_getDevice() == dev else (torch.cuda.device(dev),)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream),
                                           device=torch.device("cuda", dev))
    if stream.device.index != dev:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to cuda:{dev}")
    return torch.cuda.device(dev), torch.cuda.stream(stream)


def _within(contexts, call, *args, **kw):
    with contextlib.ExitStack() as stack:
        for c in contexts:
            stack.enter_context(c)
        return call(*args, **kw)


def _raw_stream(dev):
    return _torch()._C._cuda_getCurrentRawStream(dev)


def _kv4_pool(codes, scales, dev):
    """Addresses of a pool's codes [..., 256] and scales [..., 16], and its number of slots."""
    uint8 = _torch().uint8
    pc, psc = _addr("codes", codes, uint8, dev), _addr("scales", scales, uint8, dev)
    n = codes.numel() // KV4_CODE_BYTES
    if codes.size(-1) != KV4_CODE_BYTES or scales.size(-1) != KV4_SCALE_BYTES:
        raise ValueError(f"codes must end in {KV4_CODE_BYTES} bytes and scales in {KV4_SCALE_BYTES}, got "
                         f"{tuple(codes.shape)} and {tuple(scales.shape)}")
    if scales.numel() != n * KV4_SCALE_BYTES:
        raise ValueError(f"codes hold {n} slots, scales {scales.numel() // KV4_SCALE_BYTES}")
    return pc, psc, n


def page_plan(seen, n_new, rows, tables, free_pages, n_free, ratio: int, page_rows: int, T_cap: int, R_cap: int,
              positions=None, req=None, slots=None, seen_out=None, rows_out=None, n_free_out=None, totals=None,
              stream=None):
    """Positions, request ids, block tables and slots of one step of a batch, from its lengths, in one launch.
    seen, n_new, rows [n_req] int32: positions before the step, new ones, pooled rows held; tables
    [n_req, max_pages] int32, the new pages' entries are written in place; pages are taken from the end of
    free_pages[:n_free] (n_free [1] int32).  Returns (positions [T_cap], req [T_cap], slots [R_cap], seen_out,
    rows_out, n_free_out, totals [4] = tokens, completed rows, rows placed, pages taken); the packed
    outputs end in -1.  A request whose rows_out is below seen_out // ratio ran out of pages: it takes no more
    rows until it is retired or its seen is set back to rows * ratio.  Outputs may be passed in (when none is,
    they are views of one allocation, which lives as long as any of them); seen_out, rows_out and n_free_out may
    be their inputs."""
    torch = _torch()
    i32, dev = torch.int32, seen.get_device()
    contexts = _elsewhere(dev, stream)
    if contexts is not None:
        return _within(contexts, page_plan, seen, n_new, rows, tables, free_pages, n_free, ratio, page_rows, T_cap,
                       R_cap, positions, req, slots, seen_out, rows_out, n_free_out, totals)
    B = seen.numel()
    if tables.dim() != 2 or tables.size(0) != B:
        raise ValueError(f"tables must be [{B}, max_pages], got {tuple(tables.shape)}")
    if T_cap < 0 or R_cap < 0:
        raise ValueError(f"T_cap and R_cap must not be negative, got {T_cap} and {R_cap}")
    max_pages = tables.size(1)
    a = (_addr("seen", seen, i32, dev), _addr_n("n_new", n_new, i32, dev, B), _addr_n("rows", rows, i32, dev, B),
         _addr("tables", tables, i32, dev), _addr("free_pages", free_pages, i32, dev))
    pf = _addr_n("n_free", n_free, i32, dev, 1)
    outs = (positions, req, slots, seen_out, rows_out, n_free_out, totals)
    sizes = (T_cap, T_cap, R_cap, B, B, 1, 4)
    if positions is req is slots is seen_out is rows_out is n_free_out is totals is None:
        # the positions come first: 16-byte aligned, as the scorer and the top-k take them
        fresh = torch.empty((2 * T_cap + R_cap + 2 * B + 5,), dtype=i32, device=dev)
        at = fresh.data_ptr()
        b = [at, at + 4 * T_cap, at + 8 * T_cap]
        b += [b[2] + 4 * R_cap, b[2] + 4 * (R_cap + B), b[2] + 4 * (R_cap + 2 * B), b[2] + 4 * (R_cap + 2 * B + 1)]
        outs = fresh.split_with_sizes(sizes)
    else:
        outs = tuple([torch.empty((n,), dtype=i32, device=dev) if t is None else t for n, t in zip(sizes, outs)])
        b = [_addr_n(name, t, i32, dev, n) for name, t, n in zip(
            ("positions", "req", "slots", "seen_out", "rows_out", "n_free_out", "totals"), outs, sizes)]
    rc = (_lib or load()).ds4x_page_plan(*a, free_pages.numel(), pf, B, max_pages, page_rows, ratio, T_cap, R_cap, *b,
                                         _raw_stream(dev))
    if rc:
        _check("ds4x_page_plan", rc)
    return outs


def kv4_append(rows, slots, codes, scales, stream=None):
    """Quantises rows [n, 512] (fp16 or bf16) and writes row i to slot slots[i] of the pool codes [..., 256],
    scales [..., 16]; a slot outside the pool (the -1 of page_plan) skips its row.  Slots must be distinct."""
    torch = _torch()
    dt, dev = _kv_dtype(rows), rows.get_device()
    contexts = _elsewhere(dev, stream)
    if contexts is not None:
        return _within(contexts, kv4_append, rows, slots, codes, scales)
    n, Dkv = rows.shape
    pr = _addr("rows", rows, rows.dtype, dev)
    ps = _addr_n("slots", slots, torch.int32, dev, n)
    pc, psc, n_slots = _kv4_pool(codes, scales, dev)
    rc = (_lib or load()).ds4x_kv4_append(pr, dt, ps, n, Dkv, pc, psc, n_slots, _raw_stream(dev))
    if rc:
        _check("ds4x_kv4_append", rc)


def kv4_read(codes, scales, slots, dtype, out=None, stream=None):
    """The rows at slots [n] int32 of the pool as [n, 512] of `dtype` (float16 or bfloat16); zeros for a slot
    outside the pool."""
    torch = _torch()
    dev = codes.get_device()
    contexts = _elsewhere(dev, stream)
    if contexts is not None:
        return _within(contexts, kv4_read, codes, scales, slots, dtype, out)
    pc, psc, n_slots = _kv4_pool(codes, scales, dev)
    n, Dkv = slots.numel(), 2 * KV4_CODE_BYTES
    ps = _addr("slots", slots, torch.int32, dev)
    if out is None:
        out = torch.empty((n, Dkv), dtype=dtype, device=dev)
    elif out.shape != (n, Dkv):
        raise ValueError(f"out must be of shape {(n, Dkv)}, got {tuple(out.shape)}")
    po = _addr("out", out, dtype, dev)
    rc = (_lib or load()).ds4x_kv4_read(pc, psc, n_slots, ps, n, Dkv, po, _kv_dtype(out), _raw_stream(dev))
    if rc:
        _check("ds4x_kv4_read", rc)
    return out


def kv4_attn_workspace_bytes(T: int, max_rows: int) -> int:
    """Workspace of kv4_attn: max_rows = k_top, or max_pages * page_rows without indices."""
    return int(load().ds4x_kv4_attn_workspace_bytes(T, max_rows))


def kv4_attn(q_attn, codes, scales, tables, rows, page_rows: int, req=None, positions=None, ratio: int = 1,
             indices=None, counts=None, scale: float | None = None, out=None, lse=None, workspace=None,
             want_lse: bool = True, stream=None):
    """64-head MQA of q_attn [T, 64, 512] over rows of the paged 4-bit cache.  Token t belongs to request
    req[t] (None: request t), which holds rows[b] rows through tables[b] [max_pages].  With indices
    [T, k_top] it attends to those rows (the first counts[t] entries; -1 and rows not held are skipped; with
    k_top = 0 to none), without to every row visible at positions[t] (None: all held).  Returns (out, lse)."""
    torch = _torch()
    i32, dev = torch.int32, q_attn.get_device()
    contexts = _elsewhere(dev, stream)
    if contexts is not None:
        return _within(contexts, kv4_attn, q_attn, codes, scales, tables, rows, page_rows, req, positions, ratio,
                       indices, counts, scale, out, lse, workspace, want_lse)
    dt = _kv_dtype(q_attn)
    dtype = q_attn.dtype
    T, Hq, Dkv = shape = q_attn.shape
    pq = _addr("q_attn", q_attn, dtype, dev)
    pc, psc, n_slots = _kv4_pool(codes, scales, dev)
    n_req = rows.numel()
    prow = _addr("rows", rows, i32, dev)
    if tables.dim() != 2 or tables.size(0) != n_req:
        raise ValueError(f"tables must be [{n_req}, max_pages], got {tuple(tables.shape)}")
    max_pages = tables.size(1)
    ptab = _addr("tables", tables, i32, dev)
    preq = None if req is None else _addr_n("req", req, i32, dev, T)
    ppos = None if positions is None else _addr_n("positions", positions, i32, dev, T)
    k_top, pidx, pcnt, max_rows = 0, None, None, max_pages * page_rows
    if indices is not None:
        if indices.dim() != 2 or indices.size(0) != T:
            raise ValueError(f"indices must be [{T}, k_top], got {tuple(indices.shape)}")
        k_top = max_rows = indices.size(1)
        pidx = _addr("indices", indices, i32, dev)
        pcnt = None if counts is None else _addr_n("counts", counts, i32, dev, T)
        if k_top == 0:  # an empty tensor's address is 0, which asks for every row: no page is offered instead
            max_pages, pidx, pcnt = 0, None, None
    elif counts is not None:
        raise ValueError("counts belong to indices")
    if out is None:
        out = torch.empty_like(q_attn)
    elif out.shape != shape:
        raise ValueError(f"out must be of shape {tuple(shape)}, got {tuple(out.shape)}")
    if lse is None:
        if want_lse:
            lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    elif lse.shape != (T, Hq):
        raise ValueError(f"lse must be of shape {(T, Hq)}, got {tuple(lse.shape)}")
    lib = _lib or load()
    if workspace is None and 0 <= max_rows < 2**31:
        need = lib.ds4x_kv4_attn_workspace_bytes(T, max_rows)
        if need > 0:
            workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    pw, wbytes = None, 0
    if workspace is not None:
        pw, wbytes = _addr("workspace", workspace, workspace.dtype, dev), workspace.numel() * workspace.element_size()
    rc = lib.ds4x_kv4_attn(pq, dt, pc, psc, n_slots, ptab, prow, n_req, max_pages, page_rows, preq, ppos, ratio, pidx,
                           pcnt, T, Hq, Dkv, k_top, 1.0 / math.sqrt(Dkv) if scale is None else scale,
                           _addr("out", out, dtype, dev),
                           None if lse is None else _addr("lse", lse, torch.float32, dev), pw, wbytes,
                           _raw_stream(dev))
    if rc:
        _check("ds4x_kv4_attn", rc)
    return out, lse


def device_status(stream=None, clear: bool = True) -> int:
    return int(load().ds4x_device_status(_stream(stream), 1 if clear else 0))


def selftest_bounded_wait(timeout_ns: int, stream=None):
    _check("ds4x_selftest_bounded_wait", load().ds4x_selftest_bounded_wait(timeout_ns, _stream(stream)))


TOPK_STATIC_SCRATCH_BYTES = 4 << 20


def topk_static_scratch(scores, positions, S: int, ratio: int, k_top: int = 512, indices=None, counts=None,
                        stream=None):
    """ds4x_topk without a workspace, for callers that may not allocate device memory while they
    run (the split mode's candidate lists use a fixed array inside the library instead). The
    output tensors must be passed in by such callers; calls overlapping on the GPU must not be
    issued (they share that array)."""
    torch = _torch()
    _need(scores, torch.float32, "scores")
    T, ld = scores.shape
    _need_positions(positions, T)
    if indices is None:
        indices = torch.empty((T, k_top), dtype=torch.int32, device=scores.device)
    if counts is None:
        counts = torch.empty((T,), dtype=torch.int32, device=scores.device)
    lib = load()
    fn = lib.ds4x_topk_static_scratch
    P = ctypes.c_void_p
    fn.argtypes = [P, ctypes.c_int64, P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P, P]
    fn.restype = ctypes.c_int
    _check("ds4x_topk_static_scratch", fn(_ptr(scores), ld, _ptr(positions), T, S, ratio, k_top, _ptr(indices),
                                          _ptr(counts), _stream(stream)))
    return indices, counts
