"""PaTH attention on B200 (sm_100a): thin Python binding of libpath_attn.so.

The binding only marshals arguments: it checks dtypes, shapes and
contiguity, allocates outputs and workspace with torch when the caller does
not pass them, and calls the C ABI declared in ``include/path_attn.h`` on the
current torch CUDA stream. Every step of the computation runs in the
library's CUDA kernels; there is no CPU path. If the library is missing or no
CUDA device is present, the calls raise.

Entry points (same names as the C ABI):
- ``path_attn_fwd(q, k, v, w, beta, log_f=None, scale=None) -> (out, lse)``
- ``path_attn_bwd(q, k, v, w, beta, out, lse, dout, log_f=None, scale=None) -> dict``
- ``path_decode_step(q, k_new, v_new, w, beta, k_cache, v_cache, n_cached, scale=None,
  log_f=None, g_cache=None) -> out`` (with ``log_f``: ``path_decode_step_gated``)
- ``path_attn_prefill(q, k, v, w, beta, capacity, log_f=None, scale=None)
  -> (out, lse, k_cache, v_cache, g_cache)``
- ``path_decode_step_gated(q, k_new, v_new, w, beta, log_f, k_cache, v_cache, g_cache,
  n_cached, scale=None) -> out``
- ``path_decode_step_noalloc(q, k_new, v_new, w, beta, k_cache, v_cache, n_cached, scale=None)
  -> out``
- ``path_attn_wait_status(workspace) -> int`` (0 = no bounded wait gave up)
- ``path_attn_workspace_bytes``, ``path_decode_workspace_bytes``, ``path_status_string``
- diagnostics: ``path_kernel_launch_count()``, ``path_profile_enable(on)``,
  ``path_profile_read() -> {stage: (total_ms, count)}``
- the w / beta prologue: ``path_wbeta_fwd(x, A, Bw, f, U, b, H, beta_max=2.0) -> (w, beta)``,
  ``path_wbeta_bwd(x, A, Bw, f, U, b, H, dw, dbeta, beta_max=2.0) -> dict``,
  ``path_wbeta_workspace_bytes``
- the paged decode cache (a pool of pages, and tables on the device):
  ``path_decode_step_paged(q, k_new, v_new, w, beta, k_pages, v_pages, table, lens, rows=None)
  -> out``, ``path_decode_step_shared(..., prefix_table, prefix_len, state, rows=None) -> out``
  (a batch behind one shared prefix), ``path_pages_reserve``, ``path_pages_fork``,
  ``path_pages_free``, ``path_pages_compact``, ``path_pages_copy``, ``path_pages_store``,
  ``path_state_copy``, ``path_decode_paged_workspace_bytes``
- test hook: ``path_test_withhold_kv_load(on)`` (makes bounded waits of the forward and the
  paged decode steps give up)
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpath_attn.so")

PATH_F32, PATH_BF16, PATH_BF16_F32OUT = 0, 1, 2
PATH_ERR_PAGE = 6
_DT = {torch.float32: PATH_F32, torch.bfloat16: PATH_BF16}


def _mode(in_dtype, out_dtype):
    """path_dtype of a call from the input and output element types."""
    if in_dtype == torch.float32 and out_dtype == torch.float32:
        return PATH_F32
    if in_dtype == torch.bfloat16 and out_dtype == torch.bfloat16:
        return PATH_BF16
    if in_dtype == torch.bfloat16 and out_dtype == torch.float32:
        return PATH_BF16_F32OUT
    raise ValueError(f"unsupported dtypes: inputs {in_dtype}, outputs {out_dtype}")
_lib = None


class _StageTime(ctypes.Structure):
    """path_stage_time of the C header."""
    _fields_ = [("name", ctypes.c_char * 32), ("total_ms", ctypes.c_double),
                ("count", ctypes.c_int)]


class PathError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {path_status_string(status)} (status {status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m softmax_attention_block_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, fp, i, f, sz = (ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                            ctypes.c_size_t)
        L.path_status_string.argtypes = [i]
        L.path_status_string.restype = ctypes.c_char_p
        L.path_attn_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.path_attn_workspace_bytes.restype = sz
        L.path_decode_workspace_bytes.argtypes = [i, i, i, i, i]
        L.path_decode_workspace_bytes.restype = sz
        L.path_attn_fwd.argtypes = [vp, vp, vp, vp, fp, fp, f, i, i, i, i, i, vp, fp, vp, sz, vp]
        L.path_attn_bwd.argtypes = [vp, vp, vp, vp, fp, fp, f, i, i, i, i, i, vp, fp, vp,
                                    vp, vp, vp, vp, fp, fp, ctypes.c_uint, vp, sz, vp]
        L.path_decode_step.argtypes = [vp, vp, vp, vp, fp, f, i, i, i, i, i, i, vp, vp, vp, vp,
                                       sz, vp]
        L.path_decode_step_gated.argtypes = [vp, vp, vp, vp, fp, fp, f, i, i, i, i, i, i, vp,
                                             vp, fp, vp, vp, sz, vp]
        L.path_attn_prefill.argtypes = [vp, vp, vp, vp, fp, fp, f, i, i, i, i, i, vp, fp, vp, vp,
                                        fp, i, vp, sz, vp]
        L.path_decode_step_noalloc.argtypes = [vp, vp, vp, vp, fp, f, i, i, i, i, i, i, vp, vp,
                                               vp, vp]
        L.path_attn_wait_status.argtypes = [vp, vp]
        L.path_wbeta_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
        L.path_wbeta_workspace_bytes.restype = sz
        L.path_wbeta_fwd.argtypes = [vp, vp, vp, fp, vp, fp, f, i, i, i, i, i, i, i, vp, fp, vp, sz,
                                     vp]
        L.path_wbeta_bwd.argtypes = [vp, vp, vp, fp, vp, fp, f, i, i, i, i, i, i, i, vp, fp, vp, fp,
                                     fp, fp, fp, fp, ctypes.c_uint, vp, sz, vp]
        L.path_wbeta_fwd.restype = i
        L.path_wbeta_bwd.restype = i
        L.path_decode_paged_workspace_bytes.argtypes = [i] * 7
        L.path_decode_paged_workspace_bytes.restype = sz
        step = [vp, vp, vp, vp, fp, fp, f, i, i, i, i, vp, vp, fp, i, i, vp, i, i, vp, vp]
        L.path_decode_step_paged.argtypes = [*step, vp, vp, sz, vp]
        L.path_decode_step_shared.argtypes = [*step, vp, i, fp, fp, vp, vp, sz, vp]
        L.path_pages_reserve.argtypes = [vp, vp, vp, i, i, i, i, vp, vp, i, vp, vp]
        L.path_pages_fork.argtypes = [vp, vp, vp, vp, i, i, i, i, vp, vp, i, vp, i, vp, vp]
        L.path_pages_free.argtypes = [vp, vp, vp, vp, i, i, i, vp, i, vp]
        L.path_pages_compact.argtypes = [vp, vp, vp, i, i, i, vp, i, vp, vp]
        L.path_pages_copy.argtypes = [vp, i, vp, vp, vp, fp, i, i, i, i, i, vp]
        L.path_pages_store.argtypes = [vp, vp, fp, i, i, i, i, i, vp, vp, fp, i, i, vp, i, i, vp, vp,
                                       vp, vp]
        L.path_state_copy.argtypes = [fp, fp, i, i, i, vp, vp, i, vp]
        for fn in (L.path_decode_step_paged, L.path_decode_step_shared, L.path_pages_reserve,
                   L.path_pages_fork, L.path_pages_free, L.path_pages_compact, L.path_pages_copy,
                   L.path_pages_store, L.path_state_copy):
            fn.restype = i
        L.path_test_withhold_kv_load.argtypes = [i]
        L.path_test_withhold_kv_load.restype = i
        L.path_kernel_launch_count.restype = ctypes.c_ulonglong
        L.path_profile_enable.argtypes = [i]
        L.path_profile_enable.restype = i
        L.path_profile_read.argtypes = [ctypes.POINTER(_StageTime), i]
        L.path_profile_read.restype = i
        for fn in (L.path_attn_fwd, L.path_attn_bwd, L.path_decode_step,
                   L.path_decode_step_gated, L.path_decode_step_noalloc, L.path_attn_prefill,
                   L.path_attn_wait_status):
            fn.restype = i
        _lib = L
    return _lib


def path_status_string(status: int) -> str:
    return lib().path_status_string(int(status)).decode()


def path_attn_workspace_bytes(B, H, L, d, dtype, for_bwd=False, out_dtype=None) -> int:
    mode = _mode(dtype, out_dtype or dtype)
    return int(lib().path_attn_workspace_bytes(B, H, L, d, mode, int(bool(for_bwd))))


def path_decode_workspace_bytes(B, H, capacity, d, dtype) -> int:
    return int(lib().path_decode_workspace_bytes(B, H, capacity, d, _DT[dtype]))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _expect(name, t, shape, dtype):
    """The library reads and writes these buffers by size alone: check what it will assume."""
    if t is None or (t.shape == shape and t.dtype == dtype):
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")


def _check_dev(*ts):
    """All tensors contiguous, on one CUDA device, and that device the current one: the
    library launches on the current device's stream and resolves its own per-device
    state (the allocation-free decode's scratch array) through the current device."""
    ts = [t for t in ts if t is not None]
    for t in ts:
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        if t.device != ts[0].device:
            raise ValueError("all tensors must be on one device")
    if ts and ts[0].device.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {ts[0].device} but the current CUDA device is "
                         f"cuda:{torch.cuda.current_device()}: call under "
                         f"torch.cuda.device({ts[0].device})")


def _check_here(*ts):
    """_check_dev, its usual outcome first: contiguous tensors on the current device."""
    here = torch.cuda.current_device() if torch.cuda.is_initialized() else -1
    for t in ts:
        if t is not None and (t.get_device() != here or here < 0 or not t.is_contiguous()):
            return _check_dev(*ts)


def _room(nbytes, ws, device):
    """A workspace of nbytes() bytes, or the caller's, whose size the library checks."""
    if ws is None:
        n = nbytes()
        return torch.empty(max(n, 1), dtype=torch.uint8, device=device), n
    return ws, ws.nbytes


def _check_attn_inputs(q, k, v, w, beta, log_f):
    if q.dim() != 4:
        raise ValueError("q must be [B,H,L,d]")
    if q.dtype not in _DT:
        raise ValueError(f"q: dtype {q.dtype}, expected float32 or bfloat16")
    B, H, L, d = q.shape
    for n, t in (("k", k), ("v", v), ("w", w)):
        _expect(n, t, q.shape, q.dtype)
    _expect("beta", beta, (B, H, L), torch.float32)
    _expect("log_f", log_f, (B, H, L), torch.float32)


# the current stream's handle without a Stream object around it, where this torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _workspace(nbytes, device, ws):
    if ws is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    if ws.numel() * ws.element_size() < nbytes:
        raise ValueError("workspace too small")
    return ws


def _scale(scale, d):
    return float(d ** -0.5 if scale is None else scale)


def path_attn_fwd(q, k, v, w, beta, log_f=None, scale=None, out=None, lse=None, workspace=None,
                  out_dtype=None):
    """Forward pass. q, k, v, w: [B,H,L,d] (fp32 or bf16); beta, log_f: [B,H,L] fp32.
    out_dtype (default: q's dtype) may be torch.float32 with bf16 inputs.
    Returns (out [B,H,L,d], lse [B,H,L] fp32)."""
    _check_attn_inputs(q, k, v, w, beta, log_f)
    B, H, L, d = q.shape
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    dt = _mode(q.dtype, out.dtype)
    if lse is None:
        lse = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    _expect("out", out, q.shape, out.dtype)
    _expect("lse", lse, (B, H, L), torch.float32)
    _check_dev(q, k, v, w, beta, log_f, out, lse, workspace)
    nbytes = path_attn_workspace_bytes(B, H, L, d, q.dtype, False, out.dtype)
    ws = _workspace(nbytes, q.device, workspace)
    # the buffer's whole size: a backward-sized workspace also receives what a
    # backward that reuses it reads
    st = lib().path_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(w), _ptr(beta), _ptr(log_f),
                             _scale(scale, d), B, H, L, d, dt, _ptr(out), _ptr(lse), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream())
    if st:
        raise PathError(st, "path_attn_fwd")
    return out, lse


PATH_BWD_REUSE_FWD_WORKSPACE = 1


def path_attn_bwd(q, k, v, w, beta, out, lse, dout, log_f=None, scale=None, grads=None,
                  workspace=None, reuse_fwd_workspace=False):
    """Backward of sum(out * dout). out, dout and the returned dq, dk, dv, dw share
    out's dtype. Returns dict dq, dk, dv, dw, dbeta[, dlog_f].

    reuse_fwd_workspace: `workspace` is the buffer the matching path_attn_fwd call
    used (allocated with the backward size), inputs unchanged since; the backward
    then reuses the forward's block transforms and transported keys."""
    if reuse_fwd_workspace and workspace is None:
        raise ValueError("reuse_fwd_workspace needs the forward's workspace")
    _check_attn_inputs(q, k, v, w, beta, log_f)
    B, H, L, d = q.shape
    dt = _mode(q.dtype, out.dtype)
    if dout.dtype != out.dtype:
        raise ValueError("dout must have out's dtype")
    _expect("out", out, q.shape, out.dtype)
    _expect("dout", dout, q.shape, out.dtype)
    _expect("lse", lse, (B, H, L), torch.float32)
    if grads is None:
        grads = {n: torch.empty(q.shape, dtype=out.dtype, device=q.device)
                 for n in ("dq", "dk", "dv", "dw")}
        grads["dbeta"] = torch.empty_like(beta)
        if log_f is not None:
            grads["dlog_f"] = torch.empty_like(log_f)
    for n in ("dq", "dk", "dv", "dw"):
        _expect(n, grads[n], q.shape, out.dtype)
    _expect("dbeta", grads["dbeta"], (B, H, L), torch.float32)
    dlf = grads.get("dlog_f") if log_f is not None else None
    if log_f is not None and dlf is None:
        raise ValueError("grads needs dlog_f when log_f is given")
    _expect("dlog_f", dlf, (B, H, L), torch.float32)
    _check_dev(q, k, v, w, beta, log_f, out, lse, dout, workspace, *grads.values())
    nbytes = path_attn_workspace_bytes(B, H, L, d, q.dtype, True, out.dtype)
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().path_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(w), _ptr(beta), _ptr(log_f),
                             _scale(scale, d), B, H, L, d, dt, _ptr(out), _ptr(lse), _ptr(dout),
                             _ptr(grads["dq"]), _ptr(grads["dk"]), _ptr(grads["dv"]),
                             _ptr(grads["dw"]), _ptr(grads["dbeta"]), _ptr(dlf),
                             PATH_BWD_REUSE_FWD_WORKSPACE if reuse_fwd_workspace else 0, _ptr(ws),
                             nbytes, _stream())
    if st:
        raise PathError(st, "path_attn_bwd")
    return grads


def _check_decode(q, k_new, v_new, w, beta, k_cache, v_cache, out, log_f, g_cache):
    if k_cache.dim() != 4 or k_cache.dtype not in _DT:
        raise ValueError("k_cache must be [B,H,capacity,d], float32 or bfloat16")
    B, H, cap, d = k_cache.shape
    if (log_f is None) != (g_cache is None):
        raise ValueError("log_f and g_cache go together")
    _expect("v_cache", v_cache, k_cache.shape, k_cache.dtype)
    for n, t in (("q", q), ("k_new", k_new), ("v_new", v_new), ("w", w), ("out", out)):
        _expect(n, t, (B, H, d), k_cache.dtype)
    _expect("beta", beta, (B, H), torch.float32)
    _expect("log_f", log_f, (B, H), torch.float32)
    _expect("g_cache", g_cache, (B, H, cap), torch.float32)
    return B, H, cap, d


def path_decode_step(q, k_new, v_new, w, beta, k_cache, v_cache, n_cached, scale=None, out=None,
                     workspace=None, log_f=None, g_cache=None):
    """One decode step; updates k_cache / v_cache ([B,H,cap,d]) in place. Returns out [B,H,d].

    With the forget gate, log_f [B,H] fp32 is log f of the new position and g_cache
    [B,H,cap] fp32 the cached keys' gate biases, also updated in place
    (path_decode_step_gated)."""
    if out is None:
        out = torch.empty_like(q)
    B, H, cap, d = _check_decode(q, k_new, v_new, w, beta, k_cache, v_cache, out, log_f, g_cache)
    dt = _DT[k_cache.dtype]
    _check_dev(q, k_new, v_new, w, beta, k_cache, v_cache, out, log_f, g_cache, workspace)
    nbytes = path_decode_workspace_bytes(B, H, cap, d, k_cache.dtype)
    ws = _workspace(nbytes, q.device, workspace)
    if log_f is None:
        st = lib().path_decode_step(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(w), _ptr(beta),
                                    _scale(scale, d), B, H, d, int(n_cached), cap, dt,
                                    _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(ws), nbytes,
                                    _stream())
        where = "path_decode_step"
    else:
        st = lib().path_decode_step_gated(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(w), _ptr(beta),
                                          _ptr(log_f), _scale(scale, d), B, H, d, int(n_cached),
                                          cap, dt, _ptr(k_cache), _ptr(v_cache), _ptr(g_cache),
                                          _ptr(out), _ptr(ws), nbytes, _stream())
        where = "path_decode_step_gated"
    if st:
        raise PathError(st, where)
    return out


def path_decode_step_gated(q, k_new, v_new, w, beta, log_f, k_cache, v_cache, g_cache, n_cached,
                           scale=None, out=None, workspace=None):
    """PaTH-FoX decode step: path_decode_step with the forget gate (log_f [B,H] fp32 of the
    new position; g_cache [B,H,cap] fp32, the cached keys' gate biases, updated in place)."""
    if log_f is None or g_cache is None:
        raise ValueError("path_decode_step_gated needs log_f and g_cache")
    return path_decode_step(q, k_new, v_new, w, beta, k_cache, v_cache, n_cached, scale=scale,
                            out=out, workspace=workspace, log_f=log_f, g_cache=g_cache)


def path_decode_step_noalloc(q, k_new, v_new, w, beta, k_cache, v_cache, n_cached, scale=None,
                             out=None):
    """path_decode_step without a workspace (the library's fixed 4 MiB device scratch; see
    the C header for its limit and its sharing between calls on one device)."""
    if out is None:
        out = torch.empty_like(q)
    B, H, cap, d = _check_decode(q, k_new, v_new, w, beta, k_cache, v_cache, out, None, None)
    _check_dev(q, k_new, v_new, w, beta, k_cache, v_cache, out)
    st = lib().path_decode_step_noalloc(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(w), _ptr(beta),
                                        _scale(scale, d), B, H, d, int(n_cached), cap,
                                        _DT[k_cache.dtype], _ptr(k_cache), _ptr(v_cache),
                                        _ptr(out), _stream())
    if st:
        raise PathError(st, "path_decode_step_noalloc")
    return out


def path_attn_wait_status(workspace) -> int:
    """Waits for the current stream, then returns 0, or PATH_ERR_TIMEOUT (5) if the last
    path_attn_fwd / path_attn_bwd that used `workspace` had a bounded wait give up, or
    PATH_ERR_PAGE (6) if the last paged decode step that used it met a page, slot or length
    out of range."""
    _check_dev(workspace)
    return int(lib().path_attn_wait_status(_ptr(workspace), _stream()))


def path_kernel_launch_count() -> int:
    """Kernels this library has launched in this process so far."""
    return int(lib().path_kernel_launch_count())


def path_profile_enable(on: bool) -> bool:
    """Per-stage event timing on or off; returns the previous setting."""
    return bool(lib().path_profile_enable(int(bool(on))))


def path_profile_read(max_entries: int = 64) -> dict:
    """Stage name -> (total ms, launches) of the stages timed since the last read."""
    buf = (_StageTime * max_entries)()
    n = lib().path_profile_read(buf, max_entries)
    return {buf[i].name.decode(): (buf[i].total_ms, buf[i].count) for i in range(n)}


def path_attn_prefill(q, k, v, w, beta, capacity, log_f=None, scale=None, out=None, lse=None,
                      k_cache=None, v_cache=None, g_cache=None, workspace=None, out_dtype=None):
    """Forward over positions 0..L-1 plus the decode cache it leaves.

    Returns (out, lse, k_cache, v_cache, g_cache): out / lse as path_attn_fwd; the
    caches [B,H,capacity,d] in q's dtype with rows 0..L-1 written (k_cache row j =
    H_{L-1} ... H_{j+1} k_j, v_cache row j = v_j); g_cache [B,H,capacity] fp32 (row j =
    c_{L-1} - c_j) with the forget gate, else None. Caches the call allocates are
    zero past row L-1. Rows padded to one L need beta = 0 and log_f = 0 behind their ends, so
    that the padding's factors stay out of their keys."""
    _check_attn_inputs(q, k, v, w, beta, log_f)
    B, H, L, d = q.shape
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    dt = _mode(q.dtype, out.dtype)
    if lse is None:
        lse = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    _expect("out", out, q.shape, out.dtype)
    _expect("lse", lse, (B, H, L), torch.float32)
    _expect("k_cache", k_cache, (B, H, capacity, d), q.dtype)
    _expect("v_cache", v_cache, (B, H, capacity, d), q.dtype)
    if log_f is not None:
        _expect("g_cache", g_cache, (B, H, capacity), torch.float32)
    if k_cache is None:
        k_cache = torch.zeros((B, H, capacity, d), dtype=q.dtype, device=q.device)
    if v_cache is None:
        v_cache = torch.zeros((B, H, capacity, d), dtype=q.dtype, device=q.device)
    if log_f is not None and g_cache is None:
        g_cache = torch.zeros((B, H, capacity), dtype=torch.float32, device=q.device)
    if log_f is None:
        g_cache = None
    _check_dev(q, k, v, w, beta, log_f, out, lse, k_cache, v_cache, g_cache, workspace)
    nbytes = path_attn_workspace_bytes(B, H, L, d, q.dtype, False, out.dtype)
    ws = _workspace(nbytes, q.device, workspace)
    st = lib().path_attn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(w), _ptr(beta), _ptr(log_f),
                                 _scale(scale, d), B, H, L, d, dt, _ptr(out), _ptr(lse),
                                 _ptr(k_cache), _ptr(v_cache), _ptr(g_cache), int(capacity),
                                 _ptr(ws), nbytes, _stream())
    if st:
        raise PathError(st, "path_attn_prefill")
    return out, lse, k_cache, v_cache, g_cache


def path_test_withhold_kv_load(on: bool) -> None:
    """Test hook of the bounded waits (include/path_attn.h): while on, the tensor-core
    forward's last query tile never receives one key/value block and reports a timeout; so does
    the paged decode steps' first warp."""
    st = lib().path_test_withhold_kv_load(1 if on else 0)
    if st:
        raise PathError(st, "path_test_withhold_kv_load")


# ---------------------------------------------------------------- the paged decode cache
def _expect_pool(k_pages, v_pages, g_pages):
    shape = k_pages.shape
    if len(shape) != 4 or k_pages.dtype not in _DT:
        raise ValueError("k_pages must be [n_pages,H,page,d], float32 or bfloat16")
    _expect("v_pages", v_pages, shape, k_pages.dtype)
    if g_pages is not None:
        _expect("g_pages", g_pages, shape[:3], torch.float32)
    return shape


def _expect_table(table, **per_slot):
    shape = table.shape
    if len(shape) != 2:
        raise ValueError("table must be [n_slots,max_pages]")
    _expect("table", table, shape, torch.int32)
    slots = shape[:1]
    for n, t in per_slot.items():
        _expect(n, t, slots, torch.int32)
    return shape


def _expect_owner(owner):
    if owner.dim() != 1:
        raise ValueError("owner must be [n_pages]")
    _expect("owner", owner, owner.shape, torch.int32)
    return owner.shape[0]


def _expect_list(**lists):
    """int32 lists of one length; returns it."""
    shape = None
    for name, t in lists.items():
        if t.dim() != 1:
            raise ValueError(f"{name}: must have one dimension")
        shape = shape or t.shape
        _expect(name, t, shape, torch.int32)
    return shape[0]


def _moves(moves, most, device):
    """The caller's list of moves, or a new one of `most` pairs, and its length."""
    if moves is None:
        moves = torch.empty((max(most, 1), 2), dtype=torch.int32, device=device)
    if moves.dim() != 2:
        raise ValueError("moves must be [max_moves,2]")
    _expect("moves", moves, (moves.shape[0], 2), torch.int32)
    return moves, moves.shape[0]


def _info(info, device):
    if info is None:
        info = torch.zeros(4, dtype=torch.int32, device=device)
    _expect("info", info, (4,), torch.int32)
    return info


def path_decode_paged_workspace_bytes(B, H, max_pages, page, d, dtype, prefix_len=0) -> int:
    return int(lib().path_decode_paged_workspace_bytes(B, H, max_pages, page, d, _DT[dtype],
                                                       int(prefix_len)))


def _step_paged(where, q, k_new, v_new, w, beta, k_pages, v_pages, table, lens, rows, scale, log_f,
                g_pages, out, workspace, prefix=None):
    n_pages, H, page, d = _expect_pool(k_pages, v_pages, g_pages)
    if q.dim() != 3:
        raise ValueError("q must be [B,H,d]")
    B, dtype = q.shape[0], k_pages.dtype
    if out is None:  # an idle row's output is not written
        out = torch.empty_like(q) if rows is None else torch.zeros_like(q)
    if (log_f is None) != (g_pages is None):
        raise ValueError("log_f and g_pages go together")
    shape = (B, H, d)
    for n, t in (("q", q), ("k_new", k_new), ("v_new", v_new), ("w", w), ("out", out)):
        _expect(n, t, shape, dtype)
    _expect("beta", beta, (B, H), torch.float32)
    _expect("log_f", log_f, (B, H), torch.float32)
    n_slots, max_pages = _expect_table(table, lens=lens)
    _expect("rows", rows, (B,), torch.int32)
    prefix_len, more, extra = 0, (), ()
    if prefix is not None:
        prefix_table, prefix_len, state, g_state = prefix
        prefix_len = int(prefix_len)
        _expect_list(prefix_table=prefix_table)
        if prefix_len > prefix_table.shape[0] * page:
            raise ValueError(f"prefix_table: {prefix_table.shape[0]} pages of {page} rows do not "
                             f"hold prefix_len={prefix_len}")
        if (log_f is None) != (g_state is None):
            raise ValueError("log_f and g_state go together")
        _expect("state", state, (n_slots, H, d, d), torch.float32)
        _expect("g_state", g_state, (n_slots, H), torch.float32)
        more = (prefix_table, state, g_state)
        extra = (_ptr(prefix_table), prefix_len, _ptr(state), _ptr(g_state))
    _check_here(q, k_new, v_new, w, beta, log_f, k_pages, v_pages, g_pages, table, lens, rows, out,
               workspace, *more)
    ws, nbytes = _room(lambda: path_decode_paged_workspace_bytes(B, H, max_pages, page, d, dtype, prefix_len),
                       workspace, q.device)
    st = getattr(lib(), where)(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(w), _ptr(beta), _ptr(log_f),
                               _scale(scale, d), B, H, d, _DT[dtype], _ptr(k_pages), _ptr(v_pages),
                               _ptr(g_pages), n_pages, page, _ptr(table), n_slots, max_pages,
                               _ptr(lens), _ptr(rows), *extra, _ptr(out), _ptr(ws), nbytes,
                               _stream())
    if st:
        raise PathError(st, where)
    return out


def path_decode_step_paged(q, k_new, v_new, w, beta, k_pages, v_pages, table, lens, rows=None,
                           scale=None, log_f=None, g_pages=None, out=None, workspace=None):
    """One decode step of a ragged batch over paged caches. q, k_new, v_new, w: [B,H,d]; beta
    (and log_f): [B,H] fp32; k_pages, v_pages: [n_pages,H,page,d] (g_pages [n_pages,H,page] fp32
    with log_f), updated in place; table [n_slots,max_pages] and lens [n_slots] int32; rows [B]
    int32: the slot of each batch row (default: its own number; negative: idle, its row of out is
    left as it was). lens is not advanced. Returns out [B,H,d]."""
    return _step_paged("path_decode_step_paged", q, k_new, v_new, w, beta, k_pages, v_pages, table,
                       lens, rows, scale, log_f, g_pages, out, workspace)


def path_decode_step_shared(q, k_new, v_new, w, beta, k_pages, v_pages, table, lens, prefix_table,
                            prefix_len, state, rows=None, scale=None, log_f=None, g_pages=None,
                            g_state=None, out=None, workspace=None):
    """path_decode_step_paged for sequences that continue one prefix: prefix_len rows in the pages
    prefix_table (int32) of the same pool, which stay as they are. state [n_slots,H,d,d] fp32 (and
    g_state [n_slots,H] with the gate) holds each slot's product of Householder factors (sum of
    log_f) since the prefix ended, updated in place; path_state_copy starts a slot."""
    return _step_paged("path_decode_step_shared", q, k_new, v_new, w, beta, k_pages, v_pages, table,
                       lens, rows, scale, log_f, g_pages, out, workspace,
                       (prefix_table, prefix_len, state, g_state))


def path_pages_reserve(table, held, owner, page, rows, tokens, info=None):
    """Gives slot rows[i] the free pages it lacks to hold tokens[i] rows, or changes nothing and
    reports PATH_ERR_PAGE. Returns info [4] int32 on the device: status, moves, pages in use,
    pages given."""
    n_slots, max_pages = _expect_table(table, held=held)
    n_pages, n = _expect_owner(owner), _expect_list(rows=rows, tokens=tokens)
    info = _info(info, table.device)
    _check_here(table, held, owner, rows, tokens, info)
    st = lib().path_pages_reserve(_ptr(table), _ptr(held), _ptr(owner), n_slots, max_pages, n_pages,
                                  int(page), _ptr(rows), _ptr(tokens), n, _ptr(info), _stream())
    if st:
        raise PathError(st, "path_pages_reserve")
    return info


def path_pages_fork(table, held, lens, owner, page, parents, children, moves=None, info=None):
    """Gives each child, a slot without pages, pages for its parent's rows and the parent's length
    (negative parent: an empty child), and lists the pages to copy. Returns (moves [max_moves,2],
    info [4]) on the device, for path_pages_copy on each layer's pool."""
    n_slots, max_pages = _expect_table(table, held=held, lens=lens)
    n_pages, n = _expect_owner(owner), _expect_list(parents=parents, children=children)
    moves, most = _moves(moves, min(n * max_pages, n_pages), table.device)
    info = _info(info, table.device)
    _check_here(table, held, lens, owner, parents, children, moves, info)
    st = lib().path_pages_fork(_ptr(table), _ptr(held), _ptr(lens), _ptr(owner), n_slots, max_pages,
                               n_pages, int(page), _ptr(parents), _ptr(children), n, _ptr(moves),
                               most, _ptr(info), _stream())
    if st:
        raise PathError(st, "path_pages_fork")
    return moves, info


def path_pages_free(table, held, lens, owner, rows):
    """Frees the slots' pages: their entries and owners become -1, held and lens 0."""
    n_slots, max_pages = _expect_table(table, held=held, lens=lens)
    n_pages, n = _expect_owner(owner), _expect_list(rows=rows)
    _check_here(table, held, lens, owner, rows)
    st = lib().path_pages_free(_ptr(table), _ptr(held), _ptr(lens), _ptr(owner), n_slots, max_pages,
                               n_pages, _ptr(rows), n, _stream())
    if st:
        raise PathError(st, "path_pages_free")


def path_pages_compact(table, held, owner, moves=None, info=None):
    """Renumbers the pages in use to the front of the pool. Returns (moves, info) as
    path_pages_fork, for path_pages_copy on each layer's pool."""
    n_slots, max_pages = _expect_table(table, held=held)
    n_pages = _expect_owner(owner)
    moves, most = _moves(moves, n_pages // 2, table.device)
    info = _info(info, table.device)
    _check_here(table, held, owner, moves, info)
    st = lib().path_pages_compact(_ptr(table), _ptr(held), _ptr(owner), n_slots, max_pages, n_pages,
                                  _ptr(moves), most, _ptr(info), _stream())
    if st:
        raise PathError(st, "path_pages_compact")
    return moves, info


def path_pages_copy(moves, info, k_pages, v_pages, g_pages=None):
    """Copies the pages that path_pages_fork or path_pages_compact listed in one layer's pool."""
    n_pages, H, page, d = _expect_pool(k_pages, v_pages, g_pages)
    moves, most = _moves(moves, 0, k_pages.device)
    _expect("info", info, (4,), torch.int32)
    _check_here(moves, info, k_pages, v_pages, g_pages)
    st = lib().path_pages_copy(_ptr(moves), most, _ptr(info), _ptr(k_pages), _ptr(v_pages),
                               _ptr(g_pages), n_pages, H, page, d, _DT[k_pages.dtype], _stream())
    if st:
        raise PathError(st, "path_pages_copy")


def path_pages_store(k_cache, v_cache, k_pages, v_pages, table, rows, tokens, g_cache=None,
                     g_pages=None, info=None):
    """Writes rows 0..tokens[b]-1 of the contiguous caches [B,H,capacity,d] (path_attn_prefill's)
    into the pages of slot rows[b] (None: b), as they are: a prefill of padded rows needs beta = 0
    and log_f = 0 behind tokens[b]. info [4] int32, if given, reports PATH_ERR_PAGE in
    info[0]."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [B,H,capacity,d]")
    n_pages, H, page, d = _expect_pool(k_pages, v_pages, g_pages)
    if (g_cache is None) != (g_pages is None):
        raise ValueError("g_cache and g_pages go together")
    B, _, capacity, _ = k_cache.shape
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _expect(n, t, (B, H, capacity, d), k_pages.dtype)
    _expect("g_cache", g_cache, (B, H, capacity), torch.float32)
    n_slots, max_pages = _expect_table(table)
    _expect("rows", rows, (B,), torch.int32)
    _expect("tokens", tokens, (B,), torch.int32)
    _expect("info", info, (4,), torch.int32)
    _check_here(k_cache, v_cache, g_cache, k_pages, v_pages, g_pages, table, rows, tokens, info)
    st = lib().path_pages_store(_ptr(k_cache), _ptr(v_cache), _ptr(g_cache), B, H, d, capacity,
                                _DT[k_pages.dtype], _ptr(k_pages), _ptr(v_pages), _ptr(g_pages),
                                n_pages, page, _ptr(table), n_slots, max_pages, _ptr(rows),
                                _ptr(tokens), _ptr(info), _stream())
    if st:
        raise PathError(st, "path_pages_store")


def path_state_copy(state, parents, children, g_state=None):
    """state [n_slots,H,d,d] (and g_state [n_slots,H]) of slot parents[i] into slot children[i];
    a negative parent stands for the prefix's end (identity, 0)."""
    if state.dim() != 4:
        raise ValueError("state must be [n_slots,H,d,d]")
    n_slots, H, d, _ = state.shape
    _expect("state", state, (n_slots, H, d, d), torch.float32)
    _expect("g_state", g_state, (n_slots, H), torch.float32)
    n = _expect_list(parents=parents, children=children)
    _check_here(state, g_state, parents, children)
    st = lib().path_state_copy(_ptr(state), _ptr(g_state), n_slots, H, d, _ptr(parents),
                               _ptr(children), n, _stream())
    if st:
        raise PathError(st, "path_state_copy")


# ---------------------------------------------------------------- the w / beta prologue
def path_wbeta_workspace_bytes(B, L, D, r, H, d, dtype, for_bwd=False, out_dtype=None) -> int:
    mode = _mode(dtype, out_dtype or dtype)
    return int(lib().path_wbeta_workspace_bytes(B, L, D, r, H, d, mode, int(bool(for_bwd))))


def _check_wbeta(x, A, Bw, f, U, b, H):
    if x.dim() != 3 or x.dtype not in _DT:
        raise ValueError("x must be [B,L,D], float32 or bfloat16")
    B, L, D = x.shape
    if A.dim() != 2 or A.shape[0] != D:
        raise ValueError(f"A: shape {tuple(A.shape)}, expected ({D}, r)")
    r = A.shape[1]
    if Bw.dim() != 2 or Bw.shape[0] != r or Bw.shape[1] % H:
        raise ValueError(f"Bw: shape {tuple(Bw.shape)}, expected ({r}, H*d) with H={H}")
    d = Bw.shape[1] // H
    _expect("A", A, (D, r), x.dtype)
    _expect("Bw", Bw, (r, H * d), x.dtype)
    _expect("U", U, (D, H), x.dtype)
    _expect("f", f, (H * d, 3), torch.float32)
    _expect("b", b, (H,), torch.float32)
    return B, L, D, r, d


def path_wbeta_fwd(x, A, Bw, f, U, b, H, beta_max=2.0, w=None, beta=None, workspace=None,
                   out_dtype=None):
    """w [B,H,L,d] (out_dtype, default x's dtype) and beta [B,H,L] fp32 from x [B,L,D]:
    w = per-head L2 normalisation of the 3-tap causal convolution (filter f [H*d,3]) of
    (x A) Bw; beta = min(2 sigmoid(x U + b), beta_max)."""
    B, L, D, r, d = _check_wbeta(x, A, Bw, f, U, b, H)
    od = out_dtype or x.dtype
    if w is None:
        w = torch.empty((B, H, L, d), dtype=od, device=x.device)
    if beta is None:
        beta = torch.empty((B, H, L), dtype=torch.float32, device=x.device)
    _expect("w", w, (B, H, L, d), od)
    _expect("beta", beta, (B, H, L), torch.float32)
    mode = _mode(x.dtype, od)
    _check_dev(x, A, Bw, f, U, b, w, beta, workspace)
    nbytes = path_wbeta_workspace_bytes(B, L, D, r, H, d, x.dtype, False, od)
    ws = _workspace(nbytes, x.device, workspace)
    st = lib().path_wbeta_fwd(_ptr(x), _ptr(A), _ptr(Bw), _ptr(f), _ptr(U), _ptr(b), float(beta_max),
                              B, L, D, r, H, d, mode, _ptr(w), _ptr(beta), _ptr(ws), nbytes,
                              _stream())
    if st:
        raise PathError(st, "path_wbeta_fwd")
    return w, beta


def path_wbeta_bwd(x, A, Bw, f, U, b, H, dw, dbeta, beta_max=2.0, grads=None, workspace=None,
                   reuse_fwd_workspace=False):
    """Gradients of sum(w * dw) + sum(beta * dbeta): dict dx (dw's dtype), dA, dBw, df, dU,
    db (fp32)."""
    if reuse_fwd_workspace and workspace is None:
        raise ValueError("reuse_fwd_workspace needs the forward's workspace")
    B, L, D, r, d = _check_wbeta(x, A, Bw, f, U, b, H)
    od = dw.dtype
    _expect("dw", dw, (B, H, L, d), od)
    _expect("dbeta", dbeta, (B, H, L), torch.float32)
    if grads is None:
        dev = x.device
        grads = dict(dx=torch.empty((B, L, D), dtype=od, device=dev),
                     dA=torch.empty((D, r), dtype=torch.float32, device=dev),
                     dBw=torch.empty((r, H * d), dtype=torch.float32, device=dev),
                     df=torch.empty((H * d, 3), dtype=torch.float32, device=dev),
                     dU=torch.empty((D, H), dtype=torch.float32, device=dev),
                     db=torch.empty((H,), dtype=torch.float32, device=dev))
    _expect("dx", grads["dx"], (B, L, D), od)
    for n, shp in (("dA", (D, r)), ("dBw", (r, H * d)), ("df", (H * d, 3)), ("dU", (D, H)),
                   ("db", (H,))):
        _expect(n, grads[n], shp, torch.float32)
    mode = _mode(x.dtype, od)
    _check_dev(x, A, Bw, f, U, b, dw, dbeta, workspace, *grads.values())
    nbytes = path_wbeta_workspace_bytes(B, L, D, r, H, d, x.dtype, True, od)
    ws = _workspace(nbytes, x.device, workspace)
    st = lib().path_wbeta_bwd(_ptr(x), _ptr(A), _ptr(Bw), _ptr(f), _ptr(U), _ptr(b), float(beta_max),
                              B, L, D, r, H, d, mode, _ptr(dw), _ptr(dbeta), _ptr(grads["dx"]),
                              _ptr(grads["dA"]), _ptr(grads["dBw"]), _ptr(grads["df"]),
                              _ptr(grads["dU"]), _ptr(grads["db"]),
                              PATH_BWD_REUSE_FWD_WORKSPACE if reuse_fwd_workspace else 0, _ptr(ws),
                              nbytes, _stream())
    if st:
        raise PathError(st, "path_wbeta_bwd")
    return grads
