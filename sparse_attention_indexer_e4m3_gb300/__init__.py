"""GB300-native FP8 lightning indexer and exact top-k selector.

Python binding of the C ABI in ``include/dsa.h`` (library ``libdsa_gb300.so``, built in-tree by
``sparse_attention_indexer_e4m3_gb300.build``; the 4-bit cache's calls marshal natively, ``_marshal.so``).  This module only marshals arguments: it checks
torch tensors, passes their device pointers and the current CUDA stream, and raises
``DsaError`` on a non-OK status.  Every step of the computation runs in the library's kernels;
there is no fallback path.  If the library has not been built, every call raises.

    score[t, j] = k_scale[j] * sum_h relu(q[t, h] . k[j]) * w[t, h],   ks[t] <= j < ke[t]
    idx[t]      = the topk keys of largest score in the window, ascending, -1 padded
"""
from __future__ import annotations

import ctypes
import importlib
import os
import threading

__all__ = [
    "DsaError", "library_path", "load", "index_score", "index_score_kres", "index_score_kres_workspace_size", "topk",
    "index_topk", "index_topk_plan", "index_topk_run", "topk_workspace_size",
    "index_topk_workspace_size", "get_device_error", "status_string", "version", "MAX_TOPK", "SUPPORTED_H",
    "SUPPORTED_D", "kv4_page_bytes", "quantize_kv4", "dequantize_kv4", "sparse_attn_kv4", "sparse_attn_kv4_workspace_size", "fork_pages", "reserve_pages",
    "reserve_pages_workspace_size", "compact_pages", "compact_pages_workspace_size", "copy_pages", "SUPPORTED_KV4_D",
]

MAX_TOPK = 2048
SUPPORTED_H = (4, 8, 16, 32, 64)
SUPPORTED_D = (64, 128)
SUPPORTED_KV4_D = (64, 128, 256, 512)

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libdsa_gb300.so"
_lib = None
_lock = threading.Lock()

DSA_OK = 0
_STATUS = {0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED", 3: "DSA_ERR_WORKSPACE",
           4: "DSA_ERR_CUDA", 5: "DSA_ERR_TIMEOUT"}


class DsaError(RuntimeError):
    """A non-OK status returned by the C ABI."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)}")


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def load():
    """Load libdsa_gb300.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with "
                                   "`python -m sparse_attention_indexer_e4m3_gb300.build`")
            lib = ctypes.CDLL(path)
            p, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            lib.dsa_index_score.argtypes = [p, p, p, p, p, p, i, i, i, i, p, p]
            lib.dsa_index_score.restype = i
            lib.dsa_index_score_kres_workspace_size.argtypes = [i, i, i, i]
            lib.dsa_index_score_kres_workspace_size.restype = sz
            lib.dsa_index_score_kres.argtypes = [p, p, p, p, p, p, i, i, i, i, p, p, sz, p]
            lib.dsa_index_score_kres.restype = i
            lib.dsa_topk_workspace_size.argtypes = [i, i, i]
            lib.dsa_topk_workspace_size.restype = sz
            lib.dsa_topk.argtypes = [p, p, p, i, i, i, p, p, sz, p]
            lib.dsa_topk.restype = i
            lib.dsa_index_topk_workspace_size.argtypes = [i, i, i, i, i]
            lib.dsa_index_topk_workspace_size.restype = sz
            lib.dsa_index_topk.argtypes = [p, p, p, p, p, p, i, i, i, i, i, p, p, sz, p]
            lib.dsa_index_topk.restype = i
            lib.dsa_index_topk_plan.argtypes = [p, p, i, i, i, i, i, p, sz, p]
            lib.dsa_index_topk_plan.restype = i
            lib.dsa_index_topk_run.argtypes = [p, p, p, p, p, p, i, i, i, i, i, p, p, sz, p]
            lib.dsa_index_topk_run.restype = i
            lib.dsa_get_device_error.argtypes = [p]
            lib.dsa_get_device_error.restype = i
            lib.dsa_quantize_k.argtypes = [p, i, i, p, p, p]
            lib.dsa_quantize_k.restype = i
            lib.dsa_sparse_attn.argtypes = [p, p, p, p, i, i, i, i, i, ctypes.c_float, p, p, p]
            lib.dsa_sparse_attn_bwd.argtypes = [p, p, p, p, p, p, p, i, i, i, i, i, ctypes.c_float, p, p, p, p]
            lib.dsa_sparse_attn_bwd.restype = i
            lib.dsa_sparse_attn.restype = i
            lib.dsa_kv4_page_bytes.argtypes = [i, i]
            lib.dsa_kv4_page_bytes.restype = sz
            lib.dsa_sparse_attn_kv4_workspace_size.argtypes = [i, i, i, i]
            lib.dsa_sparse_attn_kv4_workspace_size.restype = sz
            lib.dsa_reserve_pages_workspace_size.argtypes = [i]
            lib.dsa_reserve_pages_workspace_size.restype = sz
            lib.dsa_compact_pages_workspace_size.argtypes = [i]
            lib.dsa_compact_pages_workspace_size.restype = sz
            lib.dsa_check_bounded_wait.argtypes = [p, p]
            lib.dsa_check_bounded_wait.restype = i
            lib.dsa_status_string.argtypes = [i]
            lib.dsa_status_string.restype = ctypes.c_char_p
            lib.dsa_version.argtypes = []
            lib.dsa_version.restype = i
            _lib = lib
    return _lib


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _stream_ptr(stream) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    c = _torch()._C  # the current stream's handle, without a Stream object around it
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


def _dev(t, name, dtypes):
    torch = _torch()
    try:
        if t.dtype in dtypes and t.is_cuda and t.is_contiguous():
            return t
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _shape(t, name, shape):
    """Raise unless tensor t has exactly this shape (caller buffers are never written past)."""
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _empty(shape, dtype, device, stream):
    """A new tensor for a call on `stream`, allocated for that stream: memory of the current stream's pool may still be in
    use there by what held it last.  It is not used anew before the current stream is done with it either."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    here, handle = torch.cuda.current_stream(device), int(stream.cuda_stream)
    # (an ExternalStream of handle 0 would be some other stream, not the default one)
    there = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(there):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def _check(status: int, where: str):
    if status != DSA_OK:
        raise DsaError(status, where)


def status_string(status: int) -> str:
    return load().dsa_status_string(status).decode()


def version() -> int:
    return load().dsa_version()


def _inputs(q, w, k, k_scale, ks, ke):
    torch = _torch()
    q = _dev(q, "q", (torch.uint8,))
    k = _dev(k, "k", (torch.uint8,))
    w = _dev(w, "w", (torch.float32,))
    k_scale = _dev(k_scale, "k_scale", (torch.float32,))
    ks = _dev(ks, "ks", (torch.int32,))
    ke = _dev(ke, "ke", (torch.int32,))
    if q.dim() != 3 or k.dim() != 2:
        raise ValueError("q must be [T, H, D] and k must be [N, D]")
    T, H, D = q.shape
    N = k.shape[0]
    if k.shape[1] != D or tuple(w.shape) != (T, H) or tuple(k_scale.shape) != (N,):
        raise ValueError("shape mismatch among q [T,H,D], w [T,H], k [N,D], k_scale [N]")
    if tuple(ks.shape) != (T,) or tuple(ke.shape) != (T,):
        raise ValueError("ks and ke must be [T]")
    return q, w, k, k_scale, ks, ke, T, N, H, D


def index_score(q, w, k, k_scale, ks, ke, logits=None, stream=None):
    """fp32 logits [T, N]; only in-window entries are written (others keep their value)."""
    torch = _torch()
    q, w, k, k_scale, ks, ke, T, N, H, D = _inputs(q, w, k, k_scale, ks, ke)
    if logits is None:
        logits = _empty((T, N), torch.float32, q.device, stream)
    logits = _dev(logits, "logits", (torch.float32,))
    if tuple(logits.shape) != (T, N):
        raise ValueError("logits must be [T, N]")
    st = load().dsa_index_score(q.data_ptr(), w.data_ptr(), k.data_ptr(), k_scale.data_ptr(), ks.data_ptr(),
                                ke.data_ptr(), T, N, H, D, logits.data_ptr(), _stream_ptr(stream))
    _check(st, "dsa_index_score")
    return logits


def index_score_kres_workspace_size(T: int, N: int, H: int, D: int) -> int:
    return int(load().dsa_index_score_kres_workspace_size(T, N, H, D))


def index_score_kres(q, w, k, k_scale, ks, ke, logits=None, workspace=None, stream=None):
    """index_score with the key tile resident and the query blocks streamed (same scores, same
    output contract); w must be 16-byte aligned."""
    torch = _torch()
    q, w, k, k_scale, ks, ke, T, N, H, D = _inputs(q, w, k, k_scale, ks, ke)
    if logits is None:
        logits = _empty((T, N), torch.float32, q.device, stream)
    logits = _dev(logits, "logits", (torch.float32,))
    if tuple(logits.shape) != (T, N):
        raise ValueError("logits must be [T, N]")
    need = index_score_kres_workspace_size(T, N, H, D)
    ws, nbytes = _workspace(need, _scratch(need, workspace, q.device, stream), q.device)
    st = load().dsa_index_score_kres(q.data_ptr(), w.data_ptr(), k.data_ptr(), k_scale.data_ptr(), ks.data_ptr(),
                                     ke.data_ptr(), T, N, H, D, logits.data_ptr(),
                                     ws.data_ptr() if ws is not None else None, nbytes, _stream_ptr(stream))
    _check(st, "dsa_index_score_kres")
    return logits


def topk_workspace_size(T: int, N: int, k: int) -> int:
    return int(load().dsa_topk_workspace_size(T, N, k))


def index_topk_workspace_size(T: int, N: int, H: int, D: int, k: int) -> int:
    return int(load().dsa_index_topk_workspace_size(T, N, H, D, k))


def _scratch(nbytes, workspace, device, stream):
    """The caller's workspace, or one for a call on another stream (none here for the current one: _workspace's)."""
    if workspace is not None or stream is None or nbytes == 0:
        return workspace
    return _empty(nbytes, _torch().uint8, device, stream)


def _workspace(nbytes, workspace, device):
    torch = _torch()
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    workspace = _dev(workspace, "workspace", (torch.uint8,))
    return workspace, workspace.numel()


def topk(logits, ks, ke, k: int, idx=None, workspace=None, stream=None):
    """int32 [T, k] top-k key indices per row of logits [T, N], ascending, -1 padded."""
    torch = _torch()
    logits = _dev(logits, "logits", (torch.float32,))
    ks = _dev(ks, "ks", (torch.int32,))
    ke = _dev(ke, "ke", (torch.int32,))
    if logits.dim() != 2:
        raise ValueError("logits must be [T, N]")
    T, N = logits.shape
    _shape(ks, "ks", (T,))
    _shape(ke, "ke", (T,))
    if idx is None:
        idx = _empty((T, k), torch.int32, logits.device, stream)
    idx = _dev(idx, "idx", (torch.int32,))
    _shape(idx, "idx", (T, k))
    need = topk_workspace_size(T, N, k)
    ws, wsb = _workspace(need, _scratch(need, workspace, logits.device, stream), logits.device)
    st = load().dsa_topk(logits.data_ptr(), ks.data_ptr(), ke.data_ptr(), T, N, k, idx.data_ptr(),
                         None if ws is None else ws.data_ptr(), wsb, _stream_ptr(stream))
    _check(st, "dsa_topk")
    return idx


def index_topk(q, w, k, k_scale, ks, ke, topk_k: int, idx=None, workspace=None, stream=None):
    """Fused scorer + selector: int32 [T, topk_k] without materialising the [T, N] logits."""
    torch = _torch()
    q, w, k, k_scale, ks, ke, T, N, H, D = _inputs(q, w, k, k_scale, ks, ke)
    if idx is None:
        idx = _empty((T, topk_k), torch.int32, q.device, stream)
    idx = _dev(idx, "idx", (torch.int32,))
    _shape(idx, "idx", (T, topk_k))
    need = index_topk_workspace_size(T, N, H, D, topk_k)
    ws, wsb = _workspace(need, _scratch(need, workspace, q.device, stream), q.device)
    st = load().dsa_index_topk(q.data_ptr(), w.data_ptr(), k.data_ptr(), k_scale.data_ptr(), ks.data_ptr(),
                               ke.data_ptr(), T, N, H, D, topk_k, idx.data_ptr(),
                               None if ws is None else ws.data_ptr(), wsb, _stream_ptr(stream))
    _check(st, "dsa_index_topk")
    return idx


def index_topk_plan(ks, ke, N: int, H: int, D: int, topk_k: int, workspace=None, stream=None):
    """Plan the fused path for windows ks / ke; returns the workspace holding the plan."""
    torch = _torch()
    ks = _dev(ks, "ks", (torch.int32,))
    ke = _dev(ke, "ke", (torch.int32,))
    if ks.dim() != 1:
        raise ValueError("ks must be [T]")
    T = ks.shape[0]
    _shape(ke, "ke", (T,))
    need = index_topk_workspace_size(T, N, H, D, topk_k)
    ws, wsb = _workspace(need, _scratch(need, workspace, ks.device, stream), ks.device)
    st = load().dsa_index_topk_plan(ks.data_ptr(), ke.data_ptr(), T, N, H, D, topk_k,
                                    None if ws is None else ws.data_ptr(), wsb, _stream_ptr(stream))
    _check(st, "dsa_index_topk_plan")
    return ws


def index_topk_run(q, w, k, k_scale, ks, ke, topk_k: int, workspace, idx=None, stream=None):
    """Run the fused path with a plan made by index_topk_plan for the same ks / ke / shapes."""
    torch = _torch()
    q, w, k, k_scale, ks, ke, T, N, H, D = _inputs(q, w, k, k_scale, ks, ke)
    if idx is None:
        idx = _empty((T, topk_k), torch.int32, q.device, stream)
    idx = _dev(idx, "idx", (torch.int32,))
    _shape(idx, "idx", (T, topk_k))
    ws = None if workspace is None else _dev(workspace, "workspace", (torch.uint8,))
    st = load().dsa_index_topk_run(q.data_ptr(), w.data_ptr(), k.data_ptr(), k_scale.data_ptr(), ks.data_ptr(),
                                   ke.data_ptr(), T, N, H, D, topk_k, idx.data_ptr(),
                                   None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(),
                                   _stream_ptr(stream))
    _check(st, "dsa_index_topk_run")
    return idx


def get_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status."""
    return int(load().dsa_get_device_error(_stream_ptr(stream)))


def quantize_k(k, codes=None, scale=None, stream=None):
    """e4m3 quantise-on-write of key rows: bf16 [N, D] -> (uint8 codes [N, D], fp32 scales [N])."""
    torch = _torch()
    k = _dev(k, "k", (torch.bfloat16,))
    if k.dim() != 2:
        raise ValueError("k must be [N, D]")
    N, D = k.shape
    if codes is None:
        codes = _empty((N, D), torch.uint8, k.device, stream)
    if scale is None:
        scale = _empty(N, torch.float32, k.device, stream)
    codes = _dev(codes, "codes", (torch.uint8,))
    scale = _dev(scale, "scale", (torch.float32,))
    _shape(codes, "codes", (N, D))
    _shape(scale, "scale", (N,))
    _check(load().dsa_quantize_k(k.data_ptr(), N, D, codes.data_ptr(), scale.data_ptr(), _stream_ptr(stream)),
           "dsa_quantize_k")
    return codes, scale


def sparse_attn(q, kv, idx, attn_sink=None, scale=None, out=None, lse=None, stream=None):
    """Attention of each query row over its selected keys: q bf16 [T, H, D], kv bf16 [N, D]
    (keys = values), idx int32 [T, K] (-1 = none), attn_sink fp32 [H] or None, scale default
    1 / sqrt(D).  Returns bf16 [T, H, D]; with lse (fp32 [T, H]) given, also writes the natural
    log of each softmax denominator into it (what sparse_attn_bwd takes)."""
    torch = _torch()
    q = _dev(q, "q", (torch.bfloat16,))
    kv = _dev(kv, "kv", (torch.bfloat16,))
    idx = _dev(idx, "idx", (torch.int32,))
    if q.dim() != 3 or kv.dim() != 2 or idx.dim() != 2:
        raise ValueError("shapes: q [T, H, D], kv [N, D], idx [T, K]")
    T, H, D = q.shape
    N = kv.shape[0]
    if kv.shape[1] != D or idx.shape[0] != T:
        raise ValueError("shapes: q [T, H, D], kv [N, D], idx [T, K]")
    sink_ptr = None
    if attn_sink is not None:
        attn_sink = _dev(attn_sink, "attn_sink", (torch.float32,))
        if attn_sink.shape != (H,):
            raise ValueError("attn_sink must be [H]")
        sink_ptr = attn_sink.data_ptr()
    if out is None:
        out = _empty((T, H, D), torch.bfloat16, q.device, stream)
    out = _dev(out, "out", (torch.bfloat16,))
    _shape(out, "out", (T, H, D))
    lse_ptr = None
    if lse is not None:
        lse = _dev(lse, "lse", (torch.float32,))
        _shape(lse, "lse", (T, H))
        lse_ptr = lse.data_ptr()
    sc = float(scale) if scale is not None else 1.0 / float(D) ** 0.5
    _check(load().dsa_sparse_attn(q.data_ptr(), kv.data_ptr(), sink_ptr, idx.data_ptr(), T, N, H, D, idx.shape[1],
                                  sc, out.data_ptr(), lse_ptr, _stream_ptr(stream)), "dsa_sparse_attn")
    return out


def sparse_attn_bwd(q, kv, idx, out, lse, dout, attn_sink=None, scale=None, dq=None, dkv=None, dsink=None,
                    stream=None):
    """Gradients of sparse_attn for the loss sum(dout * out): returns (dq fp32 [T, H, D], dkv fp32
    [N, D], dsink fp32 [H] or None).  out and lse are the forward's outputs (bf16 [T, H, D] and
    fp32 [T, H]), dout bf16 [T, H, D]; the other arguments as passed to sparse_attn."""
    torch = _torch()
    q = _dev(q, "q", (torch.bfloat16,))
    kv = _dev(kv, "kv", (torch.bfloat16,))
    idx = _dev(idx, "idx", (torch.int32,))
    if q.dim() != 3 or kv.dim() != 2 or idx.dim() != 2:
        raise ValueError("shapes: q [T, H, D], kv [N, D], idx [T, K]")
    T, H, D = q.shape
    N = kv.shape[0]
    if kv.shape[1] != D or idx.shape[0] != T:
        raise ValueError("shapes: q [T, H, D], kv [N, D], idx [T, K]")
    out = _dev(out, "out", (torch.bfloat16,))
    _shape(out, "out", (T, H, D))
    dout = _dev(dout, "dout", (torch.bfloat16,))
    _shape(dout, "dout", (T, H, D))
    lse = _dev(lse, "lse", (torch.float32,))
    _shape(lse, "lse", (T, H))
    sink_ptr = None
    if attn_sink is not None:
        attn_sink = _dev(attn_sink, "attn_sink", (torch.float32,))
        if attn_sink.shape != (H,):
            raise ValueError("attn_sink must be [H]")
        sink_ptr = attn_sink.data_ptr()
        if dsink is None:
            dsink = _empty(H, torch.float32, q.device, stream)
    if dq is None:
        dq = _empty((T, H, D), torch.float32, q.device, stream)
    if dkv is None:
        dkv = _empty((N, D), torch.float32, q.device, stream)
    dq = _dev(dq, "dq", (torch.float32,))
    _shape(dq, "dq", (T, H, D))
    dkv = _dev(dkv, "dkv", (torch.float32,))
    _shape(dkv, "dkv", (N, D))
    dsink_ptr = None
    if dsink is not None:
        dsink = _dev(dsink, "dsink", (torch.float32,))
        _shape(dsink, "dsink", (H,))
        dsink_ptr = dsink.data_ptr()
    sc = float(scale) if scale is not None else 1.0 / float(D) ** 0.5
    _check(load().dsa_sparse_attn_bwd(q.data_ptr(), kv.data_ptr(), sink_ptr, idx.data_ptr(), out.data_ptr(),
                                      lse.data_ptr(), dout.data_ptr(), T, N, H, D, idx.shape[1], sc, dq.data_ptr(),
                                      dkv.data_ptr(), dsink_ptr, _stream_ptr(stream)), "dsa_sparse_attn_bwd")
    return dq, dkv, (dsink if attn_sink is not None else None)


# ------------------------------------------------------------------ the 4-bit paged kv cache


def kv4_page_bytes(page_rows: int, D: int) -> int:
    """Bytes of a page of page_rows held rows of D values (0 for an unsupported page_rows or D)."""
    return int(load().dsa_kv4_page_bytes(page_rows, D))


_calls = None  # the module _marshal, once loaded and bound


def _native():
    """The native argument marshalling of the calls below, bound to the loaded library."""
    global _calls
    if _calls is None:
        lib, torch = load(), _torch()
        path = os.path.join(_HERE, "_marshal.so")
        how = "build it with `python -m sparse_attention_indexer_e4m3_gb300.build`"
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: {how}")
        try:
            m = importlib.import_module(__name__ + "._marshal")
        except ImportError as e:
            raise RuntimeError(f"{path} does not load, as if built for another torch or Python ({e}): {how}") from e
        if m.torch_version != torch.__version__.split("+")[0]:
            raise RuntimeError(f"{path} was built for torch {m.torch_version}, not {torch.__version__}: {how}")
        names = ("quantize_kv4_reserved", "dequantize_kv4", "sparse_attn_kv4", "sparse_attn_kv4_workspace_size", "fork_pages", "reserve_pages",
                 "reserve_pages_workspace_size", "compact_pages", "compact_pages_workspace_size", "copy_pages")
        m.bind(tuple(ctypes.cast(getattr(lib, "dsa_" + n), ctypes.c_void_p).value for n in names), DsaError)
        _calls = m
    return _calls


def quantize_kv4(kv, cache, table, seq, pos, stream=None, lacking=None):
    """Write bf16 rows kv [N, D] in 4 bits into the paged cache (uint8 [P, kv4_page_bytes]): row i as
    row pos[i] of sequence seq[i], whose pages are table[seq[i]] (int32 [R, M], -1 = none); rows
    whose place is not mapped are left out.  With lacking (int32 [1], from reserve_pages for these rows) nothing
    is written where it is not 0: the rows' pages may then still be shared.  Returns cache."""
    return (_calls or _native()).quantize_kv4(kv, cache, table, seq, pos, stream, lacking)


def dequantize_kv4(cache, table, seq, pos, D: int, out=None, stream=None):
    """Rows pos[i] of sequences seq[i] of the 4-bit paged cache as bf16 [N, D] (zeros where no page is
    mapped)."""
    return (_calls or _native()).dequantize_kv4(cache, table, seq, pos, D, out, stream)


def sparse_attn_kv4_workspace_size(T: int, H: int, D: int, K: int) -> int:
    return int(load().dsa_sparse_attn_kv4_workspace_size(T, H, D, K))


def sparse_attn_kv4(q, cache, table, seq, idx, start=None, attn_sink=None, scale=None, out=None, lse=None, workspace=None,
                    stream=None):
    """sparse_attn over the 4-bit paged cache: q bf16 [T, H, D]; idx int32 [T, K], entry v of token t
    naming row v - start[t] of sequence seq[t] (start int32 [T], default 0; negative or unmapped entries
    are skipped); attn_sink fp32 [H] or None, scale default 1 / sqrt(D).  Returns bf16 [T, H, D]; with
    lse (fp32 [T, H]) given, also writes the natural log of each softmax denominator into it."""
    return (_calls or _native()).sparse_attn_kv4(q, cache, table, seq, idx, start, attn_sink, scale, out, lse, workspace,
                                                 stream)


def fork_pages(table, parent, ref, table_out=None, stream=None):
    """New page table (int32 [R, M]) whose row r is table[parent[r]] (-1: the row is freed); the page
    counts ref (int32 [P]) follow in place.  table_out must not overlap table."""
    return (_calls or _native()).fork_pages(table, parent, ref, table_out, stream)


def reserve_pages_workspace_size(P: int) -> int:
    return int(load().dsa_reserve_pages_workspace_size(P))


def reserve_pages(table, ref, begin, end, page_rows: int, src=None, dst=None, lacking=None, workspace=None, stream=None):
    """Before rows [begin[r], end[r]) of each sequence are written: maps every page they cover and gives
    the sequence a page of its own where one is shared (table and ref in place).  Returns (src, dst, lacking):
    copy_pages(cache, src, dst) brings along what the replaced pages hold (int32 [2 R], -1 = none), and
    lacking (int32 [1]) is 0 or by how many pages the pool falls short (then nothing changed, and the rows
    must not be written: pass it on to quantize_kv4)."""
    return (_calls or _native()).reserve_pages(table, ref, begin, end, page_rows, src, dst, lacking, workspace, stream)


def compact_pages_workspace_size(P: int) -> int:
    return int(load().dsa_compact_pages_workspace_size(P))


def compact_pages(table, ref, src=None, dst=None, n_live=None, workspace=None, stream=None):
    """Rename the pages in use to the lowest ones (table and ref in place).  Returns (src, dst, n_live):
    copy_pages(cache, src, dst) moves the rows (int32 [P // 2], -1 = none); n_live (int32 [1]) pages are in use."""
    return (_calls or _native()).compact_pages(table, ref, src, dst, n_live, workspace, stream)


def copy_pages(pages, src, dst, stream=None):
    """pages[dst[i]] = pages[src[i]] in place for the entries whose two ids name pages (src, dst int32 [n]);
    pages is any contiguous tensor [P, ...] whose pages take a multiple of 16 bytes.  Returns pages."""
    return (_calls or _native()).copy_pages(pages, src, dst, stream)


def check_bounded_wait(stream=None):
    """Run the bounded-wait self-check; returns the device time (ns) of its expired wait and of
    the wait that returned on the abort flag.  The timeout it records is left for
    get_device_error()."""
    took = (ctypes.c_uint64 * 2)()
    _check(load().dsa_check_bounded_wait(ctypes.cast(took, ctypes.c_void_p), _stream_ptr(stream)), "dsa_check_bounded_wait")
    return int(took[0]), int(took[1])
