"""ctypes binding of the LSA C ABI (include/lsa.h).

Argument marshalling only: every step of the path runs in the CUDA kernels of
liblsa.so. The functions carry the C names and take torch CUDA tensors; outputs
and workspaces are allocated with torch when the caller does not pass them.
There is no CPU fallback: if the library is missing or a call fails, an
exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblsa.so")

LSA_OK, LSA_ERR_INVALID_ARG, LSA_ERR_UNSUPPORTED, LSA_ERR_WORKSPACE, LSA_ERR_CUDA, LSA_ERR_TIMEOUT = range(6)
LSA_BF16, LSA_E4M3, LSA_FP32 = 0, 1, 2
(LSA_OP_INDEX_FLAT, LSA_OP_INDEX_HIER, LSA_OP_SELECT, LSA_OP_SPARSE_ATTN, LSA_OP_LAYER_GROUP,
 LSA_OP_INDEX_COMPRESSED, LSA_OP_PAGED_ATTN, LSA_OP_PAGES_FORK, LSA_OP_PAGES_COPY, LSA_OP_PAGES_COMPACT) = range(10)
LSA_ROPE_SCALINGS = {"none": 0, "linear": 1, "yarn": 2}
LSA_ROPE_MAX_PAIRS = 128
LSA_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024   # static scratch of lsa_select_streaming_noalloc

EXPORTS = [
    "lsa_status_string", "lsa_last_error", "lsa_workspace_size", "lsa_index_flat", "lsa_select_streaming",
    "lsa_pool_pages", "lsa_index_hier", "lsa_sparse_attn", "lsa_layer_group", "lsa_device_status",
    "lsa_select_streaming_noalloc", "lsa_index_compressed", "lsa_pool_pages_e4m3", "lsa_index_hier_e4m3",
    "lsa_rope_plan", "lsa_rope", "lsa_pages_append", "lsa_paged_attn", "lsa_pages_reserve", "lsa_pages_fork",
    "lsa_pages_free", "lsa_pages_copy", "lsa_pages_compact",
]


class LsaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"[{status}] {msg}")
        self.status = status


class Budget(ctypes.Structure):
    _fields_ = [("k", ctypes.c_int32), ("sink", ctypes.c_int32), ("window", ctypes.c_int32)]


class IndexerIn(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("d", ctypes.c_int32),
                ("L_max", ctypes.c_int32), ("dtype", ctypes.c_int32), ("seq_len", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("q_scale", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p)]


class AttnIn(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("Hq", ctypes.c_int32), ("d_qk", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("L_max", ctypes.c_int32), ("scale", ctypes.c_float),
                ("seq_len", ctypes.c_void_p), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_row_stride", ctypes.c_int64), ("v_row_stride", ctypes.c_int64),
                ("stream_sink", ctypes.c_int32), ("stream_window", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("k_scale", ctypes.c_void_p)]


class RopePlan(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("amplitude", ctypes.c_double),
                ("freq", ctypes.c_double * LSA_ROPE_MAX_PAIRS)]


class RopeIn(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("B", "T", "H", "d", "dtype", "offset", "inverse")] + \
               [(f, ctypes.c_void_p) for f in ("seq_len", "q_len", "x")] + \
               [(f, ctypes.c_int64) for f in ("x_stride_b", "x_stride_t", "x_stride_h", "out_stride_b", "out_stride_t",
                                              "out_stride_h")]


class AppendIn(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("B", "T", "H", "d", "n_pages", "page_size", "max_pages", "dtype",
                                              "offset")] + \
               [(f, ctypes.c_void_p) for f in ("seq_len", "q_len", "table", "x", "pool")] + \
               [("page_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64), ("scales", ctypes.c_void_p)]


class PagedAttnIn(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("B", "T", "Hq", "Hkv", "d_qk", "d_v", "n_pages", "page_size",
                                              "max_pages")] + \
               [("scale", ctypes.c_float), ("kv_dtype", ctypes.c_int32)] + \
               [(f, ctypes.c_void_p) for f in ("seq_len", "q_len", "table", "q", "k", "v")] + \
               [(f, ctypes.c_int64) for f in ("k_page_stride", "k_row_stride", "v_page_stride", "v_row_stride")] + \
               [("k_scale", ctypes.c_void_p)]


class Pool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_int64), ("page_stride", ctypes.c_int64)]


class OpArgs(ctypes.Structure):
    _fields_ = [("indexer", ctypes.POINTER(IndexerIn)), ("attn", ctypes.POINTER(AttnIn)), ("budget", Budget),
                ("P", ctypes.c_int32), ("M", ctypes.c_int32), ("n_layers", ctypes.c_int32),
                ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("L_max", ctypes.c_int32),
                ("scores_external", ctypes.c_int32), ("m", ctypes.c_int32),
                ("paged", ctypes.POINTER(PagedAttnIn)), ("n", ctypes.c_int32), ("n_pages", ctypes.c_int32)]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load liblsa.so (built by kv_indexing_b200.build). Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m kv_indexing_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.lsa_status_string.restype = ctypes.c_char_p
    lib.lsa_status_string.argtypes = [i32]
    lib.lsa_last_error.restype = ctypes.c_char_p
    lib.lsa_last_error.argtypes = []
    lib.lsa_workspace_size.restype = i32
    lib.lsa_workspace_size.argtypes = [i32, ctypes.POINTER(OpArgs), ctypes.POINTER(sz)]
    lib.lsa_index_flat.restype = i32
    lib.lsa_index_flat.argtypes = [ctypes.POINTER(IndexerIn), Budget, vp, vp, vp, sz, vp]
    lib.lsa_index_compressed.restype = i32
    lib.lsa_index_compressed.argtypes = [ctypes.POINTER(IndexerIn), i32, Budget, vp, vp, vp, sz, vp]
    lib.lsa_select_streaming.restype = i32
    lib.lsa_select_streaming.argtypes = [vp, vp, i32, i32, i32, Budget, vp, vp, sz, vp]
    lib.lsa_select_streaming_noalloc.restype = i32
    lib.lsa_select_streaming_noalloc.argtypes = [vp, vp, i32, i32, i32, Budget, vp, vp]
    lib.lsa_pool_pages.restype = i32
    lib.lsa_pool_pages.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp]
    lib.lsa_pool_pages_e4m3.restype = i32
    lib.lsa_pool_pages_e4m3.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp]
    lib.lsa_index_hier_e4m3.restype = i32
    lib.lsa_index_hier_e4m3.argtypes = [ctypes.POINTER(IndexerIn), vp, vp, i32, i32, Budget, vp, vp, vp, sz, vp]
    lib.lsa_index_hier.restype = i32
    lib.lsa_index_hier.argtypes = [ctypes.POINTER(IndexerIn), vp, i32, i32, Budget, vp, vp, vp, sz, vp]
    lib.lsa_sparse_attn.restype = i32
    lib.lsa_sparse_attn.argtypes = [ctypes.POINTER(AttnIn), vp, i32, vp, vp, vp, sz, vp]
    lib.lsa_layer_group.restype = i32
    lib.lsa_layer_group.argtypes = [ctypes.POINTER(IndexerIn), vp, i32, i32, Budget, i32, ctypes.POINTER(AttnIn),
                                    ctypes.POINTER(vp), ctypes.POINTER(vp), vp, vp, sz, vp]
    f64, P = ctypes.c_double, ctypes.POINTER
    for name, args in (
            ("lsa_rope_plan", [i32, i32, f64, i32, f64, i32, f64, f64, f64, P(RopePlan)]),
            ("lsa_rope", [P(RopeIn), P(RopePlan), vp, vp]),
            ("lsa_pages_append", [P(AppendIn), P(RopePlan), vp]),
            ("lsa_paged_attn", [P(PagedAttnIn), vp, vp, vp, sz, vp]),
            ("lsa_pages_reserve", [vp, vp, vp, i32, i32, i32, i32, vp]),
            ("lsa_pages_fork", [vp, vp, vp, i32, i32, i32, i32, vp, vp, i32, P(Pool), i32, vp, sz, vp]),
            ("lsa_pages_free", [vp, vp, vp, i32, i32, i32, vp, i32, vp]),
            ("lsa_pages_copy", [P(Pool), i32, i32, vp, vp, i32, vp, sz, vp]),
            ("lsa_pages_compact", [vp, vp, i32, i32, i32, P(Pool), i32, vp, vp, vp, vp, sz, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = i32, args
    lib.lsa_device_status.restype = i32
    lib.lsa_device_status.argtypes = [vp]
    _lib = lib
    return lib


def _check(st: int):
    if st != LSA_OK:
        lib = load()
        raise LsaError(st, f"{lib.lsa_status_string(st).decode()}: {lib.lsa_last_error().decode()}")


# ---------------------------------------------------------------------------
# torch marshalling helpers
# ---------------------------------------------------------------------------


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        torch = _torch()
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _need(t, name, dtype=None, dim=None):
    torch = _torch()
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    cur = torch.cuda.current_device()
    if t.device.index != cur:   # the kernels launch on the current device and would read another GPU's memory
        raise ValueError(f"{name} is on {t.device}, but the calls launch on the current device cuda:{cur}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None:
        dts = dtype if isinstance(dtype, tuple) else (dtype,)
        if t.dtype not in dts:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dts}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dims")
    return t


def _dims(t, name, shape):
    """t's shape must equal `shape` (None = any size in that place)."""
    if len(t.shape) != len(shape) or any(want is not None and got != want for got, want in zip(t.shape, shape)):
        want = tuple("*" if n is None else n for n in shape)
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {want}")


def _out(t, name, dtype, shape):
    """A caller-supplied output (or None): a contiguous CUDA tensor on the current
    device with exactly the documented shape, since the kernels write all of it."""
    if t is None:
        return None
    _need(t, name, dtype, len(shape))
    _dims(t, name, shape)
    return t


def indexer_in(q, w, k, seq_len, q_scale=None, k_scale=None, m=1) -> IndexerIn:
    """Describe indexer tensors: q [B,T,H,d], w [B,T,H] f32, k [B,L_max,d], seq_len [B] i32.
    With m > 1, k holds one key per entry of m tokens: [B,L_max/m,d]."""
    torch = _torch()
    fp8 = q.dtype in (torch.float8_e4m3fn, torch.uint8)
    _need(q, "q", (torch.float8_e4m3fn, torch.uint8) if fp8 else torch.bfloat16, 4)
    _need(k, "k", (torch.float8_e4m3fn, torch.uint8) if fp8 else torch.bfloat16, 3)
    _need(w, "w", torch.float32, 3)
    _need(seq_len, "seq_len", torch.int32, 1)
    B, T, H, d = q.shape
    _dims(k, "k", (B, None, d))
    _dims(w, "w", (B, T, H))
    _dims(seq_len, "seq_len", (B,))
    if fp8:
        _need(q_scale, "q_scale", torch.float32, 3)
        _need(k_scale, "k_scale", torch.float32, 2)
        _dims(q_scale, "q_scale", (B, T, H))
        _dims(k_scale, "k_scale", (B, k.shape[1]))
    return IndexerIn(B, T, H, d, k.shape[1] * m, LSA_E4M3 if fp8 else LSA_BF16, _ptr(seq_len), _ptr(q),
                     _ptr(q_scale) if fp8 else None, _ptr(w), _ptr(k), _ptr(k_scale) if fp8 else None)


def attn_in(q, seq_len, scale, *, kv=None, k=None, v=None, d_v=None, stream_budget=None, kv_scale=None) -> AttnIn:
    """Describe attention tensors: q [B,T,Hq,d_qk]; MLA kv [B,L_max,d_qk] (V = first d_v
    columns) or separate k [B,L_max,d_qk], v [B,L_max,d_v]; all bf16, or an MLA kv of
    e4m3 codes (torch.float8_e4m3fn) with kv_scale [B,L_max] fp32 per token. stream_budget
    (k, sink, window) promises the index rows start with that streaming prefix."""
    torch = _torch()
    _need(q, "q", torch.bfloat16, 4)
    _need(seq_len, "seq_len", torch.int32, 1)
    B, T, Hq, d_qk = q.shape
    _dims(seq_len, "seq_len", (B,))
    ss, sw = (-1, -1) if stream_budget is None else (int(stream_budget[1]), int(stream_budget[2]))
    if kv is not None and kv.dtype == torch.float8_e4m3fn:
        _need(kv, "kv", torch.float8_e4m3fn, 3)
        _dims(kv, "kv", (B, None, None))
        if kv_scale is None:
            raise ValueError("an e4m3 kv needs kv_scale [B, L_max] float32")
        _need(kv_scale, "kv_scale", torch.float32, 2)
        if tuple(kv_scale.shape) != (kv.shape[0], kv.shape[1]):
            raise ValueError("kv_scale must be [B, L_max]")
        dv = d_v if d_v is not None else 512
        return AttnIn(B, T, Hq, d_qk, dv, kv.shape[1], float(scale), _ptr(seq_len), _ptr(q), _ptr(kv), _ptr(kv),
                      kv.shape[2], kv.shape[2], ss, sw, LSA_E4M3, _ptr(kv_scale))
    if kv_scale is not None:
        raise ValueError("kv_scale is for an e4m3 kv only")
    if kv is not None:
        _need(kv, "kv", torch.bfloat16, 3)
        _dims(kv, "kv", (B, None, None))
        dv = d_v if d_v is not None else (512 if d_qk == 576 else d_qk)
        return AttnIn(B, T, Hq, d_qk, dv, kv.shape[1], float(scale), _ptr(seq_len), _ptr(q), _ptr(kv), _ptr(kv),
                      kv.shape[2], kv.shape[2], ss, sw)
    _need(k, "k", torch.bfloat16, 3)
    _need(v, "v", torch.bfloat16, 3)
    _dims(k, "k", (B, None, None))
    _dims(v, "v", (B, k.shape[1], None))
    return AttnIn(B, T, Hq, d_qk, v.shape[2], k.shape[1], float(scale), _ptr(seq_len), _ptr(q), _ptr(k), _ptr(v),
                  k.shape[2], v.shape[2], ss, sw)


def workspace_size(op: int, *, indexer: Optional[IndexerIn] = None, attn=None, budget=(1, 0, 0), P=0, M=0,
                   n_layers=0, B=0, T=0, L_max=0, scores_external=False, m=0, paged: Optional[PagedAttnIn] = None,
                   n=0, n_pages=0) -> int:
    lib = load()
    a = OpArgs()
    keep = []
    if indexer is not None:
        a.indexer = ctypes.pointer(indexer)
    if attn is not None:
        if isinstance(attn, AttnIn):
            arr = (AttnIn * 1)(attn)
        else:
            arr = (AttnIn * len(attn))(*attn)
        keep.append(arr)
        a.attn = ctypes.cast(arr, ctypes.POINTER(AttnIn))
    a.budget = Budget(*budget)
    a.P, a.M, a.n_layers, a.B, a.T, a.L_max = P, M, n_layers, B, T, L_max
    a.scores_external = int(bool(scores_external))
    a.m = m
    if paged is not None:
        a.paged = ctypes.pointer(paged)
    a.n, a.n_pages = n, n_pages
    out = ctypes.c_size_t(0)
    _check(lib.lsa_workspace_size(op, ctypes.byref(a), ctypes.byref(out)))
    return out.value


def _workspace(nbytes: int, device, workspace=None):
    torch = _torch()
    if nbytes == 0:
        return None
    if workspace is not None:
        _need(workspace, "workspace")
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace smaller than the {nbytes} bytes required")
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------


def lsa_index_flat(q, w, k, seq_len, budget, *, q_scale=None, k_scale=None, idx=None, scores_out=None,
                   with_idx=True, workspace=None, stream=None):
    """Flat indexing. Returns idx [B,T,k] int32 (or None when with_idx is False)."""
    torch = _torch()
    lib = load()
    ii = indexer_in(q, w, k, seq_len, q_scale, k_scale)
    B, T = q.shape[0], q.shape[1]
    if with_idx and idx is None:
        idx = torch.empty((B, T, budget[0]), dtype=torch.int32, device=q.device)
    if with_idx:
        _out(idx, "idx", torch.int32, (B, T, budget[0]))
    _out(scores_out, "scores_out", torch.float32, (B, T, k.shape[1]))
    need = workspace_size(LSA_OP_INDEX_FLAT, indexer=ii, budget=budget, scores_external=scores_out is not None)
    ws = _workspace(need, q.device, workspace)
    _check(lib.lsa_index_flat(ctypes.byref(ii), Budget(*budget), _ptr(idx) if with_idx else None, _ptr(scores_out),
                              _ptr(ws), _nbytes(ws), _stream(stream)))
    return idx if with_idx else None


def lsa_index_compressed(q, w, entry_keys, seq_len, m, budget, *, q_scale=None, k_scale=None, idx=None,
                         scores_out=None, with_idx=True, workspace=None, stream=None):
    """Indexing over compressed entries of m tokens: entry_keys [B,L_max/m,d]
    (seq_len in tokens; budget in entries). Returns idx [B,T,k] entry ids (or
    None when with_idx is False)."""
    torch = _torch()
    lib = load()
    ii = indexer_in(q, w, entry_keys, seq_len, q_scale, k_scale, m=m)
    B, T = q.shape[0], q.shape[1]
    if with_idx and idx is None:
        idx = torch.empty((B, T, budget[0]), dtype=torch.int32, device=q.device)
    if with_idx:
        _out(idx, "idx", torch.int32, (B, T, budget[0]))
    _out(scores_out, "scores_out", torch.float32, (B, T, entry_keys.shape[1]))
    need = workspace_size(LSA_OP_INDEX_COMPRESSED, indexer=ii, budget=budget, m=m,
                          scores_external=scores_out is not None)
    ws = _workspace(need, q.device, workspace)
    _check(lib.lsa_index_compressed(ctypes.byref(ii), m, Budget(*budget), _ptr(idx) if with_idx else None,
                                    _ptr(scores_out), _ptr(ws), _nbytes(ws), _stream(stream)))
    return idx if with_idx else None


def lsa_select_streaming(scores, seq_len, budget, *, idx=None, workspace=None, stream=None):
    """Streaming selection over given fp32 scores [B,T,L_max]. Returns idx [B,T,k]."""
    torch = _torch()
    lib = load()
    _need(scores, "scores", torch.float32, 3)
    _need(seq_len, "seq_len", torch.int32, 1)
    B, T, L_max = scores.shape
    _dims(seq_len, "seq_len", (B,))
    if idx is None:
        idx = torch.empty((B, T, budget[0]), dtype=torch.int32, device=scores.device)
    _out(idx, "idx", torch.int32, (B, T, budget[0]))
    need = workspace_size(LSA_OP_SELECT, budget=budget, B=B, T=T, L_max=L_max)
    ws = _workspace(need, scores.device, workspace)
    _check(lib.lsa_select_streaming(_ptr(scores), _ptr(seq_len), B, T, L_max, Budget(*budget), _ptr(idx), _ptr(ws),
                                    _nbytes(ws), _stream(stream)))
    return idx


def lsa_select_streaming_noalloc(scores, seq_len, budget, *, idx=None, stream=None):
    """lsa_select_streaming with the library's static scratch instead of a
    workspace: the C entry point allocates nothing, for callers that cannot
    allocate device memory where they select. Pass `idx` [B,T,k] int32 to keep
    this call free of allocations on the Python side too. Calls on one device
    share the scratch, so they must not overlap on the GPU."""
    torch = _torch()
    lib = load()
    _need(scores, "scores", torch.float32, 3)
    _need(seq_len, "seq_len", torch.int32, 1)
    B, T, L_max = scores.shape
    _dims(seq_len, "seq_len", (B,))
    if idx is None:
        idx = torch.empty((B, T, budget[0]), dtype=torch.int32, device=scores.device)
    _out(idx, "idx", torch.int32, (B, T, budget[0]))
    _check(lib.lsa_select_streaming_noalloc(_ptr(scores), _ptr(seq_len), B, T, L_max, Budget(*budget), _ptr(idx),
                                            _stream(stream)))
    return idx


def lsa_pool_pages(k, seq_len, P, *, page_keys=None, stream=None):
    """Mean-pooled page keys [B, L_max/P, d] bf16 from keys [B, L_max, d] bf16."""
    torch = _torch()
    lib = load()
    _need(k, "k", torch.bfloat16, 3)
    _need(seq_len, "seq_len", torch.int32, 1)
    B, L_max, d = k.shape
    _dims(seq_len, "seq_len", (B,))
    if page_keys is None:
        page_keys = torch.zeros((B, L_max // P, d), dtype=torch.bfloat16, device=k.device)
    _out(page_keys, "page_keys", torch.bfloat16, (B, L_max // P, d))
    _check(lib.lsa_pool_pages(_ptr(k), _ptr(seq_len), B, L_max, d, P, _ptr(page_keys), _stream(stream)))
    return page_keys


def lsa_index_hier(q, w, k, seq_len, page_keys, P, M, budget, *, idx=None, pages_out=None, workspace=None,
                   stream=None):
    """Hierarchical indexing. Returns (idx [B,T,k], pages [B,T,M] or None)."""
    torch = _torch()
    lib = load()
    ii = indexer_in(q, w, k, seq_len)
    _need(page_keys, "page_keys", torch.bfloat16, 3)
    if P > 0:
        _dims(page_keys, "page_keys", (q.shape[0], k.shape[1] // P, q.shape[3]))
    B, T = q.shape[0], q.shape[1]
    if idx is None:
        idx = torch.empty((B, T, budget[0]), dtype=torch.int32, device=q.device)
    _out(idx, "idx", torch.int32, (B, T, budget[0]))
    _out(pages_out, "pages_out", torch.int32, (B, T, M))
    need = workspace_size(LSA_OP_INDEX_HIER, indexer=ii, budget=budget, P=P, M=M)
    ws = _workspace(need, q.device, workspace)
    _check(lib.lsa_index_hier(ctypes.byref(ii), _ptr(page_keys), P, M, Budget(*budget), _ptr(idx), _ptr(pages_out),
                              _ptr(ws), _nbytes(ws), _stream(stream)))
    return idx, pages_out


def lsa_pool_pages_e4m3(k8, k_scale, seq_len, P, *, page_codes=None, page_scales=None, stream=None):
    """FP8 page keys from e4m3 token keys k8 [B, L_max, 128] with k_scale [B, L_max]:
    (page codes [B, L_max/P, 128] e4m3, page scales [B, L_max/P] fp32)."""
    torch = _torch()
    lib = load()
    _need(k8, "k8", (torch.float8_e4m3fn, torch.uint8), 3)
    _need(k_scale, "k_scale", torch.float32, 2)
    _need(seq_len, "seq_len", torch.int32, 1)
    B, L_max, d = k8.shape
    _dims(k_scale, "k_scale", (B, L_max))
    _dims(seq_len, "seq_len", (B,))
    if page_codes is None:
        page_codes = torch.zeros((B, L_max // P, d), dtype=torch.uint8, device=k8.device).view(k8.dtype)
    if page_scales is None:
        page_scales = torch.ones((B, L_max // P), dtype=torch.float32, device=k8.device)
    _out(page_codes, "page_codes", (torch.float8_e4m3fn, torch.uint8), (B, L_max // P, d))
    _out(page_scales, "page_scales", torch.float32, (B, L_max // P))
    _check(lib.lsa_pool_pages_e4m3(_ptr(k8), _ptr(k_scale), _ptr(seq_len), B, L_max, d, P, _ptr(page_codes),
                                   _ptr(page_scales), _stream(stream)))
    return page_codes, page_scales


def lsa_index_hier_e4m3(q8, q_scale, w, k8, k_scale, seq_len, page_codes, page_scales, P, M, budget, *, idx=None,
                        pages_out=None, workspace=None, stream=None):
    """FP8 hierarchical indexing. Returns (idx [B,T,k], pages [B,T,M] or None)."""
    torch = _torch()
    lib = load()
    ii = indexer_in(q8, w, k8, seq_len, q_scale, k_scale)
    _need(page_codes, "page_codes", (torch.float8_e4m3fn, torch.uint8), 3)
    _need(page_scales, "page_scales", torch.float32, 2)
    if P > 0:
        _dims(page_codes, "page_codes", (q8.shape[0], k8.shape[1] // P, q8.shape[3]))
        _dims(page_scales, "page_scales", (q8.shape[0], k8.shape[1] // P))
    B, T = q8.shape[0], q8.shape[1]
    if idx is None:
        idx = torch.empty((B, T, budget[0]), dtype=torch.int32, device=q8.device)
    _out(idx, "idx", torch.int32, (B, T, budget[0]))
    _out(pages_out, "pages_out", torch.int32, (B, T, M))
    need = workspace_size(LSA_OP_INDEX_HIER, indexer=ii, budget=budget, P=P, M=M)
    ws = _workspace(need, q8.device, workspace)
    _check(lib.lsa_index_hier_e4m3(ctypes.byref(ii), _ptr(page_codes), _ptr(page_scales), P, M, Budget(*budget),
                                   _ptr(idx), _ptr(pages_out), _ptr(ws), _nbytes(ws), _stream(stream)))
    return idx, pages_out


def lsa_sparse_attn(q, idx, seq_len, scale, *, kv=None, k=None, v=None, d_v=None, out=None, lse=None,
                    workspace=None, stream=None, stream_budget=None, kv_scale=None):
    """Sparse attention over idx [B,T,k]. Returns (out [B,T,Hq,d_v] bf16, lse or None).
    stream_budget (k, sink, window): idx rows come from the streaming selection with
    that budget, so their sink/window prefix may be computed instead of read.
    An e4m3 MLA kv (torch.float8_e4m3fn) takes kv_scale [B, L_max] fp32."""
    torch = _torch()
    lib = load()
    ai = attn_in(q, seq_len, scale, kv=kv, k=k, v=v, d_v=d_v, stream_budget=stream_budget, kv_scale=kv_scale)
    _need(idx, "idx", torch.int32, 3)
    if tuple(idx.shape[:2]) != (ai.B, ai.T):
        raise ValueError(f"idx has shape {tuple(idx.shape)}, expected [{ai.B}, {ai.T}, k]")
    if out is None:
        out = torch.empty((ai.B, ai.T, ai.Hq, ai.d_v), dtype=torch.bfloat16, device=q.device)
    _out(out, "out", torch.bfloat16, (ai.B, ai.T, ai.Hq, ai.d_v))
    _out(lse, "lse", torch.float32, (ai.B, ai.T, ai.Hq))
    need = workspace_size(LSA_OP_SPARSE_ATTN, attn=ai, budget=(idx.shape[2], 0, 0))
    ws = _workspace(need, q.device, workspace)
    _check(lib.lsa_sparse_attn(ctypes.byref(ai), _ptr(idx), idx.shape[2], _ptr(out), _ptr(lse), _ptr(ws), _nbytes(ws),
                               _stream(stream)))
    return out, lse


def lsa_layer_group(q, w, k, seq_len, budget, layers: Sequence[dict], *, P=0, M=0, page_keys=None, outs=None,
                    lses=None, idx=None, workspace=None, stream=None):
    """One indexing pass (flat if P == 0) feeding len(layers) sparse-attention layers.

    Each layer dict: q, scale and kv (MLA) or k/v. Returns (idx, outs)."""
    torch = _torch()
    lib = load()
    ii = indexer_in(q, w, k, seq_len)
    ais = [attn_in(l["q"], seq_len, l["scale"], kv=l.get("kv"), k=l.get("k"), v=l.get("v"), d_v=l.get("d_v"),
                   kv_scale=l.get("kv_scale"))
           for l in layers]
    n = len(ais)
    if outs is None:
        outs = [torch.empty((a.B, a.T, a.Hq, a.d_v), dtype=torch.bfloat16, device=q.device) for a in ais]
    if idx is None:
        idx = torch.empty((q.shape[0], q.shape[1], budget[0]), dtype=torch.int32, device=q.device)
    _out(idx, "idx", torch.int32, (q.shape[0], q.shape[1], budget[0]))
    if len(outs) != n or (lses is not None and len(lses) != n):
        raise ValueError(f"outs and lses need one entry per layer ({n})")
    for i, a in enumerate(ais):
        _out(outs[i], f"outs[{i}]", torch.bfloat16, (a.B, a.T, a.Hq, a.d_v))
        if lses is not None:
            _out(lses[i], f"lses[{i}]", torch.float32, (a.B, a.T, a.Hq))
    if page_keys is not None:
        _out(page_keys, "page_keys", torch.bfloat16, (q.shape[0], k.shape[1] // P if P else 0, k.shape[2]))
    need = workspace_size(LSA_OP_LAYER_GROUP, indexer=ii, attn=ais, budget=budget, P=P, M=M, n_layers=n)
    ws = _workspace(need, q.device, workspace)
    arr = (AttnIn * n)(*ais)
    outp = (ctypes.c_void_p * n)(*[o.data_ptr() for o in outs])
    lsep = (ctypes.c_void_p * n)(*[(_ptr(l) if l is not None else None) for l in (lses or [None] * n)])
    _check(lib.lsa_layer_group(ctypes.byref(ii), _ptr(page_keys), P, M, Budget(*budget), n, arr, outp, lsep,
                               _ptr(idx), _ptr(ws), _nbytes(ws), _stream(stream)))
    return idx, outs


# ---------------------------------------------------------------------------
# the paged cache: rotary positions, new rows, attention, page upkeep
# ---------------------------------------------------------------------------


# A decode step makes these calls for every layer and each is a few microseconds of GPU work, so the checks of
# the binding come in two steps: _fits says in one expression whether a tensor is as it should be, and only
# where it is not do _need, _here and _dims work out what to raise.


def _made(stream, make):
    """make() on the stream that the call runs on: what it allocates must not be handed out again, nor filled,
    in the order of another stream."""
    if stream is None:
        return make()
    torch = _torch()
    with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
        return make()


def _fits(t, dtype, shape, cur):
    """t is a dense tensor of this type and shape on device `cur`."""
    return t is not None and t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous() \
        and t.device.index == cur


def _here(t, name, dtype, dim):
    """_need without the demand for dense rows: strides are passed on."""
    torch = _torch()
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    cur = torch.cuda.current_device()
    if t.device.index != cur:
        raise ValueError(f"{name} is on {t.device}, but the calls launch on the current device cuda:{cur}")
    dts = dtype if isinstance(dtype, tuple) else (dtype,)
    if t.dtype not in dts:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dts}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dims")
    return t


def _pages_of(t, name, dtype, heads, d, cur):
    """(page stride, row stride) in elements of a pool [n_pages, P, heads, d] or,
    for one head, [n_pages, P, d]: any page and row strides, dense rows."""
    if t is not None and t.is_cuda and t.dtype in dtype and t.is_contiguous() and t.device.index == cur:
        shape = t.shape
        if len(shape) == 4 and shape[2] == heads and shape[3] == d or len(shape) == 3 and heads == 1 and shape[2] == d:
            return shape[1] * heads * d, heads * d
    if t is not None and t.dim() == 3 and heads == 1:
        _here(t, name, dtype, 3)
        _dims(t, name, (None, None, d))
    else:
        _here(t, name, dtype, 4)
        _dims(t, name, (None, None, heads, d))
        if heads > 1 and t.stride(2) != d:
            raise ValueError(f"{name}: the heads of a row must be dense")
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must have a dense last dimension")
    P = t.shape[1]
    row = t.stride(1) if P > 1 else heads * d
    page = t.stride(0) if t.shape[0] > 1 else P * row
    return page, row


def _lengths(t, name, B, cur):
    if not _fits(t, _torch().int32, (B,), cur):
        _need(t, name, _torch().int32, 1)
        _dims(t, name, (B,))


def _table(table, seq_len, q_len, B, cur):
    i32 = _torch().int32
    if table is None or not _fits(table, i32, (B, table.shape[-1]), cur):
        _need(table, "table", i32, 2)
        _dims(table, "table", (B, None))
    _lengths(seq_len, "seq_len", B, cur)
    if q_len is not None:
        _lengths(q_len, "q_len", B, cur)


def lsa_rope_plan(rot_dim, theta, *, interleaved=False, scaling="none", factor=1.0, orig_len=0, beta_fast=32.0,
                  beta_slow=1.0, amplitude=0.0) -> RopePlan:
    """Frequencies of a rotary embedding of rot_dim columns, kept by the caller and passed
    to lsa_rope / lsa_pages_append. Pairs are (2i, 2i+1) if interleaved, else
    (i, i + rot_dim/2). scaling: "none", "linear" or "yarn" (with orig_len); amplitude 0
    takes the default (0.1 ln factor + 1 for yarn)."""
    if scaling not in LSA_ROPE_SCALINGS:
        raise ValueError(f"scaling {scaling!r} is not one of {sorted(LSA_ROPE_SCALINGS)}")
    plan = RopePlan()
    _check(load().lsa_rope_plan(rot_dim, int(bool(interleaved)), float(theta), LSA_ROPE_SCALINGS[scaling], float(factor),
                                orig_len, float(beta_fast), float(beta_slow), float(amplitude), ctypes.byref(plan)))
    return plan


def lsa_rope(x, plan, seq_len, *, q_len=None, offset=0, inverse=False, out=None, stream=None):
    """Rotates the columns [offset, offset + rot_dim) of x [B,T,H,d] (bf16 or fp32, any strides with
    a dense last dimension) by each token's position; the other columns are copied. inverse: the
    transposed rotation, which takes the gradient of the output to that of x. out may be x. Returns
    out; rows of padding tokens of a given out are left as they were (a new out is zero there)."""
    torch = _torch()
    cur = torch.cuda.current_device()
    if x is None or not x.is_cuda or x.device.index != cur or x.dim() != 4 or \
            x.dtype is not torch.bfloat16 and x.dtype is not torch.float32:
        _here(x, "x", (torch.bfloat16, torch.float32), 4)
    B, T, H, d = shape = x.shape
    _lengths(seq_len, "seq_len", B, cur)
    if q_len is not None:
        _lengths(q_len, "q_len", B, cur)
    if out is None:
        out = _made(stream, lambda: torch.zeros(shape, dtype=x.dtype, device=x.device))
    elif not out.is_cuda or out.device.index != cur or out.dtype is not x.dtype or out.shape != shape:
        _here(out, "out", x.dtype, 4)
        _dims(out, "out", tuple(shape))
    xs, os = x.stride(), out.stride()
    if d > 1 and (xs[3] != 1 or os[3] != 1):
        raise ValueError("x and out must have a dense last dimension")
    ri = RopeIn(B, T, H, d, LSA_FP32 if x.dtype is torch.float32 else LSA_BF16, offset, int(bool(inverse)),
                seq_len.data_ptr(), _ptr(q_len), x.data_ptr(), xs[0], xs[1], xs[2], os[0], os[1], os[2])
    _check(load().lsa_rope(ri, plan, out.data_ptr(), _stream(stream)))
    return out


def lsa_pages_append(x, table, seq_len, pool, *, q_len=None, scale_pool=None, plan=None, offset=0, stream=None):
    """Writes the new rows x [B,T,H,d] bf16 (or [B,T,d] for one head) into their pages of pool
    [n_pages,P,H,d] (or [n_pages,P,d]): bf16, or e4m3 codes (torch.float8_e4m3fn) with the row's
    scale in scale_pool [n_pages,P] fp32. plan: every head's columns [offset, offset + rot_dim) are
    rotated first. seq_len counts the new tokens. Returns pool."""
    torch = _torch()
    cur = torch.cuda.current_device()
    if x is None or not x.is_cuda or x.dtype is not torch.bfloat16 or not x.is_contiguous() or x.device.index != cur or \
            x.dim() not in (3, 4):
        _need(x, "x", torch.bfloat16, 4)
    if x.dim() == 3:
        (B, T, d), H = x.shape, 1
    else:
        B, T, H, d = x.shape
    _table(table, seq_len, q_len, B, cur)
    page, row = _pages_of(pool, "pool", (torch.bfloat16, torch.float8_e4m3fn), H, d, cur)
    n_pages, P = pool.shape[:2]
    e4m3 = pool.dtype is torch.float8_e4m3fn
    if e4m3:
        if not _fits(scale_pool, torch.float32, (n_pages, P), cur):
            _need(scale_pool, "scale_pool", torch.float32, 2)
            _dims(scale_pool, "scale_pool", (n_pages, P))
    elif scale_pool is not None:
        raise ValueError("scale_pool is for an e4m3 pool only")
    ai = AppendIn(B, T, H, d, n_pages, P, table.shape[1], LSA_E4M3 if e4m3 else LSA_BF16, offset, seq_len.data_ptr(),
                  _ptr(q_len), table.data_ptr(), x.data_ptr(), pool.data_ptr(), page, row, _ptr(scale_pool))
    _check(load().lsa_pages_append(ai, plan, _stream(stream)))
    return pool


def paged_attn_in(q, table, seq_len, scale, *, kv=None, k=None, v=None, d_v=None, kv_scale=None,
                  q_len=None) -> PagedAttnIn:
    """Describe paged attention: q [B,T,Hq,d_qk] bf16; latent rows kv [n_pages,P,576] (bf16, or
    torch.float8_e4m3fn with kv_scale [n_pages,P]), or k, v [n_pages,P,Hkv,d] bf16."""
    torch = _torch()
    cur = torch.cuda.current_device()
    if q is None or q.dim() != 4 or not _fits(q, torch.bfloat16, q.shape, cur):
        _need(q, "q", torch.bfloat16, 4)
    B, T, Hq, d_qk = q.shape
    _table(table, seq_len, q_len, B, cur)
    if kv is not None:
        if k is not None or v is not None:
            raise ValueError("give kv (latent rows) or k and v, not both")
        page, row = _pages_of(kv, "kv", (torch.bfloat16, torch.float8_e4m3fn), 1, d_qk, cur)
        n_pages, P = kv.shape[:2]
        e4m3 = kv.dtype is torch.float8_e4m3fn
        if e4m3:
            if not _fits(kv_scale, torch.float32, (n_pages, P), cur):
                _need(kv_scale, "kv_scale", torch.float32, 2)
                _dims(kv_scale, "kv_scale", (n_pages, P))
        elif kv_scale is not None:
            raise ValueError("kv_scale is for an e4m3 kv only")
        at = kv.data_ptr()
        return PagedAttnIn(B, T, Hq, 1, d_qk, d_v if d_v is not None else 512, n_pages, P, table.shape[1], scale,
                           LSA_E4M3 if e4m3 else LSA_BF16, seq_len.data_ptr(), _ptr(q_len), table.data_ptr(), q.data_ptr(),
                           at, at, page, row, page, row, _ptr(kv_scale))
    if kv_scale is not None:
        raise ValueError("kv_scale is for an e4m3 kv only")
    if k is None or v is None or k.dim() != 4 or v.dim() != 4:
        _here(k, "k", torch.bfloat16, 4)
        _here(v, "v", torch.bfloat16, 4)
    n_pages, P, Hkv = k.shape[:3]
    kp, kr = _pages_of(k, "k", (torch.bfloat16,), Hkv, d_qk, cur)
    vd = v.shape[3]
    vp, vr = _pages_of(v, "v", (torch.bfloat16,), Hkv, vd, cur)
    if v.shape != (n_pages, P, Hkv, vd if d_v is None else d_v):
        _dims(v, "v", (n_pages, P, Hkv, d_v))
    return PagedAttnIn(B, T, Hq, Hkv, d_qk, vd, n_pages, P, table.shape[1], scale, LSA_BF16, seq_len.data_ptr(), _ptr(q_len),
                       table.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), kp, kr, vp, vr, None)


def lsa_paged_attn(q, table, seq_len, scale, *, kv=None, k=None, v=None, d_v=None, kv_scale=None, q_len=None, out=None,
                   lse=None, workspace=None, stream=None):
    """Attention of the new tokens q [B,T,Hq,d_qk] over every cached token they see (causal; seq_len
    counts the new tokens). The cache is kv (latent rows, MLA) or k and v, in pages listed by table
    [B,max_pages]. Returns (out [B,T,Hq,d_v] bf16, lse or None); rows t >= q_len[b] of a given out
    are left as they were (a new out is zero there)."""
    torch = _torch()
    lib = load()
    pi = paged_attn_in(q, table, seq_len, scale, kv=kv, k=k, v=v, d_v=d_v, kv_scale=kv_scale, q_len=q_len)
    shape, cur = (pi.B, pi.T, pi.Hq, pi.d_v), q.device.index
    if out is None:
        make = torch.empty if q_len is None else torch.zeros
        out = _made(stream, lambda: make(shape, dtype=torch.bfloat16, device=q.device))
    elif not _fits(out, torch.bfloat16, shape, cur):
        _out(out, "out", torch.bfloat16, shape)
    if lse is not None and not _fits(lse, torch.float32, shape[:3], cur):
        _out(lse, "lse", torch.float32, shape[:3])
    size = _paged_bytes(cur, pi.B, pi.T, pi.Hq, pi.Hkv, pi.d_qk, pi.page_size, pi.max_pages)
    size = size if size else workspace_size(LSA_OP_PAGED_ATTN, paged=pi)
    ws = _made(stream, lambda: _workspace(size, q.device, workspace))
    _check(lib.lsa_paged_attn(pi, out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.nbytes, _stream(stream)))
    return out, lse


@functools.lru_cache(maxsize=256)
def _paged_bytes(device, B, T, Hq, Hkv, d, page_size, max_pages):
    """Workspace of a paged attention call of these sizes (0: sizes that the call itself refuses)."""
    pi = PagedAttnIn(B, T, Hq, Hkv, d, 512 if d == 576 else d, 1, page_size, max_pages, 1.0, LSA_BF16, 16, None, 16, 16, 16, 16,
                     1 << 20, Hkv * d, 1 << 20, Hkv * d, None)
    size = ctypes.c_size_t()
    ok = load().lsa_workspace_size(LSA_OP_PAGED_ATTN, OpArgs(paged=ctypes.pointer(pi)), size)
    return size.value if ok == LSA_OK else 0


def _cache(table, ref, seq_len=None):
    """(S, max_pages, n_pages, device) of a table [S,max_pages] and counts ref [n_pages], all int32."""
    i32, cur = _torch().int32, _torch().cuda.current_device()
    if table is None or table.dim() != 2 or not _fits(table, i32, table.shape, cur):
        _need(table, "table", i32, 2)
    if ref is None or ref.dim() != 1 or not _fits(ref, i32, ref.shape, cur):
        _need(ref, "ref", i32, 1)
    S, max_pages = table.shape
    if seq_len is not None:
        _lengths(seq_len, "seq_len", S, cur)
    return S, max_pages, ref.shape[0], cur


def _list(t, name, cur):
    if t is None or t.dim() != 1 or not _fits(t, _torch().int32, t.shape, cur):
        _need(t, name, _torch().int32, 1)
    return t.shape[0]


def _pools(pools, n_pages, cur):
    """Descriptors of pools [n_pages, ...]: any page stride, dense pages of a multiple of 16 bytes."""
    rows = []
    for i, t in enumerate(pools):
        if not t.is_cuda or t.device.index != cur:
            raise ValueError(f"pools[{i}] must be a CUDA tensor on the current device cuda:{cur}")
        shape = t.shape
        if len(shape) < 2 or shape[0] != n_pages:
            raise ValueError(f"pools[{i}] has shape {tuple(shape)}, expected ({n_pages}, ...)")
        strides, es = t.stride(), t.element_size()
        if n_pages > 1 and t.is_contiguous():
            rows.append((t.data_ptr(), strides[0] * es, strides[0] * es))
            continue
        page = 1
        for n, step in zip(shape[:0:-1], strides[:0:-1]):
            if step != page and n != 1:
                raise ValueError(f"pools[{i}]: a page must be contiguous")
            page *= n
        rows.append((t.data_ptr(), page * es, (strides[0] if n_pages > 1 else page) * es))
    return (Pool * max(1, len(rows)))(*rows)


def lsa_pages_reserve(table, ref, lens, page_size, *, stream=None):
    """Maps pages (the lowest free ones) until row s of table [S,max_pages] holds lens[s] tokens."""
    S, max_pages, n_pages, cur = _cache(table, ref)
    _lengths(lens, "lens", S, cur)
    _check(load().lsa_pages_reserve(table.data_ptr(), ref.data_ptr(), lens.data_ptr(), S, max_pages, n_pages, page_size,
                                    _stream(stream)))


def lsa_pages_free(table, ref, seq_len, seqs, *, stream=None):
    """Frees the sequences seqs [n]: their pages' counts - 1, rows unmapped, lengths 0."""
    S, max_pages, n_pages, cur = _cache(table, ref, seq_len)
    n = _list(seqs, "seqs", cur)
    _check(load().lsa_pages_free(table.data_ptr(), ref.data_ptr(), seq_len.data_ptr(), S, max_pages, n_pages,
                                 seqs.data_ptr(), n, _stream(stream)))


def lsa_pages_fork(table, ref, seq_len, page_size, parent, child, pools: Sequence, *, workspace=None, stream=None):
    """Makes sequences child[i] copies of parent[i]: full pages shared, a partly filled last page
    copied in every pool. Children must be free (lsa_pages_free)."""
    S, max_pages, n_pages, cur = _cache(table, ref, seq_len)
    n = _list(parent, "parent", cur)
    _lengths(child, "child", n, cur)
    arr = _pools(pools, n_pages, cur)
    ws = _made(stream, lambda: _workspace(_pages_bytes(LSA_OP_PAGES_FORK, n, 0), table.device, workspace))
    _check(load().lsa_pages_fork(table.data_ptr(), ref.data_ptr(), seq_len.data_ptr(), S, max_pages, n_pages, page_size,
                                 parent.data_ptr(), child.data_ptr(), n, arr, len(pools), _ptr(ws), _nbytes(ws),
                                 _stream(stream)))


def lsa_pages_copy(pools: Sequence, src, dst, *, workspace=None, stream=None):
    """Copies page src[i] to dst[i] in every pool [n_pages, ...]."""
    if not len(pools):
        raise ValueError("need at least one pool")
    cur = _torch().cuda.current_device()
    n_pages = pools[0].shape[0]
    n = _list(src, "src", cur)
    _lengths(dst, "dst", n, cur)
    arr = _pools(pools, n_pages, cur)
    ws = _made(stream, lambda: _workspace(_pages_bytes(LSA_OP_PAGES_COPY, n, 0), src.device, workspace))
    _check(load().lsa_pages_copy(arr, len(pools), n_pages, src.data_ptr(), dst.data_ptr(), n, _ptr(ws), _nbytes(ws),
                                 _stream(stream)))


def lsa_pages_compact(table, ref, pools: Sequence, *, table_out=None, ref_out=None, n_live=None, workspace=None,
                      stream=None):
    """Packs the live pages into the first n_live pages of every pool. table_out and ref_out default to
    table and ref themselves. Returns (table_out, ref_out, n_live [1] int32)."""
    torch = _torch()
    S, max_pages, n_pages, cur = _cache(table, ref)
    if table_out is None:
        table_out = table
    elif not _fits(table_out, torch.int32, (S, max_pages), cur):
        _out(table_out, "table_out", torch.int32, (S, max_pages))
    if ref_out is None:
        ref_out = ref
    elif not _fits(ref_out, torch.int32, (n_pages,), cur):
        _out(ref_out, "ref_out", torch.int32, (n_pages,))
    if n_live is None:
        n_live = _made(stream, lambda: torch.empty(1, dtype=torch.int32, device=table.device))
    elif not _fits(n_live, torch.int32, (1,), cur):
        _out(n_live, "n_live", torch.int32, (1,))
    arr = _pools(pools, n_pages, cur)
    ws = _made(stream, lambda: _workspace(_pages_bytes(LSA_OP_PAGES_COMPACT, 0, n_pages), table.device, workspace))
    _check(load().lsa_pages_compact(table.data_ptr(), ref.data_ptr(), S, max_pages, n_pages, arr, len(pools),
                                    table_out.data_ptr(), ref_out.data_ptr(), n_live.data_ptr(), _ptr(ws), _nbytes(ws),
                                    _stream(stream)))
    return table_out, ref_out, n_live


@functools.lru_cache(maxsize=256)
def _pages_bytes(op, n, n_pages):
    size = ctypes.c_size_t()
    _check(load().lsa_workspace_size(op, OpArgs(n=n, n_pages=n_pages), size))
    return size.value


def lsa_device_status(stream=None) -> int:
    """Synchronise and return the device status word (0 = ok); raises on timeout."""
    lib = load()
    st = lib.lsa_device_status(_stream(stream))
    _check(st)
    return st
