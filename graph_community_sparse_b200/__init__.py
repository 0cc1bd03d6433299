"""Python binding of libckv, the CommunityKV decode hot path for B200.

Argument marshalling only: every function passes raw device pointers, sizes
and the current CUDA stream to the C entry point of the same name in
``libckv.so`` (declared in include/ckv.h) and raises ``CKVError`` on a
non-zero status.  PyTorch provides device memory and streams; no computation
of the path happens here.  Importing the package fails loudly when the
library has not been built: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

__all__ = [
    "CKVError", "lib", "LIB_PATH", "CacheDesc", "GraphDesc", "SelectionDesc",
    "Graph", "Selection", "cache_desc", "new_graph", "new_selection", "new_workspace",
    "ckv_workspace_size", "ckv_build_centroids", "ckv_score_select", "ckv_sparse_decode",
    "ckv_sparse_decode_noalloc", "NOALLOC_SCRATCH_BYTES", "ckv_assign_update", "ckv_append_assign",
    "ckv_sparse_decode_append", "ckv_get_device_error", "ckv_kernel_timing", "ckv_kernel_times",
    "KERNEL_KINDS",
    "ckv_dense_decode", "ckv_status_string", "ckv_last_error",
    "ckv_abi_version", "ckv_debug_build", "load_debug_library", "DEBUG_LIB_PATH",
    "ckv_edges_workspace_size", "ckv_build_edges", "Edges", "new_edges", "DEVERR_EDGE_CAP",
    "EXPORTED", "DTYPE_F32", "DTYPE_BF16", "PER_GROUP", "PER_HEAD",
    "ASSIGN_SCORE", "ASSIGN_VOTE",
    "DEVERR_SINK_LABEL", "DEVERR_LABEL_RANGE", "DEVERR_TAIL_FULL", "DEVERR_TOKEN_CAP", "DEVERR_INDEX",
    "NEIGHBOURS",
    "Q8_INT8", "Q8_E4M3", "DEVERR_PLAN", "DEVERR_BLOCK", "DEVERR_CUT", "TableDesc", "Q8Desc", "PlanDesc", "BlockTable", "Q8Cache",
    "Plan", "block_table", "q8_cache", "new_q8_cache", "new_plan", "q8_shape", "ckv_plan_blocks", "ckv_quant_append",
    "ckv_q8_read", "ckv_q8_workspace_size", "ckv_dense_decode_q8", "ckv_sparse_decode_q8", "ckv_build_centroids_q8",
    "ckv_trim_graph_q8",
]

# the in-tree build, always: no environment variable selects another library
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libckv.so")
# the same library built with device-side index checks (build.py --debug); it
# is loaded only on request (load_debug_library)
DEBUG_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libckv_debug.so")

DTYPE_F32, DTYPE_BF16 = 0, 1
PER_GROUP, PER_HEAD = 0, 1
ASSIGN_SCORE, ASSIGN_VOTE = 0, 1
DEVERR_SINK_LABEL, DEVERR_LABEL_RANGE, DEVERR_TAIL_FULL, DEVERR_TOKEN_CAP, DEVERR_INDEX = 1, 2, 4, 8, 16
DEVERR_EDGE_CAP = 32
DEVERR_PLAN, DEVERR_BLOCK, DEVERR_CUT = 64, 128, 256
Q8_INT8, Q8_E4M3 = 0, 1
NEIGHBOURS = 8
KERNEL_KINDS = ("build", "score", "select", "attention", "merge", "update", "edges")
EXPORTED = ("ckv_workspace_size", "ckv_build_centroids", "ckv_score_select", "ckv_sparse_decode",
            "ckv_sparse_decode_noalloc", "ckv_assign_update", "ckv_append_assign", "ckv_sparse_decode_append",
            "ckv_get_device_error", "ckv_kernel_timing", "ckv_kernel_times",
            "ckv_dense_decode",
            "ckv_edges_workspace_size", "ckv_build_edges",
            "ckv_plan_blocks", "ckv_quant_append", "ckv_q8_read", "ckv_q8_workspace_size", "ckv_dense_decode_q8",
            "ckv_sparse_decode_q8", "ckv_build_centroids_q8", "ckv_trim_graph_q8",
            "ckv_status_string", "ckv_last_error", "ckv_abi_version", "ckv_debug_build")
NOALLOC_SCRATCH_BYTES = 32 << 20


class CKVError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: {ckv_status_string(status)}: {message}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"libckv.so not built at {LIB_PATH}; run `python graph_community_sparse_b200/build.py`")
lib = ctypes.CDLL(LIB_PATH)

_i32, _i64, _p, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


class CacheDesc(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("B", _i32), ("Hkv", _i32), ("Hq", _i32), ("d", _i32),
                ("T_cap", _i32), ("k", _p), ("v", _p), ("stride_b", _i64), ("stride_h", _i64),
                ("stride_t", _i64)]


class GraphDesc(ctypes.Structure):
    _fields_ = [("mode", _i32), ("S", _i32), ("Cmax", _i32), ("max_tail", _i32), ("T_cap", _i32),
                ("assign_rule", _i32), ("comm_of", _p), ("offs", _p), ("tok", _p), ("cnt", _p), ("cent", _p), ("cent_q", _p), ("cent_qs", _p),
                ("num_comm", _p), ("tail_tok", _p), ("tail_comm", _p), ("tail_len", _p),
                ("dev_err", _p), ("undo", _p), ("built", _p)]


class SelectionDesc(ctypes.Structure):
    _fields_ = [("tok_cap", _i32), ("sel_comm", _p), ("n_sel", _p), ("sel_tok", _p), ("n_tok", _p),
                ("tok_prefix", _p), ("tail_sel", _p), ("unit_prefix", _p)]


class TableDesc(ctypes.Structure):
    _fields_ = [("B", _i32), ("block", _i32), ("n_blocks", _i32), ("max_blocks", _i32), ("table", _p), ("len", _p),
                ("free_list", _p), ("n_free", _p), ("dev_err", _p)]


class Q8Desc(ctypes.Structure):
    _fields_ = [("blocks", TableDesc), ("format", _i32), ("dtype", _i32), ("Hkv", _i32), ("Hq", _i32), ("d", _i32),
                ("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p)]


class PlanDesc(ctypes.Structure):
    _fields_ = [("n_rows", _i32), ("start", _p), ("slot", _p), ("granted", _p)]


_P = ctypes.POINTER


def _declare(lib_: ctypes.CDLL) -> ctypes.CDLL:
    """Argument and result types of every entry point of a loaded libckv."""
    lib_.ckv_workspace_size.argtypes = [_P(CacheDesc), _P(GraphDesc), _P(SelectionDesc), _P(_sz)]
    lib_.ckv_build_centroids.argtypes = [_P(CacheDesc), _p, _i64, _i32, _P(GraphDesc), _p, _sz, _p]
    lib_.ckv_score_select.argtypes = [_P(CacheDesc), _P(GraphDesc), _p, _i32, _P(SelectionDesc), _p, _sz, _p]
    lib_.ckv_sparse_decode.argtypes = [_P(CacheDesc), _p, _P(GraphDesc), _P(SelectionDesc), _p, _p, _p, _sz, _p]
    lib_.ckv_sparse_decode_noalloc.argtypes = [_P(CacheDesc), _p, _P(GraphDesc), _P(SelectionDesc), _p, _p, _p]
    lib_.ckv_assign_update.argtypes = [_P(CacheDesc), _P(GraphDesc), _i32, _p, _p, _p]
    lib_.ckv_append_assign.argtypes = [_P(CacheDesc), _P(GraphDesc), _i32, _p, _p, _p, _p, _p]
    lib_.ckv_sparse_decode_append.argtypes = [_P(CacheDesc), _p, _P(GraphDesc), _P(SelectionDesc), _p, _p, _i32,
                                              _p, _p, _p, _p, _sz, _p]
    lib_.ckv_dense_decode.argtypes = [_P(CacheDesc), _p, _i32, _p, _p, _sz, _p]
    lib_.ckv_edges_workspace_size.argtypes = [_P(CacheDesc), _i32, _i32, _i32, _P(_sz)]
    lib_.ckv_build_edges.argtypes = [_P(CacheDesc), _i32, _i32, _p, _i32, _p, _p, _p, _p, _p, _p, _i32, _p, _p, _sz,
                                     _p]
    lib_.ckv_plan_blocks.argtypes = [_P(TableDesc), _p, _P(PlanDesc), _p]
    lib_.ckv_quant_append.argtypes = [_P(Q8Desc), _P(PlanDesc), _p, _p, _i32, _i64, _i64, _i64, _p]
    lib_.ckv_q8_read.argtypes = [_P(Q8Desc), _p, _i32, _p, _p, _i64, _i64, _i64, _p]
    lib_.ckv_q8_workspace_size.argtypes = [_P(Q8Desc), _P(GraphDesc), _P(SelectionDesc), _P(_sz)]
    lib_.ckv_dense_decode_q8.argtypes = [_P(Q8Desc), _p, _p, _p, _sz, _p]
    lib_.ckv_sparse_decode_q8.argtypes = [_P(Q8Desc), _p, _P(GraphDesc), _P(SelectionDesc), _p, _p, _p, _p, _p, _sz,
                                          _p]
    lib_.ckv_build_centroids_q8.argtypes = [_P(Q8Desc), _p, _i64, _i32, _p, _P(GraphDesc), _p, _sz, _p]
    lib_.ckv_trim_graph_q8.argtypes = [_P(Q8Desc), _P(GraphDesc), _p]
    lib_.ckv_get_device_error.argtypes = [_P(GraphDesc), _p, _P(ctypes.c_int32), _i32]
    lib_.ckv_kernel_timing.argtypes = [_i32]
    lib_.ckv_kernel_times.argtypes = [_P(ctypes.c_float), _P(ctypes.c_int32), _i32]
    for f in ("ckv_workspace_size", "ckv_build_centroids", "ckv_score_select", "ckv_sparse_decode",
              "ckv_sparse_decode_noalloc", "ckv_assign_update", "ckv_append_assign", "ckv_sparse_decode_append",
              "ckv_dense_decode", "ckv_get_device_error", "ckv_kernel_timing", "ckv_kernel_times",
              "ckv_edges_workspace_size", "ckv_build_edges", "ckv_plan_blocks", "ckv_quant_append", "ckv_q8_read",
              "ckv_q8_workspace_size", "ckv_dense_decode_q8", "ckv_sparse_decode_q8", "ckv_build_centroids_q8",
              "ckv_trim_graph_q8"):
        getattr(lib_, f).restype = ctypes.c_int
    lib_.ckv_status_string.argtypes = [ctypes.c_int]
    lib_.ckv_status_string.restype = ctypes.c_char_p
    lib_.ckv_last_error.argtypes = []
    lib_.ckv_last_error.restype = ctypes.c_char_p
    lib_.ckv_abi_version.argtypes = []
    lib_.ckv_abi_version.restype = ctypes.c_int32
    lib_.ckv_debug_build.argtypes = []
    lib_.ckv_debug_build.restype = ctypes.c_int32
    return lib_


_declare(lib)
_debug_lib: Optional[ctypes.CDLL] = None


def load_debug_library() -> ctypes.CDLL:
    """The debug build of the library (libckv_debug.so: every index a
    caller's array feeds to a kernel is checked on the device), loaded on
    first use, with the same entry points as `lib`.  Raises ImportError when
    it has not been built (build.py --debug)."""
    global _debug_lib
    if _debug_lib is None:
        if not os.path.exists(DEBUG_LIB_PATH):
            raise ImportError(f"libckv_debug.so not built at {DEBUG_LIB_PATH}; run "
                              "`python graph_community_sparse_b200/build.py --debug`")
        _debug_lib = _declare(ctypes.CDLL(DEBUG_LIB_PATH))
    return _debug_lib


def ckv_debug_build() -> int:
    return int(lib.ckv_debug_build())


def ckv_status_string(status: int) -> str:
    return lib.ckv_status_string(int(status)).decode()


def ckv_last_error() -> str:
    return lib.ckv_last_error().decode()


def ckv_abi_version() -> int:
    return int(lib.ckv_abi_version())


def _check(status: int, where: str) -> None:
    if status != 0:
        raise CKVError(status, where, ckv_last_error())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        if not torch.cuda.is_available():
            return None
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ----------------------------------------------------------------------------
# descriptors and buffers (device memory comes from PyTorch)
# ----------------------------------------------------------------------------

def cache_desc(K: torch.Tensor, V: torch.Tensor, Hq: int) -> CacheDesc:
    """Describe a [B, Hkv, T_cap, d] K/V cache pair (same shape and strides)."""
    if K.shape != V.shape or K.stride() != V.stride() or K.dtype != V.dtype:
        raise ValueError("K and V must share shape, strides and dtype")
    if K.dim() != 4 or K.stride(3) != 1:
        raise ValueError("K must be [B, Hkv, T_cap, d] with contiguous rows")
    dt = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}.get(K.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {K.dtype}")
    B, Hkv, T_cap, d = K.shape
    return CacheDesc(dt, B, Hkv, Hq, d, T_cap, K.data_ptr(), V.data_ptr(),
                     K.stride(0), K.stride(1), K.stride(2))


@dataclass
class Graph:
    desc: GraphDesc
    comm_of: torch.Tensor
    offs: torch.Tensor
    tok: torch.Tensor
    cnt: torch.Tensor
    cent: torch.Tensor
    cent_q: torch.Tensor
    cent_qs: torch.Tensor
    num_comm: torch.Tensor
    tail_tok: torch.Tensor
    tail_comm: torch.Tensor
    tail_len: torch.Tensor
    dev_err: torch.Tensor
    undo: Optional[torch.Tensor] = None
    built: Optional[torch.Tensor] = None

    @property
    def U(self) -> int:
        return self.num_comm.shape[0]


@dataclass
class Selection:
    desc: SelectionDesc
    sel_comm: torch.Tensor
    n_sel: torch.Tensor
    sel_tok: torch.Tensor
    n_tok: torch.Tensor
    tok_prefix: torch.Tensor
    tail_sel: torch.Tensor
    unit_prefix: torch.Tensor


def new_graph(cache: CacheDesc, mode: int, S: int, Cmax: int, max_tail: int, device="cuda",
              rule: int = ASSIGN_SCORE, undo: bool = False) -> Graph:
    """undo: with room to take tail members out again (fp32 [U, max_tail, d]), which a paged 8-bit cache's
    requests need when they lose tokens."""
    G = cache.Hq if mode == PER_HEAD else cache.Hkv
    U = cache.B * G
    i32 = dict(dtype=torch.int32, device=device)
    t = dict(
        comm_of=torch.full((U, cache.T_cap), -1, **i32),
        offs=torch.zeros((U, Cmax + 1), **i32),
        tok=torch.zeros((U, cache.T_cap), **i32),
        cnt=torch.zeros((U, Cmax), **i32),
        cent=torch.zeros((U, Cmax, cache.d), dtype=torch.float32, device=device),
        cent_q=torch.zeros((U, Cmax, cache.d), dtype=torch.int8, device=device),
        cent_qs=torch.zeros((U, Cmax), dtype=torch.float32, device=device),
        num_comm=torch.zeros((U,), **i32),
        tail_tok=torch.zeros((U, max(max_tail, 1)), **i32),
        tail_comm=torch.zeros((U, max(max_tail, 1)), **i32),
        tail_len=torch.zeros((U,), **i32),
        dev_err=torch.zeros((1,), **i32),
        built=torch.zeros((U,), **i32),
    )
    if undo:
        t["undo"] = torch.zeros((U, max(max_tail, 1), cache.d), dtype=torch.float32, device=device)
    desc = GraphDesc(mode, S, Cmax, max_tail, cache.T_cap, rule, *(t[k].data_ptr() for k in (
        "comm_of", "offs", "tok", "cnt", "cent", "cent_q", "cent_qs", "num_comm", "tail_tok", "tail_comm", "tail_len",
        "dev_err")), _ptr(t.get("undo")), t["built"].data_ptr())
    return Graph(desc, **t)


def new_selection(cache: CacheDesc, graph: Graph, tok_cap: int, device="cuda") -> Selection:
    U, Cmax = graph.U, graph.desc.Cmax
    i32 = dict(dtype=torch.int32, device=device)
    t = dict(sel_comm=torch.zeros((U, Cmax), **i32), n_sel=torch.zeros((U,), **i32),
             sel_tok=torch.zeros((U, tok_cap), **i32), n_tok=torch.zeros((U,), **i32),
             tok_prefix=torch.zeros((U, Cmax + 1), **i32),
             tail_sel=torch.zeros((U, max(graph.desc.max_tail, 1)), **i32),
             unit_prefix=torch.zeros((U + 1,), **i32))
    desc = SelectionDesc(tok_cap, *(t[k].data_ptr() for k in ("sel_comm", "n_sel", "sel_tok", "n_tok",
                                                               "tok_prefix", "tail_sel", "unit_prefix")))
    return Selection(desc, **t)


def new_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Zeroed (the library needs its first 256 bytes zero before first use
    and leaves them zero); torch's caching allocator hands out 512-byte
    aligned blocks."""
    return torch.zeros((max(int(nbytes), 256),), dtype=torch.uint8, device=device)


# ----------------------------------------------------------------------------
# the entry points
# ----------------------------------------------------------------------------

def ckv_workspace_size(cache: CacheDesc, graph: Optional[Graph] = None,
                       sel: Optional[Selection] = None) -> int:
    out = _sz(0)
    g = ctypes.byref(graph.desc) if graph is not None else None
    s = ctypes.byref(sel.desc) if sel is not None else None
    _check(lib.ckv_workspace_size(ctypes.byref(cache), g, s, ctypes.byref(out)), "ckv_workspace_size")
    return int(out.value)


def ckv_build_centroids(cache: CacheDesc, labels: torch.Tensor, T: int, graph: Graph,
                        ws: torch.Tensor, stream=None) -> None:
    if labels.dtype != torch.int32 or labels.dim() != 2 or labels.stride(1) != 1:
        raise ValueError("labels must be int32 [U, >=T] with contiguous rows")
    _check(lib.ckv_build_centroids(ctypes.byref(cache), labels.data_ptr(), labels.stride(0), T,
                                   ctypes.byref(graph.desc), ws.data_ptr(), ws.numel(), _stream(stream)),
           "ckv_build_centroids")


def ckv_score_select(cache: CacheDesc, graph: Graph, q: torch.Tensor, budget: int, sel: Selection,
                     ws: torch.Tensor, stream=None) -> None:
    _check(lib.ckv_score_select(ctypes.byref(cache), ctypes.byref(graph.desc), q.data_ptr(), budget,
                                ctypes.byref(sel.desc), ws.data_ptr(), ws.numel(), _stream(stream)),
           "ckv_score_select")


def ckv_sparse_decode(cache: CacheDesc, q: torch.Tensor, graph: Graph, sel: Selection, out: torch.Tensor,
                      nbr8: Optional[torch.Tensor], ws: torch.Tensor, stream=None) -> None:
    _check(lib.ckv_sparse_decode(ctypes.byref(cache), q.data_ptr(), ctypes.byref(graph.desc),
                                 ctypes.byref(sel.desc), out.data_ptr(), _ptr(nbr8), ws.data_ptr(),
                                 ws.numel(), _stream(stream)),
           "ckv_sparse_decode")


def ckv_sparse_decode_noalloc(cache: CacheDesc, q: torch.Tensor, graph: Graph, sel: Selection,
                              out: torch.Tensor, nbr8: Optional[torch.Tensor], stream=None) -> None:
    """ckv_sparse_decode for callers that cannot hand over a workspace: the
    scratch is a fixed 32 MiB array inside the library (see include/ckv.h).
    Calls must not overlap on the GPU."""
    _check(lib.ckv_sparse_decode_noalloc(ctypes.byref(cache), q.data_ptr(), ctypes.byref(graph.desc),
                                         ctypes.byref(sel.desc), out.data_ptr(), _ptr(nbr8), _stream(stream)),
           "ckv_sparse_decode_noalloc")


def ckv_assign_update(cache: CacheDesc, graph: Graph, pos: int, nbr8: torch.Tensor,
                      assigned: Optional[torch.Tensor], stream=None) -> None:
    _check(lib.ckv_assign_update(ctypes.byref(cache), ctypes.byref(graph.desc), pos, nbr8.data_ptr(),
                                 _ptr(assigned), _stream(stream)),
           "ckv_assign_update")


def _check_rows(cache: CacheDesc, **rows) -> None:
    shape = (cache.B, cache.Hkv, cache.d)
    for name, t in rows.items():
        if tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {shape} tensor, got {tuple(t.shape)}")


def ckv_sparse_decode_append(cache: CacheDesc, q: torch.Tensor, graph: Graph, sel: Selection, out: torch.Tensor,
                             nbr8: Optional[torch.Tensor], pos: int, k_new: torch.Tensor, v_new: torch.Tensor,
                             assigned: Optional[torch.Tensor], ws: torch.Tensor, stream=None) -> None:
    """ckv_sparse_decode + ckv_append_assign in one call (the update runs in
    the attention's merge kernel)."""
    _check_rows(cache, k_new=k_new, v_new=v_new)
    _check(lib.ckv_sparse_decode_append(ctypes.byref(cache), q.data_ptr(), ctypes.byref(graph.desc),
                                        ctypes.byref(sel.desc), out.data_ptr(), _ptr(nbr8), pos, k_new.data_ptr(),
                                        v_new.data_ptr(), _ptr(assigned), ws.data_ptr(), ws.numel(),
                                        _stream(stream)),
           "ckv_sparse_decode_append")


def ckv_kernel_timing(enable: bool) -> None:
    """Bracket every later launch with CUDA events (diagnostic; see ckv.h)."""
    _check(lib.ckv_kernel_timing(int(bool(enable))), "ckv_kernel_timing")


def ckv_kernel_times() -> dict:
    """{kind: (total ms, launches)} of the launches timed since the last read."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_float * n)()
    cnt = (ctypes.c_int32 * n)()
    _check(lib.ckv_kernel_times(ms, cnt, n), "ckv_kernel_times")
    return {k: (float(ms[i]), int(cnt[i])) for i, k in enumerate(KERNEL_KINDS)}


def ckv_get_device_error(graph, reset: bool = False, stream=None) -> int:
    """The device error word (OR of DEVERR_* bits) of a Graph, a BlockTable or
    a Q8Cache once the queued work of the stream (by default the current one of
    the word's device) is done; reset=True zeroes it afterwards."""
    code = ctypes.c_int32(0)
    dev = graph.dev_err.device
    if dev.type != "cuda":
        raise ValueError(f"ckv_get_device_error: the error word must be on a CUDA device, not {dev}")
    desc = graph.desc if isinstance(graph.desc, GraphDesc) else GraphDesc(dev_err=graph.dev_err.data_ptr())
    with torch.cuda.device(dev):
        _check(lib.ckv_get_device_error(ctypes.byref(desc), _stream(stream), ctypes.byref(code), int(reset)),
               "ckv_get_device_error")
    return int(code.value)


def ckv_append_assign(cache: CacheDesc, graph: Graph, pos: int, k_new: torch.Tensor, v_new: torch.Tensor,
                      nbr8: torch.Tensor, assigned: Optional[torch.Tensor], stream=None) -> None:
    """k_new, v_new: [B, Hkv, d] contiguous in the cache dtype; written to
    row ``pos`` of K and V by the library, then the update runs."""
    _check_rows(cache, k_new=k_new, v_new=v_new)
    _check(lib.ckv_append_assign(ctypes.byref(cache), ctypes.byref(graph.desc), pos, k_new.data_ptr(),
                                 v_new.data_ptr(), nbr8.data_ptr(), _ptr(assigned), _stream(stream)),
           "ckv_append_assign")


def ckv_dense_decode(cache: CacheDesc, q: torch.Tensor, T: int, out: torch.Tensor, ws: torch.Tensor,
                     stream=None) -> None:
    _check(lib.ckv_dense_decode(ctypes.byref(cache), q.data_ptr(), T, out.data_ptr(), ws.data_ptr(),
                                ws.numel(), _stream(stream)),
           "ckv_dense_decode")


# ----------------------------------------------------------------------------
# the prefill token graph
# ----------------------------------------------------------------------------

@dataclass
class Edges:
    """Outputs of ckv_build_edges for U graph units of a T-token prefill."""
    nbr: torch.Tensor      # int32 [U, T, 8] direct-edge key positions, best first, -1 padded
    lam: torch.Tensor      # fp32 [U, T, 8] their graph logits
    co_src: torch.Tensor   # int32 [U, pair_cap]
    co_dst: torch.Tensor   # int32 [U, pair_cap]
    co_w: torch.Tensor     # int32 [U, pair_cap]
    co_n: torch.Tensor     # int32 [U]
    dev_err: torch.Tensor  # int32 [1]
    ws: torch.Tensor

    def pairs(self, u: int):
        """Unit u's co-attention edges as (src, dst, weight) rows, sorted."""
        n = min(int(self.co_n[u].item()), self.co_src.shape[1])
        t = torch.stack([self.co_src[u, :n], self.co_dst[u, :n], self.co_w[u, :n]], dim=1)
        if n == 0:
            return t
        order = torch.argsort(t[:, 0].long() * (1 << 31) + t[:, 1].long())
        return t[order]


def ckv_edges_workspace_size(cache: CacheDesc, mode: int, S: int, T: int) -> int:
    out = _sz(0)
    _check(lib.ckv_edges_workspace_size(ctypes.byref(cache), mode, S, T, ctypes.byref(out)),
           "ckv_edges_workspace_size")
    return int(out.value)


def new_edges(cache: CacheDesc, mode: int, S: int, T: int, pair_cap: Optional[int] = None, device="cuda") -> Edges:
    """Buffers for ckv_build_edges; pair_cap defaults to 28 (T - S), which can
    never overflow."""
    U = cache.B * (cache.Hq if mode == PER_HEAD else cache.Hkv)
    cap = max(1, 28 * max(T - S, 0)) if pair_cap is None else pair_cap
    i32 = dict(dtype=torch.int32, device=device)
    return Edges(nbr=torch.empty((U, T, NEIGHBOURS), **i32),
                 lam=torch.empty((U, T, NEIGHBOURS), dtype=torch.float32, device=device),
                 co_src=torch.empty((U, cap), **i32), co_dst=torch.empty((U, cap), **i32),
                 co_w=torch.empty((U, cap), **i32), co_n=torch.empty((U,), **i32),
                 dev_err=torch.zeros((1,), **i32),
                 ws=torch.empty((max(ckv_edges_workspace_size(cache, mode, S, T), 256),), dtype=torch.uint8,
                                device=device))


def ckv_build_edges(cache: CacheDesc, mode: int, S: int, q_prefill: torch.Tensor, T: int, edges: Edges,
                    stream=None) -> None:
    """q_prefill: [B, Hq, >=T, d] bf16, contiguous rows; fills `edges`."""
    if q_prefill.dtype != torch.bfloat16 or q_prefill.dim() != 4 or not q_prefill.is_contiguous():
        raise ValueError("q_prefill must be a contiguous bf16 [B, Hq, T, d] tensor")
    if q_prefill.shape[2] != T:
        raise ValueError("q_prefill's third dimension must be T")
    _check(lib.ckv_build_edges(ctypes.byref(cache), mode, S, q_prefill.data_ptr(), T, edges.nbr.data_ptr(),
                               edges.lam.data_ptr(), edges.co_src.data_ptr(), edges.co_dst.data_ptr(),
                               edges.co_w.data_ptr(), edges.co_n.data_ptr(), edges.co_src.shape[1],
                               edges.dev_err.data_ptr(), edges.ws.data_ptr(), edges.ws.numel(), _stream(stream)),
           "ckv_build_edges")


# ----------------------------------------------------------------------------
# the paged 8-bit cache
# ----------------------------------------------------------------------------

_Q8_CODES = {torch.int8: Q8_INT8, torch.float8_e4m3fn: Q8_E4M3}
_Q8_FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_ROW_TYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _need(name: str, t: torch.Tensor, dtype, shape, device) -> int:
    """The data pointer of a tensor that has to be contiguous, of this dtype
    and shape, on this device."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} (strides {t.stride()}) on {t.device}")
    return t.data_ptr()


def _call(where: str, fn, device: torch.device, stream, *args) -> None:
    """Runs an entry point on the tensors' device: on its current stream unless
    one is given, with that device current.  The stream and the device are read
    without building torch's Stream and device objects: a decode step's calls
    are a few microseconds each on the host (8.4 with them, 5 without)."""
    if device.type != "cuda":
        raise ValueError(f"{where}: tensors must be on a CUDA device, not {device}")
    index = device.index
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status != 0:
        _check(status, where)


@dataclass
class BlockTable:
    """The blocks of a batch of requests and those that are free (ckv_table_desc)."""
    desc: TableDesc
    table: torch.Tensor      # int32 [B, max_blocks]
    len: torch.Tensor        # int32 [B]
    free_list: Optional[torch.Tensor]  # int32 [n_blocks]
    n_free: Optional[torch.Tensor]     # int32 [1]
    dev_err: torch.Tensor    # int32 [1]

    def __post_init__(self):
        self.device, self.shape, self.ref_blocks = self.len.device, self.len.shape, ctypes.byref(self.desc)

    @property
    def blocks(self) -> "BlockTable":
        return self


@dataclass
class Q8Cache:
    """A paged 8-bit cache (ckv_q8_desc); `dtype` is that of q and of the rows."""
    desc: Q8Desc
    blocks: BlockTable
    k: torch.Tensor          # int8 or float8_e4m3fn [n_blocks, Hkv, block, d]
    v: torch.Tensor
    k_scale: torch.Tensor    # fp32 [n_blocks, Hkv]
    v_scale: torch.Tensor
    dtype: torch.dtype

    def __post_init__(self):
        # what every call looks at, read once: a decode step's calls are a few
        # microseconds each on the host
        c = self.desc
        self.B, self.Hkv, self.Hq, self.d, self.device = c.blocks.B, c.Hkv, c.Hq, c.d, self.k.device
        self.q_shape, self.row_shape = torch.Size((self.B, self.Hq, self.d)), torch.Size((self.B, self.Hkv, self.d))
        self.ref, self.ref_blocks = ctypes.byref(c), ctypes.byref(self.blocks.desc)

    @property
    def dev_err(self) -> torch.Tensor:
        return self.blocks.dev_err

    @property
    def table(self) -> torch.Tensor:
        return self.blocks.table

    @property
    def len(self) -> torch.Tensor:
        return self.blocks.len


@dataclass
class Plan:
    """Where a batch of new tokens goes (ckv_plan_desc)."""
    start: torch.Tensor      # int32 [B + 1]
    slot: torch.Tensor       # int32 [n_rows]
    granted: torch.Tensor    # int32 [B]

    def __post_init__(self):
        B, dev = self.granted.shape[0], self.granted.device
        self.n_rows, self.device, self.shape = self.slot.numel(), dev, self.granted.shape
        self.desc = PlanDesc(self.slot.numel(), _need("start", self.start, torch.int32, (B + 1,), dev),
                             _need("slot", self.slot, torch.int32, (self.slot.numel(),), dev),
                             _need("granted", self.granted, torch.int32, (B,), dev))
        self.ref = ctypes.byref(self.desc)


def block_table(table: torch.Tensor, length: torch.Tensor, free_list: Optional[torch.Tensor],
                n_free: Optional[torch.Tensor], block: int, dev_err: Optional[torch.Tensor] = None,
                n_blocks: Optional[int] = None) -> BlockTable:
    """Describe existing tensors; n_blocks defaults to the free list's length."""
    if table.dim() != 2:
        raise ValueError("table must be int32 [B, max_blocks]")
    B, width = table.shape
    dev = table.device
    if dev_err is None:
        dev_err = torch.zeros((1,), dtype=torch.int32, device=dev)
    if n_blocks is None:
        if free_list is None:
            raise ValueError("n_blocks is needed without a free list")
        n_blocks = free_list.shape[0]
    desc = TableDesc(B, block, n_blocks, width, _need("table", table, torch.int32, (B, width), dev),
                     _need("length", length, torch.int32, (B,), dev),
                     None if free_list is None else _need("free_list", free_list, torch.int32, (n_blocks,), dev),
                     None if n_free is None else _need("n_free", n_free, torch.int32, (1,), dev),
                     _need("dev_err", dev_err, torch.int32, (1,), dev))
    return BlockTable(desc, table, length, free_list, n_free, dev_err)


def q8_cache(k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, table: torch.Tensor,
             length: torch.Tensor, Hq: int, dtype: torch.dtype = torch.bfloat16,
             free_list: Optional[torch.Tensor] = None, n_free: Optional[torch.Tensor] = None,
             dev_err: Optional[torch.Tensor] = None) -> Q8Cache:
    """Describe an existing pool [n_blocks, Hkv, block, d] of int8 or
    float8_e4m3fn codes with its scales, table and lengths."""
    if k.dim() != 4 or k.dtype not in _Q8_CODES:
        raise ValueError("k must be int8 or float8_e4m3fn [n_blocks, Hkv, block, d]")
    if dtype not in _ROW_TYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    n_blocks, Hkv, block, d = k.shape
    dev = k.device
    bt = block_table(table, length, free_list, n_free, block, dev_err, n_blocks)
    if table.device != dev:
        raise ValueError("the table must be on the pool's device")
    desc = Q8Desc(bt.desc, _Q8_CODES[k.dtype], _ROW_TYPES[dtype], Hkv, Hq, d, _need("k", k, k.dtype, k.shape, dev),
                  _need("v", v, k.dtype, k.shape, dev), _need("k_scale", k_scale, torch.float32, (n_blocks, Hkv), dev),
                  _need("v_scale", v_scale, torch.float32, (n_blocks, Hkv), dev))
    return Q8Cache(desc, bt, k, v, k_scale, v_scale, dtype)


def new_q8_cache(B: int, Hkv: int, Hq: int, d: int, n_blocks: int, block: int = 64, max_blocks: Optional[int] = None,
                 fmt: str = "int8", dtype: torch.dtype = torch.bfloat16, device="cuda") -> Q8Cache:
    """An empty pool: B requests of length 0, every block free (block 0 is
    taken first).  fmt: "int8" or "e4m3"."""
    if fmt not in _Q8_FORMATS:
        raise ValueError(f"unknown format {fmt!r}")
    i32 = dict(dtype=torch.int32, device=device)
    k = torch.zeros((n_blocks, Hkv, block, d), dtype=torch.uint8, device=device).view(_Q8_FORMATS[fmt])
    scale = torch.ones((n_blocks, Hkv), dtype=torch.float32, device=device)
    return q8_cache(k, torch.zeros_like(k.view(torch.uint8)).view(k.dtype), scale, scale.clone(),
                    torch.full((B, n_blocks if max_blocks is None else max_blocks), -1, **i32),
                    torch.zeros((B,), **i32), Hq, dtype,
                    torch.arange(n_blocks - 1, -1, -1, **i32), torch.full((1,), n_blocks, **i32))


def new_plan(cache, n_rows: int) -> Plan:
    """Buffers for ckv_plan_blocks on a BlockTable or Q8Cache; n_rows bounds
    the tokens that the batch may add."""
    length = cache.len
    i32 = dict(dtype=torch.int32, device=length.device)
    B = length.shape[0]
    return Plan(torch.zeros((B + 1,), **i32), torch.full((n_rows,), -1, **i32), torch.zeros((B,), **i32))


def q8_shape(cache: Q8Cache, T_cap: int) -> CacheDesc:
    """The cache's shapes, for new_graph, new_selection and ckv_score_select."""
    c = cache.desc
    return CacheDesc(c.dtype, c.blocks.B, c.Hkv, c.Hq, c.d, T_cap, None, None, 0, 0, 0)


def _of_plan(blocks: BlockTable, plan: Plan) -> None:
    if plan.shape != blocks.shape or plan.device != blocks.device:
        raise ValueError("the plan was made for another batch size or device")


def ckv_plan_blocks(cache, add: torch.Tensor, plan: Plan, stream=None) -> None:
    """Request b of a BlockTable or Q8Cache changes by add[b] tokens (int32 [B])."""
    bt = cache.blocks
    _of_plan(bt, plan)
    _call("ckv_plan_blocks", lib.ckv_plan_blocks, bt.device, stream, bt.ref_blocks,
          _need("add", add, torch.int32, bt.shape, bt.device), plan.ref)


def _rows(cache: Q8Cache, names, k: torch.Tensor, v: torch.Tensor, shape):
    """The common strides of a pair of row tensors of this shape."""
    strides, dtype, dev = k.stride(), cache.dtype, cache.device
    if (k.shape != shape or v.shape != shape or k.dtype is not dtype or v.dtype is not dtype or k.device != dev
            or v.device != dev or v.stride() != strides or strides[-1] != 1):
        raise ValueError(f"{names} must be {dtype} tensors of shape {tuple(shape)} on {dev} with contiguous rows and common "
                         f"strides, got {k.dtype} {tuple(k.shape)} {strides} on {k.device} and {v.dtype} "
                         f"{tuple(v.shape)} {v.stride()} on {v.device}")
    return strides


def ckv_quant_append(cache: Q8Cache, plan: Plan, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
    """k_new, v_new: packed rows [n_rows, Hkv, d], or padded ones [B, T, Hkv, d]
    of which request b's first granted[b] count; cache dtype, any strides with
    contiguous rows of 16-byte multiples, the same for both."""
    _of_plan(cache.blocks, plan)
    if k_new.dim() == 3:
        T_rows = sb = 0
        st, sh, _ = _rows(cache, "k_new and v_new", k_new, v_new, (plan.n_rows, cache.Hkv, cache.d))
    elif k_new.dim() == 4:
        T_rows = k_new.shape[1]
        sb, st, sh, _ = _rows(cache, "k_new and v_new", k_new, v_new, (cache.B, T_rows, cache.Hkv, cache.d))
    else:
        raise ValueError("k_new must be [n_rows, Hkv, d] or [B, T, Hkv, d]")
    if plan.n_rows == 0:
        return
    if k_new.numel() == 0:
        raise ValueError("no rows for a plan that has some")
    _call("ckv_quant_append", lib.ckv_quant_append, cache.device, stream, cache.ref, plan.ref, k_new.data_ptr(),
          v_new.data_ptr(), T_rows, sb, st, sh)


def ckv_q8_read(cache: Q8Cache, k_out: torch.Tensor, v_out: torch.Tensor, first: Optional[torch.Tensor] = None,
                stream=None) -> None:
    """Fills k_out and v_out, [B, Hkv, R, d] in the cache dtype, with positions
    first[b] .. first[b] + R - 1 (first None: from 0); zeros past a request's
    end."""
    if k_out.dim() != 4:
        raise ValueError("k_out must be [B, Hkv, R, d]")
    R = k_out.shape[2]
    sb, sh, st, _ = _rows(cache, "k_out and v_out", k_out, v_out, (cache.B, cache.Hkv, R, cache.d))
    at = None if first is None else _need("first", first, torch.int32, cache.blocks.shape, cache.device)
    _call("ckv_q8_read", lib.ckv_q8_read, cache.device, stream, cache.ref, at, R, k_out.data_ptr(), v_out.data_ptr(),
          sb, sh, st)


def ckv_q8_workspace_size(cache: Q8Cache, graph: Optional[Graph] = None, sel: Optional[Selection] = None) -> int:
    out = _sz(0)
    g = ctypes.byref(graph.desc) if graph is not None else None
    s = ctypes.byref(sel.desc) if sel is not None else None
    _check(lib.ckv_q8_workspace_size(ctypes.byref(cache.desc), g, s, ctypes.byref(out)), "ckv_q8_workspace_size")
    return int(out.value)


def _q8_attention(cache: Q8Cache, q: torch.Tensor, out: torch.Tensor, ws: torch.Tensor):
    dev = cache.device
    if ws.device != dev:
        raise ValueError("the workspace is on another device")
    return _need("q", q, cache.dtype, cache.q_shape, dev), _need("out", out, torch.float32, cache.q_shape, dev)


def ckv_dense_decode_q8(cache: Q8Cache, q: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """out [B, Hq, d] fp32: attention of q [B, Hq, d] over each request's tokens."""
    qp, op = _q8_attention(cache, q, out, ws)
    _call("ckv_dense_decode_q8", lib.ckv_dense_decode_q8, cache.device, stream, cache.ref, qp, op, ws.data_ptr(),
          ws.numel())


def ckv_sparse_decode_q8(cache: Q8Cache, q: torch.Tensor, graph: Graph, sel: Selection, out: torch.Tensor,
                         nbr8: Optional[torch.Tensor], ws: torch.Tensor, k_new: Optional[torch.Tensor] = None,
                         assigned: Optional[torch.Tensor] = None, stream=None) -> None:
    """Attention over the selected positions; with k_new [B, Hkv, d] the new
    token also joins a community (ckv_sparse_decode_append without the rows)."""
    qp, op = _q8_attention(cache, q, out, ws)
    dev = cache.device
    U = cache.B * (cache.Hq if graph.desc.mode == PER_HEAD else cache.Hkv)
    if graph.U != U or sel.n_tok.shape[0] != U or graph.dev_err.device != dev or sel.sel_tok.device != dev:
        raise ValueError("the graph and the selection must be for this cache's batch and heads, on its device")
    kp = None if k_new is None else _need("k_new", k_new, cache.dtype, cache.row_shape, dev)
    np_ = None if nbr8 is None else _need("nbr8", nbr8, torch.int32, (graph.U, NEIGHBOURS), dev)
    ap = None if assigned is None else _need("assigned", assigned, torch.int32, (graph.U,), dev)
    _call("ckv_sparse_decode_q8", lib.ckv_sparse_decode_q8, dev, stream, cache.ref, qp, ctypes.byref(graph.desc),
          ctypes.byref(sel.desc), op, np_, kp, ap, ws.data_ptr(), ws.numel())


def _of_graph(cache: Q8Cache, graph: Graph) -> None:
    U = cache.B * (cache.Hq if graph.desc.mode == PER_HEAD else cache.Hkv)
    if graph.U != U or graph.dev_err.device != cache.device:
        raise ValueError("the graph must be for this cache's batch and heads, on its device")


def ckv_build_centroids_q8(cache: Q8Cache, labels: torch.Tensor, T: int, graph: Graph, ws: torch.Tensor,
                           which: Optional[torch.Tensor] = None, stream=None) -> None:
    """Community state from labels (int32 [U, >= T], T at least the longest request) over each request's own positions
    [0, len[b]); which (int32 [B]): only the requests that are not 0 there."""
    _of_graph(cache, graph)
    dev = cache.device
    if (labels.dtype is not torch.int32 or labels.dim() != 2 or labels.shape[0] != graph.U or labels.shape[1] < T
            or labels.stride(1) != 1 or labels.device != dev):
        raise ValueError(f"labels must be int32 [{graph.U}, >= {T}] on {dev} with contiguous rows")
    if ws.device != dev:
        raise ValueError("the workspace is on another device")
    wp = None if which is None else _need("which", which, torch.int32, cache.blocks.shape, dev)
    _call("ckv_build_centroids_q8", lib.ckv_build_centroids_q8, dev, stream, cache.ref, labels.data_ptr(),
          labels.stride(0) if graph.U > 1 else labels.shape[1], T, wp, ctypes.byref(graph.desc), ws.data_ptr(), ws.numel())


def ckv_trim_graph_q8(cache: Q8Cache, graph: Graph, stream=None) -> None:
    """Takes the tokens at or past each request's length out of its communities: after a ckv_plan_blocks that may have
    refused a joined token or dropped tokens, before the next ckv_score_select.  The graph needs new_graph(undo=True)."""
    _of_graph(cache, graph)
    _call("ckv_trim_graph_q8", lib.ckv_trim_graph_q8, cache.device, stream, cache.ref, ctypes.byref(graph.desc))
