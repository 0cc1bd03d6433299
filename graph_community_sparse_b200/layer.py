"""Buffers and call sequence for one layer's CommunityKV decode state.

``LayerState`` owns (through PyTorch) the graph arrays, the selection and the
workspace for one KV cache, and issues the four library calls in decode
order.  ``PagedLayerState`` does the same over a paged 8-bit cache that requests
of different lengths share.  They compute nothing themselves.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import (ASSIGN_SCORE, ASSIGN_VOTE, PER_GROUP, PER_HEAD, Graph, Selection, cache_desc, ckv_append_assign, ckv_assign_update,
               ckv_sparse_decode_append,
               ckv_build_centroids, ckv_dense_decode, ckv_score_select, ckv_sparse_decode,
               ckv_workspace_size, new_graph, new_selection, new_workspace, NEIGHBOURS,
               CacheDesc, Plan, Q8Cache, ckv_build_centroids_q8, ckv_dense_decode_q8, ckv_plan_blocks, ckv_q8_read, ckv_q8_workspace_size,
               ckv_quant_append, ckv_sparse_decode_q8, ckv_trim_graph_q8, new_plan, q8_shape)


@contextlib.contextmanager
def _range(name: str):
    """An NVTX range around one library call, so that a profiler's timeline
    names the step's parts; a no-op when no profiler is attached."""
    torch.cuda.nvtx.range_push(name)
    try:
        yield
    finally:
        torch.cuda.nvtx.range_pop()


def _made_on(stream):
    """Tensors made inside are allocated and filled on the stream that the calls
    using them go to."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream)))


class LayerState:
    """K, V: [B, Hkv, T_cap, d] device tensors (bf16 or fp32), read in place.

    mode: "group" (one graph per KV group) or "head" (one graph per query head).
    tok_cap defaults to T_cap, which can never overflow.
    rule: how a new token picks among its neighbours' communities, "score"
    (best k . c) or "vote" (most neighbours, then the score).
    """

    def __init__(self, K: torch.Tensor, V: torch.Tensor, Hq: int, mode: str, S: int, Cmax: int,
                 max_tail: int, tok_cap: Optional[int] = None, rule: str = "score"):
        if rule not in ("score", "vote"):
            raise ValueError(f"unknown assignment rule {rule!r}")
        self.K, self.V = K, V
        self.cache = cache_desc(K, V, Hq)
        self.mode = PER_HEAD if mode == "head" else PER_GROUP
        self.graph: Graph = new_graph(self.cache, self.mode, S, Cmax, max_tail, device=K.device,
                                      rule=ASSIGN_VOTE if rule == "vote" else ASSIGN_SCORE)
        self.sel: Selection = new_selection(self.cache, self.graph, tok_cap or self.cache.T_cap,
                                            device=K.device)
        self.ws = new_workspace(ckv_workspace_size(self.cache, self.graph, self.sel), device=K.device)
        B, Hq_, d = self.cache.B, Hq, self.cache.d
        # the step's results share one allocation (out, then nbr8, then
        # assigned; all 4-byte types), so a caller reads them back with one copy
        n_out, U = B * Hq_ * d, self.graph.U
        self.results = torch.full((n_out + U * NEIGHBOURS + U,), -1, dtype=torch.int32, device=K.device)
        self.out = self.results[:n_out].view(torch.float32).view(B, Hq_, d)
        self.nbr8 = self.results[n_out: n_out + U * NEIGHBOURS].view(U, NEIGHBOURS)
        self.assigned = self.results[n_out + U * NEIGHBOURS:]
        self.T = 0

    @property
    def U(self) -> int:
        return self.graph.U

    def build(self, labels: torch.Tensor, T: int, stream=None) -> None:
        """labels: int32 [U, >=T] on the device."""
        with _range("ckv_build_centroids"):
            ckv_build_centroids(self.cache, labels, T, self.graph, self.ws, stream)
        self.T = T

    def select(self, q: torch.Tensor, budget: int, stream=None) -> None:
        with _range("ckv_score_select"):
            ckv_score_select(self.cache, self.graph, q, budget, self.sel, self.ws, stream)

    def attend(self, q: torch.Tensor, want_nbr: bool = True, stream=None) -> torch.Tensor:
        with _range("ckv_sparse_decode"):
            ckv_sparse_decode(self.cache, q, self.graph, self.sel, self.out,
                              self.nbr8 if want_nbr else None, self.ws, stream)
        return self.out

    def decode(self, q: torch.Tensor, budget: int, want_nbr: bool = True, stream=None) -> torch.Tensor:
        self.select(q, budget, stream)
        return self.attend(q, want_nbr, stream)

    def attend_append(self, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> torch.Tensor:
        """attend (neighbours into nbr8) and append in one call: the update
        runs inside the attention's merge kernel."""
        pos = self.T
        with _range("ckv_sparse_decode_append"):
            ckv_sparse_decode_append(self.cache, q, self.graph, self.sel, self.out, self.nbr8, pos,
                                     k_new.contiguous(), v_new.contiguous(), self.assigned, self.ws, stream)
        self.T += 1
        return self.out

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> torch.Tensor:
        """Write the new token's K/V rows ([B, Hkv, d]) at position T and let
        it join a community: one library call (ckv_append_assign)."""
        pos = self.T
        with _range("ckv_append_assign"):
            ckv_append_assign(self.cache, self.graph, pos, k_new.contiguous(), v_new.contiguous(), self.nbr8,
                              self.assigned, stream)
        self.T += 1
        return self.assigned

    def append_external(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> torch.Tensor:
        """Same result for a caller that writes the cache itself: the rows are
        copied with PyTorch, then ckv_assign_update reads the key from K."""
        pos = self.T
        self.K[:, :, pos].copy_(k_new)
        self.V[:, :, pos].copy_(v_new)
        with _range("ckv_assign_update"):
            ckv_assign_update(self.cache, self.graph, pos, self.nbr8, self.assigned, stream)
        self.T += 1
        return self.assigned

    def dense(self, q: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        out = torch.empty_like(self.out) if out is None else out
        with _range("ckv_dense_decode"):
            ckv_dense_decode(self.cache, q, self.T, out, self.ws, stream)
        return out


class PagedLayerState:
    """One layer's decode state over a paged 8-bit cache (`cache`, from
    new_q8_cache) that up to cache.B requests share.

    grow() takes slots for new tokens, or gives blocks back; write() quantises
    the new tokens' rows into them; dense() attends to every token.  With Cmax > 0
    it also holds community graphs over positions [0, T_cap): build(), select()
    and attend() are LayerState's, over this cache.  A decode step with graphs is
    select, attend (with the new keys, which join communities), grow, write.
    Joins are undone by the grow() that refuses their token, adds none, or gives
    it back later; a request that falls below the positions its communities were
    built over loses them (DEVERR_CUT, unless it ended) until the next build().
    What undoing takes is kept for the tail: max_tail centres (fp32) a graph unit.
    grow()'s plan buffers are used again by the next grow() of as many rows; those
    of more than KEEP_ROWS rows only live until a grow() of another number.
    """

    KEEP_ROWS = 4096

    def __init__(self, cache: Q8Cache, mode: str = "group", S: int = 0, Cmax: int = 0, max_tail: int = 0,
                 T_cap: int = 0, tok_cap: Optional[int] = None, rule: str = "score"):
        if rule not in ("score", "vote"):
            raise ValueError(f"unknown assignment rule {rule!r}")
        self.cache = cache
        dev = cache.device
        self.out = torch.empty(cache.q_shape, dtype=torch.float32, device=dev)
        self.plan: Optional[Plan] = None
        self._plans = {}  # by their number of rows, up to KEEP_ROWS: a decode step, captured or not, uses the same one again
        self.graph = self.sel = None
        if Cmax > 0:
            self.shape: CacheDesc = q8_shape(cache, T_cap)
            self.graph = new_graph(self.shape, PER_HEAD if mode == "head" else PER_GROUP, S, Cmax, max_tail, device=dev,
                                   rule=ASSIGN_VOTE if rule == "vote" else ASSIGN_SCORE, undo=True)
            self.sel = new_selection(self.shape, self.graph, tok_cap or T_cap, device=dev)
            self.nbr8 = torch.full((self.graph.U, NEIGHBOURS), -1, dtype=torch.int32, device=dev)
            self.assigned = torch.full((self.graph.U,), -1, dtype=torch.int32, device=dev)
            self.graph_ws = new_workspace(ckv_workspace_size(self.shape, self.graph, self.sel), device=dev)
        self.ws = new_workspace(ckv_q8_workspace_size(cache, self.graph, self.sel), device=dev)

    def grow(self, add: torch.Tensor, rows: int, stream=None) -> Plan:
        """Request b changes by add[b] tokens (int32 [B] on the device); rows
        bounds the tokens that this call may add.  The graphs follow."""
        plan = self._plans.get(rows)
        if plan is None and self.plan is not None and self.plan.n_rows == rows:
            plan = self.plan
        if plan is None:
            with _made_on(stream):
                plan = new_plan(self.cache, rows)
            if rows <= self.KEEP_ROWS:
                self._plans[rows] = plan
        with _range("ckv_plan_blocks"):
            ckv_plan_blocks(self.cache, add, plan, stream)
        self.plan = plan
        if self.graph is not None:
            with _range("ckv_trim_graph_q8"):
                ckv_trim_graph_q8(self.cache, self.graph, stream)
        return plan

    def write(self, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> None:
        """The rows of the last grow(): packed [rows, Hkv, d] or padded [B, T, Hkv, d]."""
        if self.plan is None:
            raise RuntimeError("write() follows grow()")
        with _range("ckv_quant_append"):
            ckv_quant_append(self.cache, self.plan, k_new, v_new, stream)

    def read(self, R: int, first: Optional[torch.Tensor] = None, stream=None):
        """Positions first[b] .. first[b] + R - 1 of every request as [B, Hkv, R, d] pairs."""
        c = self.cache
        with _made_on(stream):
            k = torch.empty((c.B, c.Hkv, R, c.d), dtype=c.dtype, device=c.device)
            v = torch.empty_like(k)
        with _range("ckv_q8_read"):
            ckv_q8_read(c, k, v, first, stream)
        return k, v

    def dense(self, q: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        out = self.out if out is None else out
        with _range("ckv_dense_decode_q8"):
            ckv_dense_decode_q8(self.cache, q, out, self.ws, stream)
        return out

    def build(self, labels: torch.Tensor, T: Optional[int] = None, requests: Optional[torch.Tensor] = None,
              stream=None) -> None:
        """Community state from labels (int32 [U, >= T], T at least the longest
        request) over each request's own positions; the centres are those of the
        values held.  requests (int32 [B] on the device): only those that are not 0
        there, e.g. a new one in the row of one that ended."""
        with _range("ckv_build_centroids_q8"):
            ckv_build_centroids_q8(self.cache, labels, labels.shape[1] if T is None else T, self.graph, self.graph_ws,
                                   requests, stream)

    def select(self, q: torch.Tensor, budget: int, stream=None) -> None:
        with _range("ckv_score_select"):
            ckv_score_select(self.shape, self.graph, q, budget, self.sel, self.graph_ws, stream)

    def attend(self, q: torch.Tensor, k_new: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention over the selection; with k_new the new tokens also join
        communities (nbr8, assigned), each at its request's length."""
        with _range("ckv_sparse_decode_q8"):
            if k_new is None:
                ckv_sparse_decode_q8(self.cache, q, self.graph, self.sel, self.out, None, self.ws, stream=stream)
            else:
                ckv_sparse_decode_q8(self.cache, q, self.graph, self.sel, self.out, self.nbr8, self.ws, k_new,
                                     self.assigned, stream)
        return self.out
