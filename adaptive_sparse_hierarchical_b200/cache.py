"""Caches for serving over include/dash_cache.h: decode on a K/V cache held in 4 bits
(Q4DecodeState) and the pages that caches share (PagePool).  All arithmetic happens in the CUDA
kernels of libdash_b200.so."""
from __future__ import annotations

import contextlib

import torch

from . import _lib as L
from .api import _st

_CONTEXT = contextlib.nullcontext()


def _within(device, stream):
    """Context in which `device` is current and allocations and copies go to `stream` (None: the
    device's current stream)."""
    if stream is None:
        return _CONTEXT if torch.cuda.current_device() == device.index else torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


def _need(t, name, device, dtype, shape=None):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device:
        raise TypeError(f"{name}: a {dtype} tensor on {device} is needed")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(shape)} is needed, not {tuple(t.shape)}")
    return t


class Q4DecodeState:
    """PagedDecodeState with keys and values held in 4 bits (17/32 bytes per element, format in
    include/dash_cache.h): pools of codes [num_pages, h_kv, page_size, d / 2] and of e4m3 scales
    [num_pages, h_kv, page_size, d / 32].  Summaries and routing use the bf16 keys as they arrive.
    gamma = 0 makes decode a dense attention over the whole cache.

    k_exp, v_exp: power-of-two exponents of the data's size (scales cover 2^-9 .. 448 times 2^exp).
    page_table (device int32 [batch, max_pages]) may be rewritten between steps, by the caller or by
    a PagePool; without one, sequence b owns pages b * max_pages and on.  Copying the tensors saves
    or restores a session."""

    def __init__(self, batch, capacity, h_q, h_kv, d, *, chunk, alpha, gamma, page_size, num_pages=None,
                 page_table=None, k_exp=0, v_exp=0, inv_sigma=1.0, device="cuda", qbar=None):
        slots = (capacity + page_size - 1) // page_size
        if page_table is None:
            page_table = torch.arange(batch * slots, dtype=torch.int32).view(batch, slots)
        if num_pages is None:
            num_pages = batch * slots
        self.page_table = page_table.to(device=device, dtype=torch.int32).contiguous()
        self.device = self.page_table.device
        self.page_size = page_size
        new = dict(dtype=torch.uint8, device=self.device)
        self.k_codes = torch.zeros((num_pages, h_kv, page_size, d // 2), **new)
        self.v_codes = torch.zeros_like(self.k_codes)
        self.k_scales = torch.zeros((num_pages, h_kv, page_size, d // 32), **new)
        self.v_scales = torch.zeros_like(self.k_scales)
        self.T = capacity // chunk
        self.kbar = torch.zeros((batch, h_kv, self.T, d), dtype=torch.float32, device=self.device)
        self.state = torch.zeros((batch, h_kv, d + 2), dtype=torch.float32, device=self.device)
        self.state[..., d] = -torch.inf
        self.seqlens = torch.zeros(batch, dtype=torch.int32, device=self.device)
        self.qbar = qbar
        self.O = torch.empty((batch, h_q, d), dtype=torch.bfloat16, device=self.device)
        self._shape = dict(batch=batch, seqlen=capacity, h_q=h_q, h_kv=h_kv, d_h=d, chunk=chunk, alpha=alpha,
                           gamma=gamma, inv_sigma=inv_sigma, dtype=L.DASH_BF16)
        self.p = L.params(**self._shape)
        self._strided = {}
        self.kv = L.q4_kv(self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.page_table,
                          page_size=page_size, k_exp=k_exp, v_exp=v_exp)
        ws = L.dash_q4_workspace_size(self.p)
        self.workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=self.device)
        self.route = None

    def _tokens(self, t, name):
        """t as [batch, n, h_kv, d] with contiguous d."""
        s = self._shape
        if t.dim() == 3:
            t = t.unsqueeze(1)
        _need(t, name, self.device, torch.bfloat16, (s["batch"], t.shape[1], s["h_kv"], s["d_h"]))
        if t.stride(3) != 1:
            raise ValueError(f"{name}: the head dimension must be contiguous")
        return t

    def _params(self, k, v):
        key = (k.stride(), v.stride())
        p = self._strided.get(key)
        if p is None:
            if len(self._strided) > 64:
                self._strided.clear()
            p = self._strided[key] = L.params(**self._shape, k_strides=_st(k), v_strides=_st(v))
        return p

    def append(self, k_new, v_new, counts=None, stream=None):
        """Append k_new, v_new [batch, n, h_kv, d] (or [batch, h_kv, d]: one token): the first
        counts[b] (device int32; None: all n) tokens of each sequence, in 4 bits, and their summaries."""
        k, v = self._tokens(k_new, "k_new"), self._tokens(v_new, "v_new")
        if k.shape[1] != v.shape[1]:
            raise ValueError("k_new and v_new hold different numbers of tokens")
        if counts is not None and not _need(counts, "counts", self.device, torch.int32, self.seqlens.shape).is_contiguous():
            raise ValueError("counts must be contiguous")
        _need(self.qbar, "qbar", self.device, torch.float32, (self._shape["h_kv"], self._shape["d_h"]))
        with _within(self.device, stream):
            L.dash_append_q4(self._params(k, v), self.kv, k, v, k.shape[1], counts, self.qbar, self.kbar, self.state,
                             self.seqlens)

    def fill(self, K0, V0, lengths, stream=None):
        """Start over with the first lengths[b] tokens of K0, V0 [batch, n, h_kv, d]."""
        with _within(self.device, stream):
            lengths = torch.as_tensor(lengths, dtype=torch.int32).to(self.device)
            self.seqlens.zero_()
            self.append(K0, V0, lengths)

    def load(self, start, n, K=None, V=None, stream=None):
        """Positions start[b] .. start[b] + n - 1 (start: a number or device int32 [batch]) in bf16:
        K, V [batch, n, h_kv, d], zeros where nothing is cached."""
        s = self._shape
        per = isinstance(start, torch.Tensor)
        if per and not _need(start, "start", self.device, torch.int32, self.seqlens.shape).is_contiguous():
            raise ValueError("start must be contiguous")
        with _within(self.device, stream):
            if K is None:
                K = torch.empty((s["batch"], n, s["h_kv"], s["d_h"]), dtype=torch.bfloat16, device=self.device)
            if V is None:
                V = torch.empty((s["batch"], n, s["h_kv"], s["d_h"]), dtype=torch.bfloat16, device=self.device)
            K, V = self._tokens(K, "K"), self._tokens(V, "V")
            if K.shape[1] != n or V.shape[1] != n:
                raise ValueError(f"K and V must hold {n} tokens")
            L.dash_load_q4(self._params(K, V), self.kv, start if per else None, 0 if per else start, n, self.seqlens, K, V)
        return K, V

    def decode(self, q, stream=None):
        """Attention of the query q [batch, h_q, d] of each sequence's last token; zeros for an empty one."""
        _need(q, "q", self.device, torch.bfloat16, self.O.shape)
        if not q.is_contiguous():
            raise ValueError("q must be contiguous")
        with _within(self.device, stream):
            L.dash_decode_q4(self.p, self.kv, q, self.kbar, self.seqlens, self.O, self.route, self.workspace)
        return self.O

    def step(self, q, k_new, v_new, stream=None):
        self.append(k_new, v_new, stream=stream)
        return self.decode(q, stream)

    def graph_step(self, q, k_new, v_new):
        """step() through a CUDA graph: the first call runs eagerly and records append + decode on
        static input buffers; later calls copy the inputs in and replay (lengths and page table are
        read on the device, so one graph serves every step)."""
        if getattr(self, "_graph", None) is None:
            out = self.step(q, k_new, v_new)
            self._ins = [t.clone(memory_format=torch.contiguous_format) for t in (q, k_new, v_new)]
            self._graph = torch.cuda.CUDAGraph()
            with torch.cuda.device(self.device), torch.cuda.graph(self._graph):
                self.step(*self._ins)
            return out
        for mine, t in zip(self._ins, (q, k_new, v_new)):
            mine.copy_(t)
        self._graph.replay()
        return self.O


class PagePool:
    """The pages that the sequences (rows) of one or more caches share: page_table [batch, max_pages]
    (-1: no page), refs [num_pages] (table entries that hold a page, 0: free) and seqlens [batch],
    device int32 tensors that are changed in place.  add() registers what pages and rows hold; every
    operation is enqueued on the current stream (or `stream`) and works on the device alone, so it can
    be captured into a CUDA graph.  A request that cannot be met changes nothing and leaves its reason
    in `status`, which check() raises."""

    REASONS = {1: "an index is outside its range, or a page is missing", 2: "a destination occurs twice or is also a source",
               3: "a destination row is not empty", 4: "not enough free pages", 5: "a length is beyond the row's pages"}

    def __init__(self, page_table, refs, seqlens, *, page_size):
        self.device = page_table.device
        for t, name, dim in ((page_table, "page_table", 2), (refs, "refs", 1), (seqlens, "seqlens", 1)):
            _need(t, name, self.device, torch.int32)
            if t.dim() != dim or not t.is_contiguous():
                raise ValueError(f"{name}: a contiguous tensor of {dim} dimensions is needed")
        if seqlens.shape[0] != page_table.shape[0]:
            raise ValueError("page_table and seqlens have different numbers of rows")
        self.page_table, self.refs, self.seqlens, self.page_size = page_table, refs, seqlens, page_size
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.used = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._arrays, self._rows, self._kept = [], [], []
        self._describe()
        ws = L.dash_pages_workspace_size(self.pg)
        self.workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=self.device)

    @classmethod
    def of(cls, states):
        """A pool for the caches `states` (PagedDecodeState or Q4DecodeState, one per layer) that were
        made with one shared page table; pages named in the table count as held."""
        first = states[0]
        num = min((s.k_codes if isinstance(s, Q4DecodeState) else s.K).shape[0] for s in states)
        held = first.page_table.long()
        refs = torch.zeros(num + 1, dtype=torch.int32, device=held.device)
        at = torch.where((held >= 0) & (held < num), held, num).flatten()
        refs.scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
        pool = cls(first.page_table, refs[:num].contiguous(), first.seqlens, page_size=first.page_size)
        for s in states:
            pool.add(s)
        return pool

    def _describe(self):
        self.pg = L.pages(self.page_table, self.refs, self.seqlens, page_size=self.page_size, arrays=self._arrays,
                          rows=self._rows)

    def add(self, state):
        """Register a cache: its pools, summaries, incomplete-chunk states and lengths."""
        if state.page_table.data_ptr() != self.page_table.data_ptr() or state.page_size != self.page_size:
            raise ValueError("the cache must have been made with this pool's page table and page size")
        pools = [state.k_codes, state.k_scales, state.v_codes, state.v_scales] if isinstance(state, Q4DecodeState) \
            else [state.K, state.V]
        for t in pools:
            self.add_pages(t)
        self.add_rows(state.kbar, unit_tokens=state.p.chunk)
        self.add_rows(state.state)
        if state.seqlens.data_ptr() != self.seqlens.data_ptr():
            self.add_rows(state.seqlens, clear=True)

    def add_pages(self, t):
        """Register a pool tensor [num_pages, ...] with contiguous pages."""
        if t.device != self.device or t.dim() < 2 or t.shape[0] < self.refs.shape[0] or not t[0].is_contiguous():
            raise ValueError("a pool is a tensor [num_pages, ...] with contiguous pages on the pool's device")
        e = t.element_size()
        self._register(t, self._arrays, L.dash_page_array(t.data_ptr(), t[0].numel() * e, t.stride(0) * e))

    def add_rows(self, t, unit_tokens=0, clear=False):
        """Register a tensor [batch, ...] with contiguous rows that fork copies, or, with unit_tokens, a
        tensor [batch, heads, units, ...] of which fork copies the first length // unit_tokens units.
        clear: free sets the rows to zero."""
        if t.device != self.device or t.shape[0] != self.page_table.shape[0]:
            raise ValueError("rows are a tensor [batch, ...] on the pool's device")
        e = t.element_size()
        if t.numel() == 0:
            return
        if unit_tokens:
            if t.dim() < 3 or not t[0, 0].is_contiguous():
                raise ValueError("a tensor [batch, heads, units, ...] with contiguous runs of units is needed")
            row = L.dash_row_array(t.data_ptr(), t.stride(0) * e, t.stride(1) * e, t[0, 0, 0].numel() * e, t.shape[1],
                                   t.shape[2], unit_tokens, clear)
        else:
            if not t[0].is_contiguous():
                raise ValueError("contiguous rows are needed")
            row = L.dash_row_array(t.data_ptr(), t.stride(0) * e, t[0].numel() * e, t[0].numel() * e, 1, 1, 0, clear)
        self._register(t, self._rows, row)

    def _register(self, t, entries, entry):
        entries.append(entry)
        self._describe()
        if L.dash_pages_workspace_size(self.pg) == 0:   # the library refuses the description
            entries.pop()
            self._describe()
            raise ValueError("sizes and strides of pages must be multiples of 16 bytes, those of rows of 4 bytes, "
                             "and rows must not overlap")
        self._kept.append(t)

    def _list(self, v, name):
        if isinstance(v, torch.Tensor):
            if v.dim() != 1 or not _need(v, name, self.device, torch.int32).is_contiguous():
                raise ValueError(f"{name}: a contiguous list is needed")
            return v
        return torch.tensor(list(v), dtype=torch.int32).to(self.device)

    def _pair(self, src, dst):
        src, dst = self._list(src, "src"), self._list(dst, "dst")
        if src.shape != dst.shape:
            raise ValueError("src and dst have different lengths")
        return src, dst

    def copy(self, src, dst, stream=None):
        """Copy the contents of pages src[i] to pages dst[i] (lists or device int32) in every pool."""
        with _within(self.device, stream):
            src, dst = self._pair(src, dst)
            L.dash_pages_copy(self.pg, src, dst, src.shape[0], self.status, self.workspace, self.workspace.shape[0])

    def reserve(self, count=1, stream=None):
        """Give rows the pages they lack for `count` more tokens (a number, or device int32 [batch])."""
        with _within(self.device, stream):
            per = None
            if isinstance(count, torch.Tensor):
                per, count = _need(count, "count", self.device, torch.int32, self.seqlens.shape), 0
                if not per.is_contiguous():
                    raise ValueError("count must be contiguous")
            L.dash_pages_reserve(self.pg, per, count, self.status, self.workspace, self.workspace.shape[0])

    def fork(self, src, dst, stream=None):
        """Make the empty rows dst[i] copies of the rows src[i]: full pages are shared, the last one is
        copied, summaries, states and lengths too."""
        with _within(self.device, stream):
            src, dst = self._pair(src, dst)
            L.dash_pages_fork(self.pg, src, dst, src.shape[0], self.status, self.workspace, self.workspace.shape[0])

    def free(self, rows, stream=None):
        """Empty the rows: pages nobody else holds become free."""
        with _within(self.device, stream):
            rows = self._list(rows, "rows")
            L.dash_pages_free(self.pg, rows, rows.shape[0], self.status)

    def compact(self, stream=None):
        """Move the used pages together at the front of the pools; returns their number (device int32)."""
        with _within(self.device, stream):
            L.dash_pages_compact(self.pg, self.used, self.workspace, self.workspace.shape[0])
        return self.used

    def check(self):
        """Raise DashError if an operation since the last check could not be carried out (synchronises)."""
        code = int(self.status.item())
        if code:
            self.status.zero_()
            raise L.DashError(f"page operation: {self.REASONS.get(code, code)}")
