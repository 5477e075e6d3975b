"""Caches for serving over include/dash_cache.h: decode on a K/V cache held in 4 bits
(Q4DecodeState) and the pages that caches share (PagePool).  All arithmetic happens in the CUDA
kernels of libdash_b200.so."""
from __future__ import annotations

import torch

from . import _lib as L
from .api import _st, _table


def _current(index):
    """Raw handle of device `index`'s current stream."""
    return torch._C._cuda_getCurrentRawStream(index)


def _within(device, stream):
    """Context in which `device` is current and allocations and copies go to `stream` (None: the
    device's current stream)."""
    if stream is None:
        return torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


def _elsewhere(index, stream):
    """Whether a call must first make another device or stream current."""
    return stream is not None or torch._C._cuda_getDevice() != index


def _need(t, name, device, dtype, shape=None):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device:
        raise TypeError(f"{name}: a {dtype} tensor on {device} is needed")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(shape)} is needed, not {tuple(t.shape)}")
    return t


def _int32(v, name):
    """A number that a C int holds (anything else would be cut down silently)."""
    if not -2**31 <= v < 2**31:
        raise ValueError(f"{name}: {v} does not fit 32 bits")
    return v


def _signature(t):
    """What the checks of an argument depend on."""
    return (t.shape, t.stride(), t.dtype, t.device) if isinstance(t, torch.Tensor) else type(t)


class Q4DecodeState:
    """PagedDecodeState with keys and values held in 4 bits (17/32 bytes per element, format in
    include/dash_cache.h): pools of codes [num_pages, h_kv, page_size, d / 2] and of e4m3 scales
    [num_pages, h_kv, page_size, d / 32].  Summaries and routing use the bf16 keys as they arrive.
    gamma = 0 makes decode a dense attention over the whole cache.

    k_exp, v_exp: power-of-two exponents of the data's size (scales cover 2^-9 .. 448 times 2^exp).
    page_table (device int32 [batch, max_pages]) may be rewritten between steps, by the caller or by
    a PagePool; without one, sequence b owns pages b * max_pages and on.  Copying the tensors saves
    or restores a session.  Tokens are written from seqlens on: a row whose pages another row shares
    is not to be moved back by hand.  Calls share the cache's workspace and output, so they go to one stream at
    a time (graphs of one cache are replayed one after another)."""

    def __init__(self, batch, capacity, h_q, h_kv, d, *, chunk, alpha, gamma, page_size, num_pages=None,
                 page_table=None, k_exp=0, v_exp=0, inv_sigma=1.0, device="cuda", qbar=None):
        slots = (capacity + page_size - 1) // page_size
        if page_table is None:
            page_table = torch.arange(batch * slots, dtype=torch.int32).view(batch, slots)
        if num_pages is None:
            num_pages = batch * slots
        _table(page_table, batch)
        self.page_table = page_table.to(device=device, dtype=torch.int32).contiguous()
        self.device = self.page_table.device
        self._index = self.device.index
        self._lib = L.load()
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
        self.O = torch.empty((batch, h_q, d), dtype=torch.bfloat16, device=self.device)
        self._shape = dict(batch=batch, seqlen=capacity, h_q=h_q, h_kv=h_kv, d_h=d, chunk=chunk, alpha=alpha,
                           gamma=gamma, inv_sigma=inv_sigma, dtype=L.DASH_BF16)
        self.p = L.params(**self._shape)
        self.qbar = qbar
        self._seen = {}   # arguments that passed the checks, by signature: their parameters
        self.kv = L.q4_kv(self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.page_table,
                          page_size=page_size, k_exp=k_exp, v_exp=v_exp)
        ws = L.dash_q4_workspace_size(self.p)
        self.workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=self.device)
        self._ws_bytes = self.workspace.shape[0]
        self.route = None
        self._held = None       # refs and status of the PagePool that the cache belongs to
        self._recorded = {}     # graph_step, by the number of inputs: graph, inputs, what it was recorded with

    @property
    def qbar(self):
        """The learned query of Stage 0, float32 [h_kv, d] (checked when it is set)."""
        return self._qbar

    @qbar.setter
    def qbar(self, q):
        s = self._shape
        if q is not None and not _need(q, "qbar", self.device, torch.float32, (s["h_kv"], s["d_h"])).is_contiguous():
            raise ValueError("qbar must be contiguous")
        self._qbar = q

    def _tokens(self, t, name):
        """t as [batch, n, h_kv, d] with contiguous d."""
        s = self._shape
        if isinstance(t, torch.Tensor) and t.dim() == 3:
            t = t.unsqueeze(1)
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise TypeError(f"{name}: a tensor [batch, tokens, h_kv, d] is needed")
        _need(t, name, self.device, torch.bfloat16, (s["batch"], t.shape[1], s["h_kv"], s["d_h"]))
        if t.stride(3) != 1:
            raise ValueError(f"{name}: the head dimension must be contiguous")
        return t

    def _rows(self, t, name):
        """t: int32 [batch], contiguous (or None)."""
        if t is not None and not _need(t, name, self.device, torch.int32, (self._shape["batch"],)).is_contiguous():
            raise ValueError(f"{name} must be contiguous")

    def _check(self, what, k, v, rows, name):
        """dash_params and token number for K/V arguments k, v and an int32 [batch] argument (or None)."""
        key = (what, _signature(k), _signature(v), _signature(rows))
        got = self._seen.get(key)
        if got is None:
            s = self._shape
            k4, v4 = self._tokens(k, "K"), self._tokens(v, "V")
            if k4.shape[1] != v4.shape[1]:
                raise ValueError("K and V hold different numbers of tokens")
            self._rows(rows, name)
            n = _int32(k4.shape[1], "tokens")
            got = self._remember(key, (L.params(**s, k_strides=_st(k4), v_strides=_st(v4)), n))
        return got

    def _remember(self, key, value):
        if len(self._seen) > 64:
            self._seen.clear()
        self._seen[key] = value
        return value

    def append(self, k_new, v_new, counts=None, stream=None):
        """Append k_new, v_new [batch, n, h_kv, d] (or [batch, h_kv, d]: one token): the first
        counts[b] (device int32; None: all n) tokens of each sequence, in 4 bits, and their summaries."""
        if _elsewhere(self._index, stream):
            with _within(self.device, stream):
                return self.append(k_new, v_new, counts)
        p, n = self._check("append", k_new, v_new, counts, "counts")
        self._append(p, n, k_new, v_new, counts)

    def _append(self, p, n, k_new, v_new, counts):
        q = self._qbar
        if q is None:
            raise TypeError("qbar is needed")
        rc = self._lib.dash_append_q4(p, self.kv, k_new.data_ptr(), v_new.data_ptr(), n,
                                      None if counts is None else counts.data_ptr(), q.data_ptr(), self.kbar.data_ptr(),
                                      self.state.data_ptr(), self.seqlens.data_ptr(), _current(self._index))
        if rc:
            L._check(rc, "dash_append_q4")

    def fill(self, K0, V0, lengths, stream=None):
        """Start over with the first lengths[b] tokens of K0, V0 [batch, n, h_kv, d], in the pages that the
        table holds.  Where a PagePool counts another row on one of those pages, nothing changes and the
        pool's check() tells (free the rows first, and reserve their pages anew)."""
        with _within(self.device, stream):
            lengths = torch.as_tensor(lengths, dtype=torch.int32).to(self.device).contiguous()
            p, n = self._check("append", K0, V0, lengths, "lengths")
            self._append(p, 0, K0, V0, lengths)   # no tokens: the library's checks, before anything changes
            if self._held is None:
                self.seqlens.zero_()
            else:
                refs, status = self._held
                ends = (lengths.clamp(0, min(n, self._shape["seqlen"])) + (self.page_size - 1)) // self.page_size
                table = self.page_table[:lengths.shape[0]]
                written = torch.arange(table.shape[1], device=self.device) < ends[:, None]
                pages = torch.where(written & (table >= 0) & (table < refs.shape[0]), table, -1).long()
                shared = ((pages >= 0) & (refs[pages.clamp(min=0)] > 1)).any()
                status.copy_(torch.where(shared & (status == 0), PagePool.SHARED, status))
                self.seqlens.mul_(shared)
                lengths = lengths * ~shared
            self._append(p, n, K0, V0, lengths)

    def load(self, start, n, K=None, V=None, stream=None):
        """Positions start[b] .. start[b] + n - 1 (start: a number or device int32 [batch]) in bf16:
        K, V [batch, n, h_kv, d], zeros where nothing is cached."""
        if _elsewhere(self._index, stream):
            with _within(self.device, stream):
                return self.load(start, n, K, V)
        rows = start if isinstance(start, torch.Tensor) else None
        if K is None and V is None:   # outputs of one's own need no checks
            got = self._seen.get(n)
            if got is None:
                s = self._shape
                like = self.O.new_empty(1).expand(s["batch"], n, s["h_kv"], s["d_h"])
                strides = (n * s["h_kv"] * s["d_h"], s["h_kv"] * s["d_h"], s["d_h"])
                got = self._remember(n, (like, L.params(**s, k_strides=strides, v_strides=strides)))
            like, p = got
            K = torch.empty_like(like, memory_format=torch.contiguous_format)
            V = torch.empty_like(like, memory_format=torch.contiguous_format)
            if _signature(rows) != self._seen.get("start"):
                self._rows(rows, "start")
                self._seen["start"] = _signature(rows)
        else:
            if K is None:
                K = torch.empty_like(V, memory_format=torch.contiguous_format)
            if V is None:
                V = torch.empty_like(K, memory_format=torch.contiguous_format)
            p, m = self._check("load", K, V, rows, "start")
            if m != n:
                raise ValueError(f"K and V must hold {n} tokens")
        rc = self._lib.dash_load_q4(p, self.kv, None if rows is None else rows.data_ptr(),
                                    0 if rows is not None else _int32(start, "start"), n, self.seqlens.data_ptr(),
                                    K.data_ptr(), V.data_ptr(), _current(self._index))
        if rc:
            L._check(rc, "dash_load_q4")
        return K, V

    def _query(self, q):
        if _signature(q) != self._seen.get("q"):
            if not _need(q, "q", self.device, torch.bfloat16, self.O.shape).is_contiguous():
                raise ValueError("q must be contiguous")
            self._seen["q"] = _signature(q)

    def decode(self, q, stream=None):
        """Attention of the query q [batch, h_q, d] of each sequence's last token; zeros for an empty one."""
        if _elsewhere(self._index, stream):
            with _within(self.device, stream):
                return self.decode(q)
        self._query(q)
        rc = self._lib.dash_decode_q4(self.p, self.kv, q.data_ptr(), self.kbar.data_ptr(), self.seqlens.data_ptr(),
                                      self.O.data_ptr(), self.route, self.workspace.data_ptr(), self._ws_bytes,
                                      _current(self._index))
        if rc:
            L._check(rc, "dash_decode_q4")
        return self.O

    def step(self, q, k_new, v_new, stream=None, counts=None):
        """append(k_new, v_new, counts), then decode(q): rows whose count is 0 take no token (and need
        no page for it); their outputs are those of their last token."""
        self._query(q)   # a query that decode would refuse: nothing is appended
        if q.data_ptr() % 16:
            raise L.DashError("dash_decode_q4: q must be 16-byte aligned")
        self.append(k_new, v_new, counts, stream)
        return self.decode(q, stream)

    def graph_step(self, q, k_new, v_new, counts=None):
        """step() through a CUDA graph: the first call runs eagerly and records append + decode on
        static input buffers; later calls copy the inputs in and replay (lengths and page table are
        read on the device, so one graph serves every step, and one more every step with counts).  A
        call that finds qbar, route or another of the tensors and descriptions that a step takes its
        addresses from replaced does as the first."""
        takes = (self._qbar, self.kbar, self.state, self.seqlens, self.O, self.workspace)
        described = (bytes(self.p), bytes(self.kv), None if self.route is None else bytes(self.route))
        args = (q, k_new, v_new) if counts is None else (q, k_new, v_new, counts)
        got = self._recorded.get(len(args))
        if got is None or got[3] != described or any(a is not b for a, b in zip(got[2], takes)):
            out = self.step(q, k_new, v_new, counts=counts)
            ins = [t.clone(memory_format=torch.contiguous_format) for t in args]
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.device(self.device), torch.cuda.graph(graph):
                self.step(*ins[:3], counts=None if counts is None else ins[3])
            self._recorded[len(args)] = graph, ins, takes, described   # (the graph keeps what it takes alive)
            return out
        graph, ins = got[:2]
        if counts is not None:
            self._rows(counts, "counts")
        for mine, t in zip(ins, args):
            if t.shape != mine.shape or t.dtype != mine.dtype:
                raise ValueError(f"the graph was recorded for {mine.dtype} {tuple(mine.shape)}")
        for mine, t in zip(ins, args):
            mine.copy_(t)
        graph.replay()
        return self.O


class PagePool:
    """The pages that the sequences (rows) of one or more caches share: page_table [batch, max_pages]
    (-1: no page), refs [num_pages] (table entries that hold a page, 0: free) and seqlens [batch],
    device int32 tensors that are changed in place.  add() registers what pages and rows hold; every
    operation is enqueued on the current stream (or `stream`) and works on the device alone, so it can
    be captured into a CUDA graph.  A request that cannot be met changes nothing and leaves its reason
    in `status`, which check() raises.  Operations share the pool's workspace and tables, so they go to
    one stream at a time."""

    REASONS = {1: "an index is outside its range, or a page is missing", 2: "a destination occurs twice or is also a source",
               3: "a destination row is not empty", 4: "not enough free pages", 5: "a length is beyond the row's pages",
               6: "a page to be filled is held by another row too"}
    SHARED = 6   # (set by the caches' fill; the others are the library's)

    def __init__(self, page_table, refs, seqlens, *, page_size):
        self.device = page_table.device
        self._index = self.device.index
        self._lib = L.load()
        self._seen = {}
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
        self._ws = (self.workspace.data_ptr(), self.workspace.shape[0])

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
        s = state.state
        if s.stride(2) != 1:
            raise ValueError("the incomplete-chunk state must be contiguous")
        before = len(self._arrays), len(self._rows), len(self._kept)
        try:
            for t in pools:
                self.add_pages(t)
            self.add_rows(state.kbar, unit_tokens=state.p.chunk)
            self._register(s, self._rows, L.dash_row_array(s.data_ptr(), s.stride(0) * 4, s.stride(1) * 4, s.shape[2] * 4,
                                                           s.shape[1], 1, 0, L.DASH_ROW_STATE))
            if state.seqlens.data_ptr() != self.seqlens.data_ptr():
                self.add_rows(state.seqlens, clear=True)
        except Exception:   # all of a cache or nothing of it
            for kept, n in zip((self._arrays, self._rows, self._kept), before):
                del kept[n:]
            self._describe()
            raise
        state._held = self.refs, self.status   # fill asks them

    def add_pages(self, t):
        """Register a pool tensor [num_pages, ...] with contiguous pages."""
        if t.device != self.device or t.dim() < 2 or t.shape[0] < self.refs.shape[0] or not t[0].is_contiguous():
            raise ValueError("a pool is a tensor [num_pages, ...] with contiguous pages on the pool's device")
        e = t.element_size()
        self._register(t, self._arrays, L.dash_page_array(t.data_ptr(), t[0].numel() * e, t.stride(0) * e))

    def add_rows(self, t, unit_tokens=0, clear=False):
        """Register a tensor [batch, ...] with contiguous rows that fork copies, or, with unit_tokens, a
        tensor [batch, heads, units, ...] of which fork copies the first length // unit_tokens units.
        clear: free sets the rows to zero (otherwise they stay)."""
        if t.device != self.device or t.shape[0] != self.page_table.shape[0]:
            raise ValueError("rows are a tensor [batch, ...] on the pool's device")
        e, clear = t.element_size(), L.DASH_ROW_ZERO if clear else L.DASH_ROW_KEPT
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
        """A list of indices as a device int32 tensor."""
        if not isinstance(v, torch.Tensor):
            return torch.tensor(list(v), dtype=torch.int32).to(self.device)
        if self._seen.get(name) != _signature(v):
            if v.dim() != 1 or not _need(v, name, self.device, torch.int32).is_contiguous():
                raise ValueError(f"{name}: a contiguous list is needed")
            self._seen[name] = _signature(v)
        return v

    def _pair(self, call, name, src, dst):
        src, dst = self._list(src, "src"), self._list(dst, "dst")
        n = src.shape[0]
        if dst.shape[0] != n:
            raise ValueError("src and dst have different lengths")
        rc = call(self.pg, src.data_ptr(), dst.data_ptr(), n, self.status.data_ptr(), *self._ws, _current(self._index))
        if rc:
            L._check(rc, name)

    def copy(self, src, dst, stream=None):
        """Copy the contents of pages src[i] to pages dst[i] (lists or device int32) in every pool."""
        if _elsewhere(self._index, stream):
            with _within(self.device, stream):
                return self.copy(src, dst)
        self._pair(self._lib.dash_pages_copy, "dash_pages_copy", src, dst)

    def reserve(self, count=1, stream=None):
        """Give rows the pages they lack for their next `count` tokens (a number, or device int32 [batch]);
        slots before the next token's are left as they are."""
        if _elsewhere(self._index, stream):
            with _within(self.device, stream):
                return self.reserve(count)
        per = None
        if isinstance(count, torch.Tensor):
            per = self._list(count, "count")
            if per.shape != self.seqlens.shape:
                raise ValueError("count: one number per row is needed")
        rc = self._lib.dash_pages_reserve(self.pg, None if per is None else per.data_ptr(), 0 if per is not None else _int32(count, "count"),
                                          self.status.data_ptr(), *self._ws, _current(self._index))
        if rc:
            L._check(rc, "dash_pages_reserve")

    def fork(self, src, dst, stream=None):
        """Make the empty rows dst[i] copies of the rows src[i]: full pages are shared, the last one is
        copied, summaries, states and lengths too."""
        if _elsewhere(self._index, stream):
            with _within(self.device, stream):
                return self.fork(src, dst)
        self._pair(self._lib.dash_pages_fork, "dash_pages_fork", src, dst)

    def free(self, rows, stream=None):
        """Empty the rows: pages nobody else holds become free; registered caches can fill the rows anew."""
        if _elsewhere(self._index, stream):
            with _within(self.device, stream):
                return self.free(rows)
        rows = self._list(rows, "rows")
        rc = self._lib.dash_pages_free(self.pg, rows.data_ptr(), rows.shape[0], self.status.data_ptr(),
                                       _current(self._index))
        if rc:
            L._check(rc, "dash_pages_free")

    def compact(self, stream=None):
        """Move the used pages together at the front of the pools; returns their number (device int32)."""
        if _elsewhere(self._index, stream):
            with _within(self.device, stream):
                return self.compact()
        rc = self._lib.dash_pages_compact(self.pg, self.used.data_ptr(), *self._ws, _current(self._index))
        if rc:
            L._check(rc, "dash_pages_compact")
        return self.used

    def check(self):
        """Raise DashError if an operation since the last check could not be carried out, on whichever
        stream it went (waits for the device)."""
        torch.cuda.synchronize(self.device)
        code = int(self.status.item())
        if code:
            self.status.zero_()
            torch.cuda.synchronize(self.device)   # later operations, on any stream, find it cleared
            raise L.DashError(f"page operation: {self.REASONS.get(code, code)}")
