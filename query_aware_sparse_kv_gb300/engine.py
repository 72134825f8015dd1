"""Buffer plumbing around the three C-ABI calls for one paged KV cache.

``PagedDecoder`` owns the device buffers a decode step needs (metadata,
workspace, selection, outputs) and issues the calls in order.  It only
allocates and passes pointers; every step of the computation runs in
libqskv.so's kernels.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import binding as B


@contextlib.contextmanager
def _on(device, stream):
    """`device` and `stream` (a stream object, a raw handle as the library's calls take it, or None: the device's
    current one) for torch's own operations."""
    if stream is not None and not hasattr(stream, "cuda_stream"):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


class PagedDecoder:
    """One decode batch over a paged KV cache resident on the GPU.

    q           [batch][Hq][d]            fp32 or bf16
    k_pool      [Npool][Hkv][P][d]        fp32 or bf16 (v_pool the same)
    page_table  [batch][max_pages] int32  physical page ids
    seq_lens    [batch] int32
    top_k       pages kept per (sequence, KV head); None = dense decode
    prefix_pages  logical pages [0, prefix_pages) every row shares (the same
                physical pages): dense decodes then run as a cascade, the
                prefix attended once per KV head for the whole batch
    scorer      "bound" (TinyServe min/max metadata, the default) or
                "centroid" (Block Top-K: fp32 mean key per page, q . centroid)
    approx_epsilon  None: exact top-K; else the lossy top-K stops refining
                once at most floor(epsilon * top_k) pages are undecided and
                samples them from the threshold bucket (seed approx_seed)
    prefill_tokens  queries that a ``prefill`` may bring (0: none); the
                workspace then grows by room for parts of tiles, about 80 MB
                with 128 dims
    """

    def __init__(self, q, k_pool, v_pool, page_table, seq_lens, top_k: Optional[int], sm_scale: float = 0.0,
                 prefix_pages: int = 0, scorer: str = "bound", approx_epsilon: Optional[float] = None,
                 approx_seed: int = 0, prefill_tokens: int = 0):
        self.approx_epsilon, self.approx_seed = approx_epsilon, approx_seed
        if scorer not in ("bound", "centroid"):
            raise ValueError(f"unknown scorer {scorer!r}")
        dev = k_pool.device
        self.q, self.k_pool, self.v_pool = q, k_pool, v_pool
        self.page_table, self.seq_lens = page_table, seq_lens
        n_pool, hkv, P, d = k_pool.shape
        batch, hq, _ = q.shape
        self.top_k = top_k
        self.sm_scale = sm_scale
        self.shape = B.make_shape(batch, hq, hkv, d, P, page_table.shape[1], n_pool)
        self.prefix_pages = int(prefix_pages)
        self.scorer = scorer
        if scorer == "centroid":
            self.meta = torch.empty((n_pool, hkv, d), dtype=torch.float32, device=dev)
        else:
            self.meta = torch.empty((n_pool, hkv, 2, d), dtype=k_pool.dtype, device=dev)
        ws = B.workspace_size(self.shape)
        if self.prefix_pages > 0:
            ws = max(ws, B.cascade_workspace_size(self.shape, self.prefix_pages))
        self.prefill_tokens = int(prefill_tokens)
        if self.prefill_tokens > 0:
            ws = max(ws, B.prefill_workspace_size(self.shape, self.prefill_tokens))
        self.workspace = torch.zeros(ws, dtype=torch.uint8, device=dev)
        k = max(int(top_k or 1), 1)
        self.selected = torch.full((batch, hkv, k), -1, dtype=torch.int32, device=dev)
        self.n_selected = torch.zeros((batch, hkv), dtype=torch.int32, device=dev)
        self.out = torch.empty((batch, hq, d), dtype=torch.float32, device=dev)
        self.lse = torch.empty((batch, hq), dtype=torch.float32, device=dev)

    # -- cache phase ---------------------------------------------------------
    def build_meta(self, page_ids: torch.Tensor, valid_tokens: torch.Tensor, stream=None):
        if self.scorer == "centroid":
            B.kv_centroid_build(self.k_pool, page_ids, valid_tokens, self.meta, self.shape, self.workspace, stream)
        else:
            B.kv_meta_build(self.k_pool, page_ids, valid_tokens, self.meta, self.shape, self.workspace, stream)

    def prefill(self, q: torch.Tensor, cu_new: torch.Tensor, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Causal attention of the rows' newest tokens, whose keys and values
        are in the pools and counted by ``seq_lens``: row b's queries are
        q[cu_new[b]:cu_new[b + 1]] of q [T][Hq][d].  Into ``out`` (q's shape
        and type; zeros to begin with if none is given), which is returned.
        Precision goes by the types, as binding.paged_prefill says."""
        if q.shape[0] > self.prefill_tokens:
            raise ValueError(f"{q.shape[0]} queries, at most {self.prefill_tokens} a prefill (prefill_tokens)")
        if out is None:
            with _on(self.k_pool.device, stream):
                out = torch.zeros(q.shape, dtype=q.dtype, device=self.k_pool.device)
        B.paged_prefill(q, self.k_pool, self.v_pool, self.page_table, self.seq_lens, cu_new, out, self.shape,
                        self.workspace, lse=lse, sm_scale=self.sm_scale, stream=stream)
        return out

    # -- indexer phase -------------------------------------------------------
    @property
    def can_refresh_in_select(self) -> bool:
        """Whether select(refresh_last=True) runs as one launch (bound scorer,
        exact top-K, bf16 KV); otherwise it is a metadata build of the last
        pages followed by the selection."""
        return self.scorer == "bound" and self.approx_epsilon is None and self.k_pool.dtype == torch.bfloat16

    def select(self, q=None, scores: Optional[torch.Tensor] = None, stream=None, refresh_last: bool = False):
        """Top-K pages per (sequence, KV head).  refresh_last: first rebuild
        the metadata of every sequence's last page (the page the new token
        went into)."""
        if refresh_last and self.can_refresh_in_select:
            B.page_select_refresh(self.q if q is None else q, self.k_pool, self.meta, self.page_table, self.seq_lens,
                                  self.top_k, self.selected, self.n_selected, self.shape, self.workspace, scores,
                                  stream)
            return
        if refresh_last:
            self.build_meta(*self._last_pages(), stream)
        if self.approx_epsilon is not None:
            B.page_select_approx(self.q if q is None else q, self.meta, self.page_table, self.seq_lens, self.top_k,
                                 self.selected, self.n_selected, self.shape, self.workspace, self.approx_epsilon,
                                 self.approx_seed, scorer=self.scorer, scores=scores, stream=stream)
            return
        fn = B.page_select_centroid if self.scorer == "centroid" else B.page_select
        fn(self.q if q is None else q, self.meta, self.page_table, self.seq_lens, self.top_k, self.selected,
           self.n_selected, self.shape, self.workspace, scores, stream)

    def _last_pages(self):
        """(physical id, valid tokens) of every sequence's last page, gathered
        on the device from the page table and the lengths (plumbing for the
        two-call refresh; no arithmetic of the method)."""
        P = self.shape.page_size
        nb = torch.clamp((self.seq_lens.long() + P - 1) // P, min=1)
        ids = self.page_table.gather(1, (nb - 1)[:, None]).squeeze(1).to(torch.int32)
        valid = (self.seq_lens.long() - (nb - 1) * P).clamp(min=1).to(torch.int32)
        return ids, valid

    def decode(self, q=None, dense: bool = False, out=None, lse=None, stream=None):
        sel = None if (dense or self.top_k is None) else self.selected
        if sel is None and self.prefix_pages > 0:
            B.cascade_paged_decode(self.q if q is None else q, self.k_pool, self.v_pool, self.page_table,
                                   self.seq_lens, self.out if out is None else out, self.shape, self.workspace,
                                   self.prefix_pages, lse=self.lse if lse is None else lse, sm_scale=self.sm_scale,
                                   stream=stream)
            return
        B.sparse_paged_decode(self.q if q is None else q, self.k_pool, self.v_pool, self.page_table, self.seq_lens,
                              self.out if out is None else out, self.shape, self.workspace, selected=sel,
                              n_selected=self.n_selected if sel is not None else None,
                              top_k=self.top_k or 0, lse=self.lse if lse is None else lse, sm_scale=self.sm_scale,
                              stream=stream)

    def step(self, q=None, last_ids=None, last_valid=None, stream=None, out=None, refresh_last: bool = False):
        """Metadata refresh of the pages being appended to, selection, decode
        (into ``out`` if given, else ``self.out``).  The refresh is either
        the listed pages (last_ids, last_valid) or, with refresh_last, every
        sequence's last page inside the selection's launch; then, where the
        selection can take the refresh (bound scorer, exact top-K, bf16 KV),
        the whole step is one call (qskv_select_decode)."""
        if refresh_last and last_ids is None and self.top_k is not None and self.can_refresh_in_select:
            B.select_decode(self.q if q is None else q, self.k_pool, self.v_pool, self.meta, self.page_table,
                            self.seq_lens, self.top_k, self.selected, self.n_selected,
                            self.out if out is None else out, self.shape, self.workspace, lse=self.lse,
                            sm_scale=self.sm_scale, stream=stream)
            return
        if last_ids is not None:
            self.build_meta(last_ids, last_valid, stream)
        if self.top_k is not None:
            self.select(q, stream=stream, refresh_last=refresh_last)
        self.decode(q, out=out, stream=stream)

    def capture_step(self, q: torch.Tensor, last_ids=None, last_valid=None, q_host: Optional[torch.Tensor] = None,
                     out_host: Optional[torch.Tensor] = None, zero_copy: bool = True, refresh_last: bool = False):
        """Record one step (metadata refresh, selection, decode) reading the
        query from the device buffer `q` into a CUDA graph, and return a
        function that replays it on the current stream.  Refill `q` in place
        before each replay; results land in ``out`` / ``lse``.

        With pinned host tensors ``q_host`` (shaped like q) and/or
        ``out_host`` (shaped like out) the graph also moves the query in and
        the output out, so a serving loop launches one graph per step and
        synchronises once: a copy node brings ``q_host`` into ``q`` first
        (the scoring grid reads the query once per page chunk, so it is read
        from device memory), refill ``q_host`` before each replay.
        zero_copy=True (default): the decode writes the output straight into
        ``out_host`` (pinned host memory is device-accessible; on GB300 the
        NVLink-C2C link makes this faster than a copy node), and ``out`` is
        not written.  zero_copy=False: a copy node from ``out`` into
        ``out_host`` last."""
        def body():
            if q_host is not None:
                q.copy_(q_host, non_blocking=True)
            if zero_copy:
                self.step(q, last_ids, last_valid, out=out_host, refresh_last=refresh_last)
                return
            self.step(q, last_ids, last_valid, refresh_last=refresh_last)
            if out_host is not None:
                out_host.copy_(self.out, non_blocking=True)

        for t in (q_host, out_host):
            if t is not None and not t.is_pinned():
                raise ValueError("host buffers of a captured step must be pinned")
        if q_host is not None and (q_host.shape != q.shape or q_host.dtype != q.dtype):
            raise ValueError("q_host must have the shape and dtype of q")
        if out_host is not None and (out_host.shape != self.out.shape or out_host.dtype != self.out.dtype):
            raise ValueError("out_host must have the shape and dtype of out")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            body()  # first use outside capture (device set-up)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            body()
        return graph.replay

    def wait(self, stream=None):
        """Block the host until all work issued so far on ``stream`` (the
        current stream by default) has run, by polling an event recorded
        behind it (a busy wait on the host), which returns slightly sooner
        than a stream synchronisation; for serving loops that wait for every
        step's output."""
        st = torch.cuda.current_stream() if stream is None else stream
        ev = getattr(self, "_wait_event", None)
        if ev is None:
            ev = self._wait_event = torch.cuda.Event()
        ev.record(st)
        while not ev.query():
            pass

    def check(self, stream=None):
        """Raise if the device flagged an out-of-range index or a timeout."""
        st = B.get_error(self.workspace, stream)
        if st != 0:
            raise B.QskvError(st, B.last_error_message())


class QuantizedPagedDecoder:
    """A decode batch over a KV cache held in 4 or 8 bits, from lengths to outputs.

    Owns the pool (4 bits: codes with a bf16 scale and minimum per group of
    ``group_size`` dims; 8 bits: e4m3 codes with a power of two per token and
    head), its page metadata, the page table and the free pages.  A step is: ``extend`` (tables and slots of the new tokens),
    ``append`` (their keys and values quantised into the pool, the touched
    pages' metadata rebuilt), ``select`` (with top_k: the pages each query
    attends to) and ``decode``; ``step`` does all of it.  Row lengths are
    also kept on the host, so a step never waits for the GPU.  (The lengths
    come from the host: ``extend`` cannot be captured into a graph; the calls
    it makes can, see binding.extend_tables.)  Calls may go to any streams, as
    long as each waits for the work of the call before it.

    batch       rows (requests); a row of length 0 is free
    max_pages   pages a row may hold
    max_tokens  new tokens a step may bring, all rows together
    top_k       pages kept per (row, KV head); None = all
    bits        4 or 8 (group_size says nothing for 8; ``prefill`` needs 8,
                whose workspace has about 80 MB for it with 128 dims)
    """

    def __init__(self, batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int, max_pages: int,
                 num_pool_pages: int, group_size: int = 64, top_k: Optional[int] = None, max_tokens: int = 8192,
                 sm_scale: float = 0.0, device="cuda", bits: int = 4):
        if bits not in (4, 8):
            raise ValueError(f"bits must be 4 or 8 (got {bits})")
        if top_k is not None and top_k < 1:
            raise ValueError(f"top_k must be None (all pages) or >= 1 (got {top_k})")
        if max_tokens < 1:
            raise ValueError(f"max_tokens must be >= 1 (got {max_tokens})")
        if not 0 <= sm_scale < float("inf"):
            raise ValueError(f"sm_scale must be finite and >= 0 (got {sm_scale})")
        self.shape = B.make_shape(batch, num_q_heads, num_kv_heads, head_dim, page_size, max_pages, num_pool_pages)
        self.group_size, self.top_k, self.sm_scale, self.max_tokens = group_size, top_k, sm_scale, max_tokens
        self.bits = bits
        # the shape as the cache's calls take it, with the group size where there is one
        self._format = (self.shape, group_size) if bits == 4 else (self.shape,)
        block = B.kvq_block_bytes(*self._format) if bits == 4 else B.kvf_block_bytes(self.shape)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)  # noqa: E731
        self.pool = torch.zeros((num_pool_pages, num_kv_heads, block), dtype=torch.uint8, device=device)
        self.page_table = torch.full((batch, max_pages), -1, dtype=torch.int32, device=device)
        self.seq_lens, self._lens_out = i32(batch), i32(batch)
        # ids from _taken on are free; written in place, so that no storage goes back while a stream may still read it
        self._free, self._taken = torch.arange(num_pool_pages, dtype=torch.int32, device=device), 0
        self.cu_new, self.slot_map, self.positions = i32(batch + 1), i32(max_tokens), i32(max_tokens)
        touched = min(max_tokens, max_tokens // page_size + 2 * batch)
        self.touched_ids, self.touched_valid = i32(touched), i32(touched)
        with torch.cuda.device(self.pool.device):
            size = max(B.kvq_workspace_size(self.shape) if bits == 4 else B.kvf_workspace_size(self.shape),
                       B.prefill_workspace_size(self.shape, max_tokens) if bits == 8 else 0,
                       B.tables_workspace_size(self.shape),
                       B.workspace_size(self.shape) if top_k is not None else 0)
        self.workspace = torch.zeros(size, dtype=torch.uint8, device=device)
        if top_k is not None:
            self.meta = torch.zeros((num_pool_pages, num_kv_heads, 2, head_dim), dtype=torch.bfloat16, device=device)
            self.selected, self.n_selected = i32(batch, num_kv_heads, top_k), i32(batch, num_kv_heads)
        self.out = torch.zeros((batch, num_q_heads, head_dim), dtype=torch.float32, device=device)
        self.lse = torch.zeros((batch, num_q_heads), dtype=torch.float32, device=device)
        self.lengths = [0] * batch  # as of the last extend
        self._new = 0  # tokens of the last extend that append has not stored yet

    def _on(self, stream):
        """The decoder's device and `stream` for torch's own operations."""
        return _on(self.pool.device, stream)

    def _pages(self, tokens: int) -> int:
        return -(-tokens // self.shape.page_size)

    @property
    def free_pages(self) -> torch.Tensor:
        """The pages that no row holds (a view of the list, of which ``extend`` takes the first)."""
        return self._free[self._taken:]

    def extend(self, new_lens, stream=None):
        """Make room for new_lens[b] more tokens of every row b: page table,
        ``slot_map`` and ``positions`` of the new tokens (rows in order),
        ``touched_ids`` / ``touched_valid`` and the new ``seq_lens``.  Raises
        ValueError, changing nothing, if they do not fit."""
        new = [int(n) for n in new_lens]
        if len(new) != self.shape.batch or min(new) < 0:
            raise ValueError(f"new_lens must be {self.shape.batch} counts >= 0")
        if self._new:
            raise ValueError(f"{self._new} tokens of the last extend are not stored yet")
        if sum(new) > self.max_tokens:
            raise ValueError(f"{sum(new)} new tokens, at most {self.max_tokens} a step")
        grown = [a + n for a, n in zip(self.lengths, new)]
        for b, n in enumerate(grown):
            if n > self.shape.max_pages * self.shape.page_size:
                raise ValueError(f"row {b} would hold {n} tokens, more than its {self.shape.max_pages} pages")
        need = sum(self._pages(n) - self._pages(a) for a, n in zip(self.lengths, grown))
        if need > self.free_pages.numel():
            raise ValueError(f"{need} pages needed, {self.free_pages.numel()} free")
        with self._on(stream):
            added = torch.tensor(new, dtype=torch.int32).to(self.pool.device, non_blocking=True)
        B.extend_tables(self.seq_lens, added, self.free_pages, self.page_table, self._lens_out, self.cu_new,
                        self.slot_map, self.shape, self.workspace, positions=self.positions,
                        touched_ids=self.touched_ids, touched_valid=self.touched_valid, stream=stream)
        self.seq_lens, self._lens_out = self._lens_out, self.seq_lens
        self._taken += need
        self.lengths, self._new = grown, sum(new)

    def append(self, k: torch.Tensor, v: torch.Tensor, stream=None):
        """Store the keys and values [n][Hkv][d] of the tokens of the last
        ``extend`` (rows in order) and, with top_k, rebuild the metadata of
        the pages they fall into."""
        if k.shape[0] != self._new:
            raise ValueError(f"{k.shape[0]} keys for the {self._new} tokens of the last extend")
        store, meta_build = (B.kvq_append, B.kvq_meta_build) if self.bits == 4 else (B.kvf_append, B.kvf_meta_build)
        store(k, v, self.slot_map[:k.shape[0]], self.pool, *self._format, self.workspace, stream)
        if self.top_k is not None:
            meta_build(self.pool, self.touched_ids, self.touched_valid, self.meta, *self._format, self.workspace, stream)
        self._new = 0

    def _check_query(self, q: torch.Tensor):
        """Refuse what is not queries of every row, as the decode's own call does (the selection's takes any address)."""
        B._dtype(q)
        B._tensor("q", q, q.dtype, (self.shape.batch, self.shape.num_q_heads, self.shape.head_dim),
                  self.pool.get_device())
        if q.data_ptr() % 16:
            raise ValueError("q must be 16-byte aligned")

    def select(self, q: torch.Tensor, stream=None):
        """The top_k pages of every (row, KV head) by their score bound."""
        if self.top_k is None:
            raise ValueError("a decoder with top_k None attends to all pages and selects none")
        self._check_query(q)
        with torch.cuda.device(self.pool.device):
            B.page_select(q, self.meta, self.page_table, self.seq_lens, self.top_k, self.selected, self.n_selected,
                          self.shape, self.workspace, None, stream)

    def decode(self, q: torch.Tensor, out=None, lse=None, stream=None):
        """Attention of q [batch][Hq][d] over the selected (or all) pages,
        into ``out`` / ``lse``."""
        sparse = self.top_k is not None
        paged_decode = B.kvq_paged_decode if self.bits == 4 else B.kvf_paged_decode
        paged_decode(q, self.pool, self.page_table, self.seq_lens, self.out if out is None else out, *self._format,
                     self.workspace, selected=self.selected if sparse else None,
                     n_selected=self.n_selected if sparse else None, top_k=self.top_k or 0,
                     lse=self.lse if lse is None else lse, sm_scale=self.sm_scale, stream=stream)

    def step(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, new_lens=None, stream=None):
        """One step: the rows' new tokens (one each by default) stored, then
        the queries' attention over what the rows hold with them.  A step
        that is refused (ValueError, TypeError, QskvError) leaves lengths,
        pages and cache as they were."""
        self._check_query(q)
        with self._undone_if_refused():
            self.extend([1] * self.shape.batch if new_lens is None else new_lens, stream)
            self.append(k, v, stream)
            if self.top_k is not None:
                self.select(q, stream)
            self.decode(q, stream=stream)

    @contextlib.contextmanager
    def _undone_if_refused(self):
        """Lengths and pages as they were if a call within raises: of the table and the pool only places past a row's end
        are new then, and the metadata of a row's last page still bounds its keys."""
        names = ("lengths", "_taken", "_new", "seq_lens", "_lens_out")
        before = [getattr(self, name) for name in names]
        try:
            yield
        except Exception:
            for name, value in zip(names, before):
                setattr(self, name, value)
            raise

    def prefill(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, new_lens, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Prompts, or chunks of them: the rows' new tokens stored, then the
        causal attention of all of them, q [sum(new_lens)][Hq][d], over what
        the rows hold (8-bit caches; all pages, whatever top_k).  Into ``out``
        (q's shape and type), which is returned.  With bf16 queries softmax
        weights are rounded to bf16, which ``step`` does not do; fp32 queries
        give ``step``'s precision.  A call that is refused leaves lengths,
        pages and cache as they were."""
        if self.bits != 8:
            raise ValueError("prefill attends to 8-bit caches (bits=8)")
        new_lens = [int(x) for x in new_lens]
        n, s = sum(new_lens), self.shape
        B._dtype(q)
        B._rows("q", q, q.dtype, n, s.num_q_heads, s.head_dim, self.pool.get_device())
        if q.data_ptr() % 16 or (n > 1 and q.stride(0) * q.element_size() % 16):
            raise ValueError("the rows of q must be 16-byte aligned")
        if n > 1 and q.stride(0) < s.num_q_heads * s.head_dim:
            raise ValueError(f"the rows of q must not overlap (strides {q.stride()})")
        for name, t, want in (("out", out, (q.dtype, q.shape)), ("lse", lse, (torch.float32, q.shape[:2]))):
            if t is not None and ((t.dtype, t.shape) != want or t.get_device() != self.pool.get_device()
                                  or not t.is_contiguous()):
                raise ValueError(f"{name} must be {want[0]} {tuple(want[1])}, contiguous and on the decoder's device")
        if out is not None and out.data_ptr() % 16:
            raise ValueError("out must be 16-byte aligned")
        if out is None:
            with self._on(stream):
                out = torch.empty(q.shape, dtype=q.dtype, device=self.pool.device)
        with self._undone_if_refused():
            self.extend(new_lens, stream)
            self.append(k, v, stream)
            B.kvf_paged_prefill(q, self.pool, self.page_table, self.seq_lens, self.cu_new, out, s, self.workspace, lse=lse,
                                sm_scale=self.sm_scale, stream=stream)
        return out

    def gather(self, row: int, dtype=torch.float32, stream=None):
        """The cached keys and values [length][Hkv][d] of a row."""
        P, n = self.shape.page_size, self.lengths[row]
        with self._on(stream):
            t = torch.arange(n, device=self.pool.device)
            slots = (self.page_table[row].long()[t // P] * P + t % P).to(torch.int32)
            k, v = (torch.empty((n, self.shape.num_kv_heads, self.shape.head_dim), dtype=dtype,
                                device=self.pool.device) for _ in range(2))
        (B.kvq_gather if self.bits == 4 else B.kvf_gather)(self.pool, slots, k, v, *self._format, self.workspace, stream)
        return k, v

    def release(self, row: int, stream=None):
        """Give a row's pages back; its length is 0 afterwards."""
        n = self._pages(self.lengths[row])
        with self._on(stream):
            self._free[self._taken - n:self._taken].copy_(self.page_table[row, :n])
            self.seq_lens[row] = 0
        self._taken -= n
        self.lengths[row] = 0

    def check(self, stream=None):
        """Raise if the device flagged an out-of-range index or a timeout."""
        with torch.cuda.device(self.pool.device):
            st = B.get_error(self.workspace, stream)
        if st != 0:
            raise B.QskvError(st, B.last_error_message())


def from_inputs(inputs: dict, device="cuda", top_k="spec", prefix_pages: int = 0,
                scorer: str = "bound", approx_epsilon: Optional[float] = None, approx_seed: int = 0) -> PagedDecoder:
    """A PagedDecoder over a workloads.make_inputs() batch copied to `device`."""
    if isinstance(top_k, str):
        top_k = inputs["top_k"]
    t = {k: inputs[k].to(device) for k in ("q", "k_pool", "v_pool", "page_table", "seq_lens")}
    return PagedDecoder(t["q"], t["k_pool"], t["v_pool"], t["page_table"], t["seq_lens"], top_k,
                        prefix_pages=prefix_pages, scorer=scorer, approx_epsilon=approx_epsilon,
                        approx_seed=approx_seed)
