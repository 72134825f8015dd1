"""Query-aware sparse paged KV decode for GB300 (sm_103a).

The computation lives in libqskv.so (CUDA kernels behind the C ABI declared
in include/qskv.h); this package is its binding:

  kv_meta_build        per-page min/max key metadata
  page_select          bound score of every page and top-K per (sequence, KV head)
  page_select_refresh  the same, after rebuilding every sequence's last-page
                       metadata in the same launch
  kv_centroid_build,   Block Top-K: per-page mean key, and q . centroid scores
  page_select_centroid   with the same top-K
  page_select_approx   either score with a lossy top-K (early exit + sampling)
  sparse_paged_decode  split-K attention over the selected pages, LSE merge
  select_decode        one step in one call: last-page refresh, scoring,
                       top-K and the sparse decode (the decode ranks its
                       own rows when they go one row per k CTAs)
  cascade_paged_decode dense decode of a batch sharing a page prefix: the
                       prefix once per KV head on the tensor cores, the rest
                       paged, LSE merge

  extend_tables        page tables, slot map and touched pages of a
                       scheduler step, from lengths and a free-page list
  kvq_append,          the KV cache in 4 bits (bf16 scale and minimum per
  kvq_gather,            group of dims): tokens stored by slot, read back as
  kvq_meta_build,        values, page metadata for the selection calls, and
  kvq_paged_decode       the decode over it (all pages or selected ones)

plus ``PagedDecoder`` and ``QuantizedPagedDecoder`` (buffer plumbing for a
whole step over a bf16 / fp32 and over a 4-bit cache) and ``workloads``
(seeded synthetic inputs).  Nothing here computes on the CPU: without the
built library every call raises.
"""
from .binding import (QSKV_BF16, QSKV_F32, QskvError, QskvLibraryMissing, Shape, cascade_paged_decode,
                      cascade_workspace_size, extend_tables, get_error, kv_centroid_build, kv_meta_build,
                      kvq_append, kvq_block_bytes, kvq_gather, kvq_meta_build, kvq_paged_decode, kvq_workspace_size,
                      last_error_message, load, make_shape, page_select, page_select_approx, page_select_refresh, page_select_centroid,
                      select_decode, sparse_paged_decode, sparse_paged_decode_noalloc, tables_workspace_size,
                      workspace_size)
from .engine import PagedDecoder, QuantizedPagedDecoder, from_inputs

__all__ = ["QSKV_BF16", "QSKV_F32", "QskvError", "QskvLibraryMissing", "Shape", "cascade_paged_decode",
           "cascade_workspace_size", "get_error", "kv_centroid_build", "kv_meta_build", "page_select_approx", "page_select_centroid",
           "last_error_message", "load", "make_shape", "page_select", "page_select_refresh", "select_decode",
           "sparse_paged_decode",
           "sparse_paged_decode_noalloc", "workspace_size",
           "extend_tables", "kvq_append", "kvq_block_bytes", "kvq_gather", "kvq_meta_build", "kvq_paged_decode",
           "kvq_workspace_size", "tables_workspace_size",
           "PagedDecoder", "QuantizedPagedDecoder", "from_inputs"]
