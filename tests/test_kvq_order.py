"""What the kernels of the 4-bit cache and the page tables read, and when: nothing before the kernel ahead has completed."""
import glob
import os
import re

import pytest
import torch

import query_aware_sparse_kv_gb300 as qskv

CSRC = os.path.join(os.path.dirname(qskv.__file__), "csrc")


def _kernels(path):
    """(name, body) of every kernel of a source file, comments left out."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"__global__[^{;]*?(\w+_kernel)\s*\([^{;]*\)\s*\{", text):
        yield m.group(1), text[m.end():text.index("\n}", m.end())]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "kvq_*.cu*")) + [os.path.join(CSRC, "tables.cu")]))
def test_a_kernel_waits_before_it_reads(path):
    text = open(path).read()
    kernels = list(_kernels(path))
    assert len(kernels) == text.count("__global__")
    for name, body in kernels:
        waits = [line.strip() for line in body.split("\n") if "pdl_wait" in line]
        assert waits == ["pdl_wait();"], name  # one, on no condition
        before = body[:body.index("pdl_wait();")]
        assert not re.search(r"__ld|units_of|pages_of|seq_of|a\.\w+\s*\[|scan_requests|Request\(", before), name


@pytest.mark.gpu
@pytest.mark.parametrize("rows,pages,top_k", [(3, 200, 0), (40, 9, 0), (500, 7, 0), (2, 30, 0), (6, 300, 40)])
def test_decode_right_behind_a_change_of_lengths_and_tables(rows, pages, top_k):
    """Lengths and page tables (and selections) written by an ordinary kernel, the decode next in the stream: it reads the
    new ones, longer and shorter."""
    g = torch.Generator().manual_seed(rows)
    d, gs, P, N = 64, 64, 16, 64
    shape = qskv.make_shape(rows, 2, 1, d, P, pages, N)
    pool = torch.zeros((N, 1, qskv.kvq_block_bytes(shape, gs)), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(qskv.kvq_workspace_size(shape), dtype=torch.uint8, device="cuda")
    kv = torch.randn((N * P, 1, d), generator=g).cuda()
    qskv.kvq_append(kv, kv, torch.arange(N * P, dtype=torch.int32, device="cuda"), pool, shape, gs, ws)
    q = torch.randn((rows, 2, d), generator=g).cuda()
    steps = [torch.randint(0, hi + 1, (rows,), generator=g).int().cuda() for hi in (pages * P, 16, pages * P, 1, pages * P)]
    tables = [torch.randint(0, N, (rows, pages), generator=g).int().cuda() for _ in steps]
    sel = torch.arange(max(top_k, 1), dtype=torch.int32, device="cuda").repeat(rows, 1, 1)

    def run(lens, table, out, counts):
        kw = dict(selected=sel, n_selected=counts, top_k=top_k) if top_k else {}
        qskv.kvq_paged_decode(q, pool, table, lens, out, shape, gs, ws, **kw)

    def counts_of(lens):
        return ((lens + P - 1) // P).clamp(max=top_k).int()[:, None].contiguous()

    want = []
    for lens, table in zip(steps, tables):
        n = counts_of(lens) if top_k else None
        torch.cuda.synchronize()
        want.append(torch.empty((rows, 2, d), device="cuda"))
        run(lens, table, want[-1], n)
    torch.cuda.synchronize()
    lens, table = torch.zeros_like(steps[0]), torch.zeros_like(tables[0])
    counts = torch.zeros((rows, 1), dtype=torch.int32, device="cuda")
    got = [torch.empty_like(want[0]) for _ in range(4 * len(steps))]
    for i, out in enumerate(got):
        table.copy_(tables[i % len(steps)])
        lens.copy_(steps[i % len(steps)])
        if top_k:
            counts.copy_(counts_of(lens))
        run(lens, table, out, counts)
    assert qskv.get_error(ws) == 0
    for i, out in enumerate(got):
        assert torch.equal(out, want[i % len(steps)]), i


@pytest.mark.gpu
@pytest.mark.parametrize("rows,pages,top_k", [(2, 40, 6), (16, 40, 6), (2, 400, 16), (300, 12, 0), (4, 300, 0)])
def test_tables_and_the_decodes_that_read_them_early(rows, pages, top_k):
    """extend_tables and, next in the stream, a step over a bf16 cache, whose kernels may read table and lengths ahead of
    their wait: as with the host waiting in between."""
    g = torch.Generator().manual_seed(pages)
    d, P, hkv = 64, 16, 2
    N = rows * pages
    shape = qskv.make_shape(rows, 2 * hkv, hkv, d, P, pages, N)
    k, v = (torch.randn((N, hkv, P, d), generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn((rows, 2 * hkv, d), generator=g).bfloat16().cuda()
    order = torch.randperm(N, generator=g).int()
    new = [torch.randint(0, pages * P // 6 + 1, (rows,), generator=g).int() for _ in range(5)]
    T = max(int(n.sum()) for n in new) + 1
    size = max(qskv.workspace_size(shape), qskv.tables_workspace_size(shape))
    full = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731

    def run(wait):
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        meta = torch.zeros((N, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
        qskv.kv_meta_build(k, torch.arange(N, dtype=torch.int32, device="cuda"), full(N) + P, meta, shape, ws)
        table, lens, other, cu, slots = torch.full_like(full(rows, pages), -1), full(rows), full(rows), full(rows + 1), full(T)
        sel, n_sel, outs, taken, held = full(rows, hkv, max(top_k, 1)), full(rows, hkv), [], 0, torch.zeros(rows).long()
        free, added = order.cuda(), [n.cuda() for n in new]
        for n, a in zip(new, added):
            qskv.extend_tables(lens, a, free[taken:], table, other, cu, slots, shape, ws)
            lens, other = other, lens
            if wait:
                torch.cuda.synchronize()
            outs.append(torch.empty((rows, 2 * hkv, d), device="cuda"))
            if top_k:
                qskv.select_decode(q, k, v, meta, table, lens, top_k, sel, n_sel, outs[-1], shape, ws)
            else:
                qskv.sparse_paged_decode(q, k, v, table, lens, outs[-1], shape, ws)
            taken += int(((held + n + P - 1) // P - (held + P - 1) // P).sum())
            held = held + n
        assert qskv.get_error(ws) == 0
        return outs

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)
