"""Calls that the 4-bit cache's documentation allows at its edges: most rows, most heads, lists wider than tables, graphs
over changing lengths, two calls at once, pages that all are bad."""
import math

import pytest
import torch

import kvq_ref as R
import query_aware_sparse_kv_gb300 as qskv

pytestmark = pytest.mark.gpu


class Cache:
    """N pages of random tokens that any row may name, and 64-bit attention over them on the GPU."""

    def __init__(self, N, hkv, d, P, gs, seed=0, size=1.0):
        g = torch.Generator().manual_seed(seed)
        f = [R.quantise(torch.randn((N, hkv, P, d), generator=g) * size, gs) for _ in range(2)]
        self.pool = R.pack(*f[0], *f[1]).cuda()
        self.k, self.v = (R.values(*x).cuda() for x in f)
        self.N, self.hkv, self.d, self.P, self.gs = N, hkv, d, P, gs

    def want(self, q, table, lens, pages=None):
        """q [B][hq][d], table [B][mp], lens [B]; pages [B][hkv][mp] (bool): the selected ones."""
        B, hq, d = q.shape
        G, mp = hq // self.hkv, table.shape[1]
        token = torch.arange(mp * self.P, device="cuda")[None] < lens[:, None]
        out = torch.zeros((B, hq, d), dtype=torch.float64, device="cuda")
        lse = torch.full((B, hq), -math.inf, dtype=torch.float64, device="cuda")
        for h in range(self.hkv):
            k, v = (x[table.long().clamp(0), h].flatten(1, 2) for x in (self.k, self.v))
            ok = token if pages is None else token & pages[:, h].repeat_interleave(self.P, 1)
            x = (q[:, h * G:h * G + G].double() @ k.transpose(1, 2) / d ** 0.5).masked_fill(~ok[:, None], -math.inf)
            some = ok.any(1)
            out[some, h * G:h * G + G] = (torch.softmax(x, -1) @ v)[some]
            lse[:, h * G:h * G + G] = torch.logsumexp(x, -1)
        return out, lse

    def check(self, out, lse, q, table, lens, pages=None):
        o, l = self.want(q, table, lens, pages)
        # a logit's error is about 2.3e-6 (24 roundings of 2^-24 on parts of up to 8); 5 times that, on values up to max |v|
        assert float((out.double() - o).abs().max()) <= 2.0 ** -16 * float(self.v.abs().max())
        none = torch.isinf(l)
        assert bool((out[none] == 0).all()) and bool((lse[none] == -math.inf).all())
        if not bool(none.all()):
            assert float((lse.double() - l)[~none].abs().max()) <= 2.0 ** -16


def _buffers(shape):
    out = torch.full((shape.batch, shape.num_q_heads, shape.head_dim), math.nan, device="cuda")
    return out, torch.full(out.shape[:2], math.nan, device="cuda"), \
        torch.zeros(qskv.kvq_workspace_size(shape), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("batch,hkv,hq,mp,d,P,gs", [
    (65535, 1, 1, 2, 64, 16, 64),     # most rows
    (1023, 64, 128, 1, 64, 32, 32),   # the same by heads
    (2, 64, 512, 5, 128, 16, 32),
    (1, 1, 8, 1, 128, 32, 128),
    (7, 16, 16, 3, 128, 32, 64),
])
def test_most_rows_and_heads(batch, hkv, hq, mp, d, P, gs):
    g = torch.Generator().manual_seed(batch)
    c = Cache(9, hkv, d, P, gs)
    shape = qskv.make_shape(batch, hq, hkv, d, P, mp, c.N)
    out, lse, ws = _buffers(shape)
    table = torch.randint(0, c.N, (batch, mp), generator=g).int().cuda()
    lens = torch.randint(0, mp * P + 1, (batch,), generator=g).int().cuda()
    q = torch.randn((batch, hq, d), generator=g).cuda()
    qskv.kvq_paged_decode(q, c.pool, table, lens, out, shape, gs, ws, lse=lse)
    assert qskv.get_error(ws) == 0
    for a in range(0, batch, 4096):
        b = slice(a, a + 4096)
        c.check(out[b], lse[b], q[b], table[b], lens[b])


def test_a_list_wider_than_the_table():
    c = Cache(12, 2, 64, 16, 32)
    shape = qskv.make_shape(3, 4, 2, 64, 16, 5, c.N)
    out, lse, ws = _buffers(shape)
    table = torch.arange(15).view(3, 5).remainder(12).int().cuda()
    lens = torch.tensor([80, 1, 33], dtype=torch.int32, device="cuda")
    sel = torch.full((3, 2, 40), -1, dtype=torch.int32)
    sel[0, 0, :5], sel[0, 1, :2] = torch.arange(5), torch.tensor([1, 4])
    sel[1, :, 0], sel[2, 0, :3] = 0, torch.arange(3)
    n = torch.tensor([[5, 2], [1, 1], [3, 0]], dtype=torch.int32)
    pages = torch.zeros((3, 2, 5), dtype=torch.bool)
    for b in range(3):
        for h in range(2):
            pages[b, h, sel[b, h, :int(n[b, h])].long()] = True
    q = torch.randn((3, 4, 64), generator=torch.Generator().manual_seed(1)).cuda()
    qskv.kvq_paged_decode(q, c.pool, table, lens, out, shape, 32, ws, lse=lse, selected=sel.cuda(), n_selected=n.cuda(),
                          top_k=40)
    assert qskv.get_error(ws) == 0
    c.check(out, lse, q, table, lens, pages.cuda())


@pytest.mark.parametrize("rows,mp", [(3, 150), (400, 6), (20, 40)])
def test_graphs_over_changing_lengths_share_a_workspace(rows, mp):
    """A dense and a selecting call, each recorded once: replayed in turn as lengths, tables, queries and lists change."""
    g = torch.Generator().manual_seed(mp)
    c = Cache(30, 1, 64, 16, 64)
    shape = qskv.make_shape(rows, 4, 1, 64, 16, mp, c.N)
    K = min(mp, 9)
    out, lse, ws = _buffers(shape)
    q = torch.zeros((rows, 4, 64), device="cuda")
    table, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((rows, mp), (rows,)))
    sel, n = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((rows, 1, K), (rows, 1)))
    kinds = [dict(), dict(selected=sel, n_selected=n, top_k=K)]
    for kw in kinds:
        qskv.kvq_paged_decode(q, c.pool, table, lens, out, shape, 64, ws, lse=lse, **kw)
    graphs = [torch.cuda.CUDAGraph() for _ in kinds]
    for graph, kw in zip(graphs, kinds):
        with torch.cuda.graph(graph):
            qskv.kvq_paged_decode(q, c.pool, table, lens, out, shape, 64, ws, lse=lse, **kw)
    for i in range(8):
        table.copy_(torch.randint(0, c.N, (rows, mp), generator=g))
        length = torch.randint(0, mp * 16 + 1, (rows,), generator=g) if i % 3 else torch.zeros(rows).long()
        lens.copy_(length)
        q.copy_(torch.randn((rows, 4, 64), generator=g))
        held = torch.arange(mp)[None] * 16 < length[:, None]
        n.copy_(held.sum(1)[:, None].clamp(max=K))
        order = torch.rand((rows, mp), generator=g).masked_fill(~held, 2).argsort(-1)[:, :K]
        sel.copy_(order[:, None])
        pages = torch.zeros((rows, 1, mp), dtype=torch.bool).scatter_(2, order[:, None], True) & held[:, None]
        out.fill_(math.nan)
        graphs[i % 2].replay()
        assert qskv.get_error(ws) == 0
        c.check(out, lse, q, table, lens, pages.cuda() if i % 2 else None)


def test_two_calls_at_once():
    """Two streams, a workspace each, many calls of both under way together: as one after another."""
    c = Cache(64, 2, 128, 16, 64)
    jobs = []
    for i, (rows, mp) in enumerate(((5, 120), (200, 9))):
        g = torch.Generator().manual_seed(i)
        shape = qskv.make_shape(rows, 8, 2, 128, 16, mp, c.N)
        jobs.append((shape, torch.randn((rows, 8, 128), generator=g).cuda(),
                     torch.randint(0, c.N, (rows, mp), generator=g).int().cuda(),
                     torch.randint(0, mp * 16 + 1, (rows,), generator=g).int().cuda(), *_buffers(shape)))
    streams = [torch.cuda.Stream() for _ in jobs]
    results = [[] for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(30):
        for s, r, (shape, q, table, lens, out, lse, ws) in zip(streams, results, jobs):
            with torch.cuda.stream(s):
                r.append(torch.empty_like(out))
                qskv.kvq_paged_decode(q, c.pool, table, lens, r[-1], shape, 64, ws, lse=lse)
    torch.cuda.synchronize()
    for r, (shape, q, table, lens, out, lse, ws) in zip(results, jobs):
        assert qskv.get_error(ws) == 0
        c.check(r[0], lse, q, table, lens)
        for x in r[1:]:
            assert torch.equal(x, r[0])


@pytest.mark.parametrize("rows,mp", [(2, 3), (2, 90), (400, 3)])
def test_rows_whose_pages_are_all_bad(rows, mp):
    """Flagged, and zeros with an lse of -inf, beside rows that are as ever."""
    c = Cache(20, 2, 64, 16, 64)
    shape = qskv.make_shape(rows, 4, 2, 64, 16, mp, c.N)
    out, lse, ws = _buffers(shape)
    g = torch.Generator().manual_seed(rows)
    table = torch.randint(0, c.N, (rows, mp), generator=g).int()
    table[::2] = torch.where(torch.rand((rows, mp), generator=g) < 0.5, -7, c.N)[::2].int()
    table, q = table.cuda(), torch.randn((rows, 4, 64), generator=g).cuda()
    lens = torch.full((rows,), mp * 16, dtype=torch.int32, device="cuda")
    qskv.kvq_paged_decode(q, c.pool, table, lens, out, shape, 64, ws, lse=lse)
    assert qskv.get_error(ws) == 5 and qskv.get_error(ws) == 0
    assert bool((out[::2] == 0).all()) and bool((lse[::2] == -math.inf).all())
    c.check(out[1::2], lse[1::2], q[1::2], table[1::2], lens[1::2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_tokens_with_odd_strides(dtype):
    """One token with any stride, one token for every slot (stride 0 is refused), heads that are not neighbours (refused)."""
    shape = qskv.make_shape(1, 3, 3, 64, 16, 1, 4)
    pool = torch.zeros((4, 3, qskv.kvq_block_bytes(shape, 32)), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    x = torch.randn((3, 64), generator=torch.Generator().manual_seed(0)).to(dtype)
    wide = torch.zeros((1, 7, 64), dtype=dtype, device="cuda")
    wide[0, 2:5] = x.cuda()
    slot = torch.tensor([37], dtype=torch.int32, device="cuda")
    for k in (wide[:, 2:5], torch.as_strided(wide, (1, 3, 64), (3, 64, 1), 128), torch.as_strided(wide, (1, 3, 64), (0, 64, 1), 128)):
        pool.zero_()
        qskv.kvq_append(k, k, slot, pool, shape, 32, ws)
        ko, vo = (torch.empty((1, 3, 64), device="cuda") for _ in range(2))
        qskv.kvq_gather(pool, slot, ko, vo, shape, 32, ws)
        want = R.values(*R.quantise(x, 32)).float()
        assert torch.equal(ko[0].cpu(), want) and torch.equal(vo[0].cpu(), want)
    slots = torch.arange(5, dtype=torch.int32, device="cuda")
    k = wide[:, 2:5].expand(5, 3, 64)
    with pytest.raises(qskv.QskvError):
        qskv.kvq_append(k, k, slots, pool, shape, 32, ws)
    with pytest.raises(ValueError):
        k = torch.zeros((5, 6, 64), dtype=dtype, device="cuda")[:, ::2]
        qskv.kvq_append(k, k, slots, pool, shape, 32, ws)


def test_tables_of_the_most_requests():
    """65535 requests, in one call's two launches; a single token's place; nothing free."""
    B, P, N = 65535, 16, 200_000
    g = torch.Generator().manual_seed(0)
    seq = torch.randint(0, 33, (B,), generator=g)
    new = torch.minimum(torch.randint(0, 20, (B,), generator=g) * torch.randint(0, 2, (B,), generator=g), 48 - seq)
    held = (seq + P - 1) // P
    table = torch.full((B, 3), -1, dtype=torch.int32)
    at = torch.cumsum(held, 0) - held
    for j in range(3):
        table[:, j] = torch.where(j < held, at + j, -1)
    free = torch.arange(int(held.sum()), N, dtype=torch.int32)
    T = int(new.sum()) + 5
    E = T // P + 2 * B
    shape = qskv.make_shape(B, 1, 1, 64, P, 3, N)
    i32 = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(qskv.tables_workspace_size(shape), dtype=torch.uint8, device="cuda")
    o = dict(page_table=table.cuda(), seq_lens_out=i32(B), cu_new=i32(B + 1), slot_map=i32(T), positions=i32(T),
             touched_ids=i32(E), touched_valid=i32(E), counts=i32(4))
    first = [o[k] for k in ("page_table", "seq_lens_out", "cu_new", "slot_map")]
    rest = {k: o[k] for k in ("positions", "touched_ids", "touched_valid", "counts")}
    for f in (free, free[:0]):
        o["page_table"].copy_(table)
        qskv.extend_tables(seq.int().cuda(), new.int().cuda(), f.cuda(), *first, shape, ws, **rest)
        want = R.tables(seq.tolist(), new.tolist(), f.tolist(), table.tolist(), P, N, T, E)
        for k in o:
            assert torch.equal(o[k].cpu(), torch.tensor(want[k], dtype=torch.int32)), k
        assert qskv.get_error(ws) == (0 if len(f) else 5)
