"""Prefill on the GPU against the 64-bit statement of prefill_ref."""
import math

import pytest
import torch

import kvf_ref as F
import prefill_ref as R
import query_aware_sparse_kv_gb300 as qskv
from test_gpu_kvf import spoil

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# (queries' type, cache): every combination there is
KINDS = [(BF16, "bf16"), (BF16, "kvf"), (F32, "fp32"), (F32, "bf16"), (F32, "kvf"), (BF16, "fp32")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from query_aware_sparse_kv_gb300 import build

    build.build()
    qskv.load()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    """Rows of old + new tokens: pools, tables and values on the CPU, what a prefill takes on the GPU."""

    def __init__(self, seed, rows, hq, hkv, d, P, dtype, cache, pad=3, q_scale=1.0, k=None, v=None, extra=0, room=0):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.hq, self.hkv, self.d, self.P, self.dtype, self.cache = rows, hq, hkv, d, P, dtype, cache
        self.lens, self.new = [o + n for o, n in rows], [n for _, n in rows]
        B, pages = len(rows), [-(-x // P) for x in self.lens]
        mp, N = max(1, max(pages)) + extra, sum(pages) + 2
        self.shape = qskv.make_shape(B, hq, hkv, d, P, mp, N)
        k = torch.randn((N, hkv, P, d), generator=g) if k is None else k(g, (N, hkv, P, d))
        v = torch.randn((N, hkv, P, d), generator=g) if v is None else v(g, (N, hkv, P, d))
        ids, at = torch.randperm(N, generator=g), 0
        self.table = torch.full((B, mp), -1, dtype=torch.int32)
        for b in range(B):
            self.table[b, :pages[b]] = ids[at:at + pages[b]].to(torch.int32)
            at += pages[b]
        if cache == "kvf":
            ku, vu = F.quantise(k), F.quantise(v)
            self.k, self.v = F.values(*ku), F.values(*vu)
            pool = F.pack(*ku, *vu)
        else:
            dt = BF16 if cache == "bf16" else F32
            k, v = k.to(dt), v.to(dt)
            self.k, self.v = k.double(), v.double()
        for b in range(B):
            if self.lens[b] % P:  # what lies past the end is no number
                page, n = int(self.table[b, pages[b] - 1]), self.lens[b] % P
                if cache == "kvf":
                    spoil(pool, page, n, d, P)
                else:
                    k[page, :, n:], v[page, :, n:] = math.nan, math.inf
        self.pools = dict(pool=pool.cuda()) if cache == "kvf" else dict(k_pool=k.cuda(), v_pool=v.cuda())
        self.T = sum(self.new) + pad
        qkv = torch.full((self.T, hq + 3, d), math.nan, dtype=dtype)  # rows of a wider projection output
        self.q = (torch.randn((self.T, hq, d), generator=g) * q_scale).to(dtype)
        qkv[:, 2:2 + hq] = self.q
        if pad:
            qkv[sum(self.new):] = math.nan
        cu = [0]
        for n in self.new:
            cu.append(cu[-1] + n)
        self.cu = cu
        self.gpu = dict(q=qkv.cuda()[:, 2:2 + hq], page_table=self.table.cuda(), seq_lens=_i32(self.lens), cu_new=_i32(cu))
        self.ws = torch.zeros(qskv.prefill_workspace_size(self.shape, self.T + room), dtype=torch.uint8, device="cuda")
        self.out = torch.full((self.T, hq, d), 7.0, dtype=dtype, device="cuda")
        self.lse = torch.full((self.T, hq), 7.0, device="cuda")

    def run(self, scale=0.0, **over):
        fn = qskv.kvf_paged_prefill if self.cache == "kvf" else qskv.paged_prefill
        fn(**{**self.gpu, **self.pools, "out": self.out, "lse": self.lse, "shape": self.shape, "workspace": self.ws,
              "sm_scale": scale, **over})

    def check(self, scale=0.0, error=0, skip=(), lens=None):
        """skip: (row, page) places that are not there; lens: other lengths than the batch's own."""
        assert qskv.get_error(self.ws) == error
        scale = scale or self.d ** -0.5
        lens = lens or self.lens
        out, lse, G = self.out.cpu().double(), self.lse.cpu().double(), self.hq // self.hkv
        n = self.cu[-1]
        assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())  # the padding is as it was
        low = self.dtype == BF16 and self.cache != "fp32"  # bf16 operands
        for b, new in enumerate(self.new):
            if not new:
                continue
            here = slice(self.cu[b], self.cu[b + 1])
            t = torch.tensor([j for j in range(lens[b]) if (b, j // self.P) not in skip], dtype=torch.long)
            page, place = self.table[b].long()[t // self.P], t % self.P
            pos = torch.searchsorted(t, lens[b] - new + torch.arange(new), right=True) - 1
            for h in range(self.hkv):
                hs = slice(h * G, (h + 1) * G)
                k, v = self.k[page, h, place], self.v[page, h, place]
                o, z, pabs, A = R.attend_rows(self.q[here, hs], k, v, pos, scale)
                vmax = float(v.abs().max()) if len(v) else 0.0
                tol, ltol = R.bounds(o, pabs, vmax, A, len(k), self.d, low)
                if self.dtype == BF16 and not low:  # fp32 arithmetic, bf16 output
                    tol = tol + 2.0 ** -8 * o.abs()
                bad = (out[here, hs] - o).abs() - tol
                assert not bool(torch.isnan(out[here, hs]).any()), (b, h)
                assert float(bad.max()) <= 0, (b, h, float(bad.max()), float(tol.flatten()[bad.argmax()]))
                there = z > -math.inf
                assert torch.equal(lse[here, hs] > -math.inf, there)
                assert float((lse[here, hs] - z)[there].abs().max() if there.any() else 0.0) <= ltol + 2.0 ** -22 * float(
                    z[there].abs().max() if there.any() else 0.0), (b, h)


ROWS = [(0, 1), (5, 0), (0, 5), (16, 1), (31, 33), (0, 130), (200, 2), (7, 64), (0, 0), (300, 17)]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("hq,hkv", [(3, 3), (4, 2), (4, 1), (16, 2)])
def test_mixed_batches(dtype, cache, d, P, hq, hkv):
    b = Batch(hq * d + P, ROWS, hq, hkv, d, P, dtype, cache)
    b.run()
    b.check()


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("rows,hq,hkv,d,P", [
    ([(0, 1)], 1, 1, 64, 16),
    ([(0, 1000)], 2, 1, 128, 16),               # whole prompts of many tiles
    ([(0, 700), (0, 3), (600, 500)], 8, 1, 64, 32),
    ([(5000, 1)], 8, 1, 128, 16),               # few queries over a long cache: its blocks in parts
    ([(9000, 40), (3, 1), (2500, 1)], 4, 2, 64, 32),
    ([(i % 40, i % 7) for i in range(300)], 4, 2, 64, 16),
])
def test_work_splits(dtype, cache, rows, hq, hkv, d, P):
    b = Batch(len(rows) + d, rows, hq, hkv, d, P, dtype, cache, room=77)
    b.run(scale=0.2)
    first = b.out.clone(), b.lse.clone()
    b.check(scale=0.2)
    b.run(scale=0.2)  # equal inputs, equal bits
    assert torch.equal(b.out, first[0]) and torch.equal(b.lse, first[1])


FEW = [
    ([(0, 1)], 2, 1, 64, 16),
    ([(0, 3), (200, 0), (255, 1), (0, 0), (131, 5)], 4, 2, 128, 16),
    ([(1000 + 100 * i, i % 3) for i in range(19)], 8, 4, 64, 16),           # each tile in parts, some rows without one
    ([(9000, 5), (1, 2), (20000, 1)], 8, 2, 128, 32),                       # a CTA has a range of one tile
    ([(3000 + 500 * (i % 5), 1) for i in range(32)], 4, 4, 64, 16),         # and of several
    ([(0, 1 + i % 2) for i in range(32)], 4, 4, 64, 32),
    ([(30000, 17)], 16, 2, 64, 16),
]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("rows,hq,hkv,d,P", FEW)
def test_few_tokens_of_few_rows(dtype, cache, rows, hq, hkv, d, P):
    """No list is made for these; the counters that they share with other calls are as they were after each."""
    b = Batch(len(rows) + d + P, rows, hq, hkv, d, P, dtype, cache, pad=1)
    b.run(scale=0.2)
    first = b.out.clone(), b.lse.clone()
    b.check(scale=0.2)
    assert not bool(b.ws[:256 + 4 * len(rows) * hkv].any())
    for _ in range(3):  # equal inputs, equal bits
        b.run(scale=0.2)
        assert torch.equal(b.out, first[0]) and torch.equal(b.lse, first[1])
    lens = [max(x - 7, 0) if i % 2 else x for i, x in enumerate(b.lens)]  # some shorter than what is new
    b.run(scale=0.2, seq_lens=_i32(lens))
    b.check(scale=0.2, lens=lens, error=5 if any(n > x for n, x in zip(b.new, lens)) else 0)


@pytest.mark.parametrize("cache", ["bf16", "kvf"])
def test_graphs_with_and_without_a_list_share_a_workspace(cache):
    """Few queries, the same ones within a longer buffer (a list is made then), and a decode over the same pages and counters,
    each captured; replayed in turn while the lengths change."""
    b = Batch(11, [(2000, 4), (40, 0), (0, 3), (9000, 5)], 8, 2, 128, 16, BF16, cache, pad=0, room=100)
    T, long_q = b.T, torch.zeros((b.T + 100, 8, 128), dtype=BF16, device="cuda")
    long_q[:T] = b.gpu["q"]
    long_out, long_lse = torch.full_like(long_q, 7.0), torch.full((T + 100, 8), 7.0, device="cuda")
    size = max(b.ws.numel(), qskv.kvf_workspace_size(b.shape), qskv.workspace_size(b.shape))
    b.ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    one = torch.randn((4, 8, 128), device="cuda").to(BF16)
    dec = torch.empty((4, 8, 128), device="cuda")

    def decode():
        if cache == "kvf":
            qskv.kvf_paged_decode(one, b.pools["pool"], b.gpu["page_table"], b.gpu["seq_lens"], dec, b.shape, b.ws)
        else:
            qskv.sparse_paged_decode(one, b.pools["k_pool"], b.pools["v_pool"], b.gpu["page_table"], b.gpu["seq_lens"], dec,
                                     b.shape, b.ws)

    calls = [b.run, lambda: b.run(q=long_q, out=long_out, lse=long_lse), decode]
    graphs = []
    for call in calls:
        call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    lens = list(b.lens)
    for cut in (0, 5, 900, 0):
        now = [max(x - cut, n) for x, n in zip(lens, b.new)]
        b.gpu["seq_lens"].copy_(_i32(now))
        decode()
        want = dec.clone()
        for order in ((0, 1, 2), (2, 0, 0), (1, 0, 2), (0, 2, 1)):
            b.out.fill_(7.0), b.lse.fill_(7.0), dec.fill_(7.0)
            for i in order:
                graphs[i].replay()
            if 0 in order:
                b.check(lens=now)
            if 2 in order:
                assert torch.equal(dec, want)
            if 1 in order:
                assert bool((long_out[T:] == 7).all())
                # two bf16 evaluations, each within 2^-8 (1 + 2^-7) of the weighted values and of the output, and little more
                assert float((long_out[:T].float() - b.out.float()).abs().max()) <= 2.1 * 2.0 ** -7 * float(b.v.abs().max())


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_unusual_values(dtype, cache):
    """Logits far apart, growing along the row, all equal; large values."""
    grow = lambda g, s: torch.randn(s, generator=g) * torch.linspace(0, 6, s[0])[:, None, None, None]  # noqa: E731
    for kw in (dict(q_scale=20.0), dict(k=grow), dict(q_scale=0.0), dict(v=lambda g, s: torch.randn(s, generator=g) * 1e4)):
        b = Batch(5, [(0, 300), (450, 20)], 4, 2, 128, 16, dtype, cache, **kw)
        b.run()
        b.check()


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_bad_pages_are_flagged_and_skipped(dtype, cache):
    b = Batch(6, [(40, 30), (100, 150), (0, 20)], 4, 2, 64, 16, dtype, cache)
    table = b.table.clone()
    table[1, 3], table[1, 12], table[0, 0] = b.shape.num_pool_pages, -1, -5
    b.run(page_table=table.cuda())
    b.check(error=5, skip={(1, 3), (1, 12), (0, 0)})


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_bad_lengths_are_flagged(dtype, cache):
    """Fewer tokens than queries: those before the first token attend to nothing; lengths out of range are clamped."""
    b = Batch(7, [(40, 30), (100, 50), (0, 20)], 4, 2, 64, 16, dtype, cache)
    lens = [70, 12, 0]
    b.run(seq_lens=_i32(lens))
    b.check(error=5, lens=lens)
    b.run(seq_lens=_i32([70, 150, -3]))
    b.check(error=5, lens=[70, 150, 0])
    b.run()
    b.check()


@pytest.mark.parametrize("dtype,cache", [(BF16, "bf16"), (BF16, "kvf"), (F32, "fp32")])
@pytest.mark.parametrize("cu", [[0, 30, 10, 500], [-4, 30, 80, 100], [0, 0, 0, 0], [50, 30, 20, 10], [0, 100, 0, 100],
                                [0, 2 ** 31 - 1, -2 ** 31, 5]])
def test_bad_packing_touches_nothing_else(dtype, cache, cu):
    b = Batch(8, [(40, 30), (100, 50), (0, 20)], 4, 2, 64, 16, dtype, cache, pad=0)
    guard = torch.full((b.T + 64, 4, 64), 7.0, dtype=dtype, device="cuda")
    b.run(cu_new=_i32(cu), out=guard[:b.T])
    assert qskv.get_error(b.ws) == (0 if cu == [0, 0, 0, 0] else 5)
    assert bool((guard[b.T:] == 7).all())
    if cu == [0, 0, 0, 0]:
        assert bool((guard == 7).all())
    b.run()
    b.check()


@pytest.mark.parametrize("dtype,cache", [(BF16, "bf16"), (BF16, "kvf"), (F32, "fp32")])
def test_more_rows_than_the_plan_keeps_at_hand(dtype, cache):
    """5000 sequences, most without new tokens, some with none at all; a long one among them, cut into parts."""
    rows = [(i % 23, 0 if i % 25 else 1 + i // 25 % 3) for i in range(5000)]
    rows[4321] = (6000, 2)
    b = Batch(15, rows, 4, 1, 64, 16, dtype, cache)
    b.run()
    b.check()


@pytest.mark.parametrize("dtype,cache", [(BF16, "bf16"), (BF16, "kvf"), (F32, "fp32")])
def test_a_captured_step_from_lengths_to_outputs(dtype, cache):
    """Tables, store and prefill in one graph, replayed over steps of other lengths: chunks of prompts and single tokens
    mixed, fewer tokens than the buffers hold, tables and workspace shared."""
    g = torch.Generator().manual_seed(21)
    B, hq, hkv, d, P, mp, N, T = 4, 8, 2, 64, 16, 40, 120, 300
    shape = qskv.make_shape(B, hq, hkv, d, P, mp, N)
    size = max(qskv.prefill_workspace_size(shape, T), qskv.tables_workspace_size(shape))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, grown, new, cu, slots, table, counts = i32(B), i32(B), i32(B), i32(B + 1), i32(T), i32(B, mp) - 1, i32(4)
    free = torch.randperm(N, generator=g).int().cuda()
    k, v = (torch.zeros((T, hkv, d), dtype=dtype, device="cuda") for _ in range(2))
    q, out = (torch.zeros((T, hq, d), dtype=dtype, device="cuda") for _ in range(2))
    if cache == "kvf":
        pools = [torch.zeros((N, hkv, qskv.kvf_block_bytes(shape)), dtype=torch.uint8, device="cuda")]
    else:
        pools = [torch.zeros((N, hkv, P, d), dtype=dtype, device="cuda") for _ in range(2)]

    def body():
        qskv.extend_tables(lens, new, free, table, grown, cu, slots, shape, ws, counts=counts)
        if cache == "kvf":
            qskv.kvf_append(k, v, slots, pools[0], shape, ws)
            qskv.kvf_paged_prefill(q, pools[0], table, grown, cu, out, shape, ws)
        else:  # the framework stores into its own caches only; a bf16 or fp32 pool is the caller's
            at = slots.long().clamp_min(0)
            live = (slots >= 0)[:, None, None]
            for pool, x in zip(pools, (k, v)):
                old = pool[at // P, :, at % P]
                pool[at // P, :, at % P] = torch.where(live, x, old)
            qskv.paged_prefill(q, *pools, table, grown, cu, out, shape, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()  # no new tokens yet
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    seen = [[torch.empty((0, hkv, d), dtype=torch.float64)] * 2 for _ in range(B)]
    # a padded place writes to slot 0's old values above, so slot 0's page is never handed out
    free.copy_(torch.cat([free[free != 0], free[free == 0]]))
    for step in ([120, 0, 33, 1], [1, 1, 1, 1], [150, 2, 1, 100], [0, 0, 0, 0], [1, 200, 1, 0]):
        n = sum(step)
        x = [torch.randn(t.shape, generator=g).to(dtype) for t in (k, v, q)]
        for t, y in zip((k, v, q), x):
            t.copy_(y)
        new.copy_(_i32(step))
        out.fill_(7.0)
        graph.replay()
        taken = int(counts[1])
        free.copy_(torch.roll(free, -taken))
        lens.copy_(grown)
        assert qskv.get_error(ws) == 0
        got, at = out.cpu(), 0
        assert bool((got[n:] == 7).all())
        for b, m in enumerate(step):
            for i in range(2):
                y = x[i][at:at + m].double()
                y = F.values(*F.quantise(y)) if cache == "kvf" and m else y
                seen[b][i] = torch.cat([seen[b][i], y])
            if m:
                kk, vv = seen[b]
                for h in range(hkv):
                    hs, pos = slice(4 * h, 4 * h + 4), len(kk) - m + torch.arange(m)
                    o, _, pabs, A = R.attend_rows(x[2][at:at + m, hs], kk[:, h], vv[:, h], pos, d ** -0.5)
                    tol, _ = R.bounds(o, pabs, float(vv.abs().max()), A, len(kk), d, dtype == BF16)
                    assert bool(((got[at:at + m, hs].double() - o).abs() <= tol).all()), (step, b, h)
            at += m


def test_refused_arguments():
    b = Batch(9, [(4, 30)], 4, 2, 64, 16, BF16, "bf16")
    for over, match in ((dict(out=b.out.float()), "out"), (dict(lse=b.lse[:-1]), "lse"), (dict(cu_new=b.gpu["cu_new"][:-1]), "cu_new"),
                        (dict(q=b.q), "q"), (dict(v_pool=b.pools["v_pool"].float()), "v_pool"), (dict(out=b.out.cpu().pin_memory()), "out"),
                        (dict(q=b.gpu["q"].transpose(1, 2).contiguous().transpose(1, 2)), "q")):
        with pytest.raises(ValueError, match=match):
            b.run(**over)
    with pytest.raises(qskv.QskvError):
        b.run(workspace=b.ws[:256])
    wide = torch.zeros((33, 4 * 64 + 4), dtype=BF16, device="cuda")[:, 4:]  # rows off the 16-byte grid
    with pytest.raises(qskv.QskvError):
        b.run(q=wide.view(33, 4, 64) if wide.is_contiguous() else wide.unflatten(1, (4, 64)))
    none = dict(q=b.gpu["q"][:0], out=b.out[:0], lse=b.lse[:0])
    b.run(**none)
    b.run(lse=None)
    got = b.out.clone()
    b.run()
    b.check()
    assert torch.equal(got, b.out)


@pytest.mark.parametrize("dtype,cache", [(BF16, "bf16"), (BF16, "kvf"), (F32, "fp32")])
def test_in_graphs_that_share_a_workspace(dtype, cache):
    """Two captured prefills of different sizes over one workspace, replayed in turn with a decode's calls between."""
    a = Batch(10, [(4000, 3), (0, 300)], 8, 1, 128, 16, dtype, cache)
    b = Batch(11, [(0, 129), (70, 40)], 8, 1, 128, 16, dtype, cache)
    size = max(a.ws.numel(), b.ws.numel(), qskv.kvq_workspace_size(a.shape), qskv.workspace_size(a.shape))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    a.ws = b.ws = ws
    graphs = []
    for x in (a, b):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            x.run()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
        x.out.fill_(7.0)
        x.lse.fill_(7.0)
    dec = torch.empty((2, 8, 128), device="cuda")
    for _ in range(3):
        for g, x in zip(graphs, (a, b)):
            g.replay()
            if cache == "kvf":
                qskv.kvf_paged_decode(torch.ones((2, 8, 128), device="cuda"), x.pools["pool"], x.gpu["page_table"],
                                      x.gpu["seq_lens"], dec, x.shape, ws)
            else:
                qskv.sparse_paged_decode(torch.ones((2, 8, 128), device="cuda"), x.pools["k_pool"], x.pools["v_pool"],
                                         x.gpu["page_table"], x.gpu["seq_lens"], dec, x.shape, ws)
    a.check()
    b.check()
    # the replayed graphs follow what their buffers hold: fewer queries, other lengths
    n = 200
    a.gpu["cu_new"].copy_(_i32([0, 0, n]))
    a.gpu["seq_lens"].copy_(_i32([17, 250]))
    a.out.fill_(7.0)
    a.lse.fill_(7.0)
    graphs[0].replay()
    a.new, a.cu, a.lens = [0, n], [0, 0, n], [17, 250]
    # the tokens of row 1 lie in its pages up to 250
    a.check()


def test_offsets_past_32_bits():
    """A pool of over 4 GiB, its last pages; and on a stream of its own."""
    d, P, H, N = 128, 32, 8, 33_000
    shape = qskv.make_shape(1, H, H, d, P, 3, N)
    k, v = (torch.empty((N, H, P, d), dtype=torch.float32, device="cuda") for _ in range(2))
    assert k.numel() * 4 > 2 ** 32 and k.numel() * 2 > 2 ** 31
    g = torch.Generator().manual_seed(1)
    for dtype in (F32, BF16):
        if dtype == BF16:
            N = 66_000
            shape = qskv.make_shape(1, H, H, d, P, 3, N)
            k, v = (x.view(BF16).view(N, H, P, d) for x in (k, v))
            assert k.numel() * 2 > 2 ** 32
        pages = [N - 1, N - 3, N - 2]
        kx, vx = (torch.randn((3, H, P, d), generator=g).to(dtype) for _ in range(2))
        k[pages], v[pages] = kx.cuda(), vx.cuda()
        q = torch.randn((70, H, d), generator=g).to(dtype)
        ws = torch.zeros(qskv.prefill_workspace_size(shape, 70), dtype=torch.uint8, device="cuda")
        out = torch.empty((70, H, d), dtype=dtype, device="cuda")
        qc, table, lens, cu = q.cuda(), _i32([pages]), _i32([90]), _i32([0, 70])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        qskv.paged_prefill(qc, k, v, table, lens, cu, out, shape, ws, stream=side)
        side.synchronize()
        assert qskv.get_error(ws) == 0
        for h in range(H):
            kk, vv = (x[:, h].reshape(-1, d)[:90].double() for x in (kx, vx))
            o, _, pabs, A = R.attend_rows(q[:, h:h + 1], kk, vv, 20 + torch.arange(70), d ** -0.5)
            tol, _ = R.bounds(o, pabs, float(vv.abs().max()), A, 90, d, dtype == BF16)
            assert bool(((out[:, h:h + 1].cpu().double() - o).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,P", [(64, 16), (64, 32), (128, 16), (128, 32)])
def test_every_number_of_an_8_bit_cache(dtype, d, P):
    """Rows of one token: the output is its value, whatever code and power, and the lse its key's dim that the query asks for."""
    g = torch.Generator().manual_seed(d + P)
    B, H, G = 96, 2, 8
    codes = [torch.randint(0, 256, (B, H, P, d), generator=g) for _ in range(2)]
    codes = [torch.where((u & 127) == 127, u - 1, u) for u in codes]
    # (a logit of 2^20 keeps 2^-4 in fp32, which is as far as this asks for)
    powers = [torch.randint(-100, 12, (B, H, P), generator=g), torch.randint(-100, 120, (B, H, P), generator=g)]
    powers[1][::2] = torch.randint(-12, 14, powers[1][::2].shape, generator=g)
    pool = F.pack(codes[0], powers[0], codes[1], powers[1]).cuda()
    k, v = F.values(codes[0], powers[0])[:, :, 0], F.values(codes[1], powers[1])[:, :, 0]
    shape = qskv.make_shape(B, H * G, H, d, P, 1, B)
    table, lens, cu = _i32([[b] for b in range(B)]), _i32([1] * B), _i32(list(range(B + 1)))
    ws = torch.zeros(qskv.prefill_workspace_size(shape, B), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((B, H * G, d), dtype=dtype, device="cuda"), torch.empty((B, H * G), device="cuda")
    dims = torch.randint(0, d, (B, H * G), generator=g)
    q = torch.zeros((B, H * G, d), dtype=dtype).scatter_(2, dims[..., None], 1.0)
    qskv.kvf_paged_prefill(torch.zeros_like(q).cuda(), pool, table, lens, cu, out, shape, ws, lse=lse, sm_scale=1.0)
    assert torch.equal(out.cpu().double(), v.repeat_interleave(G, 1)) and bool((lse == 0).all())
    qskv.kvf_paged_prefill(q.cuda(), pool, table, lens, cu, out, shape, ws, lse=lse, sm_scale=1.0)
    assert qskv.get_error(ws) == 0
    want = k.repeat_interleave(G, 1).gather(2, dims[..., None])[..., 0]
    # scaled by log2 e and back by ln 2: two constants, two products and their sum, 2^-24 each; the weight's exponent 2^-22
    assert bool(((lse.cpu().double() - want).abs() <= 5 * 2.0 ** -24 * want.abs() + 2.0 ** -22).all())


# --------------------------------------------------- with what calls it --
def test_paged_decoder_prefills_and_decodes():
    """PagedDecoder.prefill over bf16 pools; a decode step's output is the prefill's of the last token."""
    b = Batch(12, [(0, 200), (64, 33), (10, 1)], 8, 2, 128, 16, BF16, "bf16", pad=0)
    last = torch.tensor([n - 1 for n in b.cu[1:]])
    q = b.gpu["q"][last.cuda()].contiguous()
    dec = qskv.PagedDecoder(q, b.pools["k_pool"], b.pools["v_pool"], b.gpu["page_table"], b.gpu["seq_lens"], None,
                            prefill_tokens=b.T)
    out = dec.prefill(b.gpu["q"], b.gpu["cu_new"], lse=b.lse)
    b.out, b.ws = out, dec.workspace
    b.check()
    dec.decode()
    dec.check()
    # both within their own bounds of the exact value: bf16 weights and a bf16 output here, bf16 weights there
    diff = (out[last.cuda()].float() - dec.out).abs()
    assert float(diff.max()) <= 4 * 2.0 ** -8 * float(b.v.abs().max())
    with pytest.raises(ValueError, match="prefill_tokens"):
        dec.prefill(torch.zeros((b.T + 1, 8, 128), dtype=BF16, device="cuda"), b.gpu["cu_new"])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_batch_prefilled_and_served_from_an_8_bit_cache(dtype):
    """Prompts in chunks through QuantizedPagedDecoder.prefill, then single tokens through step."""
    g = torch.Generator().manual_seed(13)
    dec = qskv.QuantizedPagedDecoder(3, 8, 2, 128, 16, max_pages=30, num_pool_pages=60, top_k=None, max_tokens=400, bits=8)
    seen = [[torch.empty((0, 2, 128))] * 2 for _ in range(3)]

    def bring(new):
        k, v = (torch.randn((sum(new), 2, 128), generator=g).to(dtype) for _ in range(2))
        at = 0
        for b, n in enumerate(new):
            for i, x in enumerate((k, v)):
                seen[b][i] = torch.cat([seen[b][i], x[at:at + n].float()])
            at += n
        return k.cuda(), v.cuda()

    def check(q, out, new):
        at = 0
        for b, n in enumerate(new):
            if n:
                kc, vc = (F.values(*F.quantise(x)) for x in seen[b])
                for h in range(2):
                    hs, pos = slice(4 * h, 4 * h + 4), len(kc) - n + torch.arange(n)
                    o, _, pabs, A = R.attend_rows(q[at:at + n, hs], kc[:, h], vc[:, h], pos, 128 ** -0.5)
                    tol, _ = R.bounds(o, pabs, float(vc.abs().max()), A, len(kc), 128, out.dtype == BF16)
                    assert bool(((out[at:at + n, hs].cpu().double() - o).abs() <= tol).all()), (b, h)
            at += n

    for new in ([150, 0, 17], [100, 70, 0], [1, 60, 3]):
        q = torch.randn((sum(new), 8, 128), generator=g).to(dtype)
        out = dec.prefill(q.cuda(), *bring(new), new)
        dec.check()
        check(q, out, new)
    q = torch.randn((3, 8, 128), generator=g).to(dtype)
    dec.step(q.cuda(), *bring([1, 1, 1]))
    dec.check()
    check(q, dec.out, [1, 1, 1])
    before = list(dec.lengths), dec.free_pages.numel()
    k, v = (torch.zeros((5, 2, 128), dtype=dtype, device="cuda") for _ in range(2))
    q = torch.zeros((5, 8, 128), dtype=dtype, device="cuda")
    for args, match in (((q[:4], k, v, [5, 0, 0]), "q"), ((q, k[:4], v, [5, 0, 0]), "keys"), ((q, k, v.double(), [5, 0, 0]), "v")):
        with pytest.raises(ValueError, match=match):
            dec.prefill(*args)
    with pytest.raises(ValueError, match="out"):
        dec.prefill(q, k, v, [5, 0, 0], out=q[:3])
    assert before == (list(dec.lengths), dec.free_pages.numel())
    four = qskv.QuantizedPagedDecoder(3, 8, 2, 128, 16, max_pages=30, num_pool_pages=60)
    with pytest.raises(ValueError, match="bits"):
        four.prefill(q, k, v, [5, 0, 0])
