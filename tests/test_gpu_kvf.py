"""The 8-bit paged cache on the GPU against the 64-bit statements of kvf_ref."""
import math

import pytest
import torch

import kvf_ref as R
import query_aware_sparse_kv_gb300 as qskv
from kvq_ref import attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from query_aware_sparse_kv_gb300 import build

    build.build()
    qskv.load()


def _ws(n=256):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _data(g, *shape):
    """Rows of very different ranges: plain, shifted, tiny, huge, constant, ties, zeros, below the smallest power."""
    x = torch.randn(shape, generator=g)
    kind = torch.randint(0, 8, shape[:-1] + (1,), generator=g)
    x = torch.where(kind == 1, x + 40, x)
    x = torch.where(kind == 2, x * 1e-6, x)
    x = torch.where(kind == 3, x * 1e9, x)
    x = torch.where(kind == 4, torch.full_like(x, -448.0), x)
    x = torch.where(kind == 5, torch.round(x * 16) * 1.0625, x)  # halves of a code's step among them
    x = torch.where(kind == 6, torch.zeros_like(x), x)
    return torch.where(kind == 7, x * 1e-32, x)


# ------------------------------------------------------ append and gather --
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P,H,n,kind", [(16, 3, 1, "any"), (16, 1, 37, "any"), (32, 2, 200, "runs"), (32, 5, 33, "any"),
                                        (16, 8, 5003, "runs"), (32, 8, 4100, "runs")])
def test_append_stores_exactly_and_gather_reads_back(dtype, d, P, H, n, kind):
    """Every byte of the pool: the reference's where a token went, as before elsewhere.  Runs start at any place of a
    page, so pairs of tokens lie across threads; the long ones take several tokens a thread."""
    g = torch.Generator().manual_seed(n * d + P)
    if kind == "runs":
        length = 61
        runs = -(-n // length)
        per = -(-(length + P) // P)
        N = runs * per + 3
        i = torch.arange(n)
        at = i % length + torch.randint(0, P, (runs,), generator=g)[i // length]
        slots = (torch.randperm(N, generator=g)[i // length * per + at // P] * P + at % P).to(torch.int32)
    else:
        N = n // 4 + 6
        slots = torch.randperm(N * P, generator=g)[:n].to(torch.int32)
    shape = qskv.make_shape(1, H, H, d, P, 1, N)
    k, v = _data(g, n, H, d).to(dtype), _data(g, n, H, d).to(dtype)
    skip = torch.rand(n, generator=g) < 0.1
    slots[skip] = -1 - torch.randint(0, 1000, (int(skip.sum()),), generator=g).to(torch.int32)
    before = torch.randint(0, 256, (N, H, qskv.kvf_block_bytes(shape)), generator=g, dtype=torch.uint8)
    pool, ws = before.cuda(), _ws()
    qkv = torch.full((n, 3 * H + 1, d), float("nan"), dtype=dtype, device="cuda")  # rows of a wider projection output
    qkv[:, H:2 * H], qkv[:, 2 * H:3 * H] = k.cuda(), v.cuda()
    qskv.kvf_append(qkv[:, H:2 * H], qkv[:, 2 * H:3 * H], slots.cuda(), pool, shape, ws)
    assert qskv.get_error(ws) == 0
    new = [R.quantise(x) for x in (k, v)]
    live = slots >= 0
    page, t = slots[live].long() // P, slots[live].long() % P
    want = before.clone()
    key, val, kp, vp = R.places(d, P)
    heads = torch.arange(H)[None, :]
    for codes, powers, (u, e) in ((key, kp, new[0]), (val, vp, new[1])):
        want[page[:, None, None], heads[:, :, None], codes[t][:, None, :]] = u[live].to(torch.uint8)
        want[page[:, None], heads, powers[t][:, None]] = (e[live] + 127).to(torch.uint8)
    got = pool.cpu()
    if not torch.equal(got, want):
        # a zero's sign is not part of the format
        bad = torch.nonzero(got != want)
        assert False, (len(bad), bad[:5].tolist(), got[tuple(bad[0])].item(), want[tuple(bad[0])].item())
    for out_dtype in (torch.float32, torch.bfloat16):
        ko, vo = (torch.full((n, H, d), float("nan"), dtype=out_dtype, device="cuda") for _ in range(2))
        qskv.kvf_gather(pool, slots.cuda(), ko, vo, shape, ws)
        assert qskv.get_error(ws) == 0
        for o, x in ((ko, new[0]), (vo, new[1])):
            exact = torch.where(live[:, None, None], R.values(*x), torch.zeros((), dtype=torch.float64))
            assert torch.equal(o.cpu().double(), exact)  # both types hold every value


def test_gather_repeated_and_unordered_slots():
    shape = qskv.make_shape(1, 2, 2, 64, 16, 1, 4)
    g = torch.Generator().manual_seed(5)
    f = [R.quantise(torch.randn((4, 2, 16, 64), generator=g)) for _ in range(2)]
    pool, ws = R.pack(*f[0], *f[1]).cuda(), _ws()
    slots = _i32([63, 5, 5, 0, 63, -1, 17])
    ko, vo = (torch.empty((7, 2, 64), device="cuda") for _ in range(2))
    qskv.kvf_gather(pool, slots, ko, vo, shape, ws)
    for o, x in ((ko, f[0]), (vo, f[1])):
        val = R.values(*x).float().transpose(1, 2).reshape(64, 2, 64)  # [slot][H][d]
        val = torch.cat([val, torch.zeros((1, 2, 64))])
        assert torch.equal(o.cpu(), val[[63, 5, 5, 0, 63, 64, 17]])


def test_slots_past_the_pool_are_flagged_and_skipped():
    shape = qskv.make_shape(1, 2, 2, 64, 16, 1, 4)
    pool, ws = _ws(4 * 2 * qskv.kvf_block_bytes(shape)).view(4, 2, -1), _ws()
    k = torch.ones((3, 2, 64), device="cuda")
    slots = _i32([64, 3, 2 ** 31 - 1])
    qskv.kvf_append(k, k, slots, pool, shape, ws)
    assert qskv.get_error(ws) == 5 and qskv.get_error(ws) == 0
    ko, vo = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    qskv.kvf_gather(pool, slots, ko, vo, shape, ws)
    assert qskv.get_error(ws) == 5
    for o in (ko, vo):
        assert o[1].eq(1).all() and o[0].eq(0).all() and o[2].eq(0).all()


def test_nothing_to_store_or_read():
    shape = qskv.make_shape(1, 2, 2, 64, 16, 1, 4)
    pool, ws = _ws(4 * 2 * qskv.kvf_block_bytes(shape)).view(4, 2, -1), _ws()
    none, k = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty((0, 2, 64), device="cuda")
    qskv.kvf_append(k, k, none, pool, shape, ws)
    qskv.kvf_gather(pool, none, k, k, shape, ws)
    qskv.kvf_meta_build(pool, none, none, torch.empty((4, 2, 2, 64), device="cuda"), shape, ws)
    assert qskv.get_error(ws) == 0 and int(pool.sum()) == 0


def test_offsets_past_32_bits():
    """A pool of over 4 GiB: the last page stored, read, summarised and attended."""
    d, P, H, N = 128, 32, 8, 70_000
    shape = qskv.make_shape(1, H, H, d, P, 1, N)
    pool = torch.empty((N, H, qskv.kvf_block_bytes(shape)), dtype=torch.uint8, device="cuda")
    assert pool.numel() > 2 ** 32
    ws = _ws(qskv.kvf_workspace_size(shape))
    g = torch.Generator().manual_seed(1)
    k, v = torch.randn((20, H, d), generator=g), torch.randn((20, H, d), generator=g)
    slots = ((N - 1) * P + torch.arange(20)).to(torch.int32).cuda()
    qskv.kvf_append(k.cuda(), v.cuda(), slots, pool, shape, ws)
    ko, vo = torch.empty((20, H, d), device="cuda"), torch.empty((20, H, d), device="cuda")
    qskv.kvf_gather(pool, slots, ko, vo, shape, ws)
    kx, vx = (R.values(*R.quantise(x)) for x in (k, v))
    assert torch.equal(ko.cpu(), kx.float()) and torch.equal(vo.cpu(), vx.float())
    meta = torch.zeros((N, H, 2, d), device="cuda")
    qskv.kvf_meta_build(pool, _i32([N - 1]), _i32([20]), meta, shape, ws)
    assert torch.equal(meta[-1, :, 0].cpu(), kx.float().amin(0)) and torch.equal(meta[-1, :, 1].cpu(), kx.float().amax(0))
    q = torch.randn((1, H, d), generator=g)
    out = torch.empty((1, H, d), device="cuda")
    qskv.kvf_paged_decode(q.cuda(), pool, _i32([[N - 1]]), _i32([20]), out, shape, ws)
    assert qskv.get_error(ws) == 0
    for h in range(H):
        o, _ = attend(q[0, h:h + 1], kx[:, h], vx[:, h], d ** -0.5)
        assert (out[0, h].cpu().double() - o[0]).abs().max() < R.attend_bounds(q[0, h:h + 1], kx[:, h], vx[:, h], d ** -0.5)[0]


# ------------------------------------------------------------- metadata --
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 32])
def test_metadata_is_that_of_the_cached_keys(d, P):
    g = torch.Generator().manual_seed(d + P)
    N, H = 9, 3
    shape = qskv.make_shape(1, H, H, d, P, 1, N)
    f = [R.quantise(_data(g, N, H, P, d)) for _ in range(2)]
    ids, valid = [3, -1, 0, 8, 5, -7], [P, 0, 1, P - 1, 7, 99]
    k = R.values(*f[0])
    pool = R.pack(*f[0], *f[1])
    key, _, kp, _ = R.places(d, P)
    for i, n in zip(ids, valid):  # what lies past a page's tokens is no number
        if i >= 0:
            pool[i][:, key[n:].flatten()] = R.NAN
            pool[i][:, kp[n:]] = 255
    pool, ws = pool.cuda(), _ws()
    for dtype in (torch.float32, torch.bfloat16):
        meta = torch.full((N, H, 2, d), 123.0, dtype=dtype, device="cuda")
        qskv.kvf_meta_build(pool, _i32(ids), _i32(valid), meta, shape, ws)
        assert qskv.get_error(ws) == 0
        got = meta.cpu().double()
        for p in range(N):
            if p not in ids:
                assert bool((got[p] == 123.0).all())
                continue
            n = valid[ids.index(p)]
            assert torch.equal(got[p, :, 0], k[p, :, :n].amin(1)) and torch.equal(got[p, :, 1], k[p, :, :n].amax(1))


def test_metadata_of_bad_entries_is_flagged_and_left():
    shape = qskv.make_shape(1, 2, 2, 64, 16, 1, 4)
    pool, ws = _ws(4 * 2 * qskv.kvf_block_bytes(shape)).view(4, 2, -1), _ws()
    meta = torch.full((4, 2, 2, 64), 5.0, device="cuda")
    for ids, valid in (([4], [1]), ([1], [0]), ([1], [17])):
        qskv.kvf_meta_build(pool, _i32(ids), _i32(valid), meta, shape, ws)
        assert qskv.get_error(ws) == 5
    assert bool((meta == 5).all())


@pytest.mark.parametrize("d,P,H,entries", [(64, 16, 3, 60000), (64, 32, 1, 3001), (128, 16, 5, 30000), (128, 32, 8, 999)])
def test_metadata_of_long_lists(d, P, H, entries):
    """Odd numbers of heads; full, part filled, skipped and bad entries next to one another."""
    g = torch.Generator().manual_seed(entries)
    N = 61
    shape = qskv.make_shape(1, H, H, d, P, 1, N)
    f = [R.quantise(torch.randn((N, H, P, d), generator=g)) for _ in range(2)]
    pool, ws = R.pack(*f[0], *f[1]).cuda(), _ws()
    filled = torch.randint(1, P + 1, (N,), generator=g)
    filled[::2] = P
    k = R.values(*f[0])
    for bad in (False, True):
        ids = torch.randint(0, N - 1, (entries,), generator=g)  # a page listed again is given the same count again
        valid = filled[ids]
        ids[5::7] = -1
        if bad:
            ids[3::101], valid[4::103] = N, P + 1
        meta = torch.full((N, H, 2, d), 123.0, device="cuda")
        qskv.kvf_meta_build(pool, ids.int().cuda(), valid.int().cuda(), meta, shape, ws)
        assert qskv.get_error(ws) == (5 if bad else 0)
        want = torch.full((N, H, 2, d), 123.0, dtype=torch.float64)
        for p in range(N):
            if bool(((ids == p) & (valid <= P)).any()):
                x = k[p, :, :int(filled[p])]
                want[p] = torch.stack([x.amin(1), x.amax(1)], 1)
        assert torch.equal(meta.cpu().double(), want)


# --------------------------------------------------------------- decode --
def spoil(pool, page, first, d, P):
    """A page's places from `first` on become anything: not-a-number codes, extreme powers."""
    key, val, kp, vp = R.places(d, P)
    pool[page][:, key[first:].flatten()] = R.NAN
    pool[page][:, val[first:].flatten()] = 255
    pool[page][:, kp[first:]] = 255
    pool[page][:, vp[first:]] = 0


class Batch:
    """A random batch: pool, tables and values on the CPU, what the decode takes on the GPU."""

    def __init__(self, seed, lens, hq, hkv, d, P, dtype, k=None, v=None, q_scale=1.0, extra=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hkv, self.d, self.P = lens, hq, hkv, d, P
        B, n = len(lens), [-(-x // P) for x in lens]
        self.mp = max(1, max(n)) + extra
        N = sum(n) + 2
        self.shape = qskv.make_shape(B, hq, hkv, d, P, self.mp, N)
        k = torch.randn((N, hkv, P, d), generator=g) if k is None else k(g, (N, hkv, P, d))
        v = torch.randn((N, hkv, P, d), generator=g) if v is None else v(g, (N, hkv, P, d))
        k, v = R.quantise(k), R.quantise(v)
        self.k, self.v = R.values(*k), R.values(*v)
        pool = R.pack(*k, *v)
        ids = torch.randperm(N, generator=g)
        self.table = torch.full((B, self.mp), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :n[b]] = ids[at:at + n[b]].to(torch.int32)
            at += n[b]
            if lens[b] % P:
                spoil(pool, int(self.table[b, n[b] - 1]), lens[b] % P, d, P)
        self.q = (torch.randn((B, hq, d), generator=g) * q_scale).to(dtype)
        self.pool, self.n = pool, n
        self.gpu = dict(q=self.q.cuda(), pool=pool.cuda(), page_table=self.table.cuda(), seq_lens=_i32(lens))
        self.ws = _ws(qskv.kvf_workspace_size(self.shape))
        self.out = torch.full((B, hq, d), float("nan"), device="cuda")
        self.lse = torch.full((B, hq), float("nan"), device="cuda")

    def decode(self, selected=None, top_k=0, scale=0.0, **over):
        kw = dict(self.gpu, out=self.out, lse=self.lse, workspace=self.ws, shape=self.shape)
        if selected is not None:  # lists [B][H] of pages
            sel = torch.full((len(self.lens), self.hkv, top_k), -1, dtype=torch.int32)
            for b, row in enumerate(selected):
                for h, pages in enumerate(row):
                    sel[b, h, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
            kw.update(selected=sel.cuda(), top_k=top_k, n_selected=_i32([[len(p) for p in row] for row in selected]))
        kw.update(over)
        qskv.kvf_paged_decode(sm_scale=scale, **kw)

    def check(self, selected=None, scale=0.0):
        assert qskv.get_error(self.ws) == 0
        out, lse, G = self.out.cpu().double(), self.lse.cpu().double(), self.hq // self.hkv
        scale = scale or self.d ** -0.5
        for b, h in [(b, h) for b in range(len(self.lens)) for h in range(self.hkv)]:
            pages = selected[b][h] if selected is not None else range(self.n[b])
            at = [(int(self.table[b, j]), t) for j in pages for t in range(min(self.P, self.lens[b] - j * self.P))]
            hs = slice(h * G, (h + 1) * G)
            if not at:
                assert bool((out[b, hs] == 0).all()) and bool((lse[b, hs] == -math.inf).all())
                continue
            p, t = ([x[i] for x in at] for i in (0, 1))
            kx, vx = self.k[p, h, t], self.v[p, h, t]
            o, z = attend(self.q[b, hs], kx, vx, scale)
            tol, ltol = R.attend_bounds(self.q[b, hs], kx, vx, scale)
            err, lerr = float((out[b, hs] - o).abs().max()), float((lse[b, hs] - z).abs().max())
            assert err <= tol and lerr <= ltol + 2.0 ** -22 * float(z.abs().max()), (b, h, len(at), err, tol, lerr, ltol)


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 100, 257]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("hq,hkv", [(3, 3), (4, 2), (4, 1), (16, 2)])
def test_decode_over_all_pages(dtype, d, P, hq, hkv):
    b = Batch(hq * d + P, LENS, hq, hkv, d, P, dtype)
    b.decode()
    b.check()


@pytest.mark.parametrize("d,P,hq,hkv", [(64, 16, 2, 2), (128, 16, 8, 2), (128, 32, 8, 1), (64, 32, 3, 3)])
def test_decode_over_selected_pages(d, P, hq, hkv):
    g = torch.Generator().manual_seed(3)
    b = Batch(9, [0, 5, 16, 300, 1000], hq, hkv, d, P, torch.bfloat16)
    sel = []
    for n in b.n:
        row = []
        for h in range(hkv):
            m = min(n, int(torch.randint(0, 20, (1,), generator=g)))  # rows that select nothing among them
            row.append(sorted(torch.randperm(n, generator=g)[:m].tolist()))
        sel.append(row)
    sel[4][0] = sorted(set(sel[4][0] + [b.n[4] - 1]))  # the partial last page
    b.decode(selected=sel, top_k=24)
    b.check(selected=sel)
    b.decode(selected=sel, top_k=24, scale=0.37)
    b.check(selected=sel, scale=0.37)


@pytest.mark.parametrize("lens,hq,hkv,d,P", [
    ([5000], 8, 1, 128, 16),             # one row over the whole GPU
    ([40_000], 2, 2, 64, 32),
    ([1, 9000, 0, 3, 2500], 4, 2, 128, 32),
    ([20] * 700, 4, 2, 64, 16),          # many short rows, whole ones a warp
    (list(range(0, 400, 3)), 16, 2, 128, 16),
    ([50 + i % 70 for i in range(400)], 8, 8, 64, 32),
])
def test_decode_work_splits(lens, hq, hkv, d, P):
    b = Batch(len(lens), lens, hq, hkv, d, P, torch.float32)
    b.decode()
    first = b.out.clone(), b.lse.clone()
    b.check()
    b.decode()  # tickets are back at zero; equal inputs give equal bits
    assert torch.equal(b.out, first[0]) and torch.equal(b.lse, first[1])


@pytest.mark.parametrize("case", ["large", "steps", "zeros", "mixed", "sharp", "zero_queries"])
def test_decode_of_unusual_values(case):
    """Keys and values of very different powers, all-zero values, logits far apart."""
    def ranges(g, s):
        return torch.randn(s, generator=g) * 2.0 ** torch.randint(-20, 20, s[:-1] + (1,), generator=g)

    def zeros(g, s):
        return torch.randn(s, generator=g) * (torch.rand(s[:-1] + (1,), generator=g) < 0.5)

    k = {"large": lambda g, s: torch.randn(s, generator=g) * 1e3, "sharp": lambda g, s: torch.randn(s, generator=g) * 30,
         "steps": lambda g, s: torch.randn(s, generator=g) * torch.linspace(0, 4, s[0])[:, None, None, None]}.get(case)
    v = {"large": lambda g, s: torch.randn(s, generator=g) * 1e15, "steps": ranges, "mixed": ranges, "zeros": zeros,
         "zero_queries": zeros}.get(case)
    q_scale = {"large": 1e-3, "zero_queries": 0.0}.get(case, 1.0)
    for d, P, hq, hkv in ((128, 16, 8, 1), (64, 32, 2, 2)):
        b = Batch(17, [0, 3, 40, 333, 2000], hq, hkv, d, P, torch.float32, k=k, v=v, q_scale=q_scale)
        b.decode()
        b.check()
    if case == "zeros":  # only zeros: their power is the smallest there is
        b = Batch(18, [5, 700], 4, 1, 128, 16, torch.bfloat16, v=lambda g, s: torch.zeros(s))
        b.decode()
        b.check()
        assert bool((b.out == 0).all())


def test_bad_pages_and_lengths_are_flagged_and_skipped():
    b = Batch(4, [40, 50, 20], 2, 1, 64, 16, torch.float32)
    table = b.table.clone()
    table[1, 1] = b.shape.num_pool_pages  # outside the pool
    b.decode(page_table=table.cuda())
    assert qskv.get_error(b.ws) == 5
    keep = [j for j in range(4) if j != 1]
    sel = [[list(range(3))], [keep], [list(range(2))]]
    b.check(selected=sel)
    b.decode(seq_lens=_i32([40, -3, b.mp * 16 + 1]))
    assert qskv.get_error(b.ws) == 5
    b.decode(selected=[[[0, 3]], [[2]], [[1]]], top_k=2)  # page 3 of a row of 3
    assert qskv.get_error(b.ws) == 5
    b.check(selected=[[[0]], [[2]], [[1]]])


def test_pinned_host_buffers_and_no_lse():
    b = Batch(5, [100, 7], 4, 2, 128, 16, torch.bfloat16)
    q, out = b.q.pin_memory(), torch.full((2, 4, 128), float("nan")).pin_memory()
    b.decode()
    b.decode(q=q, out=out, lse=None)
    torch.cuda.synchronize()
    assert torch.equal(out, b.out.cpu())


def test_on_a_side_stream_and_in_a_graph():
    """The whole cache path on a stream of its own, captured and replayed with other inputs."""
    shape = qskv.make_shape(2, 8, 2, 128, 16, 4, 10)
    g = torch.Generator().manual_seed(8)
    pool = torch.zeros((10, 2, qskv.kvf_block_bytes(shape)), dtype=torch.uint8, device="cuda")
    ws = _ws(qskv.kvf_workspace_size(shape))
    k, v = (torch.zeros((50, 2, 128), device="cuda") for _ in range(2))
    q = torch.zeros((2, 8, 128), device="cuda")
    slots, table, lens = _i32(list(range(50))), _i32([[0, 1, 2, -1], [3, -1, -1, -1]]), _i32([48, 2])
    out, lse = torch.empty((2, 8, 128), device="cuda"), torch.empty((2, 8), device="cuda")

    def body():
        qskv.kvf_append(k, v, slots, pool, shape, ws)
        qskv.kvf_paged_decode(q, pool, table, lens, out, shape, ws, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for _ in range(2):
        x = [torch.randn(t.shape, generator=g) for t in (k, v, q)]
        for t, y in zip((k, v, q), x):
            t.copy_(y)
        graph.replay()
        got = out.clone(), lse.clone()
        body()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
        kx, vx = (R.values(*R.quantise(y)) for y in x[:2])
        o, _ = attend(x[2][0, :4], kx[:48, 0], vx[:48, 0], 128 ** -0.5)
        assert (out[0, :4].cpu().double() - o).abs().max() <= R.attend_bounds(x[2][0, :4], kx[:48, 0], vx[:48, 0], 128 ** -0.5)[0]
    assert qskv.get_error(ws) == 0


# --------------------------------------------------- all of them together --
@pytest.mark.parametrize("top_k", [None, 3])
def test_a_batch_served_from_an_8_bit_cache(top_k):
    """QuantizedPagedDecoder with bits=8: prompts, single tokens, a row released and taken again."""
    g = torch.Generator().manual_seed(11)
    dec = qskv.QuantizedPagedDecoder(3, 8, 2, 128, 16, max_pages=12, num_pool_pages=30, top_k=top_k, max_tokens=256, bits=8)
    seen = [[torch.empty((0, 2, 128))] * 2 for _ in range(3)]
    for new in ([100, 0, 17], [1, 1, 1], [1, 60, 1], [5, 0, 3]):
        k, v = (torch.randn((sum(new), 2, 128), generator=g).bfloat16() for _ in range(2))
        q = torch.randn((3, 8, 128), generator=g).bfloat16()
        dec.step(q.cuda(), k.cuda(), v.cuda(), new)
        dec.check()
        at = 0
        for b, n in enumerate(new):
            for i, x in enumerate((k, v)):
                seen[b][i] = torch.cat([seen[b][i], x[at:at + n].float()])
            at += n
            kc, vc = (R.values(*R.quantise(x)) for x in seen[b])
            gk, gv = dec.gather(b)
            assert torch.equal(gk.cpu().double(), kc) and torch.equal(gv.cpu().double(), vc)
            for h in range(2):
                pages = range(-(-len(kc) // 16)) if top_k is None else dec.selected[b, h, :int(dec.n_selected[b, h])].tolist()
                assert top_k is None or len(pages) == min(top_k, -(-len(kc) // 16))
                t = [i for j in pages for i in range(j * 16, min(len(kc), j * 16 + 16))]
                hs = slice(4 * h, 4 * h + 4)
                if not t:
                    assert bool((dec.out[b, hs] == 0).all())
                    continue
                o, _ = attend(q[b, hs], kc[t, h], vc[t, h], 128 ** -0.5)
                tol = R.attend_bounds(q[b, hs], kc[t, h], vc[t, h], 128 ** -0.5)[0]
                assert (dec.out[b, hs].cpu().double() - o).abs().max() <= tol
        if new[1] == 60:
            dec.release(1)
            seen[1] = [torch.empty((0, 2, 128))] * 2
    with pytest.raises(ValueError, match="bits"):
        qskv.QuantizedPagedDecoder(3, 8, 2, 128, 16, max_pages=12, num_pool_pages=30, bits=6)
