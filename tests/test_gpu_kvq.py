"""The 4-bit paged cache on the GPU against the 64-bit statements of kvq_ref."""
import math

import pytest
import torch

import kvq_ref as R
import query_aware_sparse_kv_gb300 as qskv

pytestmark = pytest.mark.gpu

FORMATS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from query_aware_sparse_kv_gb300 import build

    build.build()
    qskv.load()


def _ws(n=256):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _data(g, *shape):
    """Rows of very different ranges: plain, shifted, tiny, huge, constant, two-valued."""
    x = torch.randn(shape, generator=g)
    kind = torch.randint(0, 7, shape[:-1] + (1,), generator=g)
    x = torch.where(kind == 1, x + 40, x)
    x = torch.where(kind == 2, x * 1e-6, x)
    x = torch.where(kind == 3, x * 1e6, x)
    x = torch.where(kind == 4, torch.full_like(x, -3.3), x)
    x = torch.where(kind == 5, torch.sign(x) * 0.75, x)  # m / s is a half: ties
    return torch.where(kind == 6, x * 1e-33, x)  # the scale is below 2^-100


# ------------------------------------------------------ append and gather --
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,gs", FORMATS)
@pytest.mark.parametrize("P,H,n,view", [(16, 3, 1, False), (16, 1, 37, True), (32, 2, 200, True), (32, 5, 33, False)])
def test_append_stores_exactly_and_gather_reads_back(dtype, d, gs, P, H, n, view):
    g = torch.Generator().manual_seed(n * d + gs + P)
    N = n // 4 + 6
    shape = qskv.make_shape(1, H, H, d, P, 1, N)
    k, v = _data(g, n, H, d).to(dtype), _data(g, n, H, d).to(dtype)
    slots = torch.randperm(N * P, generator=g)[:n].to(torch.int32)
    skip = torch.rand(n, generator=g) < 0.2
    slots[skip] = -1 - torch.randint(0, 1000, (int(skip.sum()),), generator=g).to(torch.int32)
    before = torch.randint(0, 256, (N, H, qskv.kvq_block_bytes(shape, gs)), generator=g, dtype=torch.uint8)
    pool, ws = before.cuda(), _ws()
    if view:  # the tokens' rows inside a wider projection output
        qkv = torch.full((n, 3 * H + 1, d), float("nan"), dtype=dtype, device="cuda")
        qkv[:, H:2 * H], qkv[:, 2 * H:3 * H] = k.cuda(), v.cuda()
        kc, vc = qkv[:, H:2 * H], qkv[:, 2 * H:3 * H]
    else:
        kc, vc = k.cuda(), v.cuda()
    qskv.kvq_append(kc, vc, slots.cuda(), pool, shape, gs, ws)
    assert qskv.get_error(ws) == 0
    # the untouched words are as before, the written ones are the reference's bits
    want = R.unpack(before, d, P, gs)
    new = [R.quantise(x, gs) for x in (k, v)]
    live = slots >= 0
    page, t = slots[live].long() // P, slots[live].long() % P
    for w, x in zip(want, new):
        for field, y in zip(w, x):
            field[page, :, t] = y[live]
    got = R.unpack(pool.cpu(), d, P, gs)
    for a, b, name in zip(got, want, ("keys", "values")):
        for x, y, f in zip(a, b, ("codes", "scales", "minima")):
            assert torch.equal(x.nan_to_num(1.5), y.nan_to_num(1.5)), (name, f)
    for out_dtype in (torch.float32, torch.bfloat16):
        ko, vo = (torch.full((n, H, d), float("nan"), dtype=out_dtype, device="cuda") for _ in range(2))
        qskv.kvq_gather(pool, slots.cuda(), ko, vo, shape, gs, ws)
        assert qskv.get_error(ws) == 0
        for o, x in ((ko, new[0]), (vo, new[1])):
            want_values = torch.where(live[:, None, None], R.values(*x), torch.zeros((), dtype=torch.float64))
            assert torch.equal(o.cpu(), want_values.float().to(out_dtype))  # m + s u rounded to fp32, then to out's type


def test_gather_repeated_and_unordered_slots():
    shape = qskv.make_shape(1, 2, 2, 64, 16, 1, 4)
    g = torch.Generator().manual_seed(5)
    f = [R.quantise(torch.randn((4, 2, 16, 64), generator=g), 32) for _ in range(2)]
    pool, ws = R.pack(*f[0], *f[1]).cuda(), _ws()
    slots = torch.tensor([63, 5, 5, 0, 63, -1, 17], dtype=torch.int32)
    ko, vo = (torch.empty((7, 2, 64), device="cuda") for _ in range(2))
    qskv.kvq_gather(pool, slots.cuda(), ko, vo, shape, 32, ws)
    for o, x in ((ko, f[0]), (vo, f[1])):
        val = R.values(*x).float().transpose(1, 2).reshape(64, 2, 64)  # [slot][H][d]
        val = torch.cat([val, torch.zeros((1, 2, 64))])
        assert torch.equal(o.cpu(), val[[63, 5, 5, 0, 63, 64, 17]])


def test_slots_past_the_pool_are_flagged_and_skipped():
    shape = qskv.make_shape(1, 2, 2, 64, 16, 1, 4)
    pool, ws = _ws(4 * 2 * qskv.kvq_block_bytes(shape, 64)).view(4, 2, -1), _ws()
    k = torch.ones((3, 2, 64), device="cuda")
    slots = torch.tensor([64, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    qskv.kvq_append(k, k, slots, pool, shape, 64, ws)
    assert qskv.get_error(ws) == 5 and qskv.get_error(ws) == 0
    ko, vo = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    qskv.kvq_gather(pool, slots, ko, vo, shape, 64, ws)
    assert qskv.get_error(ws) == 5
    for o in (ko, vo):
        assert o[1].eq(1).all() and o[0].eq(0).all() and o[2].eq(0).all()


def test_nothing_to_store_or_read():
    shape = qskv.make_shape(1, 2, 2, 64, 16, 1, 4)
    pool, ws = _ws(4 * 2 * qskv.kvq_block_bytes(shape, 64)).view(4, 2, -1), _ws()
    none, k = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty((0, 2, 64), device="cuda")
    qskv.kvq_append(k, k, none, pool, shape, 64, ws)
    qskv.kvq_gather(pool, none, k, k, shape, 64, ws)
    qskv.kvq_meta_build(pool, none, none, torch.empty((4, 2, 2, 64), device="cuda"), shape, 64, ws)
    assert qskv.get_error(ws) == 0 and int(pool.sum()) == 0


def test_offsets_past_32_bits():
    """A pool of over 4 GiB: the last page stored, read, summarised and attended."""
    d, gs, P, H = 128, 128, 32, 8
    N = 130_000
    shape = qskv.make_shape(1, H, H, d, P, 1, N)
    pool = torch.empty((N, H, qskv.kvq_block_bytes(shape, gs)), dtype=torch.uint8, device="cuda")
    assert pool.numel() > 2 ** 32
    ws = _ws(qskv.kvq_workspace_size(shape))
    g = torch.Generator().manual_seed(1)
    k, v = torch.randn((20, H, d), generator=g), torch.randn((20, H, d), generator=g)
    slots = ((N - 1) * P + torch.arange(20)).to(torch.int32).cuda()
    qskv.kvq_append(k.cuda(), v.cuda(), slots, pool, shape, gs, ws)
    ko, vo = torch.empty((20, H, d), device="cuda"), torch.empty((20, H, d), device="cuda")
    qskv.kvq_gather(pool, slots, ko, vo, shape, gs, ws)
    kx, vx = (R.values(*R.quantise(x, gs)) for x in (k, v))
    assert torch.equal(ko.cpu(), kx.float()) and torch.equal(vo.cpu(), vx.float())
    meta = torch.zeros((N, H, 2, d), device="cuda")
    last = torch.tensor([N - 1], dtype=torch.int32, device="cuda")
    qskv.kvq_meta_build(pool, last, torch.tensor([20], dtype=torch.int32, device="cuda"), meta, shape, gs, ws)
    assert torch.equal(meta[-1, :, 0].cpu(), kx.float().amin(0)) and torch.equal(meta[-1, :, 1].cpu(), kx.float().amax(0))
    q = torch.randn((1, H, d), generator=g)
    out = torch.empty((1, H, d), device="cuda")
    qskv.kvq_paged_decode(q.cuda(), pool, last.view(1, 1), torch.tensor([20], dtype=torch.int32, device="cuda"), out,
                          shape, gs, ws)
    assert qskv.get_error(ws) == 0
    for h in range(H):
        o, _ = R.attend(q[0, h:h + 1], kx[:, h], vx[:, h], d ** -0.5)
        assert (out[0, h].cpu().double() - o[0]).abs().max() < 1e-4


# ------------------------------------------------------------- metadata --
@pytest.mark.parametrize("d,gs", FORMATS)
@pytest.mark.parametrize("P", [16, 32])
def test_metadata_bounds_the_cached_keys(d, gs, P):
    g = torch.Generator().manual_seed(d + gs)
    N, H = 9, 3
    shape = qskv.make_shape(1, H, H, d, P, 1, N)
    f = [R.quantise(_data(g, N, H, P, d), gs) for _ in range(2)]
    pool, ws = R.pack(*f[0], *f[1]).cuda(), _ws()
    ids = torch.tensor([3, -1, 0, 8, 5, -7], dtype=torch.int32)
    valid = torch.tensor([P, 0, 1, P - 1, 7, 99], dtype=torch.int32)
    k = R.values(*f[0])
    for dtype in (torch.float32, torch.bfloat16):
        meta = torch.full((N, H, 2, d), 123.0, dtype=dtype, device="cuda")
        qskv.kvq_meta_build(pool, ids.cuda(), valid.cuda(), meta, shape, gs, ws)
        assert qskv.get_error(ws) == 0
        got = meta.cpu().double()
        for p in range(N):
            if p not in ids.tolist():
                assert bool((got[p] == 123.0).all())
                continue
            n = int(valid[ids.tolist().index(p)])
            lo, hi = k[p, :, :n].float().double().amin(1), k[p, :, :n].float().double().amax(1)
            if dtype == torch.float32:
                assert torch.equal(got[p, :, 0], lo) and torch.equal(got[p, :, 1], hi)
            else:  # the nearest bf16 outwards: a step (2^-7 of the value, 2^-133 for subnormals) away at most
                for x, y, s in ((got[p, :, 0], lo, -1), (got[p, :, 1], hi, 1)):
                    assert bool(((x - y) * s >= 0).all())
                    assert bool(((x - y).abs() < 2.0 ** -7 * y.abs() + 2.0 ** -133).all())
                    exact = y.float().to(torch.bfloat16).double() == y
                    assert torch.equal(x[exact], y[exact])


def test_metadata_of_bad_entries_is_flagged_and_left():
    shape = qskv.make_shape(1, 2, 2, 64, 16, 1, 4)
    pool, ws = _ws(4 * 2 * qskv.kvq_block_bytes(shape, 64)).view(4, 2, -1), _ws()
    meta = torch.full((4, 2, 2, 64), 5.0, device="cuda")
    for ids, valid in (([4], [1]), ([1], [0]), ([1], [17])):
        t = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (ids, valid)]
        qskv.kvq_meta_build(pool, *t, meta, shape, 64, ws)
        assert qskv.get_error(ws) == 5
    assert bool((meta == 5).all())


@pytest.mark.parametrize("d, gs, P, entries", [(64, 32, 16, 90000), (64, 64, 32, 3001), (128, 128, 16, 80000),
                                               (128, 32, 32, 20000)])
def test_metadata_of_long_lists(d, gs, P, entries):
    """Many tiles a warp, odd numbers of heads; full, part filled, skipped and bad entries next to one another."""
    g = torch.Generator().manual_seed(entries)
    N, H = 61, 3
    shape = qskv.make_shape(1, H, H, d, P, 1, N)
    f = [R.quantise(torch.randn((N, H, P, d), generator=g), gs) for _ in range(2)]
    pool, ws = R.pack(*f[0], *f[1]).cuda(), _ws()
    filled = torch.randint(1, P + 1, (N,), generator=g)
    filled[::2] = P
    k = R.values(*f[0]).float()
    want = torch.full((N, H, 2, d), 123.0)
    for bad in (False, True):
        ids = torch.randint(0, N - 1, (entries,), generator=g)  # a page listed again is given the same count again
        valid = filled[ids]
        ids[5::7] = -1
        if bad:
            ids[3::1001], valid[4::1009] = N, P + 1
        meta = torch.full((N, H, 2, d), 123.0, device="cuda")
        qskv.kvq_meta_build(pool, ids.int().cuda(), valid.int().cuda(), meta, shape, gs, ws)
        assert qskv.get_error(ws) == (5 if bad else 0)
        for p in range(N):
            listed = bool(((ids == p) & (valid <= P)).any())
            x = k[p, :, :int(filled[p])]
            want[p] = torch.stack([x.amin(1), x.amax(1)], 1) if listed else 123.0
        assert torch.equal(meta.cpu(), want)


# --------------------------------------------------------------- decode --
def _garbage(pool, page, first, d, P, gs):
    """The params of a page's places from `first` on become NaN, infinities and the type's extremes."""
    w = pool.view(torch.int32)
    W, ng = d // 8, d // gs
    bad = torch.tensor([0x7FC07FC0, 0x7F807F80, -8323200, 0x7F7F7F7F], dtype=torch.int64).to(torch.int32)
    for r in range(2 * ng):
        for t in range(first, P):
            w[page, :, 2 * P * W + r * P + t] = bad[(r + t) % 4]


class Batch:
    """A random batch: pool, tables and fields on the CPU, what decode takes on the GPU."""

    def __init__(self, seed, lens, hq, hkv, d, P, gs, dtype, k=None, v=None, q_scale=1.0, extra=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hkv, self.d, self.P, self.gs = lens, hq, hkv, d, P, gs
        B, n = len(lens), [-(-x // P) for x in lens]
        self.mp = max(1, max(n)) + extra
        N = sum(n) + 2
        self.shape = qskv.make_shape(B, hq, hkv, d, P, self.mp, N)
        k = torch.randn((N, hkv, P, d), generator=g) if k is None else k(g, (N, hkv, P, d))
        v = torch.randn((N, hkv, P, d), generator=g) if v is None else v(g, (N, hkv, P, d))
        self.k, self.v = R.quantise(k, gs), R.quantise(v, gs)
        pool = R.pack(*self.k, *self.v)
        ids = torch.randperm(N, generator=g)
        self.table = torch.full((B, self.mp), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            self.table[b, :n[b]] = ids[at:at + n[b]].to(torch.int32)
            at += n[b]
            if lens[b] % P:
                _garbage(pool, int(self.table[b, n[b] - 1]), lens[b] % P, d, P, gs)
        self.q = (torch.randn((B, hq, d), generator=g) * q_scale).to(dtype)
        self.pool, self.n = pool, n
        self.gpu = dict(q=self.q.cuda(), pool=pool.cuda(), page_table=self.table.cuda(),
                        seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        self.ws = _ws(qskv.kvq_workspace_size(self.shape))
        self.out = torch.full((B, hq, d), float("nan"), device="cuda")
        self.lse = torch.full((B, hq), float("nan"), device="cuda")

    def decode(self, selected=None, top_k=0, scale=0.0, **over):
        kw = dict(self.gpu, out=self.out, lse=self.lse, workspace=self.ws, shape=self.shape, group_size=self.gs)
        if selected is not None:  # lists [B][H] of pages
            sel = torch.full((len(self.lens), self.hkv, top_k), -1, dtype=torch.int32)
            for b, row in enumerate(selected):
                for h, pages in enumerate(row):
                    sel[b, h, :len(pages)] = torch.tensor(pages, dtype=torch.int32)
            kw.update(selected=sel.cuda(), top_k=top_k,
                      n_selected=torch.tensor([[len(p) for p in row] for row in selected], dtype=torch.int32).cuda())
        kw.update(over)
        qskv.kvq_paged_decode(sm_scale=scale, **kw)

    def check(self, selected=None, scale=0.0, rows=None):
        assert qskv.get_error(self.ws) == 0
        out, lse, G = self.out.cpu().double(), self.lse.cpu().double(), self.hq // self.hkv
        scale = scale or self.d ** -0.5
        kx, vx = R.values(*self.k), R.values(*self.v)
        for b, h in rows or [(b, h) for b in range(len(self.lens)) for h in range(self.hkv)]:
            pages = selected[b][h] if selected is not None else range(self.n[b])
            at = [(int(self.table[b, j]), t) for j in pages for t in range(min(self.P, self.lens[b] - j * self.P))]
            p, t = ([x[i] for x in at] for i in (0, 1))
            hs = slice(h * G, (h + 1) * G)
            o, l = R.attend(self.q[b, hs], kx[p, h, t], vx[p, h, t], scale)
            if not at:
                assert bool((out[b, hs] == 0).all()) and bool((lse[b, hs] == -math.inf).all())
                continue
            tol, ltol = R.attend_bounds(self.q[b, hs], self.k[2][p, h, t], self.k[1][p, h, t], self.v[2][p, h, t],
                                        self.v[1][p, h, t], scale, len(at))
            err, lerr = float((out[b, hs] - o).abs().max()), float((lse[b, hs] - l).abs().max())
            assert err <= tol and lerr <= ltol + 2.0 ** -22 * float(l.abs().max()), (b, h, len(at), err, tol, lerr, ltol)


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 100, 257]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,gs", FORMATS)
@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("hq,hkv", [(3, 3), (4, 2), (4, 1), (16, 2)])
def test_decode_over_all_pages(dtype, d, gs, P, hq, hkv):
    b = Batch(hq * d + gs, LENS, hq, hkv, d, P, gs, dtype)
    b.decode()
    b.check()


@pytest.mark.parametrize("d,gs,P,hq,hkv", [(64, 64, 16, 2, 2), (128, 128, 16, 8, 2), (128, 32, 32, 8, 1)])
def test_decode_over_selected_pages(d, gs, P, hq, hkv):
    g = torch.Generator().manual_seed(3)
    b = Batch(9, [0, 5, 16, 300, 1000], hq, hkv, d, P, gs, torch.bfloat16)
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


@pytest.mark.parametrize("lens,hq,hkv,d,P,gs", [
    ([5000], 8, 1, 128, 16, 128),        # one row over the whole GPU
    ([40_000], 2, 2, 64, 32, 32),
    ([3000, 1, 20_000, 0, 7], 4, 2, 128, 32, 64),
    ([1] * 700, 2, 2, 64, 16, 64),       # more rows than warps, one token each
    ([37] * 300 + [0] * 100 + [2000], 4, 4, 64, 16, 32),
    ([i * 7 % 41 for i in range(900)] + [500], 1, 1, 64, 16, 32),  # more sequences than the prefix has entries
    ([i * 13 % 190 for i in range(170)], 16, 2, 64, 16, 64),     # whole rows to warps, 8 heads, empty ones
    ([i * 29 % 350 for i in range(110)], 4, 4, 128, 32, 128),    # the same, pages of 32
])
def test_decode_splits_and_joins(lens, hq, hkv, d, P, gs):
    b = Batch(17, lens, hq, hkv, d, P, gs, torch.float32)
    b.decode()
    rows = [(i, h) for i in sorted({0, 1, 2, len(lens) // 2, len(lens) - 1} & set(range(len(lens)))) for h in range(hkv)]
    b.check(rows=rows)
    first = b.out.clone()
    for _ in range(3):  # no order of arrival shows
        b.decode()
        assert torch.equal(b.out, first)


@pytest.mark.parametrize("P,top_k,most", [(16, 5, 190), (16, 20, 700), (32, 40, 900)])
def test_decode_over_selected_pages_of_many_rows(P, top_k, most):
    """More rows than a wave of CTAs: short selections to warps whole, longer ones split evenly; some rows empty, some
    selecting nothing."""
    g = torch.Generator().manual_seed(top_k)
    lens = [0 if i % 17 == 0 else i * 37 % most for i in range(200)]
    b = Batch(31, lens, 4, 2, 64, P, 64, torch.bfloat16)
    sel = [[sorted(torch.randperm(n, generator=g)[:min(n, (i * 3 + h) % (top_k + 1))].tolist()) for h in range(2)]
           for i, n in enumerate(b.n)]
    b.decode(selected=sel, top_k=top_k)
    b.check(selected=sel)


def test_decode_with_a_wider_table_and_without_lse():
    b = Batch(2, [33, 64], 4, 2, 64, 16, 64, torch.float32, extra=37)
    b.decode()
    b.check()
    out = b.out.clone()
    b.decode(lse=None)
    assert torch.equal(out, b.out)


def _sink(g, shape):
    """Values of very different scale from token to token, some zero, some constant over the head."""
    x = torch.randn(shape, generator=g) * 10.0 ** (12 * torch.rand(shape[:-1] + (1,), generator=g) - 6)
    x[:, :, 3] = 0
    x[:, :, 5] = 0.25
    return x


@pytest.mark.parametrize("d,gs,hq", [(64, 32, 1), (128, 128, 4), (128, 64, 8)])
@pytest.mark.parametrize("q_scale", [1e-4, 1.0, 30.0])
def test_decode_with_values_of_every_scale(d, gs, hq, q_scale):
    """Sharp and flat softmaxes over values whose scale varies by 10^12 between tokens; the error is still relative to
    the weights' own values: the bound uses sum p (|m| + 15 s), not the largest value."""
    b = Batch(23, [200, 500], hq, 1, d, 16, gs, torch.float32, v=_sink, q_scale=q_scale)
    b.decode()
    assert qskv.get_error(b.ws) == 0
    out = b.out.cpu().double()
    kx, vx = R.values(*b.k), R.values(*b.v)
    for i, n in enumerate(b.lens):
        at = [(int(b.table[i, t // 16]), t % 16) for t in range(n)]
        p, t = ([x[j] for x in at] for j in (0, 1))
        x = b.q[i].double() @ kx[p, 0, t].T * d ** -0.5
        w = torch.softmax(x, -1)
        want = w @ vx[p, 0, t]
        ng = d // gs
        size = (b.v[2][p, 0, t].abs() + 15 * b.v[1][p, 0, t])  # [T][ng]
        kabs = (b.k[2][p, 0, t].abs() + 15 * b.k[1][p, 0, t]).amax(0).repeat_interleave(gs, -1)
        A = float((b.q[i].double().abs() @ kabs).max()) * d ** -0.5
        # 2 (d + 16) A roundings in the exponent on each token's own share, T in the sums; a weight's two
        # halves lose what is below 2^-25 of a 2^8 reference within 2^12: 2^-20 of the largest share
        share = (w[:, :, None] * size[None]).sum(1)
        top = (w[:, :, None] * size[None]).amax(1)
        tol = (2 * (d + 16) * A + n + 32) * 2.0 ** -24 * share + 2.0 ** -20 * top.amax(-1, keepdim=True)
        assert bool(((out[i] - want).abs() <= tol.repeat_interleave(gs, -1) * (1 if ng else 1)).all()), i


def test_decode_flags_bad_indices():
    b = Batch(4, [40, 20], 2, 2, 64, 16, 64, torch.float32)
    table = b.table.clone()
    table[0, 1] = int(b.shape.num_pool_pages)  # one past the pool: that page is skipped
    b.decode(page_table=table.cuda())
    assert qskv.get_error(b.ws) == 5
    keep = [[[0, 2]] * 2, [[0, 1]] * 2]
    assert qskv.get_error(b.ws) == 0
    b.check(selected=keep)
    b.decode(seq_lens=torch.tensor([-3, 20], dtype=torch.int32, device="cuda"))
    assert qskv.get_error(b.ws) == 5
    assert bool((b.out[0] == 0).all())
    b.decode(selected=[[[0, 3]] * 2, [[1]] * 2], top_k=4)  # page 3 of 3
    assert qskv.get_error(b.ws) == 5
    b.decode()
    b.check()


def test_decode_reads_and_writes_pinned_memory():
    b = Batch(6, [100, 3], 4, 2, 128, 16, 64, torch.bfloat16)
    q, out = b.q.pin_memory(), torch.empty(b.out.shape).pin_memory()
    b.decode(q=q, out=out)
    torch.cuda.synchronize()
    b.out.copy_(out)
    b.check()


def test_calls_on_another_stream_and_captured():
    """Append and decode recorded once, replayed with new tokens; a second graph shares the workspace."""
    b = Batch(8, [64, 30], 4, 2, 64, 16, 32, torch.float32)
    k, v = torch.zeros((1, 2, 64), device="cuda"), torch.zeros((1, 2, 64), device="cuda")
    page = int(b.table[1, 1])
    slot = torch.tensor([page * 16 + 14], dtype=torch.int32, device="cuda")  # token 30 of row 1
    b.gpu["seq_lens"][1] = 31

    def body():
        qskv.kvq_append(k, v, slot, b.gpu["pool"], b.shape, 32, b.ws)
        b.decode()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        body()
    torch.cuda.current_stream().wait_stream(s)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr in graphs:
        with torch.cuda.graph(gr):
            body()
    b.lens = [64, 31]
    gen = torch.Generator().manual_seed(0)
    for i in range(4):
        kn, vn = torch.randn((1, 2, 64), generator=gen), torch.randn((1, 2, 64), generator=gen)
        k.copy_(kn), v.copy_(vn)
        graphs[i % 2].replay()
        for f, x in ((b.k, kn), (b.v, vn)):
            for dst, src in zip(f, R.quantise(x, 32)):
                dst[page, :, 14] = src[0]
        b.check()


def test_refusals_on_device():
    b = Batch(1, [20], 2, 2, 64, 16, 64, torch.float32)
    for over in (dict(q=b.gpu["q"][:, :1]), dict(q=b.gpu["q"].half()), dict(pool=b.gpu["pool"][1:]),
                 dict(page_table=b.gpu["page_table"].long()), dict(out=b.out.double()), dict(group_size=32),
                 dict(seq_lens=b.gpu["seq_lens"].cpu()), dict(workspace=b.ws.cpu()),
                 dict(q=b.gpu["q"].transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            b.decode(**over)
    with pytest.raises(qskv.QskvError):
        b.decode(workspace=b.ws[:0])
    k = torch.zeros((2, 2, 64), device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    args = (b.gpu["pool"], b.shape, 64, b.ws)
    for bad in ((k, k.bfloat16(), slots), (k, k[:1], slots), (k.half(), k.half(), slots), (k, k, slots.long()),
                (k.transpose(1, 2).contiguous().transpose(1, 2), k, slots), (k, k.cpu(), slots)):
        with pytest.raises((ValueError, TypeError)):
            qskv.kvq_append(*bad, *args)
    assert qskv.get_error(b.ws) == 0


# ---------------------------------------------------------------- tables --
def _run_tables(seq, new, free, table, P, N, T, E=None, hkv=2):
    B, mp = len(seq), len(table[0])
    E = E or max(1, min(T, T // P + 2 * B))
    shape = qskv.make_shape(B, hkv, hkv, 64, P, mp, N)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    full = lambda n: torch.full((n,), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    o = dict(page_table=t(table), seq_lens_out=full(B), cu_new=full(B + 1), slot_map=full(T), positions=full(T),
             touched_ids=full(E), touched_valid=full(E), counts=full(4))
    ws = _ws(qskv.tables_workspace_size(shape))
    args = (t(seq), t(new), t(free))
    rest = {k: v for k, v in o.items() if k not in ("page_table", "seq_lens_out", "cu_new", "slot_map")}
    qskv.extend_tables(*args, o["page_table"], o["seq_lens_out"], o["cu_new"], o["slot_map"], shape, ws, **rest)
    want = R.tables(seq, new, free, table, P, N, T, E)
    got = {k: v.cpu() for k, v in o.items()}
    for k in o:
        assert torch.equal(got[k], torch.tensor(want[k], dtype=torch.int32)), k
    # without the optional outputs the rest is the same
    again = t(table)
    qskv.extend_tables(*args, again, o["seq_lens_out"], o["cu_new"], o["slot_map"], shape, ws)
    assert torch.equal(again.cpu(), got["page_table"]) and torch.equal(o["slot_map"].cpu(), got["slot_map"])
    return qskv.get_error(ws), want


def _requests(seed, B, P, mp, most):
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi: torch.randint(lo, hi + 1, (B,), generator=g).tolist()  # noqa: E731
    cap = mp * P
    seq = [min(x, cap) for x in r(0, cap)]
    new = [min(x if z < 2 else z // 4, cap - s) for x, z, s in zip(r(0, most), r(0, 7), seq)]
    need = sum(-(-(s + n) // P) for s, n in zip(seq, new))
    ids = torch.randperm(need + 5, generator=g).tolist()
    table, at = [], 0
    for s in seq:
        n = -(-s // P)
        table.append(ids[at:at + n] + [-1] * (mp - n))
        at += n
    return seq, new, ids[at:], table, need + 5


@pytest.mark.parametrize("P", [16, 32])
@pytest.mark.parametrize("B,mp,most", [(1, 1, 16), (1, 40, 600), (5, 7, 100), (300, 20, 40), (2048, 6, 30),
                                       (2049, 6, 30), (4032, 4, 20), (4033, 4, 20), (5000, 4, 20)])
def test_tables(P, B, mp, most):
    seq, new, free, table, N = _requests(B + P, B, P, mp, most)
    T = max(1, sum(new))
    assert _run_tables(seq, new, free, table, P, N, T)[0] == 0
    assert _run_tables(seq, new, free, table, P, N, T + 33)[0] == 0  # padded places


@pytest.mark.parametrize("B", [40, 2100, 4100])
def test_tables_refuse_in_order(B):
    seq, new, free, table, N = _requests(B, B, 16, 8, 60)
    err, want = _run_tables(seq, new, free[:len(free) // 2], table, 16, N, sum(new))  # pages run out
    assert err == 5 and want["counts"][3] > 0
    err, want = _run_tables(seq, new, free, table, 16, N, sum(new) // 2)  # tokens run out
    assert err == 5 and want["counts"][3] > 0
    err, want = _run_tables(seq, new, [], table, 16, N, sum(new))  # no free page at all
    assert err == 5


def test_tables_with_bad_lengths_and_pages():
    table = [[0, 1, -1, -1], [2, -1, -1, -1], [99, -1, -1, -1], [-1] * 4, [3, -1, -1, -1]]
    # a length past the table, a negative one, a negative addition, a bad page in the table and one in the free list
    err, want = _run_tables([65, -1, 5, 0, 4], [1, 2, 3, 20, 2], [50, 7, 8], table, 16, 40, 40)
    assert err == 5 and want["counts"][3] == 2
    err, want = _run_tables([30, 10, 5, 0, 4], [40, -2, 0, 0, 2], [5, 7, 8], table, 16, 100, 60)
    assert err == 5 and want["seq_lens_out"] == [30, 10, 5, 0, 6]


def test_tables_with_no_new_tokens():
    err, want = _run_tables([3, 0], [0, 0], [], [[1], [-1]], 16, 4, 9)
    assert err == 0 and want["counts"] == [0, 0, 0, 0]


def test_tables_of_long_prompts():
    mp = 9000
    err, _ = _run_tables([0, 100, 17], [140_001, 1, 0], list(range(50, 9000)), [[-1] * mp, list(range(7)) + [-1] * (mp - 7),
                         [20, 21] + [-1] * (mp - 2)], 16, 10_000, 140_010)
    assert err == 0


def test_tables_share_the_decodes_workspace():
    """More requests than one CTA scans: the tables' scratch leaves the decode's row counters alone."""
    B, P, mp, N = 4100, 16, 200, 800
    shape = qskv.make_shape(B, 1, 1, 64, P, mp, N)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = _ws(max(qskv.kvq_workspace_size(shape), qskv.tables_workspace_size(shape)))
    g = torch.Generator().manual_seed(2)
    f = [R.quantise(torch.randn((N, 1, P, 64), generator=g), 64) for _ in range(2)]
    pool = R.pack(*f[0], *f[1]).cuda()
    new = i32(B)
    new[0], new[7], new[4099] = 3000, 2900, 3100
    table, lens, cu, slots = torch.full((B, mp), -1, dtype=torch.int32, device="cuda"), i32(B), i32(B + 1), i32(9000)
    q, outs = torch.randn((B, 1, 64), device="cuda"), []
    for _ in range(3):
        qskv.extend_tables(i32(B), new, torch.arange(N, dtype=torch.int32, device="cuda"), table, lens, cu, slots, shape, ws)
        outs.append(torch.empty((B, 1, 64), device="cuda"))
        qskv.kvq_paged_decode(q, pool, table, lens, outs[-1], shape, 64, ws)
        assert qskv.get_error(ws) == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]) and bool((outs[0][[0, 7, 4099]] != 0).any())
    kx, vx = R.values(*f[0]), R.values(*f[1])
    at = [(j // P, j % P) for j in range(3000)]
    p, t = ([x[i] for x in at] for i in (0, 1))
    o, _ = R.attend(q[0].cpu(), kx[p, 0, t], vx[p, 0, t], 64 ** -0.5)
    tol, _ = R.attend_bounds(q[0].cpu(), f[0][2][p, 0, t], f[0][1][p, 0, t], f[1][2][p, 0, t], f[1][1][p, 0, t], 64 ** -0.5,
                             3000)
    assert float((outs[0][0].cpu().double() - o).abs().max()) <= tol


# ------------------------------------------------------------- in a run --
def test_a_serving_run_together():
    """Prefill of two requests and four decode steps: tables, append, metadata, selection and decode in turn, against
    the reference on the same cache; the third request joins late."""
    P, d, gs, hkv, hq, B, mp, N, K = 16, 64, 32, 2, 4, 3, 12, 40, 3
    shape = qskv.make_shape(B, hq, hkv, d, P, mp, N)
    g = torch.Generator().manual_seed(42)
    free = torch.randperm(N, generator=g).to(torch.int32)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    T, E = 200, 18
    table, lens, lens_out, cu, slots, pos = i32(B, mp), i32(B), i32(B), i32(B + 1), i32(T), i32(T)
    ids, valid, counts = i32(E), i32(E), i32(4)
    pool = torch.zeros((N, hkv, qskv.kvq_block_bytes(shape, gs)), dtype=torch.uint8, device="cuda")
    meta = torch.zeros((N, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    ws = _ws(max(qskv.workspace_size(shape), qskv.kvq_workspace_size(shape), qskv.tables_workspace_size(shape)))
    sel, nsel = i32(B, hkv, K), i32(B, hkv)
    scores = torch.zeros((B, hkv, mp), device="cuda")
    out, lse = torch.zeros((B, hq, d), device="cuda"), torch.zeros((B, hq), device="cuda")
    kept = [(torch.zeros((0, hkv, d)), torch.zeros((0, hkv, d))) for _ in range(B)]
    for new in ([100, 17, 0], [1, 1, 0], [1, 0, 50], [1, 1, 1], [0, 1, 1]):
        n = sum(new)
        nl = torch.tensor(new, dtype=torch.int32, device="cuda")
        k, v = torch.randn((T, hkv, d), generator=g), torch.randn((T, hkv, d), generator=g)
        q = torch.randn((B, hq, d), generator=g)
        qskv.extend_tables(lens, nl, free.cuda(), table, lens_out, cu, slots, shape, ws, positions=pos, touched_ids=ids,
                           touched_valid=valid, counts=counts)
        lens.copy_(lens_out)
        free = free[int(counts[1]):]
        qskv.kvq_append(k.cuda(), v.cuda(), slots, pool, shape, gs, ws)
        qskv.kvq_meta_build(pool, ids, valid, meta, shape, gs, ws)
        qskv.page_select(q.cuda(), meta, table, lens, K, sel, nsel, shape, ws, scores)
        qskv.kvq_paged_decode(q.cuda(), pool, table, lens, out, shape, gs, ws, selected=sel, n_selected=nsel, top_k=K,
                              lse=lse)
        assert qskv.get_error(ws) == 0
        at = 0
        for b in range(B):
            kept[b] = tuple(torch.cat([x, y[at:at + new[b]]]) for x, y in zip(kept[b], (k, v)))
            at += new[b]
            length = len(kept[b][0])
            assert int(lens[b]) == length
            for h in range(hkv):
                G = hq // hkv
                kf, vf = (R.quantise(x[:, h], gs) for x in kept[b])
                kx, vx = R.values(*kf), R.values(*vf)
                pages = sel[b, h, :int(nsel[b, h])].tolist()
                n_b = -(-length // P)
                assert len(pages) == min(K, n_b)
                qs = q[b, h * G:(h + 1) * G]
                for j in range(n_b):  # the score bounds every logit of its page (2^-20: fp32 sums of 64 terms)
                    best = float((qs.double() @ kx[j * P:(j + 1) * P].T).max())
                    assert float(scores[b, h, j]) >= best - 2.0 ** -20 * float((qs.abs().double() @ kx.abs().amax(0)).max())
                rows = [t for j in pages for t in range(j * P, min(length, (j + 1) * P))]
                o, l = R.attend(qs, kx[rows], vx[rows], d ** -0.5)
                got = out[b, h * G:(h + 1) * G].cpu().double()
                if not rows:
                    assert bool((got == 0).all())
                    continue
                tol, _ = R.attend_bounds(qs, kf[2][rows], kf[1][rows], vf[2][rows], vf[1][rows], d ** -0.5, len(rows))
                assert float((got - o).abs().max()) <= tol


def test_quantized_decoder_runs_a_batch():
    """The engine's class over prefill, steps, a row given back and taken again: every output against the reference."""
    g = torch.Generator().manual_seed(7)
    B, hq, hkv, d, P, gs = 3, 8, 2, 128, 16, 64
    for top_k in (None, 2):
        dec = qskv.QuantizedPagedDecoder(B, hq, hkv, d, P, max_pages=9, num_pool_pages=20, group_size=gs, top_k=top_k,
                                         max_tokens=400)
        kept = [[torch.zeros((0, hkv, d))] * 2 for _ in range(B)]
        for new in ([40, 0, 90], [1, 1, 1], [1, 17, 0], None, [0, 1, 1]):
            if new is None:
                dec.release(0)
                kept[0] = [torch.zeros((0, hkv, d))] * 2
                continue
            n = sum(new)
            k, v = (torch.randn((n, hkv, d), generator=g).bfloat16() for _ in range(2))
            q = torch.randn((B, hq, d), generator=g).bfloat16()
            dec.step(q.cuda(), k.cuda(), v.cuda(), new)
            dec.check()
            at = 0
            for b in range(B):
                kept[b] = [torch.cat([x, y[at:at + new[b]].float()]) for x, y in zip(kept[b], (k, v))]
                at += new[b]
                n_b = -(-len(kept[b][0]) // P)
                for h in range(hkv):
                    kf, vf = (R.quantise(x[:, h], gs) for x in kept[b])
                    pages = list(range(n_b)) if top_k is None else dec.selected[b, h, :min(top_k, n_b)].tolist()
                    rows = [t for j in pages for t in range(j * P, min(len(kept[b][0]), (j + 1) * P))]
                    qs = q[b, h * 4:h * 4 + 4]
                    o, l = R.attend(qs, R.values(*kf)[rows], R.values(*vf)[rows], d ** -0.5)
                    if not rows:
                        assert bool((dec.out[b] == 0).all()) and bool(torch.isinf(dec.lse[b]).all())
                        continue
                    tol, _ = R.attend_bounds(qs, kf[2][rows], kf[1][rows], vf[2][rows], vf[1][rows], d ** -0.5, len(rows))
                    assert float((dec.out[b, h * 4:h * 4 + 4].cpu().double() - o).abs().max()) <= tol
        assert dec.lengths == [0, 19, 92]
        with pytest.raises(ValueError, match="14 pages needed, 12 free"):  # 2 + 6 of 20 are held
            dec.extend([144, 80, 0])
        with pytest.raises(ValueError, match="401 new tokens"):
            dec.extend([300, 101, 0])
        with pytest.raises(ValueError, match="row 2"):
            dec.extend([0, 0, 53])
        with pytest.raises(ValueError, match="1 keys for the 0 tokens"):
            dec.append(k.cuda()[:1], v.cuda()[:1])
        assert dec.lengths == [0, 19, 92]
        side = torch.cuda.Stream()  # the same on a stream that is not the current one
        side.wait_stream(torch.cuda.current_stream())
        dec.extend([0, 2, 0], stream=side)
        with pytest.raises(ValueError, match="2 tokens of the last extend"):
            dec.extend([1, 0, 0])
        dec.append(k.cuda()[:2], v.cuda()[:2], stream=side)
        got = dec.gather(1, stream=side)
        side.synchronize()
        for x, y in zip(got, (k, v)):
            assert torch.equal(x[-2:].cpu(), R.values(*R.quantise(y[:2], gs)).float())
