"""Prefill without a GPU: the reference by hand, sizes, and every refusal of the calls."""
import ctypes
import math

import pytest
import torch

import prefill_ref as R
import query_aware_sparse_kv_gb300 as qskv
from query_aware_sparse_kv_gb300 import build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
SHAPE = (2, 8, 2, 128, 16, 8, 16)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return qskv.load()


@pytest.fixture(scope="module")
def base():
    buf = ctypes.create_string_buffer(1 << 16)
    yield (ctypes.addressof(buf) + 255) // 256 * 256


def test_reference_by_hand():
    """Two tokens, keys 0 and ln 3 along q: the second query weighs the values 1/4 and 3/4, the first sees one."""
    q = torch.tensor([[[1.0]], [[1.0]]])
    k, v = torch.tensor([[0.0], [math.log(3)]], dtype=torch.float64), torch.tensor([[4.0], [8.0]]).double()
    out, lse, pabs, A = R.attend_rows(q, k, v, torch.tensor([0, 1]), 1.0)
    assert torch.allclose(out.flatten(), torch.tensor([4.0, 7.0]).double())
    assert torch.allclose(lse.flatten(), torch.tensor([0.0, math.log(4)]).double())
    assert torch.equal(pabs, out) and abs(A - math.log(3)) < 1e-12
    out, lse, _, _ = R.attend_rows(q, k, v, torch.tensor([-2, -1]), 1.0)  # before the first token
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_refusals(lib, base):
    p, odd = ctypes.c_void_p(base), ctypes.c_void_p(base + 4)
    s = ctypes.byref(qskv.make_shape(*SHAPE))
    row = 8 * 128

    def call(q=p, qt=1, qs=row, k=p, v=p, kt=1, pt=p, sl=p, cu=p, n=3, shape=s, scale=0.0, out=p, lse=None):
        return lib.qskv_paged_prefill(q, qt, qs, k, v, kt, pt, sl, cu, n, shape, scale, out, lse, p, 1 << 40, None)

    def call8(q=p, qt=1, qs=row, pool=p, pt=p, sl=p, cu=p, n=3, shape=s, scale=0.0, out=p, lse=None):
        return lib.qskv_kvf_paged_prefill(q, qt, qs, pool, pt, sl, cu, n, shape, scale, out, lse, p, 1 << 40, None)

    common = [dict(q=None), dict(pt=None), dict(sl=None), dict(cu=None), dict(out=None), dict(q=odd), dict(out=odd),
              dict(cu=ctypes.c_void_p(base + 2)), dict(lse=ctypes.c_void_p(base + 1)), dict(scale=-1.0),
              dict(scale=float("inf")), dict(scale=float("nan")), dict(n=-1), dict(qs=row - 8), dict(qs=row + 4)]
    for kw in common + [dict(k=None), dict(v=odd), dict(k=odd)]:
        assert call(**kw) == INVALID, kw
    for kw in common + [dict(pool=None), dict(pool=odd)]:
        assert call8(**kw) == INVALID, kw
    unsupported = [dict(qt=3), dict(n=2 ** 28), dict(shape=ctypes.byref(qskv.make_shape(2, 8, 2, 96, 16, 8, 16))),
                   dict(shape=ctypes.byref(qskv.make_shape(2, 48, 4, 128, 16, 8, 16)))]
    for kw in unsupported + [dict(kt=5)]:
        assert call(**kw) == UNSUPPORTED, kw
    for kw in unsupported:
        assert call8(**kw) == UNSUPPORTED, kw
    assert call(n=0) == OK and call8(n=0) == OK  # nothing to do
    assert lib.qskv_prefill_workspace_size(None, 4) == 0
    assert lib.qskv_prefill_workspace_size(s, -1) == 0
    with pytest.raises(qskv.QskvError):
        qskv.prefill_workspace_size(qskv.make_shape(2, 8, 2, 96, 16, 8, 16), 4)


def test_binding_refuses_host_tensors(lib):
    shape = qskv.make_shape(*SHAPE)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    k, q = torch.zeros((16, 2, 16, 128)), torch.zeros((3, 8, 128))
    pool = torch.zeros((16, 2, 16 * 258), dtype=torch.uint8)
    with pytest.raises(ValueError, match="k_pool"):
        qskv.paged_prefill(q, k, k, i32(2, 8), i32(2), i32(3), q, shape, i32(64))
    with pytest.raises(ValueError, match="pool"):
        qskv.kvf_paged_prefill(q, pool, i32(2, 8), i32(2), i32(3), q, shape, i32(64))


def line(blocks, heads, ctas, least=8):
    """Items of a call without a list, as the kernel cuts them: (row, head, block0, block1, part, parts, place) per CTA."""
    units = [None if b is None else max(b, 1) for b in blocks]  # None: a row without queries
    even = sum(u or 0 for u in units) * heads >= least * ctas
    if not even:
        units = [u and -(-u // least) * least for u in units]
    before, total = [], 0
    for u in units:
        before.append(total)
        total += u or 0
    total *= heads
    ranges = ctas if even else total // least
    size, more = (total // ranges, total % ranges) if ranges else (0, 0)
    begin = lambda r: r * size + min(r, more)  # noqa: E731
    of = lambda x: x // (size + 1) if x < more * (size + 1) else more + (x - more * (size + 1)) // size  # noqa: E731
    work = [[] for _ in range(ctas)]
    for c in range(ctas):
        for r in range(c, ranges, ctas):
            at, end = begin(r), begin(r + 1)
            while at < end:
                row, step = 0, 16
                while step:
                    i = row + step - 1
                    done = before[i] + (units[i] or 0) if i < len(units) else total // heads
                    if done * heads <= at:
                        row += step
                    step //= 2
                off = at - before[row] * heads
                head, block = divmod(off, units[row])
                take = min(units[row] - block, end - at)
                first, last = of(at - block), of(at - block + units[row] - 1)
                work[c].append((row, head, min(block, blocks[row]), min(block + take, blocks[row]), r - first,
                                last - first + 1, row * heads + head + first))
                at += take
    return work


@pytest.mark.parametrize("blocks,heads", [
    ([1], 1), ([0], 3), ([None], 2), ([None, 3, None, 0, 9, None], 2), ([8, 16, 17, 7, 1], 4), ([800, 1, 300], 8),
    ([5000], 1), ([100000, 0, None, 7], 16), ([40] * 32, 4), ([None] * 31 + [65], 2), ([3] * 19, 8), ([8] * 19, 8),
    ([9] * 19, 8), ([1216], 1), ([1215], 1), ([1217, None, 4], 1)])
@pytest.mark.parametrize("ctas", [152, 148, 7])
def test_ranges_of_a_call_without_a_list(blocks, heads, ctas):
    """Every block of every tile is in one part, parts count up and fit their places, CTAs have about as much to do."""
    if len(blocks) * heads > ctas:
        return
    work = line(blocks, heads, ctas)
    tiles = {}
    for items in work:
        for row, head, b0, b1, part, parts, place in items:
            tiles.setdefault((row, head), []).append((part, parts, b0, b1, place))
    assert set(tiles) == {(r, h) for r, b in enumerate(blocks) if b is not None for h in range(heads)}
    places = set()
    for (row, head), parts in tiles.items():
        parts.sort()
        assert [p[0] for p in parts] == list(range(len(parts))) and all(p[1] == len(parts) for p in parts)
        edges = [0] + [p[3] for p in parts]
        assert [p[2] for p in parts] == edges[:-1] and edges[-1] == blocks[row]
        assert len({p[4] for p in parts}) == 1
        if len(parts) > 1:
            mine = set(range(parts[0][4], parts[0][4] + len(parts)))
            assert not mine & places and max(mine) < 4 * ctas + heads
            places |= mine
    loads = [sum(i[3] - i[2] for i in items) for items in work]
    total = sum(loads)
    if total >= 8 * ctas:
        assert max(loads) <= -(-total // ctas) + 1
    else:
        assert max(loads) <= 16
