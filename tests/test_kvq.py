"""The 4-bit cache and the page tables without a GPU: the reference's own
consistency, sizes, and every refusal of the C calls and of the binding."""
import ctypes

import pytest
import torch

import kvq_ref as R
import query_aware_sparse_kv_gb300 as qskv
from query_aware_sparse_kv_gb300 import build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return qskv.load()


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(1 << 16)
    base = (ctypes.addressof(buf) + 255) // 256 * 256
    return buf, base


SHAPE = (2, 8, 2, 128, 16, 8, 16)


@pytest.mark.parametrize("d,gs", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("P", [16, 32])
def test_block_bytes_and_reference_round_trip(lib, d, gs, P):
    shape = qskv.make_shape(1, 2, 2, d, P, 1, 3)
    assert qskv.kvq_block_bytes(shape, gs) == P * (d + 8 * d // gs) == 4 * R.block_words(d, P, gs)
    g = torch.Generator().manual_seed(d + gs + P)
    f = [R.quantise(torch.randn((3, 2, P, d), generator=g), gs) for _ in range(2)]
    back = R.unpack(R.pack(*f[0], *f[1]), d, P, gs)
    for a, b in zip(f, back):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    key, val = R.places(d, P)
    for t in range(P):  # every word has one place
        assert sorted(key[t].tolist()) == sorted(val[t].tolist()) == list(range(d // 8))


def test_reference_quantiser_is_within_half_a_step():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((50, 128), generator=g) * 10 ** (4 * torch.rand((50, 1), generator=g) - 2)
    u, s, m = R.quantise(x, 32)
    step = s.repeat_interleave(32, -1)
    # half a step, plus the top of the range: s and m are off by half a bf16 step (2^-9 of 15 s and of |m|)
    slack = step / 2 + 2.0 ** -9 * (15 * step + m.abs().repeat_interleave(32, -1))
    assert bool(((R.values(u, s, m) - x.double()).abs() <= slack).all())


def test_group_size_refusals(lib):
    for d, gs in ((64, 128), (128, 16), (128, 0), (128, -32), (128, 48), (64, 256)):
        shape = qskv.make_shape(1, 2, 2, d, 16, 1, 3)
        assert lib.qskv_kvq_block_bytes(ctypes.byref(shape), gs) == 0
        with pytest.raises(qskv.QskvError):
            qskv.kvq_block_bytes(shape, gs)


def test_cache_call_refusals(lib, mem):
    _, base = mem
    p, odd = ctypes.c_void_p(base), ctypes.c_void_p(base + 4)
    s = ctypes.byref(qskv.make_shape(*SHAPE))
    bad = ctypes.byref(qskv.make_shape(2, 8, 2, 96, 16, 8, 16))
    app, gat, met = lib.qskv_kvq_append, lib.qskv_kvq_gather, lib.qskv_kvq_meta_build
    row = 2 * 128
    assert app(p, p, 1, row, row, p, 0, p, s, 64, p, 256, None) == OK  # nothing to do
    assert app(p, p, 1, row, row, p, -1, p, s, 64, p, 256, None) == INVALID
    assert app(p, p, 1, row, row, p, 2, p, bad, 64, p, 256, None) == UNSUPPORTED
    assert app(p, p, 1, row, row, p, 2, p, s, 48, p, 256, None) == UNSUPPORTED
    assert app(p, p, 5, row, row, p, 2, p, s, 64, p, 256, None) == UNSUPPORTED
    assert app(None, p, 1, row, row, p, 2, p, s, 64, p, 256, None) == INVALID
    assert app(p, p, 1, row, row, None, 2, p, s, 64, p, 256, None) == INVALID
    assert app(odd, p, 1, row, row, p, 2, p, s, 64, p, 256, None) == INVALID
    assert app(p, p, 1, row - 8, row, p, 2, p, s, 64, p, 256, None) == INVALID  # rows overlap
    assert app(p, p, 1, row, row + 4, p, 2, p, s, 64, p, 256, None) == INVALID  # 8 bytes off
    assert app(p, p, 0, row, row + 2, p, 2, p, s, 64, p, 256, None) == INVALID
    assert app(p, p, 1, row, row, p, 2, p, s, 64, None, 256, None) == WORKSPACE
    assert app(p, p, 1, row, row, p, 2, p, s, 64, p, 255, None) == WORKSPACE
    assert app(p, p, 1, row, row, p, 2, p, s, 64, odd, 256, None) == WORKSPACE
    assert gat(p, p, 0, p, p, 1, s, 64, p, 256, None) == OK
    assert gat(p, p, -1, p, p, 1, s, 64, p, 256, None) == INVALID
    assert gat(p, p, 2, p, None, 1, s, 64, p, 256, None) == INVALID
    assert gat(p, p, 2, odd, p, 1, s, 64, p, 256, None) == INVALID
    assert gat(p, p, 2, p, p, 2, s, 64, p, 256, None) == UNSUPPORTED
    assert gat(p, p, 2, p, p, 1, s, 33, p, 256, None) == UNSUPPORTED
    assert gat(p, p, 2, p, p, 1, s, 64, None, 256, None) == WORKSPACE
    assert met(p, p, p, 0, p, 1, s, 64, p, 256, None) == OK
    assert met(p, p, p, -3, p, 1, s, 64, p, 256, None) == INVALID
    assert met(p, None, p, 1, p, 1, s, 64, p, 256, None) == INVALID
    assert met(p, p, p, 1, odd, 1, s, 64, p, 256, None) == INVALID
    assert met(p, p, p, 1, p, 9, s, 64, p, 256, None) == UNSUPPORTED
    assert met(p, p, p, 1, p, 1, s, 64, p, 128, None) == WORKSPACE
    assert lib.qskv_last_error_message().decode()


def test_decode_refusals(lib, mem):
    _, base = mem
    p, odd = ctypes.c_void_p(base), ctypes.c_void_p(base + 4)
    s = ctypes.byref(qskv.make_shape(*SHAPE))
    dec = lib.qskv_kvq_paged_decode

    def call(q=p, qt=1, pool=p, pt=p, sl=p, shape=s, gs=64, sel=None, ns=None, k=0, scale=0.0, out=p, lse=None, ws=p,
             n=1 << 30):
        return dec(q, qt, pool, pt, sl, shape, gs, sel, ns, k, scale, out, lse, ws, n, None)

    for kw in (dict(q=None), dict(pool=None), dict(pt=None), dict(sl=None), dict(out=None), dict(q=odd),
               dict(pool=odd), dict(out=odd), dict(lse=ctypes.c_void_p(base + 2)), dict(sel=p), dict(sel=p, ns=p),
               dict(sel=p, ns=p, k=-1), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(qt=3), dict(gs=96), dict(shape=ctypes.byref(qskv.make_shape(2, 6, 2, 128, 16, 8, 16))),
               dict(shape=ctypes.byref(qskv.make_shape(8191, 8, 8, 128, 16, 40000, 16))),  # units past 2^31
               dict(sel=p, ns=p, k=2 ** 30)):
        assert call(**kw) == UNSUPPORTED, kw
    bad = qskv.make_shape(0, 8, 2, 128, 16, 8, 16)
    assert lib.qskv_kvq_workspace_size(ctypes.byref(bad)) == 0


def test_extend_tables_refusals(lib, mem):
    _, base = mem
    p, odd = ctypes.c_void_p(base), ctypes.c_void_p(base + 2)
    o = ctypes.c_void_p(base + 1024)  # seq_lens_out, apart from the inputs
    s = ctypes.byref(qskv.make_shape(*SHAPE))

    def call(sl=p, nl=p, fp=p, nf=4, pt=p, shape=s, so=o, cu=p, sm=p, pos=p, T=8, ti=p, tv=p, E=64, ct=p, ws=p, n=256):
        return lib.qskv_extend_tables(sl, nl, fp, nf, pt, shape, so, cu, sm, pos, T, ti, tv, E, ct, ws, n, None)

    for kw in (dict(sl=None), dict(nl=None), dict(fp=None), dict(pt=None), dict(so=None), dict(cu=None),
               dict(sm=None), dict(nf=-1), dict(nf=2 ** 31 - 1), dict(T=0), dict(T=-5), dict(T=2 ** 31 - 1),
               dict(ti=None), dict(tv=None), dict(so=p), dict(sl=odd), dict(ct=odd),
               dict(E=3)):  # min(8 tokens, 8 / 16 + 2 * 2) = 4 pages may be touched
        assert call(**kw) == INVALID, kw
    assert call(shape=ctypes.byref(qskv.make_shape(2, 8, 2, 128, 24, 8, 16))) == UNSUPPORTED
    small = qskv.make_shape(4032, 8, 2, 128, 16, 8, 16)
    large = qskv.make_shape(4033, 8, 2, 128, 16, 8, 16)
    assert lib.qskv_tables_workspace_size(ctypes.byref(small)) == 256
    # behind the counters of its 2 * 4033 rows, so that the decode's stay zero in a shared workspace
    assert lib.qskv_tables_workspace_size(ctypes.byref(large)) >= 256 + 2 * 4033 * 4 + 3 * 4034 * 4
    assert lib.qskv_tables_workspace_size(ctypes.byref(qskv.make_shape(0, 8, 2, 128, 16, 8, 16))) == 0


def test_binding_refuses_host_tensors(lib):
    """Every call names the tensor that is not on the GPU, before the library is reached."""
    shape = qskv.make_shape(*SHAPE)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    pool = torch.zeros((16, 2, qskv.kvq_block_bytes(shape, 64)), dtype=torch.uint8)
    k = torch.zeros((3, 2, 128))
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="pool"):
        qskv.kvq_append(k, k, i32(3), pool, shape, 64, ws)
    with pytest.raises(ValueError, match="pool"):
        qskv.kvq_gather(pool, i32(3), k, k, shape, 64, ws)
    with pytest.raises(ValueError, match="pool"):
        qskv.kvq_meta_build(pool, i32(1), i32(1), torch.zeros((16, 2, 2, 128)), shape, 64, ws)
    with pytest.raises(ValueError, match="pool"):
        qskv.kvq_paged_decode(torch.zeros((2, 8, 128)), pool, i32(2, 8), i32(2), torch.zeros((2, 8, 128)), shape, 64, ws)
    with pytest.raises(ValueError, match="page_table"):
        qskv.extend_tables(i32(2), i32(2), i32(4), i32(2, 8), i32(2), i32(3), i32(8), shape, ws)


def test_reference_tables_by_hand():
    """16-token pages, a table of 4: request 0 fills its page and takes one, 1 adds nothing, 2 does not fit."""
    r = R.tables([14, 5, 0], [4, 0, 40], [9, 8, 7], [[3, -1, -1, -1], [2, -1, -1, -1], [-1] * 4], 16, 16, 64, 10)
    assert r["page_table"] == [[3, 9, -1, -1], [2, -1, -1, -1], [-1] * 4]
    assert r["seq_lens_out"] == [18, 5, 0] and r["cu_new"] == [0, 4, 4, 44]
    assert r["slot_map"][:5] == [62, 63, 144, 145, -1] and r["positions"][:5] == [14, 15, 16, 17, -1]
    assert r["touched_ids"][:3] == [3, 9, -1] and r["touched_valid"][:3] == [16, 2, 0]
    assert r["counts"] == [44, 1, 2, 1]
