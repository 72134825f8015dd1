"""The 8-bit cache without a GPU: the reference's own consistency, sizes, and every refusal of the calls."""
import ctypes
import glob
import os
import re

import pytest
import torch

import kvf_ref as R
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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 32])
def test_block_bytes_and_reference_round_trip(lib, d, P):
    shape = qskv.make_shape(1, 2, 2, d, P, 1, 3)
    assert qskv.kvf_block_bytes(shape) == P * (2 * d + 2)
    every = torch.cat([x.flatten() for x in R.places(d, P)])
    assert sorted(every.tolist()) == list(range(P * (2 * d + 2)))  # every byte is one number's place
    g = torch.Generator().manual_seed(d + P)
    f = [R.quantise(torch.randn((3, 2, P, d), generator=g)) for _ in range(2)]
    back = R.unpack(R.pack(*f[0], *f[1]), d, P)
    for a, b in zip(f, back):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_reference_codes_are_torch_s():
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(4000, generator=g) * 2.0 ** torch.randint(-12, 8, (4000,), generator=g),
                   R.number(torch.arange(0x7F)).float(), torch.tensor([0.0, -0.0, 448.0, -448.0]),
                   ((R.number(torch.arange(0x7E)) + R.number(torch.arange(1, 0x7F))) / 2).float()])  # every tie
    x = x.clamp(-448, 448)
    assert torch.equal(R.code(x.double()), x.to(torch.float8_e4m3fn).view(torch.uint8).long())


def test_reference_quantiser():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((50, 128), generator=g) * 10 ** (8 * torch.rand((50, 1), generator=g) - 4)
    u, e = R.quantise(x)
    top = x.double().abs().amax(-1)
    assert bool((top <= 448 * torch.exp2(e.double())).all() and (top > 224 * torch.exp2(e.double())).all())
    # half a step of 3 bits of fraction, or of the smallest codes' 2^-9
    slack = torch.maximum(x.double().abs() * 2.0 ** -4, torch.exp2(e.double() - 10)[:, None])
    assert bool(((R.values(u, e) - x.double()).abs() <= slack).all())
    assert R.quantise(torch.zeros(1, 64))[1].item() == -100
    for y, want in ((448.0, 0), (448.5, 1), (224.0, -1), (2.0 ** -120, -100), (3.0e38, 119)):
        assert R.quantise(torch.full((1, 64), y))[1].item() == want


def test_cache_call_refusals(lib, base):
    p, odd = ctypes.c_void_p(base), ctypes.c_void_p(base + 4)
    s = ctypes.byref(qskv.make_shape(*SHAPE))
    bad = ctypes.byref(qskv.make_shape(2, 8, 2, 96, 16, 8, 16))
    app, gat, met = lib.qskv_kvf_append, lib.qskv_kvf_gather, lib.qskv_kvf_meta_build
    row = 2 * 128
    assert lib.qskv_kvf_block_bytes(bad) == 0 and lib.qskv_kvf_block_bytes(None) == 0
    assert app(p, p, 1, row, row, p, 0, p, s, p, 256, None) == OK  # nothing to do
    assert app(p, p, 1, row, row, p, -1, p, s, p, 256, None) == INVALID
    assert app(p, p, 1, row, row, p, 2, p, bad, p, 256, None) == UNSUPPORTED
    assert app(p, p, 5, row, row, p, 2, p, s, p, 256, None) == UNSUPPORTED
    assert app(None, p, 1, row, row, p, 2, p, s, p, 256, None) == INVALID
    assert app(p, p, 1, row, row, None, 2, p, s, p, 256, None) == INVALID
    assert app(odd, p, 1, row, row, p, 2, p, s, p, 256, None) == INVALID
    assert app(p, p, 1, row - 8, row, p, 2, p, s, p, 256, None) == INVALID  # rows overlap
    assert app(p, p, 1, row, row + 4, p, 2, p, s, p, 256, None) == INVALID  # 8 bytes off
    assert app(p, p, 1, row, row, p, 2, p, s, None, 256, None) == WORKSPACE
    assert app(p, p, 1, row, row, p, 2, p, s, p, 255, None) == WORKSPACE
    assert app(p, p, 1, row, row, p, 2, p, s, odd, 256, None) == WORKSPACE
    assert gat(p, p, 0, p, p, 1, s, p, 256, None) == OK
    assert gat(p, p, -1, p, p, 1, s, p, 256, None) == INVALID
    assert gat(p, p, 2, p, None, 1, s, p, 256, None) == INVALID
    assert gat(p, p, 2, odd, p, 1, s, p, 256, None) == INVALID
    assert gat(p, p, 2, p, p, 2, s, p, 256, None) == UNSUPPORTED
    assert gat(p, p, 2, p, p, 1, s, None, 256, None) == WORKSPACE
    assert met(p, p, p, 0, p, 1, s, p, 256, None) == OK
    assert met(p, p, p, -3, p, 1, s, p, 256, None) == INVALID
    assert met(p, None, p, 1, p, 1, s, p, 256, None) == INVALID
    assert met(p, p, p, 1, odd, 1, s, p, 256, None) == INVALID
    assert met(p, p, p, 1, p, 9, s, p, 256, None) == UNSUPPORTED
    assert met(p, p, p, 1, p, 1, s, p, 128, None) == WORKSPACE


def test_decode_refusals(lib, base):
    p, odd = ctypes.c_void_p(base), ctypes.c_void_p(base + 4)
    s = ctypes.byref(qskv.make_shape(*SHAPE))

    def call(q=p, qt=1, pool=p, pt=p, sl=p, shape=s, sel=None, ns=None, k=0, scale=0.0, out=p, lse=None, n=1 << 30):
        return lib.qskv_kvf_paged_decode(q, qt, pool, pt, sl, shape, sel, ns, k, scale, out, lse, p, n, None)

    for kw in (dict(q=None), dict(pool=None), dict(pt=None), dict(sl=None), dict(out=None), dict(q=odd),
               dict(pool=odd), dict(out=odd), dict(lse=ctypes.c_void_p(base + 2)), dict(sel=p), dict(sel=p, ns=p),
               dict(sel=p, ns=p, k=-1), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(qt=3), dict(shape=ctypes.byref(qskv.make_shape(2, 6, 2, 128, 16, 8, 16))),
               dict(shape=ctypes.byref(qskv.make_shape(8191, 8, 8, 128, 16, 40000, 16))),  # 2^31 units and more
               dict(shape=ctypes.byref(qskv.make_shape(8191, 8, 8, 128, 32, 20000, 16))),  # two units a page
               dict(sel=p, ns=p, k=2 ** 30)):
        assert call(**kw) == UNSUPPORTED, kw
    bad = qskv.make_shape(0, 8, 2, 128, 16, 8, 16)
    assert lib.qskv_kvf_workspace_size(ctypes.byref(bad)) == 0
    with pytest.raises(qskv.QskvError):
        qskv.kvf_block_bytes(bad)


def test_binding_refuses_host_tensors(lib):
    shape = qskv.make_shape(*SHAPE)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    pool = torch.zeros((16, 2, qskv.kvf_block_bytes(shape)), dtype=torch.uint8)
    k, ws = torch.zeros((3, 2, 128)), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="pool"):
        qskv.kvf_append(k, k, i32(3), pool, shape, ws)
    with pytest.raises(ValueError, match="pool"):
        qskv.kvf_gather(pool, i32(3), k, k, shape, ws)
    with pytest.raises(ValueError, match="pool"):
        qskv.kvf_meta_build(pool, i32(1), i32(1), torch.zeros((16, 2, 2, 128)), shape, ws)
    with pytest.raises(ValueError, match="pool"):
        qskv.kvf_paged_decode(torch.zeros((2, 8, 128)), pool, i32(2, 8), i32(2), torch.zeros((2, 8, 128)), shape, ws)


CSRC = os.path.join(os.path.dirname(qskv.__file__), "csrc")


@pytest.mark.parametrize("path", sorted(p for f in ("kvf_*.cu*", "prefill_*.cu")
                                        for p in glob.glob(os.path.join(CSRC, f))))
def test_a_kernel_waits_before_it_reads(path):
    """Nothing of the caller's is read before the kernel ahead in the stream has completed."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    found = 0
    for m in re.finditer(r"__global__[^{;]*?(\w+_kernel)\s*\([^{;]*\)\s*\{", text):
        body = text[m.end():text.index("\n}", m.end())]
        waits = [line.strip() for line in body.split("\n") if "pdl_wait" in line]
        assert waits == ["pdl_wait();"], m.group(1)
        before = body[:body.index("pdl_wait();")]
        assert not re.search(r"__ld|\ba\.\w+\s*\[", before), m.group(1)
        found += 1
    assert found == text.count("__global__")
