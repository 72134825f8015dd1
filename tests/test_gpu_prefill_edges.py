"""Prefill calls at the edges of what include/qskv.h allows: two at once, the most rows, shared pages, odd addresses."""
import pytest
import torch

import query_aware_sparse_kv_gb300 as qskv
from test_gpu_prefill import BF16, F32, KINDS, Batch, _i32, _lib  # noqa: F401

pytestmark = pytest.mark.gpu

SIX = [(0, 300), (2000, 3), (700, 130), (0, 1), (5, 0), (40, 64)]


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_two_calls_at_once(dtype, cache):
    """On two streams, each with a workspace of its own: with a list of tiles and without one, and the same pools."""
    a = Batch(1, SIX, 8, 2, 128, 16, dtype, cache)
    b = Batch(2, [(3000, 4), (9000, 2)], 8, 2, 128, 16, dtype, cache)
    c = Batch(1, SIX, 8, 2, 128, 16, dtype, cache)
    c.pools, c.gpu = a.pools, a.gpu
    for x in (a, b, c):
        x.run()
    torch.cuda.synchronize()
    want = [x.out.clone() for x in (a, b, c)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for x, s in zip((a, b, c), streams):
            x.run(stream=s)
    torch.cuda.synchronize()
    for x, y in zip((a, b, c), want):
        x.check()
        assert torch.equal(x.out, y)


@pytest.mark.parametrize("dtype,cache", [(BF16, "bf16"), (BF16, "kvf"), (F32, "fp32")])
def test_the_most_rows(dtype, cache):
    """65535 rows, most of one token; outputs of single tokens are their values, and a few longer rows are checked whole."""
    B = 65535
    rows = [(0, 1)] * B
    for i in (0, 4095, 4096, 40000, B - 1):
        rows[i] = (70, 40)
    b = Batch(3, rows, 1, 1, 64, 16, dtype, cache)
    b.run()
    assert qskv.get_error(b.ws) == 0
    out, cu = b.out.cpu().double(), torch.tensor(b.cu)
    one = torch.tensor([n == 1 for _, n in rows])
    want = b.v[b.table[:, 0].long(), 0, 0]
    tol = 2.0 ** -8 if dtype == BF16 else 2.0 ** -21
    assert bool(((out[cu[:-1], 0] - want).abs()[one] <= tol * want.abs()[one]).all())
    keep = [i for i in range(B) if not one[i]]
    for i in keep:
        x = Batch.__new__(Batch)
        x.__dict__.update(b.__dict__, new=[40], lens=[110], table=b.table[i:i + 1], cu=[0, 40],
                          q=b.q[cu[i]:cu[i] + 40], out=b.out[cu[i]:cu[i] + 40], lse=b.lse[cu[i]:cu[i] + 40])
        x.check()


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_rows_that_share_pages(dtype, cache):
    """Three rows over one prompt's pages, each with its own last page; a page may also be a row's twice."""
    b = Batch(4, [(200, 20), (200, 20), (200, 20)], 4, 2, 64, 16, dtype, cache)
    for r in (1, 2):
        b.table[r, :13] = b.table[0, :13]
    b.table[2, 5] = b.table[2, 2]
    b.run(page_table=b.table.cuda())
    b.check()


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("rows", [SIX, [(100, 2), (0, 3)]])
@pytest.mark.parametrize("d", [64, 128])
def test_addresses_off_the_larger_grids(dtype, cache, rows, d):
    """q, pools and out on 16 bytes only, token strides of an odd number of 16 bytes, sums and index arrays on 4 bytes."""
    b = Batch(5, rows, 4, 2, d, 16, dtype, cache)

    def moved(x, by):
        flat = torch.zeros(x.numel() + by, dtype=x.dtype, device="cuda")
        flat[by:] = x.reshape(-1)
        return flat[by:].view(x.shape)

    vec = 16 // b.q.element_size()
    stride = 4 * d + 3 * vec
    flat = torch.full((b.T * stride + vec,), float("nan"), dtype=dtype, device="cuda")
    q = flat[vec:].as_strided((b.T, 4, d), (stride, d, 1))
    q.copy_(b.gpu["q"])
    b.pools = {k: moved(x, 16 // x.element_size()) for k, x in b.pools.items()}
    b.out, b.lse = moved(b.out, vec), moved(b.lse, 1)
    index = {k: moved(b.gpu[k], 1) for k in ("page_table", "seq_lens", "cu_new")}
    assert q.data_ptr() % 32 == b.out.data_ptr() % 32 == 16 and b.lse.data_ptr() % 8 == 4
    b.run(q=q, **index)
    b.check()
