"""Every block of a long row counts once: prefill over keys of zeros, where an output is how many tokens of each run of blocks
a query sees, over how many it sees.  A block that is left out, read twice, from another page or from an earlier call shows as
a wrong count, whatever the row's length."""
import pytest
import torch

import kvf_ref as F
import query_aware_sparse_kv_gb300 as qskv
from test_gpu_prefill import KINDS

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from query_aware_sparse_kv_gb300 import build

    build.build()
    qskv.load()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


ROWS = [
    # few tokens of few rows, which need no list: the blocks lie on a line that the CTAs share out
    ([(9000, 5), (1, 2), (20000, 1)], 8, 2, 128, 32),      # a CTA has a range of one tile
    ([(30000, 17)], 16, 2, 64, 16),
    ([(3000 + 500 * (i % 5), 1) for i in range(32)], 4, 4, 64, 16),  # and of several
    ([(1000 + 100 * i, i % 3) for i in range(19)], 8, 4, 64, 32),    # fewer blocks than the CTAs' least share
    ([(1216 * 128 - 1, 1)], 1, 1, 128, 16),                # as many blocks as make 152 CTAs' shares even, and one less
    ([(1215 * 128 - 1, 1)], 1, 1, 128, 16),
    # a list, its long tiles in parts
    ([(20000, 300)], 4, 2, 128, 16),
    ([(9000, 40), (3, 1), (2500, 1), (0, 700)], 4, 2, 64, 32),
    ([(0, 5000)], 8, 1, 128, 16),
    ([(i * 150, 1 + i % 2 * 90) for i in range(40)], 4, 4, 64, 16),
]


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("rows,hq,hkv,d,P,lead", [(*x, 0) for x in ROWS] + [(*ROWS[i], 37) for i in (0, 2, 7)])
def test_every_block_counts_once(dtype, cache, rows, hq, hkv, d, P, lead):
    """lead: rows of q before the first sequence's, as behind the last one: left as they are."""
    g = torch.Generator().manual_seed(len(rows) + d + P)
    G, B = hq // hkv, len(rows)
    lens, new = [o + n for o, n in rows], [n for _, n in rows]
    pages = [-(-x // P) for x in lens]
    mp, N = max(pages), sum(pages) + 1
    run = 128 * -(-max(lens) // (128 * hkv * d))  # tokens of a run of blocks; each has a dim of one head
    ids = torch.randperm(N, generator=g)
    table = torch.full((B, mp), -1, dtype=torch.int32)
    v = torch.zeros((2, N, hkv, P, d), dtype=torch.float32 if cache == "fp32" else torch.bfloat16)  # two kinds of values
    at = 0
    for b in range(B):
        mine = ids[at:at + pages[b]]
        table[b, :pages[b]] = mine.to(torch.int32)
        at += pages[b]
        t = torch.arange(pages[b] * P)
        name = t // run
        for kind, x in enumerate((name, hkv * d - 1 - name)):
            v[kind, mine[t // P], x // d, t % P, x % d] = 1.0
    k = torch.zeros(v.shape[1:], dtype=v.dtype)
    cu = [lead]
    for n in new:
        cu.append(cu[-1] + n)
    T = cu[-1] + 3
    shape = qskv.make_shape(B, hq, hkv, d, P, mp, N)
    size = qskv.prefill_workspace_size(shape, T)
    room = torch.zeros(size + 4096, dtype=torch.uint8, device="cuda")
    room[size:] = 0xA5
    ws = room[:size]
    q = torch.randn((T, hq, d), generator=g).to(dtype).cuda()
    args = (table.cuda(), _i32(lens), _i32(cu))
    seen = torch.cat([torch.arange(o, o + n) for o, n in rows]) + 1  # tokens that a query sees
    start = torch.arange(hkv * d) * run
    count = (seen[:, None] - start).clamp(0, run).double() / seen[:, None]  # [queries][runs]
    for kind in (0, 1, 0):
        # in this order: the outputs of a kind are not those of the call before
        if cache == "kvf":
            pools = [F.pack(*F.quantise(k.double()), *F.quantise(v[kind].double())).cuda()]
        else:
            pools = [k.cuda(), v[kind].cuda()]
        out = torch.full((T, hq, d), 7.0, dtype=dtype, device="cuda")
        lse = torch.full((T, hq), 7.0, device="cuda")
        fn = qskv.kvf_paged_prefill if cache == "kvf" else qskv.paged_prefill
        fn(q, *pools, *args, out, shape, ws, lse=lse)
        assert qskv.get_error(ws) == 0
        out, lse = out.cpu().double(), lse.cpu().double()
        for x in (out, lse):
            assert bool((x[:lead] == 7).all()) and bool((x[cu[-1]:] == 7).all())
        want = (count if kind == 0 else count.flip(1)).view(-1, hkv, 1, d).expand(-1, -1, G, -1).reshape(-1, hq, d)
        # every weight is 1 and every count exact: a division, the parts' shares (a power of two of a difference of logarithms
        # of at most 15, 2^-19) and the output's own rounding
        tol = (2.0 ** -17 + (2.0 ** -8 if dtype == BF16 else 0.0)) * want
        bad = (out[lead:cu[-1]] - want).abs() > tol
        assert not bool(bad.any()), (kind, torch.nonzero(bad)[:5].tolist(), int(bad.sum()))
        assert float((lse[lead:cu[-1]] - torch.log(seen.double())[:, None]).abs().max()) <= 2.0 ** -19
        assert bool((room[size:] == 0xA5).all())
