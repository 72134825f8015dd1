"""Prefill at the ends of what include/qskv.h allows: the largest logits beside the largest values."""
import os
import re

import pytest
import torch

import kvf_ref as F
import query_aware_sparse_kv_gb300 as qskv
from test_gpu_prefill import KINDS

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HEADER = os.path.join(os.path.dirname(qskv.__file__), os.pardir, "include", "qskv.h")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from query_aware_sparse_kv_gb300 import build

    build.build()
    qskv.load()


def limit():
    """N of the 2^N that a logit must be below with bf16 operands, as the header says."""
    text = re.sub(r"\s*\n \*\s*", " ", open(HEADER).read())
    return int(re.search(r"with bf16 queries over a bf16 or 8-bit cache.{0,400}?every logit must then be below 2\^(\d+)", text,
                         re.I).group(1))


def worst(top):
    """A bf16 number times an e4m3 one, below 2^top, whose product with log2 e rounds down (up) the furthest."""
    a = 2.0 ** ((top + 1) // 2) * (1 + torch.arange(128).double() / 128) / 2
    b = 2.0 ** (top // 2) * (1 + torch.arange(8).double() / 8) / 2
    s = (a[:, None] * b[None, :]).flatten()
    sc = torch.tensor(1.4426950408889634).float().double()
    off = s * sc - (s * sc).float().double()  # (33 bits: exact in double)
    off[s < 2.0 ** (top - 1)] = 0.0
    for i in (int(off.argmax()), int(off.argmin())):
        yield float(a[i // 8]), float(b[i % 8])


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("d,P", [(64, 32), (128, 16)])
@pytest.mark.parametrize("rows", [[(200, 3)], [(0, 300), (900, 2)]])
def test_largest_logits_and_values(dtype, cache, sign, d, P, rows):
    """Equal keys, so that the outputs are means of equal values of just below 2^72 (2^60 in 8 bits): as they are, up to their
    rounding."""
    big = -1.75 * 2.0 ** (59 if cache == "kvf" else 71)
    low = dtype == BF16 and cache != "fp32"
    H, T, B = 2, sum(n for _, n in rows), len(rows)
    lens = [o + n for o, n in rows]
    pages = -(-max(lens) // P)
    shape = qskv.make_shape(B, 2 * H, H, d, P, pages, B * pages)
    for x, y in worst(limit()) if low else [(1.75 * 2.0 ** 59, 1.75 * 2.0 ** 59)]:
        k, v = torch.zeros((B * pages, H, P, d)), torch.full((B * pages, H, P, d), big)
        q = torch.zeros((T, 2 * H, d), dtype=dtype)
        if low:
            k[..., 0], q[..., 0] = sign * y, x
        else:  # every dim: the sum of products is 3.06 * 2^118 times d, below 2^127
            k[:], q[:] = sign * y, x
        if cache == "kvf":
            pools = [F.pack(*F.quantise(k), *F.quantise(v)).cuda()]
        else:
            dt = BF16 if cache == "bf16" else F32
            pools = [k.to(dt).cuda(), v.to(dt).cuda()]
        cu = [0]
        for _, n in rows:
            cu.append(cu[-1] + n)
        i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
        table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
        ws = torch.zeros(qskv.prefill_workspace_size(shape, T), dtype=torch.uint8, device="cuda")
        out = torch.empty((T, 2 * H, d), dtype=dtype, device="cuda")
        lse = torch.empty((T, 2 * H), device="cuda")
        fn = qskv.kvf_paged_prefill if cache == "kvf" else qskv.paged_prefill
        scale = 1.0 if low else 0.0
        fn(q.cuda(), *pools, table, i32(lens), i32(cu), out, shape, ws, lse=lse, sm_scale=scale)
        assert qskv.get_error(ws) == 0
        # weights are equal: their rounding is one factor of all, which their unrounded sum does not have (2^-8), and the
        # output's (2^-8); fp32: sums of up to 902 terms, and the division
        tol = (2.0 ** -7 + 2.0 ** -13) if low else 2.0 ** -13 + (2.0 ** -8 if dtype == BF16 else 0.0)
        assert float((out.cpu().double() / big - 1).abs().max()) <= tol
        l = sign * x * y * (1 if low else d ** 0.5)
        assert float((lse.cpu().double() / l - 1).abs().max()) <= 2.0 ** -20
