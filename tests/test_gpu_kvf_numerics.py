"""How exact the decode over the 8-bit cache is where logits are far apart, or large, and values are of any size."""
import math

import pytest
import torch

import kvf_ref as R
import query_aware_sparse_kv_gb300 as qskv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from query_aware_sparse_kv_gb300 import build

    build.build()
    qskv.load()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def decode(q, k, v, scale, rows=1, P=16):
    """`rows` equal rows of q [Hq][d] over the 8-bit tokens k, v [T][Hkv][d]: out, lse of every row, and the cached values."""
    T, hkv, d = k.shape
    N = -(-T // P)
    shape = qskv.make_shape(rows, len(q), hkv, d, P, N, N)
    pool = torch.zeros((N, hkv, qskv.kvf_block_bytes(shape)), dtype=torch.uint8, device="cuda")
    ws = torch.zeros(qskv.kvf_workspace_size(shape), dtype=torch.uint8, device="cuda")
    qskv.kvf_append(k.cuda(), v.cuda(), torch.arange(T, dtype=torch.int32, device="cuda"), pool, shape, ws)
    out, lse = torch.empty((rows,) + q.shape, device="cuda"), torch.empty((rows, len(q)), device="cuda")
    qskv.kvf_paged_decode(q.cuda().repeat(rows, 1, 1), pool, _i32([list(range(N))] * rows), _i32([T] * rows), out, shape, ws,
                          lse=lse, sm_scale=scale)
    assert qskv.get_error(ws) == 0
    return out.cpu().double(), lse.cpu().double(), *(R.values(*R.quantise(x)) for x in (k, v))


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("power", [14, 15, 16, 40, 58])
@pytest.mark.parametrize("size", [-90, -8, 0, 24, 59])
@pytest.mark.parametrize("rows,hq,T", [(3, 4, 100), (1, 8, 3000), (700, 2, 40)])
def test_logits_and_values_of_any_finite_size(sign, power, size, rows, hq, T):
    """Equal keys and queries of up to 2^58, values of up to 2^59: every logit the same, up to 2^122 in magnitude; the outputs
    are the mean.  A weight is one exponential within 2^-22, held within 2^-22 or 2^-33 of the largest (its power times a code
    is at most twice the largest value); sums of T terms, one division, and as many roundings again where parts are joined."""
    g = torch.Generator().manual_seed(power)
    big = 2.0 ** power
    v = (torch.rand((T, 1, 64), generator=g) * 2 - 1) * 2.0 ** size
    out, lse, _, v = decode(torch.full((hq, 64), big), torch.full((T, 1, 64), sign * big), v, 0.0, rows)
    tol = (2.0 ** -20 + 2.0 ** -32 + 2 * (T + 32) * 2.0 ** -24) * float(v.abs().max())
    assert float((out - v[:, 0].mean(0)).abs().max()) <= tol
    l = sign * big * big * 64 / 8
    assert float((lse - l).abs().max()) <= 2.0 ** -20 * abs(l)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("far", [44.0, 88.0, 96.0, 104.0, 112.0, 120.0])
@pytest.mark.parametrize("low", [-92, -96, -100])
def test_weights_keep_their_bits_beside_a_token_of_tiny_values(first, d, far, low):
    """One token with a logit `far` (in powers of two) above the others and values of 2^low or zeros: weights times powers are
    within 2^-22 of themselves or 2^-33 of their head's largest, besides the exponential's 2^-22.  Every other token has a dim
    of its own, so an output is one weight times 448 times its power."""
    steps = [-0.375, -0.875, -1.375, -2.75, -3.25, -3.75, -5.5, -6.5, -7.5, -9.0, -11.0, -13.0, -15.0]
    T = len(steps) + 1
    k, v = torch.zeros((T, 1, d)), torch.zeros((T, 1, d))
    k[0, 0, 0] = far
    k[1:, 0, 0] = torch.tensor(steps)
    v[0] = 1.75 * 2.0 ** (low + 8) if low > -100 else 0.0
    v[torch.arange(1, T), 0, torch.arange(1, T)] = 1.75
    if not first:
        k, v = k.flip(0), v.flip(0)
    q = torch.zeros((2, d))
    q[:, 0] = 1.0
    out, _, kc, vc = decode(q, k, v, math.log(2))
    x = kc[:, 0, 0]  # logits, in powers of two up to the scale's rounding: 2^-24 of 120
    f = R.quantise(v)[1].double()[:, 0]
    p = torch.exp2(x - x.max())
    W = p * torch.exp2(f)
    want = (p @ vc[:, 0]) / p.sum()
    # of each token's weight: the exponential, the logit's rounding (2^-24 times 2 roundings of up to 120: 2^-16), the halves
    tol = (2.0 ** -21 + 2.0 ** -15) * W + 2.0 ** -33 * W.max()
    tol = (tol[:, None] * 448 * (vc[:, 0] != 0)).sum(0) / p.sum() + 2.0 ** -21 * want.abs()
    assert bool(((out[0] - want).abs() <= tol).all()), float(((out[0] - want).abs() / tol).nan_to_num().max())
