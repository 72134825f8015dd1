"""What the 4-bit decode's sums and references have to stand: logits and values of every order, and fp32 precision that a
lost fp16 half would break."""
import math

import pytest
import torch

import kvq_ref as R
import query_aware_sparse_kv_gb300 as qskv

gpu = pytest.mark.gpu
P = 32
ROWS = 320  # more rows than CTAs, of at most 12 pages: a warp takes whole rows, tile after tile


class Case:
    """`rows` sequences over the same cached tokens k, v [T][hkv][d] (their pages are shared); q [hq][d] of all of them,
    or [rows][hq][d]."""

    def __init__(self, q, k, v, gs, rows=ROWS, dtype=torch.float32):
        T, hkv, d = k.shape
        self.T, self.hkv, self.d, self.gs, self.rows = T, hkv, d, gs, rows
        n = -(-T // P)
        pad = torch.zeros((n * P - T, hkv, d), dtype=k.dtype)
        f = [R.quantise(torch.cat([x, pad]).unflatten(0, (n, P)).transpose(1, 2), gs) for x in (k, v)]
        self.pool = R.pack(*f[0], *f[1])
        # the cached values, [T][hkv][d] in 64 bits
        self.k, self.v = (R.values(*x).transpose(1, 2).flatten(0, 1)[:T] for x in f)
        self.q = q.expand((rows,) + q.shape[-2:]).contiguous().to(dtype)
        self.shape = qskv.make_shape(rows, q.shape[-2], hkv, d, P, n, n)

    def run(self, scale):
        B, hq, d = self.q.shape
        n = self.shape.max_pages
        ws = torch.zeros(qskv.kvq_workspace_size(self.shape), dtype=torch.uint8, device="cuda")
        out, lse = torch.full((B, hq, d), math.nan, device="cuda"), torch.full((B, hq), math.nan, device="cuda")
        table = torch.arange(n, dtype=torch.int32).repeat(B, 1).cuda()
        qskv.kvq_paged_decode(self.q.cuda(), self.pool.cuda(), table,
                              torch.full((B,), self.T, dtype=torch.int32, device="cuda"), out, self.shape, self.gs, ws,
                              lse=lse, sm_scale=scale)
        assert qskv.get_error(ws) == 0
        return out.cpu().double(), lse.cpu().double()

    def exact(self, scale, row=0):
        G = self.q.shape[1] // self.hkv
        r = [R.attend(self.q[row, h * G:(h + 1) * G], self.k[:, h], self.v[:, h], scale) for h in range(self.hkv)]
        return torch.cat([x[0] for x in r]), torch.cat([x[1] for x in r])


def _steps(T, heads, d, logits):
    """Queries and keys of `heads` heads of one group whose logits, in binary orders with a scale of 1, are
    logits [heads][T]: head h reads 32 dims of d, the last 32 from head d / 32 - 1 on, which hold its logit (a bf16
    number) in every place."""
    q, k = torch.zeros((heads, d)), torch.zeros((T, 1, d))
    for h in range(heads):
        at = 32 * min(h, d // 32 - 1)
        q[h, at:at + 32] = math.log(2) / 32
        k[:, 0, at:at + 32] = logits[h][:, None]
    return q, k


@gpu
@pytest.mark.parametrize("heads,gap,strong,late", [(2, 100, 15000.0, 30.0), (4, 100, 15000.0, 30.0), (8, 100, 15000.0, 30.0),
                                                  (2, 105, 4e5, 1000.0), (2, 60, 30.0, 3e-5), (8, 4, 1.0, 1.0)])
def test_a_head_keeps_its_sums_while_another_ones_logits_rise(heads, gap, strong, late):
    """The first head has 64 tokens of values 0 and `strong`, then ones of `gap` binary orders less weight and values up to
    `late`; the last head's logits rise by 14 orders a tile, so that the references move at every step.  The strong tokens'
    logits are zeros, hence their weights equal."""
    T = 12 * P
    g = torch.Generator().manual_seed(heads + gap)
    t = torch.arange(T)
    logits = [torch.where(t < 64, 0, -gap).float()] + [(t // 16 * 14.0)] * (heads - 1)
    q, k = _steps(T, heads, 128, logits)
    v = torch.rand((T, 1, 128), generator=g)
    v = torch.where(t[:, None, None] < 64, (v > 0.1).float() * strong, v * late)
    c = Case(q, k, v, 32)
    out, lse = c.run(1.0)
    o, l = c.exact(1.0)
    # weights of powers of two of logits that are sums of 32 equal products (off by 2^-22 of them at most), 384 tokens' sums
    # of 2^-24 each, two fp16 halves 2^-22: all below 2^-14 of the largest value where logits reach 336, 2^-18 for the first
    top = float(c.v.abs().max())
    assert bool(torch.isfinite(out).all())
    assert float((out[:, 0] - o[0]).abs().max()) <= 2.0 ** -18 * top
    assert float((out - o).abs().max()) <= 2.0 ** -14 * top
    assert float((lse - l).abs().max()) <= 2.0 ** -14


def _relative(out, o):
    """Root mean square of the errors over that of the outputs."""
    return float((out - o).pow(2).mean().sqrt() / o.pow(2).mean().sqrt())


# The bound on it.  A logit of order 1 is a sum of a few parts of up to about 8 (a group's scale times its codes, its minimum
# times the query's sum) with some 24 roundings of half a step, 2^-24: 8 sqrt(24) 2^-24 = 2.3e-6 by their root mean square.
# Weights carry that and their two halves' 2^-22; tokens' errors are independent and add up as the outputs themselves do.
PRECISION = 2.0 ** -18


def _fp32(c, scale, halve_q=None, halve_w=None):
    """The rows' outputs by plain fp32 torch; queries or weights rounded to a shorter type where one is given."""
    G = c.q.shape[1] // c.hkv
    outs = []
    for h in range(c.hkv):
        q = c.q[:, h * G:(h + 1) * G].float()
        if halve_q is not None:
            q = q.to(halve_q).float()
        x = q @ c.k[:, h].float().T * scale
        p = torch.exp(x - x.amax(-1, keepdim=True))
        w = p if halve_w is None else p.to(halve_w).float()
        outs.append(w @ c.v[:, h].float() / p.sum(-1, keepdim=True))
    return torch.cat(outs, 1).double()


def _plain_case(seed, d, gs, hq, hkv, dtype, rows=4, T=300):
    g = torch.Generator().manual_seed(seed)
    return Case(torch.randn((rows, hq, d), generator=g), torch.randn((T, hkv, d), generator=g),
                torch.randn((T, hkv, d), generator=g), gs, rows=rows, dtype=dtype)


def test_the_precision_bound_takes_fp32_and_refuses_a_lost_half():
    c = _plain_case(1, 128, 64, 8, 2, torch.float32)
    o = torch.stack([c.exact(128 ** -0.5, r)[0] for r in range(c.rows)])
    assert _relative(_fp32(c, 128 ** -0.5), o) < PRECISION / 4
    for kw in (dict(halve_q=torch.float16), dict(halve_q=torch.bfloat16), dict(halve_w=torch.float16),
               dict(halve_w=torch.bfloat16)):
        assert _relative(_fp32(c, 128 ** -0.5, **kw), o) > PRECISION * 8, kw


FORMATS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,gs", FORMATS)
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("rows", [4, ROWS])
def test_outputs_have_fp32_precision(dtype, d, gs, hq, hkv, rows):
    c = _plain_case(d + gs + hq, d, gs, hq, hkv, dtype, rows=rows)
    out, _ = c.run(d ** -0.5)
    some = range(0, rows, max(1, rows // 8))
    o = torch.stack([c.exact(d ** -0.5, r)[0] for r in some])
    assert _relative(out[list(some)], o) <= PRECISION


@gpu
@pytest.mark.parametrize("lead", [0.0, 0.5])
@pytest.mark.parametrize("small", [1e-3, 1e-6, 1e-9])
@pytest.mark.parametrize("d,gs,hq", [(64, 32, 2), (128, 128, 4), (128, 64, 8)])
def test_small_values_after_tokens_of_one_value(lead, small, d, gs, hq):
    """The first 40 tokens' values are all zero (or all a half) over the head, scales of zero; the others' are small.  With a
    lead of a half the small values are looked at as what the outputs hold beside its share."""
    g = torch.Generator().manual_seed(hq)
    T = 300
    v = torch.randn((T, 1, d), generator=g) * small
    v[:40] = lead
    c = Case(torch.randn((hq, d), generator=g), torch.randn((T, 1, d), generator=g), v, gs)
    out, _ = c.run(d ** -0.5)
    o, _ = c.exact(d ** -0.5)
    if lead:  # an output is rounded against that share: no more than PRECISION of it
        assert float((out - o).abs().max()) <= PRECISION * 8 * float(o.abs().max())
    else:
        for r in (0, ROWS // 2, ROWS - 1):
            assert _relative(out[r], o) <= PRECISION


@gpu
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("power", [40, 52, 58])
@pytest.mark.parametrize("rows,hq", [(3, 4), (ROWS, 8)])
def test_logits_of_any_finite_size(sign, power, rows, hq):
    """Equal keys and queries of up to 2^58: every logit the same, up to 2^122 in magnitude; the outputs are the mean."""
    g = torch.Generator().manual_seed(power)
    big = 2.0 ** power
    T = 100
    c = Case(torch.full((hq, 64), big), torch.full((T, 1, 64), sign * big), torch.randn((T, 1, 64), generator=g), 64, rows=rows)
    out, lse = c.run(0.0)
    o = c.v[:, 0].mean(0)
    assert float((out - o).abs().max()) <= 2.0 ** -18 * float(c.v.abs().max())
    l = sign * big * big * 64 / 8
    assert float((lse - l).abs().max()) <= 2.0 ** -20 * abs(l)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,gs", FORMATS)
@pytest.mark.parametrize("hq", [1, 4, 8])
@pytest.mark.parametrize("outlier", [1, 2 ** 4, 2 ** 8, 2 ** 12])
def test_logits_with_one_outlying_query_dim(dtype, d, gs, hq, outlier):
    """Rows of one token: the lse is the logit itself.  One query entry is `outlier` times the others.

    The largest entry is at least 2^13 / 1.07 units, every entry held as two fp16 halves within 2^-9 and 2^-14 of them (its
    own and the one it shares a product with): 2^-21.8 of the largest.  The tensor cores cut the 16 products and the sum of
    an instruction to 2^-23 of the largest product, at most 15 of the largest entry.  Both on codes of up to 15:
    2^-21 max |q| sum 15 s.  The rest is fp32: 20 roundings, on partial sums of at most A = sum |q| (|m| + s u)."""
    g = torch.Generator().manual_seed(d + gs + hq)
    q = torch.randn((ROWS, hq, d), generator=g)
    q[:, :, 5] *= outlier
    k = torch.randn((1, 1, d), generator=g)
    c = Case(q, k, torch.randn((1, 1, d), generator=g), gs, dtype=dtype)
    _, lse = c.run(1.0)
    u, s, m = R.quantise(k[0, 0], gs)
    s, m = (x.repeat_interleave(gs, -1) for x in (s, m))
    q = c.q.double()
    tol = 2.0 ** -21 * q.abs().amax(-1) * 15 * s.sum() + 20 * 2.0 ** -24 * (q.abs() @ (m.abs() + s * u))
    assert bool(((lse - q @ c.k[0, 0]).abs() <= tol).all())
