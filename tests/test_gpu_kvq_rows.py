"""Decodes of so many short rows over the 4-bit cache that a warp takes several of them, one after another."""
import math

import pytest
import torch

import kvq_ref as R
import query_aware_sparse_kv_gb300 as qskv

pytestmark = pytest.mark.gpu


def _check(out, lse, q, k, v, valid, scale):
    """out [n][G][d], lse [n][G] of queries q and tokens k, v [n][T][d] (double, on the GPU), those of `valid` [n][T]."""
    x = (q @ k.transpose(1, 2) * scale).masked_fill(~valid[:, None], -math.inf)
    some = valid.any(1)
    want = torch.where(some[:, None, None], torch.softmax(x, -1), 0) @ v
    # a logit's error is about 2.3e-6 (24 roundings of 2^-24 on parts of up to 8); 5 times that, on values up to max |v|
    assert float((out.double() - want).abs().max()) <= 2.0 ** -16 * float(v.abs().max())
    assert bool((out[~some] == 0).all()) and bool((lse[~some] == -math.inf).all())
    assert float((lse.double() - torch.logsumexp(x, -1))[some].abs().max()) <= 2.0 ** -16


@pytest.mark.parametrize("batch,hkv,G,d,gs,P,pages,top_k", [
    (2600, 2, 4, 64, 64, 16, 3, 0),
    (2500, 1, 8, 128, 128, 32, 7, 0),
    (1900, 4, 2, 64, 32, 16, 12, 0),
    (2600, 1, 8, 64, 64, 16, 13, 0),    # 13 to 32 pages go to warps whole only where every warp gets a row
    (1250, 4, 4, 128, 64, 32, 32, 0),
    (2000, 4, 1, 64, 64, 32, 40, 5),
    (900, 3, 8, 128, 32, 16, 50, 12),
    (1300, 2, 4, 128, 128, 32, 33, 20),
])
def test_a_warp_takes_rows_in_turn(batch, hkv, G, d, gs, P, pages, top_k):
    g = torch.Generator().manual_seed(batch + pages)
    N, hq = 48, hkv * G
    shape = qskv.make_shape(batch, hq, hkv, d, P, pages, N)
    f = [R.quantise(torch.randn((N, hkv, P, d), generator=g), gs) for _ in range(2)]
    pool = R.pack(*f[0], *f[1]).cuda()
    kx, vx = (R.values(*x).cuda() for x in f)
    table = torch.randint(0, N, (batch, pages), generator=g, dtype=torch.int32).cuda()  # rows share pages
    lens = torch.randint(0, pages * P + 1, (batch,), generator=g)
    lens[::11], lens[5::23], lens[7::29] = 0, 1, pages * P
    q = torch.randn((batch, hq, d), generator=g).cuda()
    out, lse = torch.full((batch, hq, d), math.nan, device="cuda"), torch.full((batch, hq), math.nan, device="cuda")
    ws = torch.zeros(qskv.kvq_workspace_size(shape), dtype=torch.uint8, device="cuda")
    kw = {}
    held = torch.arange(pages)[None] * P < lens[:, None]  # [batch][pages]
    listed = held[:, None].expand(batch, hkv, pages)
    if top_k:
        n = torch.minimum(held.sum(1)[:, None], torch.randint(0, top_k + 1, (batch, hkv), generator=g))
        order = torch.rand((batch, hkv, pages), generator=g).masked_fill(~listed, 2).argsort(-1)
        listed = torch.zeros((batch, hkv, pages), dtype=torch.bool).scatter_(2, order, torch.arange(pages) < n[..., None])
        selected = torch.full((batch, hkv, top_k), -1, dtype=torch.int32)
        for b, h, j in listed.nonzero().tolist():
            selected[b, h, int((selected[b, h] >= 0).sum())] = j
        kw = dict(selected=selected.cuda(), n_selected=n.int().cuda(), top_k=top_k)
    qskv.kvq_paged_decode(q, pool, table, lens.int().cuda(), out, shape, gs, ws, lse=lse, **kw)
    assert qskv.get_error(ws) == 0
    token = (torch.arange(pages * P)[None] < lens[:, None]).cuda()
    for h in range(hkv):
        hs = slice(h * G, (h + 1) * G)
        valid = token & listed[:, h].repeat_interleave(P, 1).cuda()
        for a in range(0, batch, 250):
            b = slice(a, a + 250)
            k, v = (x[table[b].long(), h].flatten(1, 2) for x in (kx, vx))
            _check(out[b, hs], lse[b, hs], q[b, hs].double(), k, v, valid[b], d ** -0.5)
