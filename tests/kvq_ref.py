"""Plain statements of the 4-bit cache and the page tables, in 64 bits, for the tests.

Packing works on unpacked fields (codes, scales, minima) and moves them to
their places by the rules stated in include/qskv.h; nothing here calls the
library.
"""
import math

import torch


def places(d, P):
    """(key place, value place) [P][d/8] of each code word within its token's row."""
    key = torch.empty((P, d // 8), dtype=torch.long)
    val = torch.empty((P, d // 8), dtype=torch.long)
    for t in range(P):
        for w in range(d // 8):
            i, r = divmod(w, 4)
            key[t, w] = r * (d // 32) + i
            x = (t // 2) % 4 if d == 128 else (t // 4) % 2
            val[t, w] = 4 * (i ^ x) + r
    return key, val


def block_words(d, P, gs):
    return (P * d + 8 * P * (d // gs)) // 4


def round_bits(x, bits=8):
    """x >= 0 (double) to `bits` significant bits, to nearest even, once."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(torch.ldexp(m, torch.full_like(e, bits))), e - bits)


def quantise(x, gs):
    """x [..., d] -> codes [..., d] (long), s, m [..., d/gs] (double, bf16 values)."""
    g = x.double().unflatten(-1, (-1, gs))
    m = g.amin(-1).float().to(torch.bfloat16).double()
    step = ((g.amax(-1) - m) / 15).clamp_min(0)
    s = torch.where(step >= 2.0 ** -100, round_bits(step), torch.zeros_like(step))
    q = (g - m[..., None]) / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    u = torch.where((s > 0)[..., None], torch.round(q).clamp(0, 15), torch.zeros_like(q))
    return u.long().flatten(-2), s, m


def values(u, s, m):
    n = u.shape[-1] // s.shape[-1]
    return m.repeat_interleave(n, -1) + s.repeat_interleave(n, -1) * u.double()


def _bf16_bits(x):
    return x.float().to(torch.bfloat16).view(torch.int16).long() & 0xFFFF


def pack(ku, ks, km, vu, vs, vm):
    """Fields [N][H][P][...] -> pool bytes [N][H][block]."""
    N, H, P, d = ku.shape
    ng = ks.shape[-1]
    pool = torch.zeros((N, H, block_words(d, P, d // ng)), dtype=torch.long)
    sh = torch.arange(0, 32, 4)
    W = d // 8
    for which, (u, s, m, place) in enumerate(zip((ku, vu), (ks, vs), (km, vm), places(d, P))):
        word = (u.unflatten(-1, (W, 8)) << sh).sum(-1)
        at = (torch.arange(P)[:, None] * W + place + which * P * W).flatten()
        pool[:, :, at] = word.flatten(-2)
        p0 = 2 * P * W + which * ng * P
        pool[:, :, p0:p0 + ng * P] = (_bf16_bits(s) | (_bf16_bits(m) << 16)).transpose(-1, -2).flatten(-2)
    pool = torch.where(pool >= 2 ** 31, pool - 2 ** 32, pool).to(torch.int32)
    return pool.view(torch.uint8)


def unpack(pool, d, P, gs):
    """Pool bytes [N][H][block] -> ((u, s, m) of keys, (u, s, m) of values), fields [N][H][P][...]."""
    w = pool.contiguous().view(torch.int32).long() & 0xFFFFFFFF
    W, ng = d // 8, d // gs
    sh = torch.arange(0, 32, 4)
    out = []
    for which, place in enumerate(places(d, P)):
        at = (torch.arange(P)[:, None] * W + place + which * P * W).flatten()
        u = ((w[..., at].unflatten(-1, (P, W))[..., None] >> sh) & 15).flatten(-2)
        p0 = 2 * P * W + which * ng * P
        par = w[..., p0:p0 + ng * P].unflatten(-1, (ng, P)).transpose(-1, -2)
        s = (par & 0xFFFF).to(torch.int16).view(torch.bfloat16).double()
        m = (par >> 16).to(torch.int16).view(torch.bfloat16).double()
        out.append((u, s, m))
    return out


def attend(q, k, v, scale):
    """q [G][d], k, v [T][d] doubles -> out [G][d], lse [G] (0 and -inf for no token)."""
    if k.shape[0] == 0:
        return torch.zeros(q.shape, dtype=torch.float64), torch.full((q.shape[0],), -math.inf, dtype=torch.float64)
    x = q.double() @ k.T * scale
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    z = p.sum(-1, keepdim=True)
    return p @ v / z, (top + torch.log(z))[:, 0]


def attend_bounds(q, km, ks, vm, vs, scale, T):
    """How far an fp32 evaluation may be off (out, lse), for one row's heads.

    Logits: a dot product of d terms, each split off its group's m + s u, in
    any order of fp32 additions: (d + 16) roundings of 2^-24 on the absolute
    sum A.  A change of every logit by at most e changes the output by at most
    2 e max|v| and the lse by e.  Weights: exp2 within 2^-22, two fp16 halves
    within 2^-22, sums of T terms.
    """
    d = q.shape[-1]
    n = d // ks.shape[-1]
    kabs = (km.abs() + 15 * ks).amax(0).repeat_interleave(n, -1)
    A = float((q.double().abs() @ kabs).amax() * scale)
    vmax = float((vm.abs() + 15 * vs).max())
    e = 2.0 ** -24
    return (2 * (d + 16) * A + T + 32) * e * vmax, ((d + 16) * A + T + 32 + 4 * A) * e


def tables(seq_lens, new_lens, free, table, P, n_pool, max_tokens, max_touched):
    """What qskv_extend_tables writes, request by request (lists and a copy of the table)."""
    B, mp = len(seq_lens), len(table[0])
    table = [list(r) for r in table]
    r = dict(page_table=table, seq_lens_out=list(seq_lens), cu_new=[0], slot_map=[-1] * max_tokens,
             positions=[-1] * max_tokens, touched_ids=[-1] * max_touched, touched_valid=[0] * max_touched)
    taken = touched = refused = tokens = pages = 0
    for b in range(B):
        old, new = seq_lens[b], new_lens[b]
        first = tokens
        tokens += max(new, 0)
        r["cu_new"].append(min(tokens, max_tokens))
        valid = old >= 0 and new >= 0 and old + new <= mp * P
        if valid:
            pages += -(-(old + new) // P) - -(-old // P)
        if new == 0 and valid:
            continue
        if not valid or tokens > max_tokens or pages > len(free):
            refused += new != 0
            continue
        for t in range(old, old + new):
            if t % P == 0:
                table[b][t // P] = free[taken] if 0 <= free[taken] < n_pool else -1
                taken += 1
            page = table[b][t // P]
            good = 0 <= page < n_pool
            if t == old or t % P == 0:
                r["touched_ids"][touched] = page if good else -1
                r["touched_valid"][touched] = min(P, old + new - t // P * P) if good else 0
                touched += 1
            r["slot_map"][first + t - old] = page * P + t % P if good else -1
            r["positions"][first + t - old] = t
        r["seq_lens_out"][b] = old + new
    r["counts"] = [min(tokens, max_tokens), taken, touched, refused]
    return r
