"""Plain statements of the 8-bit cache, in 64 bits, for the tests.

Codes are bytes, numbers come from their bits; packing moves them to their
places by the rules stated in include/qskv.h.  Nothing here calls the library.
"""
import functools

import torch

NAN = 0x7F  # e4m3's not-a-number


def part_bytes(d):
    return 16 * (2 * d + 2)


@functools.lru_cache
def places(d, P):
    """Bytes within a block of [P][d] key codes, [P][d] value codes, [P] key and [P] value powers, written out."""
    key, val = torch.empty((P, d), dtype=torch.long), torch.empty((P, d), dtype=torch.long)
    kp, vp = torch.empty(P, dtype=torch.long), torch.empty(P, dtype=torch.long)
    for tok in range(P):
        part, t = divmod(tok, 16)
        base, p = part * part_bytes(d), t // 2
        f = (p & 1) + 2 * (p & 2) if d == 128 else 2 * (p % 4)
        for i in range(d):
            c = i // 16
            key[tok, i] = base + t * d + 16 * (c ^ (4 * (t % 2)) if d == 128 else c) + i % 16
            val[tok, i] = base + 16 * d + p * 2 * d + 16 * ((i // 8) ^ f) + 2 * (i % 8) + t % 2
        kp[tok], vp[tok] = base + 32 * d + t, base + 32 * d + 16 + t
    return key, val, kp, vp


def number(u):
    """The numbers of e4m3 bytes, doubles."""
    u = u.long()
    e, m = (u >> 3) & 15, (u & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    x = torch.where((u & 0x7F) == NAN, torch.full_like(x, float("nan")), x)
    return torch.where(u >= 128, -x, x)


_GRID = number(torch.arange(NAN))  # 0 .. 448, ascending


def code(y):
    """Doubles of at most 448 in magnitude -> e4m3 bytes, to nearest, ties to even (by looking at both neighbours)."""
    a = y.abs()
    hi = torch.searchsorted(_GRID, a.contiguous()).clamp(max=NAN - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = a - _GRID[lo], _GRID[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    u = torch.where(_GRID[hi] == a, hi, torch.where(up, hi, lo))
    return u + 128 * (torch.signbit(y)).long()


def quantise(x):
    """x [..., d] -> codes [..., d], e [...] (long)."""
    x = x.double()
    top = x.abs().amax(-1)
    e = torch.full(top.shape, -100, dtype=torch.long)
    for k in range(-100, 120):  # the smallest e that holds the largest magnitude
        e = torch.where(top > 448.0 * 2.0 ** (k - 1), torch.full_like(e, k), e)
    return code(x * torch.exp2(-e.double())[..., None]), e


def values(u, e):
    return number(u) * torch.exp2(e.double())[..., None]


def pack(ku, ke, vu, ve):
    """Fields [N][H][P][...] -> pool bytes [N][H][block]."""
    N, H, P, d = ku.shape
    pool = torch.zeros((N, H, P // 16 * part_bytes(d)), dtype=torch.long)
    for at, x in zip(places(d, P), (ku, vu, ke + 127, ve + 127)):
        pool[:, :, at.flatten()] = x.flatten(2)
    return pool.to(torch.uint8)


def unpack(pool, d, P):
    """Pool bytes [N][H][block] -> (codes, e) of keys, (codes, e) of values, fields [N][H][P][...]."""
    x = pool.long()
    key, val, kp, vp = places(d, P)
    return (x[..., key], x[..., kp] - 127), (x[..., val], x[..., vp] - 127)


def attend_bounds(q, k, v, scale):
    """How far an fp32 evaluation may be off (out, lse), for one row's heads over tokens k, v [T][d].

    Logits: d products in any order of fp32 additions, the query within 2^-22:
    (d + 16) roundings of 2^-24 on the absolute sum A.  A change of every
    logit by at most e changes the output by at most 2 e max|v| and the lse by
    e.  Weights: exp2 within 2^-22, two fp16 halves within 2^-22, sums of T
    terms.
    """
    T, d = k.shape
    A = float((q.double().abs() @ k.abs().T).amax() * scale)
    e = 2.0 ** -24
    return (2 * (d + 16) * A + T + 32) * e * float(v.abs().max()), ((d + 16) * A + T + 32 + 4 * A) * e
