"""Causal attention of every row's newest tokens, in 64 bits, and how far an evaluation may be off."""
import math

import torch


def attend_rows(q, k, v, pos, scale):
    """q [n][G][d], k, v [T][d] doubles, pos [n] -> out [n][G][d], lse [n][G], sum_t p_t |v_t| [n][G][d], and the largest
    sum_i |q_i k_i| scale of a (query, key) pair that counts."""
    if len(k) == 0:
        none = torch.zeros(q.shape, dtype=torch.float64)
        return none, torch.full(q.shape[:2], -math.inf, dtype=torch.float64), none, 0.0
    x = torch.einsum("ngd,td->ngt", q.double(), k) * scale
    off = torch.arange(len(k))[None, :] > pos[:, None]
    x = x.masked_fill(off[:, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top.masked_fill(top == -math.inf, 0.0))
    z = p.sum(-1, keepdim=True)
    p = p / z.clamp_min(1e-300)
    A = torch.einsum("ngd,td->ngt", q.double().abs(), k.abs()) * scale
    A = float(A.masked_fill(off[:, None, :], 0.0).max()) if A.numel() else 0.0
    return p @ v, (top + torch.log(z))[..., 0], p @ v.abs(), A


def bounds(o, pabs, vmax, A, T, d, bf16):
    """Elementwise bound of out, and of lse.

    fp32 arithmetic: logits within (d + 16) roundings of 2^-24 on A, the
    largest sum of absolute products; a change of every logit by at most e
    changes an output by at most 2 e max|v|, the lse by e; exp2 within 2^-22;
    sums of T terms.  Where fp32 products are sums of products of bf16 parts
    each is within 4 roundings, and their sum in steps of 16 within d / 8 of
    them, T / 8 for the outputs: less.  With bf16 operands in addition each weight is rounded
    (2^-8 of it, so 2^-8 sum p|v|) and the output (2^-8 of it); the weights'
    sum is taken before their rounding.
    """
    e = 2.0 ** -24
    tol = (2 * (d + 16) * A + T + 32) * e * vmax
    if bf16:
        # second-order terms: 1 + 2^-7
        return (2.0 ** -8 * pabs + 2.0 ** -8 * o.abs()) * (1 + 2.0 ** -7) + tol * (1 + 2.0 ** -7), ((d + 16) * A + T + 32 + 4 * A) * e
    return torch.full_like(o, tol), ((d + 16) * A + T + 32 + 4 * A) * e
