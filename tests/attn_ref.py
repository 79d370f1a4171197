"""Softmax attention in 64 bits on the CPU, with bounds on what the kernels may be off by.

The bound of an output element follows from the kernels' arithmetic, with u the half step of the
tensors' type (eps / 2) and A = sum_j p_j |v_j| / sum_j p_j:
  - the output's own rounding: u |o| (and the smallest subnormal of float16),
  - the rounding of each p_j to the type before the second product: u A; float16 loses whole bits of
    p_j below 2^-14, at most 2^-25 per key relative to the largest p, which the sum is at least,
  - float32 scores: a dot product of dim terms is off by at most dim 2^-24 sum_d |q_d k_d|, its
    multiplication with the scale, the subtraction of the maximum and exp2 by 2^-22 + 2^-22 |s|
    more, and p_j by as much relative to itself; numerator and denominator both: twice,
  - float32 sums over n keys and the joins: 2 (n + 64) 2^-24 A.
"""
import math

import torch


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rows(q, k, v, last, scale, dtype):
    """Rows q [n, d] over k, v [m, d] (float64); row i sees keys 0 .. last[i] - 1.  Returns (o, tol); a row that sees
    nothing is zero."""
    n, d = q.shape
    m = k.shape[0]
    if m == 0:
        z = torch.zeros(n, v.shape[1], dtype=torch.float64)
        return z, z
    seen = torch.arange(m)[None, :] < last[:, None]
    s = (q @ k.T) * scale
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.max(1, keepdim=True).values
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.exp(s - top)
    p = torch.where(seen, p, torch.zeros_like(p))
    total = p.sum(1, keepdim=True)
    safe = torch.where(total > 0, total, torch.ones_like(total))
    vv = torch.nan_to_num(v, 0.0, 0.0, 0.0) if not torch.isfinite(v).all() else v
    o, a = p @ vv / safe, p @ vv.abs() / safe
    u = half_step(dtype)
    mag = torch.where(seen, (q.abs() @ k.abs().T) * scale, torch.zeros_like(s))
    mag = torch.nan_to_num(mag, 0.0, 0.0, 0.0).max(1, keepdim=True).values
    ds = d * 2.0 ** -24 * mag + 2.0 ** -22 * (1 + 2 * mag)
    vmax = vv.abs().max() if vv.numel() else 0.0
    tol = u * o.abs() + (u + 2 * ds + 2 * (m + 64) * 2.0 ** -24) * a
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 + m * 2.0 ** -25 * vmax / safe
    # a row's own rounding may meet the other errors at a step's border
    return o, tol * (1 + 2 * u) + 1e-30


def prompt(q, k, v, lengths, scale=None):
    """Packed causal attention: (o, tol), each [tokens, heads, dim] float64."""
    t, h, d = q.shape
    g = k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, tol = torch.zeros(t, h, d, dtype=torch.float64), torch.zeros(t, h, d, dtype=torch.float64)
    q64, k64, v64 = (x.detach().cpu().double() for x in (q, k, v))
    at = 0
    for n in lengths:
        for i in range(h):
            j = i // (h // g)
            o[at:at + n, i], tol[at:at + n, i] = rows(q64[at:at + n, i], k64[at:at + n, j], v64[at:at + n, j],
                                                      torch.arange(1, n + 1), scale, q.dtype)
        at += n
    return o, tol


def decode(q, keys, values, scale=None):
    """One query row [heads, dim] per entry of keys / values, lists of [tokens, kv_heads, dim]."""
    b, h, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    o, tol = torch.zeros(b, h, d, dtype=torch.float64), torch.zeros(b, h, d, dtype=torch.float64)
    for i in range(b):
        g = keys[i].shape[1]
        n = keys[i].shape[0]
        for j in range(g):
            sl = slice(j * (h // g), (j + 1) * (h // g))
            o[i, sl], tol[i, sl] = rows(q[i, sl].detach().cpu().double(), keys[i][:, j].double(), values[i][:, j].double(),
                                        torch.full((h // g,), n), scale, q.dtype)
    return o, tol


def check(got, ref, tol, what=""):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, what
    off = (got - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((off / tol.clamp_min(1e-300)).max()),
                           [int(x) for x in bad.nonzero()[0]])
