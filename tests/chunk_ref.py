"""Attention of chunks over a cache, and norms and rotations of heads, in 64 bits on the CPU, with bounds on what the kernels
may be off by.

Attention: with u the half step of the tensors' type, p the weights and A = sum_j p_j |v_j| / sum_j p_j, an output element may
be off by
  - its own rounding: u |o| (and half the smallest subnormal of float16),
  - the rounding of each p_j to the type before the second product: u A; float16 loses whole bits of p_j below 2^-14, at most
    2^-25 for a key relative to the largest p, which the sum is at least,
  - the scores' errors ds_j, by which p_j is off relative to itself, in numerator and denominator:
    sum_j p_j ds_j (|v_j| + |o|) / sum_j p_j.  ds_j is dim 2^-24 sum_d |q_d k_d| scale for the dot product, and 2^-22 of all
    that is added, multiplied and subtracted on the way (the score, the bias, the reference point) and of 1 for exp2; a cap
    adds 2^-21 cap, which is documented, and takes no more than that because its slope is at most 1,
  - float32 sums over m keys and the joins: 2 (m + 64) 2^-24 A.

Norm and rotation: inv = 1 / sqrt(sum / dim + eps) is off by (dim / 2 + 8) 2^-24 relative (a float32 sum of dim squares, halved
by the root, and a few operations), a cosine or sine by 6 2^-24 (angle: 2^-24 of at most pi / 4 twice; series below 2^-25;
roundings of its five operations), each product and sum by 2^-24: with a, b the values of a pair
  u |y| + m (|a| + |b|) ((dim / 2 + 8) norm + 10) 2^-24
"""
import math

import numpy as np
import torch


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rows(q, k, v, lo, hi, pos, scale, cap, slope, dtype):
    """Rows q [n, d] over k, v [m, d] (float64); row i, at place pos[i], sees keys lo[i] .. hi[i] - 1.  (o, tol)."""
    n, d = q.shape
    m = k.shape[0]
    if m == 0:
        z = torch.zeros(n, v.shape[1], dtype=torch.float64)
        return z, z
    j = torch.arange(m)[None, :]
    seen = (j >= lo[:, None]) & (j < hi[:, None])
    x = (q @ k.T) * scale
    mag = torch.nan_to_num((q.abs() @ k.abs().T) * scale, 0.0, 0.0, 0.0)
    extra = 0.0
    if cap:
        x = cap * torch.tanh(x / cap)
        extra = 2.0 ** -21 * cap
    bias = slope * (j - pos[:, None]).double()
    x = torch.where(seen, x + bias, torch.full_like(x, -math.inf))
    top = x.max(1, keepdim=True).values
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.where(seen, torch.exp(x - top), torch.zeros_like(x))
    total = p.sum(1, keepdim=True)
    safe = torch.where(total > 0, total, torch.ones_like(total))
    vv = torch.nan_to_num(v, 0.0, 0.0, 0.0)
    o, a = p @ vv / safe, p @ vv.abs() / safe
    u = half_step(dtype)
    ds = d * 2.0 ** -24 * mag + 2.0 ** -22 * (1 + mag + bias.abs() + top.abs()) + extra
    pd = p * ds
    tol = u * o.abs() + (u + 2 * (m + 64) * 2.0 ** -24) * a + (pd @ vv.abs() + o.abs() * pd.sum(1, keepdim=True)) / safe
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 + m * 2.0 ** -25 * vv.abs().max() / safe
    return o, tol * (1 + 2 * u) + 1e-30


def chunk(q, keys, values, counts, scale=None, cap=0.0, slopes=None, window=0):
    """Packed chunks q [tokens, heads, dim]; keys[i], values[i] [tokens of the slot, kv_heads, dim]: (o, tol)."""
    t, h, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    o, tol = torch.zeros(t, h, d, dtype=torch.float64), torch.zeros(t, h, d, dtype=torch.float64)
    q64, at = q.detach().cpu().double(), 0
    for k, v, c in zip(keys, values, counts):
        n, g = k.shape[0], k.shape[1]
        pos = torch.arange(n - c, n)
        hi = (pos + 1).clamp_min(0)
        lo = (pos + 1 - window).clamp_min(0) if window else torch.zeros(c, dtype=torch.long)
        k64, v64 = k.double(), v.double()
        for i in range(h):
            sl = 0.0 if slopes is None else float(slopes[i])
            o[at:at + c, i], tol[at:at + c, i] = rows(q64[at:at + c, i], k64[:, i // (h // g)], v64[:, i // (h // g)], lo, hi,
                                                      pos, scale, cap, sl, q.dtype)
        at += c
    return o, tol


def frequencies(rotary, base, rule, factor=1.0, trained=0.0, low=1.0, high=32.0):
    """(radians a token of each pair, magnitude), from the definition."""
    out, mag = [], 1.0
    for i in range(rotary // 2):
        f = base ** (-2.0 * i / rotary)
        if rule == "linear":
            f /= factor
        elif rule == "base":
            f = (base * factor ** (rotary / (rotary - 2.0))) ** (-2.0 * i / rotary)
        elif rule == "bands":
            turns = trained * f / (2 * math.pi)
            if turns <= low:
                f /= factor
            elif turns < high:
                s = (turns - low) / (high - low)
                f = (1 - s) * f / factor + s * f
        elif rule == "ramp":
            def pair(turns):
                return rotary * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
            a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rotary - 1)
            s = 1 - min(1.0, max(0.0, (i - a) / (b - a if b != a else 0.001)))
            f = f / factor * (1 - s) + f * s
            mag = 0.1 * math.log(factor) + 1
        out.append(f)
    return out, mag


def turn(x, pos, freqs, layout, magnitude=1.0, norm=None, eps=1e-6):
    """Heads x [tokens, heads, dim] normed and turned at positions pos: (y, tol).  Angles in numpy's long double, whose 64
    bits hold a position's product with a frequency to 2^-33 of a radian."""
    y = x.detach().cpu().double()
    t, h, d = y.shape
    u, r = half_step(x.dtype), 2 * len(freqs)
    normed = 0.0
    if norm is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * norm.detach().cpu().double()
        normed = d / 2 + 8
    tol = y.abs() * normed * 2.0 ** -24 + (y.abs() * 4 * 2.0 ** -24 if normed else 0.0)
    if r:
        two_pi = np.longdouble("6.283185307179586476925286766559")
        turns = np.array([int(p) for p in pos], dtype=np.longdouble)[:, None] * (np.array(freqs, dtype=np.longdouble) / two_pi)
        angle = (turns - np.floor(turns)) * two_pi
        cos, sin = (torch.from_numpy(f(angle).astype(np.float64))[:, None, :] * magnitude for f in (np.cos, np.sin))
        first = torch.arange(r // 2) if layout == "half" else torch.arange(0, r, 2)
        second = first + (r // 2 if layout == "half" else 1)
        a, b = y[..., first], y[..., second]
        y, tol = y.clone(), tol.clone()
        y[..., first], y[..., second] = a * cos - b * sin, a * sin + b * cos
        off = magnitude * (a.abs() + b.abs()) * (normed + 10) * 2.0 ** -24
        tol[..., first] = off
        tol[..., second] = off
        if norm is None:
            tol[..., r:] = 0.0
    tol = tol + (u * y.abs() if norm is not None else torch.where(torch.arange(d) < r, u * y.abs(), torch.zeros_like(y)))
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    return y, tol * (1 + 2 * u)


def check(got, ref, tol, what=""):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, what
    off = (got - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((off / tol.clamp_min(1e-300)).max()), [int(x) for x in bad.nonzero()[0]])
