"""The window cache and core attention in 64 bits, from their definitions (include/lsa.h), with the
bounds that the GPU tests hold the kernels to.

A rounding to a type is off by at most half a step, `eps / 2` relative (bf16 2^-8, f16 2^-11, fp32
2^-24, E4M3 2^-4, and half the least subnormal step absolute).
"""
import math

import torch

E4M3 = torch.float8_e4m3fn


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------------------------------ append

def rotate(x, pos, inv_freq, interleaved):
    """x [H][D] double at position pos; returns (y, bound factor): |x1| + |x2| of each element's pair."""
    y, mag = x.clone(), torch.zeros_like(x)
    if inv_freq is None:
        return y, mag
    R = 2 * inv_freq.numel()
    a = pos * inv_freq.double()
    c, s = torch.cos(a), torch.sin(a)
    one, two = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    x1, x2 = x[:, one], x[:, two]
    y[:, one] = x1 * c - x2 * s
    y[:, two] = x2 * c + x1 * s
    mag[:, one] = mag[:, two] = x1.abs() + x2.abs()
    return y, mag


# cos and sin of an angle reduced in fp64 and rounded to fp32 turns (2^-25 of a half turn, times pi:
# 1e-7), from a function within 2 ulp (2.4e-7), then two products and a sum in fp32 (3 * 2^-24 = 1.8e-7)
ROTATION = 6e-7


def pow2_scale(amax):
    """Least 2^e >= 2^-64 with amax <= 448 * 2^e."""
    if amax <= 448 * 2.0 ** -64:
        return 2.0 ** -64
    e = math.ceil(math.log2(amax / 448))
    while amax > 448 * 2.0 ** e:
        e += 1
    while amax <= 448 * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** e


def e4m3_bound(x, scale):
    """How far a value's E4M3 code times its scale may be from it."""
    return torch.maximum(x.abs() * 2.0 ** -4, torch.full_like(x, scale * 2.0 ** -10))


# --------------------------------------------------------------------------------------- attention

def visible(pos, end, window, n_sink):
    """Key positions that a query at pos sees, of a cache of `end` tokens."""
    return [j for j in range(min(pos + 1, end)) if window == 0 or j > pos - window or j < n_sink]


def attend(q, K, V, scale):
    """One query head q [D] over keys K, V [n][D] (double): out, lse, and what bounds their error:
    A = sum_j w_j |v_j| and the largest sum_i |q_i k_i| * scale."""
    if K.shape[0] == 0:
        z = torch.zeros(q.shape[0], dtype=torch.float64)
        return z, -math.inf, z.clone(), 0.0
    x = (K @ q) * scale
    w = torch.softmax(x, 0)
    return w @ V, float(torch.logsumexp(x, 0)), w @ V.abs(), float((K.abs() @ q.abs()).max()) * scale


def attend_bounds(out, A, mag, n, D, q_dtype, p_dtype):
    """(bound on |out|'s error, bound on |lse|'s error).

    A score is a sum of D products in fp32 scaled twice: off by delta = (D + 3) 2^-24 sum|q k| scale.  The
    running maximum and the exponent in base 2 add three roundings of numbers up to 1.5 |score|: 5 * 2^-24
    mag.  exp2 is within 2 ulp (2^-22).  A weight is off by delta relative, in the sum of n weights as
    well (n fp32 additions at most, n 2^-24), the value product sums n terms; probabilities are rounded to
    p_dtype once (None: not at all), the result once to q_dtype."""
    u = 2.0 ** -24
    delta = (D + 8) * u * mag + 4 * u
    rel = 2 * delta + 3 * n * u + (half_step(p_dtype) if p_dtype is not None else 0.0) + 8 * u
    return rel * A + half_step(q_dtype) * (out.abs() + rel * A) + 1e-30, delta + n * u + 8 * u * (1 + mag)
