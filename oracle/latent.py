"""Float64 restatement of rotary positions and of latent attention, with the
bounds that roundings set on a kernel's results.

Nothing here uses the library: angles come from float64 cos / sin, attention
from explicit sums over the rows that a block table names.
"""
import numpy as np

F32 = 2.0 ** -24        # half a float32 step, relative
BF16 = 2.0 ** -8        # half a bf16 step, relative


def frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_context=None,
                fast=32.0, slow=1.0):
    """(radians a position of every pair, magnitude)."""
    f = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling == "linear":
        return np.array(f) / factor, 1.0
    if scaling == "ntk":
        stretched = base * factor ** (rot_dim / (rot_dim - 2.0))
        return np.array([stretched ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]), 1.0
    if scaling == "by_parts":
        out = []
        for x in f:
            turns = original_context * x / (2 * np.pi)
            keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
            out.append(keep * x + (1 - keep) * x / factor)
        return np.array(out), 0.1 * np.log(factor) + 1.0
    return np.array(f), 1.0


def rotate(x, positions, freqs, layout, magnitude=1.0):
    """x [T][H][D] float64, its first 2 * len(freqs) elements a head rotated; and what a
    float32 computation of each element may be off by.

    The angle reaches the kernel as a float32 number of half turns in [-1, 1):
    off by at most pi * 2^-24 rad < 2^-22.  Sine and cosine are off by at most
    2^-23 more, the magnitude's product, the two products and the sum round by
    2^-24 each: under 2^-20 (|x| + |y|) m in all.
    """
    x = np.asarray(x, np.float64)
    y, off = x.copy(), np.zeros_like(x)
    n = len(freqs)
    a = np.asarray(positions, np.float64)[:, None] * np.asarray(freqs)[None]
    c, s = np.cos(a)[:, None] * magnitude, np.sin(a)[:, None] * magnitude
    if layout == "half":
        u, w = np.arange(n), np.arange(n) + n
    else:
        u, w = 2 * np.arange(n), 2 * np.arange(n) + 1
    y[..., u] = x[..., u] * c - x[..., w] * s
    y[..., w] = x[..., u] * s + x[..., w] * c
    off[..., u] = off[..., w] = (np.abs(x[..., u]) + np.abs(x[..., w])) * magnitude * 2.0 ** -20
    return y, off


def gather(rows, table, n):
    """Rows of positions 0 .. n - 1 of one sequence: rows [N][B_p][W], table of block ids."""
    bp = rows.shape[1]
    return np.stack([rows[int(table[j // bp]), j % bp] for j in range(n)]) if n else \
        np.zeros((0, rows.shape[2]))


def attend(q, keys, scale, latent_dim, seen):
    """(out, bound) of q [R][W] against keys [n][W]; row r sees its first seen[r] keys.

    bound: what a kernel with float32 sums, probabilities rounded to bf16 (and
    their sum taken of the rounded values) and one rounding of the output may be
    off by.  With w the weights, o the output and A = sum_j w_j |v_j - o|:
      - relative errors e_j of the probabilities move the output by at most
        max|e| / (1 - max|e|) A: 2^-8 for the rounding and, for a score off by d,
        e^d - 1; a float32 dot product of W terms is off by at most
        W 2^-23 sum |q k| (sums that truncate included), the base-2 exponent
        and its argument by 2^-20 (1 + |s - m|);
      - the float32 sum of n terms is off by at most n 2^-23 sum_j w_j |v_j|;
      - the output's rounding by 2^-8 of its value.
    """
    q, keys = np.asarray(q, np.float64), np.asarray(keys, np.float64)
    out = np.zeros((len(q), latent_dim))
    bound = np.zeros((len(q), latent_dim))
    for r in range(len(q)):
        n = int(seen[r])
        if n <= 0:
            continue
        k = keys[:n]
        s = scale * (k @ q[r])
        top = s.max()
        w = np.exp(s - top)
        w /= w.sum()
        v = k[:, :latent_dim]
        o = w @ v
        d = abs(scale) * k.shape[1] * 2.0 ** -23 * (np.abs(k) @ np.abs(q[r])) \
            + 2.0 ** -20 * (1 + np.abs(s - top))
        e = np.expm1(d) + BF16
        e = np.minimum(e, 0.5)
        spread = (w * e / (1 - e.max())) @ np.abs(v - o)
        b = spread + n * 2.0 ** -23 * (w @ np.abs(v))
        out[r], bound[r] = o, b + BF16 * (np.abs(o) + b) + 2.0 ** -133
    return out, bound
