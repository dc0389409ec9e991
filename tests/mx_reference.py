"""Microscaled FP4 in float64 NumPy, written from the format's definition: test infrastructure.

A block is 32 consecutive values of a row.  With amax its largest magnitude, its scale is
2^e, e = floor(log2(amax)) - 2 (at least -126; 0 for a zero block); each value is the nearest
of 0, .5, 1, 1.5, 2, 3, 4, 6 times the scale, ties to the even code, larger ones to 6.  A block
with a NaN or an infinity is NaN.
"""

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode(v):
    """[..., K] -> (codes uint8 [..., K], exponents int [..., K / 32]; exponent 128 marks a NaN block)."""
    b = np.asarray(v, dtype=np.float64).reshape(*v.shape[:-1], -1, 32)
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(amax)
    e = np.where(bad | (amax == 0), 0, np.frexp(np.where(bad, 1.0, amax))[1] - 3)
    e = np.where((amax > 0) & ~bad, np.maximum(e, -126), e)
    a = np.abs(np.where(bad[..., None], 0.0, b)) / np.exp2(e.astype(np.float64))[..., None]
    # distance to every level; at equal distance the even code
    d = np.abs(a[..., None] - LEVELS)
    code = np.argmin(d * 2 + (np.arange(8) % 2) * 1e-12 * (d == d.min(-1, keepdims=True)), axis=-1).astype(np.uint8)
    code = np.where(np.signbit(b) & ~bad[..., None], code | 8, code).astype(np.uint8)
    return code.reshape(v.shape), np.where(bad, 128, e)


def decode(codes, exps):
    c = codes.reshape(*exps.shape, 32)
    scale = np.where(exps == 128, np.nan, np.exp2(np.minimum(exps, 127).astype(np.float64)))
    v = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0) * scale[..., None]
    return v.reshape(codes.shape)


def quantise(v):
    return decode(*encode(np.asarray(v, dtype=np.float64)))


def image(codes, exps):
    """The packed image of [n][rows][K]: per 16 rows and 512 values, runs of 128 values, then scales."""
    n, R, K = codes.shape
    S, G = -(-K // 128), -(-K // 512)
    out = []
    for m in range(n):
        for f in range(R // 16):
            for g in range(G):
                steps = min(4, S - 4 * g)
                scales = np.full((64, 4), 127, np.uint8)
                for s in range(steps):
                    run = np.zeros((64, 16), np.uint8)
                    for lane in range(64):
                        k0 = g * 512 + s * 128 + (lane // 16) * 32
                        if k0 < K:
                            c = codes[m, f * 16 + lane % 16, k0:k0 + 32]
                            run[lane] = c[0::2] | (c[1::2] << 4)
                            scales[lane, s] = exps[m, f * 16 + lane % 16, k0 // 32] + 127
                    out.append(run.reshape(-1))
                out.append(scales.reshape(-1))
    return np.concatenate(out).reshape(n, -1)


def silu(z):
    return z / (1.0 + np.exp(-z))


def grouped_ffn(x, perm, offsets, wg, wu, wd):
    """(rows, slack): the grouped experts on quantised x and h, weights as decoded values; slack: how far a
    row may be off where h lies so near a rounding border that its fp32 sums decide the side."""
    a = quantise(x)[perm]
    rows, slack = np.zeros((len(perm), wd.shape[1])), np.zeros((len(perm), wd.shape[1]))
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if lo == hi:
            continue
        r = a[lo:hi]
        g, u = r @ wg[e].T, r @ wu[e].T
        h = silu(g) * u
        # fp32 sums of K products: K roundings of at most 2^-24 of the partial sums' magnitudes
        c = x.shape[1] * 2.0 ** -24
        dg, du = c * (np.abs(r) @ np.abs(wg[e]).T), c * (np.abs(r) @ np.abs(wu[e]).T)
        dh = 1.1 * dg * np.abs(u) + np.abs(silu(g)) * du + 2.0 ** -20 * np.abs(h)
        rows[lo:hi] = quantise(h) @ wd[e].T
        slack[lo:hi] = np.abs(quantise(h + dh) - quantise(h - dh)) @ np.abs(wd[e]).T
    return rows, slack
