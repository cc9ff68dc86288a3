"""Plain 64-bit forms of the operators of tf_qcache.h, and what may separate a
kernel's outputs from them. Written from the definitions in numpy; they share
no code with the kernels or the binding."""

import numpy as np

import spec_oracle as so

UNIT = so.UNIT


def to_bf16(x):
    """fp32 numbers rounded to bf16 (nearest, ties to even), as fp32."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    return r.view(np.float32)


def quantise(x, bits):
    """(whole numbers, factors) of rows x [..., d] of 16-bit elements (given in
    64 bits). A quotient in fp64 is a tie exactly where the true one is."""
    most = 2 ** (bits - 1) - 1
    with np.errstate(all="ignore"):
        top = np.abs(x).max(-1)
        s = to_bf16((top.astype(np.float32) / np.float32(most)).astype(np.float32)).astype(np.float64)
        bad = ~np.isfinite(x).all(-1)
        c = np.where((s > 0)[..., None], np.rint(x / np.where(s > 0, s, 1.0)[..., None]), 0.0)
        c = np.where(bad[..., None], 0.0, np.clip(c, -most, most))
    return c.astype(np.int64), np.where(bad, np.nan, s)


def pack(c, bits):
    if bits == 8:
        return (c + 128).astype(np.uint8)
    u = (c + 8).astype(np.uint8)
    return u[..., 0::2] + 16 * u[..., 1::2]


def unpack(codes, bits):
    if bits == 8:
        return codes.astype(np.float64) - 128
    return np.stack([codes % 16, codes // 16], -1).reshape(codes.shape[:-1] + (-1,)).astype(np.float64) - 8


def norm_rope(x, weight, positions, inv_freq, eps, interleaved, hadamard):
    """Rows x [b, n, h, d] in 64 bits; what bounds the error of the parts of a
    row: the result and the largest magnitudes that went into each element."""
    d = x.shape[-1]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) if eps is not None else x.copy()
    y = y * weight
    mag = np.abs(y)
    r = 2 * len(inv_freq)
    if r:
        t = positions.astype(np.float64)[..., None, None] * inv_freq
        first = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
        second = first + (1 if interleaved else r // 2)
        a, c = y[..., first], y[..., second]
        y[..., first], y[..., second] = a * np.cos(t) - c * np.sin(t), c * np.cos(t) + a * np.sin(t)
        both = np.abs(a) + np.abs(c)
        mag[..., first], mag[..., second] = both, both
    if hadamard:
        h = np.ones((1, 1))
        while len(h) < d:
            h = np.block([[h, h], [h, -h]])
        y = y @ h / np.sqrt(d)
        mag = np.broadcast_to(mag.sum(-1, keepdims=True) / np.sqrt(d), mag.shape)
    return y, mag


def norm_rope_bound(y, mag, dtype, positions, inv_freq, d):
    """fp32: the mean square of d elements is off by (d + 2) 2^-24 of itself
    (half of it in the root), rsqrt, eps and the products by some 2^-22;
    cosine and sine by 2^-22 and by what the angle is off, in fp64 (2^-52 of
    pos * freq, twice) and as a fraction of a turn in fp32 (2^-24 * 2 pi); a
    Hadamard sum by log2(d) + 1 roundings. Then one rounding to the dtype."""
    far = (np.abs(positions).max() * (np.abs(inv_freq).max() if len(inv_freq) else 0.0)) * 2.0 ** -51
    rel = (d / 2 + 1) * 2.0 ** -24 + 2.0 ** -21 + 2 * np.pi * 2.0 ** -24 + far + (np.log2(d) + 1) * 2.0 ** -24
    tiny = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134
    return rel * mag + UNIT[dtype] * (np.abs(y) + rel * mag) + tiny


def attend(q, kc, ks, vc, vs, seen, scale, bits):
    """One sequence over whole numbers kc, vc [slots, kh, d] and factors ks, vs
    [slots, kh]: so.attend's answers, and per row the largest p |s| of a
    value. A score's error: products with whole numbers that have the bias
    added (so that a sum goes through larger numbers), the factor and the
    scale, in fp32."""
    k, v = kc * ks[..., None], vc * vs[..., None]
    out, lse, mag, err = so.attend(q, k, v, seen, scale)
    n, h, d = q.shape
    group = h // kc.shape[1]
    top = np.zeros((n, h))
    bias = 2.0 ** (bits - 1)
    for i in range(n):
        cols = np.flatnonzero(seen[i])
        for x in range(h if len(cols) else 0):
            wide = (np.abs(kc[cols, x // group]) + bias) * np.abs(ks[cols, x // group])[:, None]
            err[i, x] = (2 * d + 4) * 2.0 ** -24 * abs(scale) * (wide @ np.abs(q[i, x])).max()
            if np.isfinite(lse[i, x]):
                p = np.exp(scale * (k[cols, x // group] @ q[i, x]) - lse[i, x])
                top[i, x] = (p * np.abs(vs[cols, x // group])).max()
    return out, lse, mag, err, top


def attend_bounds(out, lse, mag, err, top, dtype, slots, bits):
    """Largest |difference| allowed: a score error e moves weight and sum by
    exp(+-e) each; the weights with their factor are rounded to 11 bits
    (2^-11, or 2^-25 of the row's largest one where they are subnormal), the
    result to the dtype; the fp32 sums add slots * 2^-23 at most (sums of
    matrix instructions may be cut off instead of rounded), exp 2^-21."""
    rel = 2 * err[..., None] + 2.0 ** -11 + slots * 2.0 ** -23 + 2.0 ** -21
    tiny = slots * 2.0 ** -25 * top[..., None] * 2.0 ** (bits - 1) + (2.0 ** -25 if dtype == "fp16" else 0.0)
    return 1.1 * rel * mag + UNIT[dtype] * np.abs(out) + tiny + 1e-30, \
        1.1 * err + slots * 2.0 ** -23 + 2.0 ** -21 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))
