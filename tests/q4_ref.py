"""The 4-bit cache format and decode attention over it in plain float64 numpy, written from
include/dash_cache.h, and the rounding bounds that the tests hold the kernels to."""
import numpy as np


def e4m3_round(x):
    """x >= 0 (or NaN) to the nearest e4m3 number, ties to even, at most 448."""
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.maximum(x, 2.0 ** -6)))
        step = np.exp2(np.maximum(e - 3, -9))
        return np.minimum(np.round(x / step) * step, 448.0)


def e4m3_bytes(v):
    """The bytes of e4m3 numbers >= 0 (NaN: 0x7f)."""
    table = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)])
    table[127] = np.inf   # the code of NaN
    out = np.searchsorted(table, np.where(np.isnan(v), 0, v)).astype(np.uint8)
    return np.where(np.isnan(v), 0x7f, out).astype(np.uint8)


def quantise(x, exp):
    """(codes 0..15, scales) of float64 x [..., d]."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32) * 2.0 ** -exp
    top = np.abs(g).max(-1)
    s = np.where(np.isfinite(top), e4m3_round(np.where(np.isfinite(top), top, 0) / 7), np.nan)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.clip(np.round(g / s[..., None]), -7, 7)
    q = np.where(s[..., None] > 0, q, 0)
    return (q + 8).astype(np.uint8).reshape(x.shape), s


def values(codes, scales, exp):
    g = codes.reshape(*codes.shape[:-1], codes.shape[-1] // 32, 32).astype(np.float64) - 8
    return (g * scales[..., None]).reshape(codes.shape) * 2.0 ** exp


def rows(codes, keys):
    """Bytes of rows of codes [..., d] in the pools' order."""
    b = codes[..., 0::2] | (codes[..., 1::2] << 4)
    if not keys:
        return b
    ng = codes.shape[-1] // 32
    w = b.reshape(*b.shape[:-1], ng, 4, 4)
    return np.swapaxes(w, -3, -2).reshape(b.shape)


def summary(k, qbar):
    """Eq. 4 over keys k [n, d]: (summary, base-2 maximum, weight sum, weighted sum)."""
    a = k @ qbar / np.sqrt(k.shape[1]) * np.log2(np.e)
    m = a.max()
    w = np.exp2(a - m)
    return w @ k / w.sum(), m, w.sum(), w @ k


def attend(q, k, v, bias, k_scale, v_scale):
    """q [g, d], values k, v [n, d] of the cache, bias [n] (-inf: not attended).  Returns o [g, d] and the
    bound of a kernel's error before the output's rounding: k_scale, v_scale [n, d / 32] are the keys' and values'
    scales (times 2^exp)."""
    d = q.shape[1]
    z = q @ k.T / np.sqrt(d) + bias
    zm = z.max(1, keepdims=True)
    p = np.exp(z - zm)
    l = p.sum(1, keepdims=True)
    o = p @ v / l
    # logits, per scale group of the key (its scale s times codes u - 8): fp32 sums of 32 products with codes up to
    # 15, and 8 sum(q) taken off: |terms| below 23 sum|q|, a handful (8) of truncations of 2^-23 each; the query is
    # exact to 2^-27 of its largest element, sum(q) to 2^-22
    on = np.isfinite(bias)
    qs = np.abs(q).reshape(len(q), -1, 32).sum(2)                       # [g, groups]
    unit = 2.0 ** -20 * 23 * qs + 2.0 ** -27 * 7 * 32 * np.abs(q).max(1, keepdims=True)
    dz = (unit @ k_scale[on].T).max(1) / np.sqrt(d)                     # [g]
    dz = dz + 2.0 ** -20 * (np.abs(zm[:, 0]) + np.abs(z[:, on] - zm).max(1))   # scaling, bias, exp2 argument
    # weights: 2^-11 relative for f16 (2^-25 absolute below its normals, against weights of at least 1/64 at the
    # maximum), the error of the exponent, fp32 sums of n terms
    rel = 2.0 ** -11 + 2 * dz + 2.0 ** -20
    mass = p @ np.abs(v) / l
    err = rel[:, None] * (mass + np.abs(o)) + 2.0 ** -19 * np.abs(v[on]).sum(0) / l
    # the weights times the values' scales, rounded to f16 (2^-12 relative), meet codes u of up to |u - 8| + 8, and 8
    # times the unrounded sum comes off: 2^-12 p s u <= 2^-12 p (|v| + 8 s).  Below f16's normals the product is off
    # by 2^-25, where the largest scale at weight 1 gives 1 or more (2^-9 * 2^9, or 2^(e - 7) * 2^(15 - e)): codes up
    # to 15 make 15 * 2^-25 of that scale a token.  The sums of the products with u and with 8 run in fp32 and
    # truncate by 2^-23 a step at most: two sums of up to 15 p s, in n / 16 steps shared by eight warps or more, and
    # the merges: 2^-23 (n / 128 + 32) 30 p s
    on_s = np.where(on[:, None], v_scale, 0.0)
    heavy = np.repeat(p @ on_s / l, 32, axis=1)
    err = err + 2.0 ** -12 * (mass + 8 * heavy) + 2.0 ** -21 * on.sum() * on_s.max() / l
    err = err + 2.0 ** -23 * (on.sum() / 128 + 32) * 30 * heavy
    return o, err
