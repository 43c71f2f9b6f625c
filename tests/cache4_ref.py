"""The 4-bit KV cache in 64-bit arithmetic on the CPU, written from the
definitions in include/msa_cache4.h and sharing nothing with the kernels: codes
are found by searching the table of the format's values, scales by trying
exponents, attention is a dense softmax over the slots each row may attend.

A pool is a dict of uint8 arrays: k_codes, v_codes [pages, Hkv, block, d / 2],
k_scale, v_scale [pages, Hkv, block, d / 32].
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
LARGEST = 1.75 * 2.0 ** 127
GROUP = 32


def code_of(x):
    """The nearest code of each |x| <= 7, ties to the even one, with its sign bit."""
    a = np.minimum(np.abs(x), 6.0)
    hi = np.clip(np.searchsorted(E2M1, a), 0, 7)
    lo = np.maximum(hi - 1, 0)
    up, down = E2M1[hi] - a, a - E2M1[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code + 8 * np.signbit(x)).astype(np.uint8)


def exponent_of(amax):
    e = -126
    while amax > 7 * 2.0 ** e:
        e += 1
    return e


def pack(row):
    """Codes [d / 2] and scales [d / 32] of one slot's key or value."""
    if not np.isfinite(row).all() or np.abs(row).max() > LARGEST:
        return np.zeros(len(row) // 2, np.uint8), np.full(len(row) // GROUP, 255, np.uint8)
    codes, scale = [], []
    largest = exponent_of(np.abs(row).max())
    for g in row.reshape(-1, GROUP):
        e = exponent_of(np.abs(g).max()) if g.any() else largest
        c = code_of(g / 2.0 ** e)
        codes.append(c[0::2] | c[1::2] << 4)
        scale.append(e + 127)
    return np.concatenate(codes), np.array(scale, np.uint8)


def unpack(codes, scale):
    """Values [..., d]; a scale of 255 gives NaN."""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    val = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return val * np.repeat(s, GROUP, axis=-1)


def append(pool, k, v, cu, table, lens):
    block = pool["k_codes"].shape[2]
    for b, n in enumerate(lens):
        first = n - (cu[b + 1] - cu[b])
        for i in range(cu[b + 1] - cu[b]):
            page, at = table[b][(first + i) // block], (first + i) % block
            for h in range(k.shape[1]):
                for x, src in (("k", k), ("v", v)):
                    c, s = pack(src[cu[b] + i, h])
                    pool[x + "_codes"][page, h, at] = c
                    pool[x + "_scale"][page, h, at] = s


def held(pool, x, table_row, h, n):
    """Values of a sequence's n slots [n, d]."""
    block = pool["k_codes"].shape[2]
    pages = [table_row[j] for j in range(-(-n // block))]
    if not pages:
        return np.zeros((0, 2 * pool["k_codes"].shape[3]))
    val = unpack(pool[x + "_codes"][pages, h], pool[x + "_scale"][pages, h])
    return val.reshape(-1, val.shape[-1])[:n]


def attention(pool, q, table, lens, window, scale):
    """out, lse, and for error bounds: absolute weighted values (like out), the
    largest sum of |q k| scale over a row's slots, slots per row, the largest
    product of weight and value of a row, and the largest product that a small weight's rounding is taken of: 2^5 times that of the row's
    largest weight and largest value, or 2^13 times its largest product."""
    hkv = pool["k_codes"].shape[1]
    B, T, Hq, d = q.shape
    g = Hq // hkv
    out, absv = np.zeros((B, T, Hq, d)), np.zeros((B, T, Hq, d))
    lse = np.full((B, Hq, T), -np.inf)
    s1, count, top, unit = (np.zeros((B, T, Hq)) for _ in range(4))
    for b in range(B):
        n = lens[b]
        for h in range(hkv):
            k, v = held(pool, "k", table[b], h, n), held(pool, "v", table[b], h, n)
            for t in range(T):
                p = n - T + t
                if p < 0:
                    continue
                at = np.arange(max(0, p - window + 1), p + 1)
                for i in range(h * g, (h + 1) * g):
                    row = q[b, t, i]
                    s = (k[at] @ row) * scale
                    m = s.max() if np.isfinite(s).all() else 0.0
                    e = np.exp(s - m)
                    w = e / e.sum()
                    out[b, t, i] = w @ v[at]
                    absv[b, t, i] = w @ np.abs(v[at])
                    lse[b, i, t] = m + np.log(e.sum())
                    s1[b, t, i] = (np.abs(k[at]) @ np.abs(row)).max() * scale
                    count[b, t, i] = len(at)
                    size = np.abs(v[at]).max(axis=1)
                    top[b, t, i] = (w * size).max()
                    unit[b, t, i] = min(2.0 ** 5 * w.max() * size.max(), 2.0 ** 13 * top[b, t, i])
    return out, lse, absv, s1, count, top, unit
