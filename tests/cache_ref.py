"""The 8-bit KV cache in 64-bit arithmetic on the CPU, written from the
definitions in include/msa_cache.h and sharing nothing with the kernels: the
e4m3 rounding searches the table of the format's values, attention is a dense
softmax over the slots each row may attend, selection and eviction are sorts.

A pool is a dict of float64 arrays: k_codes, v_codes [pages, Hkv, block, d]
(the values of the codes), k_scale, v_scale [pages, Hkv], k_mean [pages, Hkv,
d].
"""
from __future__ import annotations

import math

import numpy as np

# The 127 finite magnitudes of e4m3 (7 exponent/mantissa bits, bias 7).
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)
                 if (e, m) != (15, 7)])


def round_e4m3(x):
    """Nearest value of the format, ties to the even code, for |x| <= 448."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3, a), 0, len(E4M3) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.copysign(E4M3[code], x)


def scale_of_block(val):
    if not np.isfinite(val).all():
        return math.nan
    amax = float(np.abs(val).max()) if val.size else 0.0
    if amax == 0.0:
        return 0.0
    e = math.frexp(amax)[1] - 12
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -126)


def codes_of(val, s):
    if math.isnan(s) or s == 0.0:
        return np.zeros_like(val)
    return round_e4m3(val / s)


def round_bf16(x):
    """Nearest bf16, ties to even: 8 significant bits, steps of 2^-133 at the least."""
    x = np.asarray(x, dtype=np.float64)
    step = np.maximum(np.frexp(x)[1] - 8, -133)
    return np.ldexp(np.rint(np.ldexp(x, -step)), step)


def write_block(pool, x, page, h, val, least, block):
    s = scale_of_block(val)
    s = math.nan if math.isnan(s) or math.isnan(least) else max(s, least)
    c = codes_of(val, s)
    pool[x + "_codes"][page, h, :len(val)] = c
    pool[x + "_scale"][page, h] = s
    if x == "k" and len(val) == block:
        pool["k_mean"][page, h] = round_bf16(c.mean(axis=0) * s)


def append(pool, k, v, cu, table, lens):
    block = pool["k_codes"].shape[2]
    for b, n in enumerate(lens):
        new = cu[b + 1] - cu[b]
        first = n - new
        for j in range(first // block, -(-n // block) if new else 0):
            lo, hi = j * block, min(n, (j + 1) * block)
            old = max(0, first - lo)
            page = table[b][j]
            for h in range(k.shape[1]):
                for x, src in (("k", k), ("v", v)):
                    s = pool[x + "_scale"][page, h] if old else 0.0
                    before = pool[x + "_codes"][page, h, :old] * s if old else np.zeros((0, k.shape[2]))
                    fresh = src[cu[b] + lo + old - first:cu[b] + hi - first, h]
                    write_block(pool, x, page, h, np.concatenate([before, fresh]), s, block)


def held(pool, x, table_row, h, n):
    """Values of a sequence's n slots [n, d]."""
    block, d = pool["k_codes"].shape[2:]
    pages = [table_row[j] for j in range(-(-n // block))]
    val = pool[x + "_codes"][pages, h] * pool[x + "_scale"][pages, h][:, None, None]
    return val.reshape(-1, d)[:n]


def select(pool, q, table, lens, window, top_k):
    """Chosen blocks [batch][n_q][Hkv] -> ascending list."""
    hkv, block = pool["k_codes"].shape[1:3]
    B, T, Hq, _ = q.shape
    g = Hq // hkv
    out = []
    for b in range(B):
        rows = []
        for t in range(T):
            p = lens[b] - T + t
            n = (p - window + 1) // block if p >= window else 0
            per = []
            for h in range(hkv):
                mean = pool["k_mean"][[table[b][j] for j in range(n)], h] if n else np.zeros((0, q.shape[3]))
                s = mean @ q[b, t, h * g:(h + 1) * g].sum(axis=0)
                s = np.where(np.isnan(s), -np.inf, s)
                per.append(sorted(np.lexsort((np.arange(n), -s))[:top_k].tolist()))
            rows.append(per)
        out.append(rows)
    return out


def attention(pool, q, table, lens, window, scale, sel=None):
    """out, lse, and for error bounds: absolute weighted values (like out),
    the largest sum of |q k| scale over a row's slots, slots per row, and the
    weights [batch, Hkv, max slots]."""
    hkv, block = pool["k_codes"].shape[1:3]
    B, T, Hq, d = q.shape
    g = Hq // hkv
    out, absv = np.zeros((B, T, Hq, d)), np.zeros((B, T, Hq, d))
    lse = np.full((B, Hq, T), -np.inf)
    s1 = np.zeros((B, T, Hq))
    count = np.zeros((B, T, Hq))
    weights = np.zeros((B, hkv, len(table[0]) * block))
    for b in range(B):
        n = lens[b]
        for h in range(hkv):
            if n == 0:
                continue
            k, v = held(pool, "k", table[b], h, n), held(pool, "v", table[b], h, n)
            for t in range(T):
                p = n - T + t
                if p < 0:
                    continue
                at = np.arange(max(0, p - window + 1), p + 1)
                if sel is not None:
                    far = [np.arange(l * block, (l + 1) * block) for l in sel[b][t][h]]
                    at = np.concatenate(far + [at]).astype(np.int64)
                for i in range(h * g, (h + 1) * g):
                    row = q[b, t, i]
                    s = (k[at] @ row) * scale
                    m = s.max() if np.isfinite(s).any() else 0.0
                    e = np.exp(s - m)
                    w = e / e.sum()
                    out[b, t, i] = w @ v[at]
                    absv[b, t, i] = w @ np.abs(v[at])
                    lse[b, i, t] = m + np.log(e.sum())
                    s1[b, t, i] = (np.abs(k[at]) @ np.abs(row)).max() * scale
                    count[b, t, i] = len(at)
                    weights[b, h, at] += w
    return out, lse, absv, s1, count, weights


def evict(pool, table, lens, weights, dst, budget, recent):
    """new_lens, kept [batch][Hkv] lists, kept weights likewise; writes the pool."""
    hkv, block = pool["k_codes"].shape[1:3]
    new_lens, kept, kept_w = [], [], []
    for b, n in enumerate(lens):
        K = min(n, budget)
        r = min(K, recent)
        new_lens.append(K)
        kept.append([])
        kept_w.append([])
        for h in range(hkv):
            w = weights[b, h, :n - r]
            best = np.lexsort((np.arange(n - r), -np.where(np.isnan(w), np.inf, w)))[:K - r]
            keep = np.concatenate([np.sort(best), np.arange(n - r, n)]).astype(np.int64)
            kept[b].append(keep)
            kept_w[b].append(weights[b, h, keep])
            if K == 0:
                continue
            for x in ("k", "v"):
                val = held(pool, x, table[b], h, n)[keep]
                for j in range(-(-K // block)):
                    write_block(pool, x, dst[b][j], h, val[j * block:(j + 1) * block], 0.0, block)
    return new_lens, kept, kept_w
