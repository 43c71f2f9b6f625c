"""The 8-bit KV cache on the GPU against its 64-bit reference.

What is held in 8 bits, scales, block means, selections and evictions must be
equal to the reference's; attention is held to bounds derived from the
arithmetic (see ``bounds``)."""
import math

import numpy as np
import pytest
import torch

import long_context_sparse_landmark_gb300 as msa
from tests import cache_ref as R
from tests.gpu_helpers import binding, check_guards, gempty, gfull

pytestmark = pytest.mark.gpu

DEV = "cuda"
F8 = torch.float8_e4m3fn


def new_cache(pages, hkv, d, block, fill=0x7F):
    """A pool in guarded memory, every byte of it `fill` (0x7f: NaN codes)."""
    codes = [gfull((pages, hkv, block, d), fill, torch.uint8) for _ in range(2)]
    scale = [gfull((pages, hkv), float("nan")) for _ in range(2)]
    return msa.KVCache(codes[0].view(F8), codes[1].view(F8), scale[0], scale[1],
                       gfull((pages, hkv, d), float("nan"), torch.bfloat16))


def pool_of(cache):
    """The cache as the reference's pool."""
    return {"k_codes": cache.k_codes.float().cpu().double().numpy(),
            "v_codes": cache.v_codes.float().cpu().double().numpy(),
            "k_scale": cache.k_scale.cpu().double().numpy(),
            "v_scale": cache.v_scale.cpu().double().numpy(),
            "k_mean": cache.k_mean.float().cpu().double().numpy()}


def tables(lens, block, rng, extra=0, width=0):
    """Distinct pages in random order, -1 where a row has none; the pages left over."""
    need = [-(-n // block) for n in lens]
    pages = rng.permutation(sum(need) + extra)
    most = max(1, width, max(need))
    t = np.full((len(lens), most), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = pages[at:at + k]
        at += k
    return t, pages[at:]


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


def same_pool(cache, pool):
    got = pool_of(cache)
    for name, want in pool.items():
        np.testing.assert_array_equal(got[name], want, err_msg=name)


def filled(lens, hkv, d, block, seed, extra=0, width=0, kscale=1.0, dtype=torch.bfloat16):
    """A cache that holds random tokens, through cache_append, and its reference."""
    rng = np.random.default_rng(seed)
    t, free = tables(lens, block, rng, extra + 1, width)
    cache = new_cache(int(t.max(initial=0)) + extra + 2 + len(free), hkv, d, block)
    total = sum(lens)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    k = (torch.randn((total, hkv, d), generator=gen, device=DEV) * kscale).to(dtype)
    v = torch.randn((total, hkv, d), generator=gen, device=DEV).to(dtype)
    cu = np.concatenate([[0], np.cumsum(lens)])
    msa.cache_append(cache, k, v, i32(cu), i32(t), i32(lens), max(lens))
    torch.cuda.synchronize()
    assert binding().device_status() == 0
    return cache, pool_of(cache), t, free


def bounds(ref, d, bf16_in, out_dtype):
    """How far out and lse may be off.

    Scores: a sum of d exact products; each fp32 step rounds (tensor cores:
    truncates) by at most 2^-23 of the absolute sum, the scalings by four half
    steps more: ds = (d + 4) 2^-23 S1, S1 the largest sum of |q k| scale.
    Weights: relative error 2 ds, two exponentials (2 ulp each), the sums'
    steps (one per slot at most, 2^-23 each), and 2^-11 for the rounding to
    halves with bf16 queries, whose subnormals (below 2^-28 of the largest)
    add 2^-39 of the largest |value| a slot.  Output: half a step of its type."""
    out, lse, absv, s1, count, _ = ref
    ds = (d + 4) * 2.0 ** -23 * s1
    rel = 2 * ds + 2.0 ** -20 + count * 2.0 ** -23 + (2.0 ** -11 if bf16_in else 0.0)
    half = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -24
    tol_o = absv * rel[..., None] * (1 + half) + np.abs(out) * half
    tol_l = (ds + 2.0 ** -20 + count * 2.0 ** -24).transpose(0, 2, 1)
    return tol_o, tol_l + np.abs(np.where(np.isfinite(lse), lse, 0.0)) * 2.0 ** -22


def check_attention(out, lse, ref, d, bf16_in, vmax):
    tol_o, tol_l = bounds(ref, d, bf16_in, out.dtype)
    if bf16_in:
        tol_o = tol_o + ref[4][..., None] * 2.0 ** -39 * vmax
    o, l = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    empty = np.isneginf(ref[1])
    assert np.array_equal(np.isneginf(l), empty)
    assert not o[empty.transpose(0, 2, 1)].any()
    err = np.abs(o - ref[0])
    assert np.isfinite(o).all() and (err <= tol_o).all(), (
        f"out: worst {np.nanmax(err / np.maximum(tol_o, 1e-300)):.3g} of the bound")
    fin = ~empty
    errl = np.abs(l - np.where(fin, ref[1], 0))[fin]
    assert (errl <= tol_l[fin]).all(), f"lse: worst {np.max(errl / tol_l[fin]):.3g} of the bound"


# -- append ------------------------------------------------------------------

@pytest.mark.parametrize("hkv,d,block,dtype,before,new", [
    (1, 64, 32, "bf16", [0], [1]),
    (1, 128, 64, "bf16", [63], [1]),              # completes a block
    (2, 128, 64, "f32", [64], [1]),               # starts one
    (3, 64, 32, "f32", [5, 0, 31], [40, 0, 1]),   # one sequence gets nothing
    (2, 128, 128, "bf16", [100, 7, 0], [300, 1, 128]),
    (1, 128, 256, "f32", [255, 0], [2, 513]),
    (8, 128, 64, "bf16", [1000, 999], [129, 64]),
])
def test_append_equals_the_definition(hkv, d, block, dtype, before, new):
    rng = np.random.default_rng(hkv * 1000 + block)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    lens = [a + b for a, b in zip(before, new)]
    t, _ = tables(lens, block, rng, 2)
    cache = new_cache(int(t.max()) + 3, hkv, d, block)
    pool = pool_of(cache)
    at = [0] * len(lens)
    for part in (before, new):
        if not sum(part):
            continue
        at = [a + b for a, b in zip(at, part)]
        cu = np.concatenate([[0], np.cumsum(part)])
        k = torch.as_tensor(rng.normal(size=(sum(part), hkv, d)) * np.exp(rng.normal(size=(sum(part), 1, 1))),
                            device=DEV).to(dt)
        v = torch.as_tensor(rng.normal(size=(sum(part), hkv, d)) * 1e-3, device=DEV).to(dt)
        msa.cache_append(cache, k, v, i32(cu), i32(t), i32(at), max(part))
        R.append(pool, k.double().cpu().numpy(), v.double().cpu().numpy(), cu, t, at)
        same_pool(cache, pool)   # slots past the lengths keep their NaN codes
    msa.cache_append(cache, k, v, i32(cu), i32(t), i32(at), max(part) + 0)
    same_pool(cache, pool)       # the same tokens again: nothing changes
    assert binding().device_status() == 0


def test_append_one_by_one_with_growing_scales():
    """Each token larger than the last: the block's scale grows and its old
    codes are rounded again, down to subnormals and zeros."""
    rng = np.random.default_rng(5)
    cache = new_cache(3, 2, 64, 32)
    pool = pool_of(cache)
    k = (rng.normal(size=(40, 2, 64)) * 1.7 ** np.arange(40)[:, None, None]).astype(np.float32)
    v = k[::-1].copy()
    kt, vt = torch.as_tensor(k, device=DEV), torch.as_tensor(v, device=DEV)
    t = np.array([[2, 0]], dtype=np.int32)
    for i in range(40):
        msa.cache_append(cache, kt[i:i + 1], vt[i:i + 1], i32([0, 1]), i32(t), i32([i + 1]), 1)
        R.append(pool, k[i:i + 1].astype(np.float64), v[i:i + 1].astype(np.float64), [0, 1], t, [i + 1])
    same_pool(cache, pool)


@pytest.mark.parametrize("special", [0.0, 448.0, 448.0 * 2 ** 5 + 64, 2.0 ** -133, 3.3e38, math.nan,
                                     math.inf, -math.inf])
def test_append_of_special_values(special):
    rng = np.random.default_rng(6)
    cache = new_cache(4, 1, 64, 32)
    pool = pool_of(cache)
    k = rng.normal(size=(70, 1, 64)).astype(np.float32)
    k[32:64] = 0.0
    k[40, 0, 3] = special
    t = np.array([[3, 1, 0]], dtype=np.int32)
    kt = torch.as_tensor(k, device=DEV)
    msa.cache_append(cache, kt, kt, i32([0, 50]), i32(t), i32([50]), 70)
    R.append(pool, k[:50].astype(np.float64), k[:50].astype(np.float64), [0, 50], t, [50])
    same_pool(cache, pool)
    # the rest joins the block that holds the special value
    msa.cache_append(cache, kt[50:], kt[50:], i32([0, 20]), i32(t), i32([70]), 20)
    R.append(pool, k[50:].astype(np.float64), k[50:].astype(np.float64), [0, 20], t, [70])
    same_pool(cache, pool)


def test_append_of_nothing_and_padded_rows():
    cache = new_cache(2, 1, 64, 32)
    pool = pool_of(cache)
    k = torch.randn((4, 1, 64), device=DEV)
    msa.cache_append(cache, k[:0], k[:0], i32([0, 0]), i32([[0]]), i32([0]), 0)
    msa.cache_append(cache, k, k, i32([0, 0, 0]), i32([[0], [-1]]), i32([0, 0]), 4)
    same_pool(cache, pool)
    assert binding().device_status() == 0


# -- attention ---------------------------------------------------------------

ATTN = [
    # lens, n_q, hkv, group, d, block, window
    ([1], 1, 1, 1, 64, 32, None),
    ([1, 0, 2], 1, 2, 4, 128, 64, None),            # a padded sequence
    ([3], 5, 1, 2, 64, 32, None),                   # more query tokens than slots: empty rows
    ([33, 31, 64], 1, 1, 8, 128, 32, None),
    ([700, 65, 300, 1], 1, 2, 8, 128, 64, None),
    ([1001, 517], 2, 3, 5, 128, 64, None),          # 10 rows: two tiles of 8 or one of 16
    ([257, 900], 4, 2, 8, 128, 128, None),          # 32 rows
    ([2500], 1, 4, 16, 64, 256, None),
    ([2047], 1, 1, 4, 64, 32, None),
    ([900, 130, 40], 1, 2, 8, 128, 64, 1),
    ([900, 130, 40], 3, 2, 4, 128, 64, 100),        # window edges inside chunks
    ([1300, 64], 8, 1, 2, 64, 64, 33),
    ([600], 1, 2, 24, 128, 64, None),               # more heads than a tile
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,n_q,hkv,group,d,block,window", ATTN)
def test_attention(lens, n_q, hkv, group, d, block, window, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cache, pool, t, _ = filled(lens, hkv, d, block, seed=sum(lens) + d, width=max(lens) // block + 3)
    q = torch.randn((len(lens), n_q, hkv * group, d), device=DEV,
                    generator=torch.Generator(device=DEV).manual_seed(1)).to(dt)
    w0 = torch.rand((len(lens), hkv, t.shape[1] * block + 8), device=DEV) * 0.01
    w = gempty(w0.shape)
    w.copy_(w0)
    ref = R.attention(pool, q.double().cpu().numpy(), t, lens, window or 1 << 30, 1 / math.sqrt(d))
    vmax = max(np.abs(R.held(pool, "v", t[b], h, n)).max(initial=0) for b, n in enumerate(lens) for h in range(hkv))
    for out_dtype in (dt, torch.float32 if dt == torch.bfloat16 else torch.bfloat16):
        out, lse = msa.cache_attention(q, cache, i32(t), i32(lens), window=window, out_dtype=out_dtype,
                                       weights=w if out_dtype == dt else None)
        torch.cuda.synchronize()
        assert binding().device_status() == 0
        check_attention(out, lse, ref, d, dtype == "bf16", vmax)
    # weights: a sum of probabilities of relative error 2 ds + 2^-20 + n 2^-23 each
    ds = (d + 4) * 2.0 ** -23 * ref[3].max(initial=0)
    rows = n_q * group
    add = np.zeros(w0.shape)
    add[..., :t.shape[1] * block] = ref[5]
    want = w0.double().cpu().numpy() + add
    tol = add * (2 * ds + 2.0 ** -20 + max(lens) * 2.0 ** -23 + rows * 2.0 ** -24) + want * 2.0 ** -24
    err = np.abs(w.double().cpu().numpy() - want)
    assert (err <= tol + 1e-30).all(), np.max(err / (tol + 1e-30))
    check_guards()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_long_sequences_is_cut_and_joined(dtype):
    """Sequences longer than a CTA's share beside short ones."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    lens = [9000, 17, 0, 4100, 64]
    cache, pool, t, _ = filled(lens, 2, 128, 64, seed=9)
    q = torch.randn((5, 1, 8, 128), device=DEV).to(dt)
    ref = R.attention(pool, q.double().cpu().numpy(), t, lens, 1 << 30, 1 / math.sqrt(128))
    out, lse = msa.cache_attention(q, cache, i32(t), i32(lens))
    check_attention(out, lse, ref, 128, dtype == "bf16", 6.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_slot_outweighs_a_long_tail(dtype):
    """A sink that takes most of the weight and thousands of slots at 2^-20
    of it that share the rest: the small weights keep their precision."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n, d = 6000, 128
    rng = np.random.default_rng(10)
    k = np.zeros((n, 1, d), dtype=np.float32)
    q = np.zeros((1, 1, 8, d), dtype=np.float32)
    q[..., 0] = 1.0
    k[:, 0, 0] = 1.0
    k[0, 0, 0] = 1.0 + 14.0 * math.sqrt(d)
    v = rng.normal(size=(n, 1, d)).astype(np.float32) + 1.0
    v[0] = 0.01
    t, _ = tables([n], 64, rng, 1)
    cache = new_cache(int(t.max()) + 2, 1, d, 64)
    kt, vt = torch.as_tensor(k, device=DEV), torch.as_tensor(v, device=DEV)
    msa.cache_append(cache, kt, vt, i32([0, n]), i32(t), i32([n]), n)
    pool = pool_of(cache)
    ref = R.attention(pool, q.astype(np.float64), t, [n], 1 << 30, 1 / math.sqrt(d))
    out, lse = msa.cache_attention(torch.as_tensor(q, device=DEV).to(dt), cache, i32(t), i32([n]),
                                   out_dtype=torch.float32)
    check_attention(out, lse, ref, d, dtype == "bf16", 6.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("big,small", [(1e30, 1e-30), (1e4, 1e-3)])
def test_values_of_very_different_blocks(dtype, big, small):
    """Neighbouring blocks whose values (and scales) are apart by up to 2^200."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    lens, d = [192], 64
    rng = np.random.default_rng(11)
    k = rng.normal(size=(192, 1, d)).astype(np.float32)
    v = rng.uniform(1, 2, size=(192, 1, d)).astype(np.float32)
    v[:64] *= small
    v[64:128] = 0.0
    v[128:] *= big
    cache = new_cache(4, 1, d, 64)
    t = np.array([[2, 0, 3]], dtype=np.int32)
    kt, vt = torch.as_tensor(k, device=DEV), torch.as_tensor(v, device=DEV)
    msa.cache_append(cache, kt, vt, i32([0, 192]), i32(t), i32([192]), 192)
    pool = pool_of(cache)
    q = torch.randn((1, 1, 4, d), device=DEV).to(dt)
    for n in (64, 128, 192):   # only small values, with zeros, all
        ref = R.attention(pool, q.double().cpu().numpy(), t, [n], 1 << 30, 0.125)
        out, lse = msa.cache_attention(q, cache, i32(t), i32([n]), out_dtype=torch.float32)
        check_attention(out, lse, ref, d, dtype == "bf16", big * 2 if n == 192 else small * 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_poisoned_blocks_reach_only_rows_that_attend_them(dtype):
    """A NaN key or value makes the rows that attend its block NaN, and no
    other: neither rows of other windows nor other sequences and heads."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    lens, d, block = [130, 130], 64, 32
    rng = np.random.default_rng(12)
    k, v = rng.normal(size=(2, 260, 2, d)).astype(np.float32)
    k[20, 0, 1] = np.nan       # sequence 0, head 0, block 0
    v[129, 1, 0] = np.inf      # sequence 0, head 1, block 4: the last two slots
    t, _ = tables(lens, block, rng, 1)
    cache = new_cache(int(t.max()) + 2, 2, d, block)
    kt, vt = torch.as_tensor(k, device=DEV), torch.as_tensor(v, device=DEV)
    msa.cache_append(cache, kt, vt, i32([0, 130, 260]), i32(t), i32(lens), 130)
    pool = pool_of(cache)
    q = torch.randn((2, 4, 4, d), device=DEV).to(dt)
    for window, nan00 in ((None, True), (70, False)):
        out, lse = msa.cache_attention(q, cache, i32(t), i32(lens), window=window)
        nan = np.isnan(out.float().cpu().numpy()).all(axis=3)
        some = np.isnan(out.float().cpu().numpy()).any(axis=3)
        want = np.zeros((2, 4, 4), dtype=bool)
        want[0, :, :2] = nan00
        want[0, 2:, 2:] = True      # positions 128 and 129
        assert np.array_equal(nan, want) and np.array_equal(some, want)
        for x in ("k", "v"):       # the reference without the poison
            pool[x + "_scale"] = np.nan_to_num(pool[x + "_scale"], nan=1.0)
        ref = R.attention(pool, q.double().cpu().numpy(), t, lens, window or 1 << 30, 0.125)
        tol = bounds(ref, d, dtype == "bf16", out.dtype)[0] + 1e-9
        ok = np.abs(out.double().cpu().numpy() - ref[0])[~want] <= tol[~want]
        assert ok.all()


def test_queries_of_any_size():
    """Rows of very large, very small and zero queries beside each other."""
    lens, d = [300], 128
    cache, pool, t, _ = filled(lens, 1, d, 64, seed=13, kscale=1e-3)
    q = torch.randn((1, 1, 6, d), device=DEV)
    q *= torch.tensor([1e4, 1e-4, 1e-36, 0.0, 1e2, 1.0], device=DEV)[None, None, :, None]
    for dt in (torch.bfloat16, torch.float32):
        ref = R.attention(pool, q.to(dt).double().cpu().numpy(), t, lens, 1 << 30, 0.1)
        out, lse = msa.cache_attention(q.to(dt), cache, i32(t), i32(lens), scale=0.1)
        check_attention(out, lse, ref, d, dt == torch.bfloat16, 6.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e4, 1e8, 1e12])
def test_scores_far_beyond_an_exponential(dtype, size):
    """Scores whose rounding is many units: the largest takes all, finitely."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    lens, d = [500], 64
    cache, pool, t, _ = filled(lens, 2, d, 64, seed=14)
    q = torch.randn((1, 1, 8, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)) * size
    q = q.to(dt)
    ref = R.attention(pool, q.double().cpu().numpy(), t, lens, 1 << 30, 0.125)
    out, lse = msa.cache_attention(q, cache, i32(t), i32(lens))
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    # one slot leads every row by more than the scores' rounding
    assert np.abs(out.double().cpu().numpy() - ref[0]).max() <= np.abs(ref[0]).max() * 2.0 ** -7
    assert np.abs(lse.double().cpu().numpy() / ref[1] - 1).max() <= (d + 4) * 2.0 ** -22 * (ref[3].max() / np.abs(ref[1]).min())


# -- selection ---------------------------------------------------------------

def selected(sel, cnt):
    sel, cnt = sel.cpu().numpy(), cnt.cpu().numpy()
    out = [[[sel[b, t, h, :cnt[b, t, h]].tolist() for h in range(sel.shape[2])] for t in range(sel.shape[1])]
           for b in range(sel.shape[0])]
    for idx in np.ndindex(*cnt.shape):
        assert (sel[idx][cnt[idx]:] == -1).all()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,n_q,hkv,group,d,block,window,top_k", [
    ([1], 1, 1, 1, 64, 32, 1, 1),
    ([33, 0, 32], 1, 1, 4, 64, 32, 1, 1),
    ([700, 65, 301], 1, 2, 8, 128, 64, 100, 3),
    ([1001, 517], 3, 3, 5, 128, 32, 33, 7),
    ([3000], 6, 2, 8, 128, 128, 512, 4),
    ([2000, 1000], 2, 1, 2, 64, 256, 1, 100),       # fewer candidates than top_k
    ([900], 1, 2, 8, 64, 64, 5000, 4),              # no candidate
])
def test_select_and_attend(lens, n_q, hkv, group, d, block, window, top_k, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cache, pool, t, _ = filled(lens, hkv, d, block, seed=sum(lens) + top_k)
    q = torch.randn((len(lens), n_q, hkv * group, d), device=DEV,
                    generator=torch.Generator(device=DEV).manual_seed(2)).to(dt)
    qn = q.double().cpu().numpy()
    sel, cnt = msa.cache_block_select(q, cache, i32(t), i32(lens), window, top_k)
    want = R.select(pool, qn, t, lens, window, top_k)
    assert selected(sel, cnt) == want
    ref = R.attention(pool, qn, t, lens, window, 1 / math.sqrt(d), sel=want)
    out, lse = msa.cache_topk_attention(q, cache, i32(t), i32(lens), window, top_k)
    torch.cuda.synchronize()
    assert binding().device_status() == 0
    check_attention(out, lse, ref, d, dtype == "bf16", 6.0)


def mean_cache(means, block=32):
    """A cache of one full sequence whose block means are given [n, Hkv, d]."""
    n, hkv, d = means.shape
    cache = msa.KVCache.empty(n + 1, hkv, d, block)
    cache.k_mean[:n].copy_(torch.as_tensor(means, device=DEV).to(torch.bfloat16))
    return cache, np.arange(n, dtype=np.int32)[None], [n * block + 1]


@pytest.mark.parametrize("n,top_k", [(40, 7), (1500, 700), (3000, 1), (1200, 1199), (41500, 600)])
def test_equal_scores_go_to_the_lower_block(n, top_k):
    """All blocks alike: few, more than the list of near ties holds, and more
    than shared memory holds keys."""
    cache, t, lens = mean_cache(np.ones((n, 2, 64)))
    q = torch.randn((1, 1, 4, 64), device=DEV)
    t = np.concatenate([t, [[n]]], axis=1)
    sel, cnt = msa.cache_block_select(q, cache, i32(t), i32(lens), 1, top_k)
    assert selected(sel, cnt)[0][0] == [list(range(top_k))] * 2


@pytest.mark.parametrize("n", [100, 2500, 41000])
def test_scores_that_fp32_cannot_tell_apart(n):
    """Large parts that cancel leave differences below fp32's rounding of the
    terms: the choice is that of 64 bits."""
    rng = np.random.default_rng(n)
    d = 64
    means = np.zeros((n, 1, d))
    big = R.round_bf16(rng.normal(size=(n, d // 2 - 1)) * 1000)
    means[:, 0, 0:d - 2:2], means[:, 0, 1:d - 2:2] = big, -big   # cancels exactly
    means[:, 0, d - 2] = R.round_bf16(rng.integers(1, 256, n) * 2.0 ** -14)
    cache, t, lens = mean_cache(means)
    t = np.concatenate([t, [[n]]], axis=1)
    q = torch.ones((1, 1, 2, d), device=DEV, dtype=torch.bfloat16)
    pool = {"k_codes": np.zeros((1, 1, 32, d)), "k_mean": np.concatenate([means, means[:1]])}
    for top_k in (1, 17, n // 2):
        sel, cnt = msa.cache_block_select(q, cache, i32(t), i32(lens), 1, top_k)
        want = R.select(pool, q.double().cpu().numpy(), t, lens, 1, top_k)
        assert selected(sel, cnt) == want


def test_head_sums_beyond_fp32():
    """The heads' sum overflows 32 bits, the 64-bit scores order the blocks."""
    n = 70
    rng = np.random.default_rng(24)
    means = np.zeros((n, 1, 64))
    means[:, 0, 0] = rng.permutation(n) * 2.0 ** -6
    cache, t, lens = mean_cache(means)
    t = np.concatenate([t, [[n]]], axis=1)
    q = torch.zeros((1, 1, 4, 64), device=DEV, dtype=torch.bfloat16)
    q[..., 0] = 2.0 ** 127
    sel, cnt = msa.cache_block_select(q, cache, i32(t), i32(lens), 1, 9)
    best = sorted(np.argsort(-means[:, 0, 0])[:9].tolist())
    assert sel[0, 0, 0].tolist() == best and cnt.item() == 9


def test_not_a_number_ranks_last():
    means = np.random.default_rng(3).normal(size=(50, 1, 64))
    means[7] = np.nan
    means[11] = np.nan
    cache, t, lens = mean_cache(means)
    t = np.concatenate([t, [[50]]], axis=1)
    q = torch.randn((1, 1, 1, 64), device=DEV)
    pool = {"k_codes": np.zeros((1, 1, 32, 64)), "k_mean": np.concatenate([R.round_bf16(means), means[:1]])}
    for top_k in (5, 48, 49):
        sel, cnt = msa.cache_block_select(q, cache, i32(t), i32(lens), 1, top_k)
        assert selected(sel, cnt) == R.select(pool, q.double().cpu().numpy(), t, lens, 1, top_k)


def test_attention_over_a_given_selection():
    """A caller's own, shorter list; a bad entry is recorded and stays in bounds."""
    B = binding()
    lens, d, block = [1000], 128, 64
    cache, pool, t, _ = filled(lens, 2, d, block, seed=20)
    q = torch.randn((1, 1, 8, d), device=DEV).to(torch.bfloat16)
    sel = i32([[[[2, 5, 9], [0, 1, -1]]]])
    cnt = i32([[[3, 2]]])
    out, lse = torch.empty_like(q), torch.empty((1, 8, 1), device=DEV)
    ws = torch.empty((B.cache_attn_select_workspace_size(cache.ref, t.shape[1], 1, 1, 8, q.dtype),),
                     dtype=torch.uint8, device=DEV)
    B.cache_attn_select(cache.ref, q, i32(t), i32(lens), 100, sel, cnt, 0.1, out, lse, ws)
    assert B.device_status() == 0
    ref = R.attention(pool, q.double().cpu().numpy(), t, lens, 100, 0.1, sel=[[[[2, 5, 9], [0, 1]]]])
    check_attention(out, lse, ref, d, True, 6.0)
    B.cache_attn_select(cache.ref, q, i32(t), i32(lens), 100, i32([[[[2, 5, 99], [0, 1, -1]]]]), cnt, 0.1,
                        out, lse, ws)
    assert B.device_status() == B.MSA_ERR_INVALID_ARG


# -- eviction ----------------------------------------------------------------

def check_evict(cache, pool, t, lens, w, dst, budget, recent):
    ref = R.evict(pool, t, lens, w.double().cpu().numpy(), dst, budget, recent)
    new_lens, kept, new_w = msa.cache_evict(cache, i32(t), i32(lens), w, i32(dst), budget, recent)
    torch.cuda.synchronize()
    assert binding().device_status() == 0
    assert new_lens.cpu().tolist() == ref[0]
    kept, new_w = kept.cpu().numpy(), new_w.cpu().double().numpy()
    for b in range(len(lens)):
        for h in range(kept.shape[1]):
            K = ref[0][b]
            np.testing.assert_array_equal(kept[b, h, :K], ref[1][b][h])
            assert (kept[b, h, K:] == -1).all()
            np.testing.assert_array_equal(new_w[b, h, :K], ref[2][b][h])
            assert not new_w[b, h, K:].any()
    same_pool(cache, pool)


@pytest.mark.parametrize("lens,hkv,d,block,budget,recent", [
    ([1], 1, 64, 32, 1, 0),
    ([0, 5, 40], 2, 64, 32, 33, 4),        # empty, shorter than the budget, longer
    ([200, 199], 1, 128, 64, 64, 64),      # the recent ones alone
    ([700, 64], 3, 128, 64, 100, 0),
    ([4160], 2, 128, 64, 4096, 512),
    ([1000, 3000], 1, 64, 256, 300, 17),
    ([20000, 17000], 2, 64, 64, 1000, 100),  # split over a cluster
])
def test_evict(lens, hkv, d, block, budget, recent):
    nb = -(-budget // block)
    cache, pool, t, free = filled(lens, hkv, d, block, seed=sum(lens), extra=nb * len(lens))
    dst = free[:nb * len(lens)].reshape(len(lens), nb)
    w = torch.rand((len(lens), hkv, t.shape[1] * block), device=DEV)
    check_evict(cache, pool, t, lens, w, dst, budget, recent)


@pytest.mark.parametrize("kind", ["equal", "few values", "zeros", "special"])
@pytest.mark.parametrize("n", [500, 20001])
def test_evict_ties_and_special_weights(kind, n):
    block, budget = 32, 130
    cache, pool, t, free = filled([n], 1, 64, block, seed=n, extra=5)
    dst = free[:5].reshape(1, 5)
    w = torch.zeros((1, 1, t.shape[1] * block), device=DEV)
    if kind == "equal":
        w += 0.25
    elif kind == "few values":
        w[0, 0] = torch.randint(0, 3, w.shape[2:], device=DEV) * 0.5
    elif kind == "special":
        w[0, 0] = torch.rand(w.shape[2:], device=DEV) - 0.5
        w[0, 0, 3], w[0, 0, 9], w[0, 0, 12], w[0, 0, 13], w[0, 0, 14] = (
            math.inf, -math.inf, 1e-45, 0.0, -0.0)
    check_evict(cache, pool, t, [n], w, dst, budget, 10)


def test_evict_of_rows_longer_than_shared_memory():
    n, budget = 400_003, 777
    cache, pool, t, free = filled([n], 1, 64, 256, seed=31, extra=4)
    w = torch.randint(0, 50_000, (1, 1, t.shape[1] * 256), device=DEV).float() / 64   # many ties
    check_evict(cache, pool, t, [n], w, free[:4].reshape(1, 4), budget, 50)


@pytest.mark.parametrize("tiny", [2.0 ** -9, 2.0 ** -8, 1.75 * 2.0 ** -7, 2.0 ** -6])
def test_evict_leaves_only_tiny_codes_of_a_block(tiny):
    """The new scale is far below the old one when the outlier is evicted."""
    rng = np.random.default_rng(33)
    k = rng.choice([0.0, tiny, -tiny, 2.0 ** -9], size=(128, 1, 64)).astype(np.float32)
    k[:, 0, 0] = tiny
    k[::32, 0, 5] = 448.0                # every block's scale is 1
    t, dst = np.array([[0, 1, 2, 3]], dtype=np.int32), np.array([[6, 4]], dtype=np.int32)
    cache = new_cache(8, 1, 64, 32)
    kt = torch.as_tensor(k, device=DEV)
    msa.cache_append(cache, kt, kt, i32([0, 128]), i32(t), i32([128]), 128)
    w = torch.rand((1, 1, 128), device=DEV) + 1
    w[..., ::32] = 0
    check_evict(cache, pool_of(cache), t, [128], w, dst, 50, 8)


def test_evict_of_poisoned_blocks():
    """Kept slots of a NaN block make their new block NaN."""
    rng = np.random.default_rng(30)
    k = rng.normal(size=(96, 1, 64)).astype(np.float32)
    k[40, 0, 0] = np.nan
    t = np.array([[0, 1, 2]], dtype=np.int32)
    cache = new_cache(6, 1, 64, 32)
    kt = torch.as_tensor(k, device=DEV)
    msa.cache_append(cache, kt, kt, i32([0, 96]), i32(t), i32([96]), 96)
    w = torch.rand((1, 1, 96), device=DEV)
    check_evict(cache, pool_of(cache), t, [96], w, np.array([[5, 4]], dtype=np.int32), 60, 8)


# -- together ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_serving_loop(dtype):
    """Prompt, tokens with weights, eviction into new pages, more tokens with
    selected blocks: every step against the reference."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    hkv, g, d, block, budget, recent = 2, 4, 128, 32, 96, 16
    rng = np.random.default_rng(40)
    gen = torch.Generator(device=DEV).manual_seed(40)
    rand = lambda *s: torch.randn(s, generator=gen, device=DEV).to(dt)  # noqa: E731
    cache = new_cache(64, hkv, d, block)
    pages = rng.permutation(64).astype(np.int32)
    t, dst = pages[:16].reshape(2, 8), pages[16:32].reshape(2, 8)
    pool = pool_of(cache)
    lens = [140, 77]
    k, v = rand(217, hkv, d), rand(217, hkv, d)
    cu = [0, 140, 217]
    msa.cache_append(cache, k, v, i32(cu), i32(t), i32(lens), 140)
    R.append(pool, k.double().cpu().numpy(), v.double().cpu().numpy(), cu, t, lens)
    w = torch.zeros((2, hkv, 8 * block), device=DEV)

    def step(table, window, top_k, weights):
        k, v, q = rand(2, hkv, d), rand(2, hkv, d), rand(2, 1, hkv * g, d)
        for b in range(2):
            lens[b] += 1
        msa.cache_append(cache, k, v, i32([0, 1, 2]), i32(table), i32(lens), 1)
        R.append(pool, k.double().cpu().numpy(), v.double().cpu().numpy(), [0, 1, 2], table, lens)
        qn = q.double().cpu().numpy()
        if top_k:
            out, lse = msa.cache_topk_attention(q, cache, i32(table), i32(lens), window, top_k)
            ref = R.attention(pool, qn, table, lens, window, 1 / math.sqrt(d),
                              sel=R.select(pool, qn, table, lens, window, top_k))
        else:
            out, lse = msa.cache_attention(q, cache, i32(table), i32(lens), weights=weights)
            ref = R.attention(pool, qn, table, lens, 1 << 30, 1 / math.sqrt(d))
        check_attention(out, lse, ref, d, dtype == "bf16", 6.0)

    for _ in range(4):
        step(t, None, 0, w)
    assert abs(float(w.double().sum()) - 4 * 2 * hkv * g) < 1e-3   # rows' weights sum to one
    same_pool(cache, pool)
    new = R.evict(pool, t, lens, w.double().cpu().numpy(), dst[:, :3], budget, recent)
    got, kept, w = msa.cache_evict(cache, i32(t), i32(lens), w, i32(dst[:, :3]), budget, recent)
    lens = list(new[0])
    assert got.cpu().tolist() == lens == [96, 81]
    for _ in range(40):
        step(dst, 20, 2, None)
    same_pool(cache, pool)
    assert binding().device_status() == 0


def test_calls_on_a_side_stream():
    lens = [500, 90]
    cache, pool, t, _ = filled(lens, 2, 128, 64, seed=50)
    q = torch.randn((2, 1, 8, 128), device=DEV).to(torch.bfloat16)
    want = msa.cache_attention(q, cache, i32(t), i32(lens))
    tt, tl = i32(t), i32(lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [msa.cache_attention(q, cache, tt, tl, stream=side) for _ in range(3)]
    top = msa.cache_topk_attention(q, cache, tt, tl, 50, 2, stream=side)
    side.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    torch.testing.assert_close(top[0], msa.cache_topk_attention(q, cache, tt, tl, 50, 2)[0], rtol=0, atol=0)


def test_calls_on_two_streams_and_two_graphs_at_once():
    """Calls that overlap have workspaces of their own."""
    lens = [9000, 300, 4096]
    cache, _, t, _ = filled(lens, 2, 128, 64, seed=51)
    tt, tl = i32(t), i32(lens)
    qs = [torch.randn((3, n, 16, 128), device=DEV).to(torch.bfloat16) for n in (1, 2)]

    def calls(q):
        w = torch.zeros((3, 2, t.shape[1] * 64), device=DEV)
        return (*msa.cache_attention(q, cache, tt, tl, weights=w), w,
                *msa.cache_topk_attention(q, cache, tt, tl, 100, 9))

    want = [calls(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    graphs, held = [torch.cuda.CUDAGraph() for _ in qs], []
    for q, g in zip(qs, graphs):
        with torch.cuda.graph(g):
            held.append(calls(q))
    got = [[], []]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls(qs[i]))
                graphs[1 - i].replay()
        torch.cuda.synchronize()
    for i in range(2):
        for run in (*got[i], held[i]):
            for x, y in zip(run, want[i]):
                assert torch.equal(x, y)


def test_a_step_replays_from_a_graph():
    """Append, attention with weights, top-k attention and eviction captured
    once: replays on new inputs, longer sequences and other pages give the
    eager calls' bits."""
    hkv, d, block = 2, 128, 64
    lens = [254, 131]
    cache, _, t, free = filled(lens, hkv, d, block, seed=60, extra=8, width=6)
    t[0, 4:6], t[1, 3:5] = free[:2], free[2:4]
    tt, tl = i32(t), i32([255, 132])
    dst = i32(free[4:8].reshape(2, 2))
    k, v = (torch.randn((2, hkv, d), device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((2, 1, 8, d), device=DEV).to(torch.bfloat16)
    w = torch.zeros((2, hkv, 6 * block), device=DEV)
    cu = i32([0, 1, 2])

    def step():
        msa.cache_append(cache, k, v, cu, tt, tl, 1)
        a = msa.cache_attention(q, cache, tt, tl, weights=w)
        b = msa.cache_topk_attention(q, cache, tt, tl, 64, 1)
        return (*a, *b, *msa.cache_evict(cache, tt, tl, w, dst, 100, 10))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    for n in ([255, 132], [256, 133], [257, 134]):   # every slot up to these has been written
        tl.copy_(i32(n))
        q.normal_()
        k.normal_()
        w.zero_()
        eager = [x.clone() for x in step()]
        w.zero_()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(captured, eager):
            assert torch.equal(x, y)
    assert binding().device_status() == 0


def test_pages_that_do_not_exist_and_lengths_that_cannot_be():
    """Recorded in the status word; neighbours are served as usual."""
    B = binding()
    lens = [100, 100]
    cache, pool, t, _ = filled(lens, 1, 64, 32, seed=70)
    q = torch.randn((2, 1, 4, 64), device=DEV).to(torch.bfloat16)
    want = msa.cache_attention(q, cache, i32(t), i32(lens))
    bad = t.copy()
    bad[1, 1] = cache.n_pages
    out, lse = msa.cache_attention(q, cache, i32(bad), i32(lens))
    assert B.device_status() == B.MSA_ERR_INVALID_ARG
    assert torch.equal(out[0], want[0][0])
    # the slots of the missing page are left out
    gap = np.concatenate([np.arange(32), np.arange(64, 100)])
    kk, vv = (R.held(pool, x, t[1], 0, 100)[gap] for x in "kv")
    s = kk @ q[1, 0].double().cpu().numpy().T * 0.125
    p = np.exp(s - s.max(axis=0))
    p /= p.sum(axis=0)
    assert np.abs(out[1, 0].double().cpu().numpy() - p.T @ vv).max() < 0.02
    before = pool_of(cache)
    k = torch.randn((2, 1, 64), device=DEV)
    bad = t.copy()
    bad[:, 3] = [-7, 1 << 30]
    msa.cache_append(cache, k, k, i32([0, 1, 2]), i32(bad), i32([101, 101]), 1)
    assert B.device_status() == B.MSA_ERR_INVALID_ARG
    same_pool(cache, before)
    for cu, ln, most in (([0, 1, 2], [1 << 20, -3], 2), ([0, 3, 2], [101, 101], 2), ([0, 1, 2], [0, 101], 2), ([-1, 1, 2], [101, 0], 2)):
        msa.cache_append(cache, k, k, i32(cu), i32(np.full_like(t, -1)), i32(ln), most)
        assert B.device_status() == B.MSA_ERR_INVALID_ARG
        same_pool(cache, before)
    msa.cache_attention(q, cache, i32(t), i32([-5, 100]))
    assert B.device_status() == B.MSA_ERR_INVALID_ARG


@pytest.mark.large
def test_rejected_drafts_are_dropped_by_the_length():
    """Lengths go back by some drafts and other tokens take their slots."""
    cache, pool, t, free = filled([61, 30], 2, 64, 32, seed=61, extra=2, width=3)
    t[0, 2], t[1, 1] = free[:2]
    rng = np.random.default_rng(62)
    q = torch.as_tensor(rng.normal(size=(2, 1, 4, 64)), device=DEV).to(torch.bfloat16)
    lens = [61, 30]
    for new, back in ((4, 3), (4, 4), (2, 0), (4, 1)):
        k, v = (torch.as_tensor(rng.normal(size=(2 * new, 2, 64)) * 4, device=DEV).to(torch.bfloat16)
                for _ in range(2))
        lens, cu = [n + new for n in lens], [0, new, 2 * new]
        msa.cache_append(cache, k, v, i32(cu), i32(t), i32(lens), new)
        R.append(pool, k.double().cpu().numpy(), v.double().cpu().numpy(), cu, t, lens)
        lens = [n - back for n in lens]
        out, lse = msa.cache_attention(q, cache, i32(t), i32(lens))
        ref = R.attention(pool, q.double().cpu().numpy(), t, lens, 1 << 30, 1 / 8)
        check_attention(out, lse, ref, 64, True, 30.0)
    same_pool(cache, pool)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes of codes: pages at its far end."""
    hkv, d, block = 8, 128, 256
    pages = (1 << 32) // (hkv * d * block) + 3
    codes = torch.zeros((2, pages, hkv, block, d), dtype=torch.uint8, device=DEV)
    cache = msa.KVCache(codes[0], codes[1], torch.zeros((pages, hkv), device=DEV),
                        torch.zeros((pages, hkv), device=DEV),
                        torch.zeros((pages, hkv, d), dtype=torch.bfloat16, device=DEV))
    t = np.array([[pages - 1, 0, pages - 2]], dtype=np.int32)
    k, v = (torch.randn((600, hkv, d), device=DEV).to(torch.bfloat16) for _ in range(2))
    small = new_cache(3, hkv, d, block)
    msa.cache_append(cache, k, v, i32([0, 600]), i32(t), i32([600]), 600)
    msa.cache_append(small, k, v, i32([0, 600]), i32([[2, 0, 1]]), i32([600]), 600)
    q = torch.randn((1, 2, 64, d), device=DEV).to(torch.bfloat16)
    for call in (lambda c, tt: msa.cache_attention(q, c, tt, i32([600])),
                 lambda c, tt: msa.cache_topk_attention(q, c, tt, i32([600]), 40, 1)):
        for x, y in zip(call(cache, i32(t)), call(small, i32([[2, 0, 1]]))):
            assert torch.equal(x, y)


def test_python_refusals():
    """Wrong types, shapes, devices and layouts raise before anything runs."""
    lens = [40]
    cache, _, t, _ = filled(lens, 2, 64, 32, seed=80)
    tt, tl = i32(t), i32(lens)
    q = torch.zeros((1, 1, 4, 64), device=DEV)
    k = torch.zeros((1, 2, 64), device=DEV)
    cu = i32([0, 1])
    w = torch.zeros((1, 2, t.shape[1] * 32), device=DEV)

    def refused(error, call, *a, **kw):
        with pytest.raises(error):
            call(*a, **kw)

    refused(TypeError, msa.cache_attention, q.half(), cache, tt, tl)
    refused(TypeError, msa.cache_attention, q, cache, tt.long(), tl)
    refused(TypeError, msa.cache_attention, q, cache, tt, tl.long())
    refused(TypeError, msa.cache_attention, q, cache, tt, tl, out_dtype=torch.float16)
    refused(TypeError, msa.cache_attention, q, cache, tt, tl, weights=w.double())
    refused(ValueError, msa.cache_attention, q.cpu(), cache, tt, tl)
    refused(ValueError, msa.cache_attention, q[0], cache, tt, tl)
    refused(ValueError, msa.cache_attention, q[..., :32], cache, tt, tl)
    refused(ValueError, msa.cache_attention, torch.zeros((1, 1, 64, 4), device=DEV).transpose(2, 3), cache, tt, tl)
    refused(ValueError, msa.cache_attention, q, cache, tt[0], tl)
    refused(ValueError, msa.cache_attention, q, cache, tt, i32([40, 40]))
    refused(ValueError, msa.cache_attention, q, cache, tt, tl, weights=w[:, :1])
    refused(msa.binding.MsaError, msa.cache_attention, q, cache, tt, tl, weights=w[:, :, :-1].contiguous())
    refused(msa.binding.MsaError, msa.cache_attention, q, cache, tt, tl, window=0)
    refused(msa.binding.MsaError, msa.cache_attention, q, cache, tt, tl, scale=-1.0)
    refused(msa.binding.MsaError, msa.cache_attention, q[:, :, :3].contiguous(), cache, tt, tl)
    refused(msa.binding.MsaError, msa.cache_topk_attention, q, cache, tt, tl, 1, 0)
    refused(msa.binding.MsaError, msa.cache_block_select, q, cache, tt, tl, 0, 1)
    refused(TypeError, msa.cache_append, cache, k.half(), k.half(), cu, tt, tl, 1)
    refused(TypeError, msa.cache_append, cache, k, k.bfloat16(), cu, tt, tl, 1)
    refused(ValueError, msa.cache_append, cache, k, k, i32([0, 1, 1]), tt, tl, 1)
    refused(msa.binding.MsaError, msa.cache_append, cache, k, k, cu, tt, tl, 2)
    refused(ValueError, msa.cache_evict, cache, tt, tl, w, i32([0]), 4, 1)
    refused(ValueError, msa.cache_evict, cache, tt, tl, w, i32([[0]]), 0, 0)
    refused(msa.binding.MsaError, msa.cache_evict, cache, tt, tl, w, i32([[0]]), 33, 0)
    refused(msa.binding.MsaError, msa.cache_evict, cache, tt, tl, w, i32([[0]]), 4, 5)
    refused(TypeError, msa.KVCache, cache.k_codes.float(), cache.v_codes, cache.k_scale, cache.v_scale, cache.k_mean)
    refused(ValueError, msa.KVCache, cache.k_codes, cache.v_codes[:1], cache.k_scale, cache.v_scale, cache.k_mean)
    refused(msa.binding.MsaError, msa.cache_attention, torch.zeros((1, 1, 4, 32), device=DEV),
            msa.KVCache.empty(2, 2, 32, 32), tt, tl)


# -- values and scores of any size -------------------------------------------

def check_in_fp32(cache, t, lens, q, dtype, scale=1.0):
    """Attention with an fp32 output against the reference, relative to each
    row's own weighted values: halves' subnormals are 2^-39 of the row's largest
    weighted block (values of one size in a block: twice a slot's at most)."""
    q = q.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    ref = R.attention(pool_of(cache), q.double().cpu().numpy(), t, lens, 1 << 30, scale)
    out, lse = msa.cache_attention(q, cache, i32(t), i32(lens), scale=scale, out_dtype=torch.float32)
    tol_o, tol_l = bounds(ref, q.shape[3], dtype == "bf16", torch.float32)
    tol_o = tol_o + 2.0 ** -149
    if dtype == "bf16":
        tol_o += ref[4][..., None] * 2.0 ** -38 * ref[2]
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(o).all() and np.isfinite(l).all()
    err = np.abs(o - ref[0])
    assert (err <= tol_o).all(), f"out: worst {np.max(err / tol_o):.3g} of the bound"
    err = np.abs(l - ref[1])
    assert (err <= tol_l).all(), f"lse: worst {np.max(err / tol_l):.3g} of the bound"


def long_sequence(n, k, v, d=128, block=64, seed=91):
    """One sequence of one KV head: keys and values [n, d]."""
    rng = np.random.default_rng(seed)
    nb = -(-n // block)
    cache, t = new_cache(nb, 1, d, block), rng.permutation(nb).astype(np.int32)[None]
    kt, vt = (torch.as_tensor(x[:, None], device=DEV).float() for x in (k, v))
    msa.cache_append(cache, kt, vt, i32([0, n]), i32(t), i32([n]), n)
    return cache, t, [n]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [500, 9000])
def test_values_near_the_end_of_the_range(n, dtype):
    """A sequence that several CTAs share: their parts are joined without
    multiplying values by anything above 1."""
    rng = np.random.default_rng(92)
    cache, t, lens = long_sequence(n, rng.normal(size=(n, 128)), rng.uniform(1, 2, size=(n, 128)) * 1e36)
    check_in_fp32(cache, t, lens, torch.randn((1, 1, 8, 128), device=DEV), dtype, 1 / math.sqrt(128))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("first", [True, False])
def test_parts_of_little_weight_and_great_values(first, dtype):
    """Half of a sequence leads by 2^130 in weight and trails by 2^200 in
    value: the other half's parts make the output."""
    rng = np.random.default_rng(93)
    n, d = 8192, 128
    lead = (np.arange(n) < n // 2) == first
    k = rng.normal(size=(n, d)) * 0.25
    k[:, 0] = np.where(lead, 90.0, 0.0)
    v = rng.uniform(1, 2, size=(n, d)) * np.where(lead, 1e-30, 1e30)[:, None]
    q = torch.randn((1, 1, 8, d), device=DEV) * 0.05
    q[..., 0] = 1.0
    check_in_fp32(*long_sequence(n, k, v), q, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [70, 8100])
def test_poison_of_no_weight_reaches_its_rows(at, dtype):
    """A NaN value whose slot's weight is below fp32, in a part before or after
    those that lead."""
    rng = np.random.default_rng(94)
    n, d = 8192, 128
    k = rng.normal(size=(n, d)) * 0.25
    k[:, 0] = np.where((np.arange(n) < 4096) == (at < 4096), 0.0, 200.0)
    v = rng.normal(size=(n, d))
    v[at, 3] = np.nan
    cache, t, lens = long_sequence(n, k, v)
    q = torch.randn((1, 1, 8, d), device=DEV) * 0.05
    q[..., 0] = 1.0
    out, _ = msa.cache_attention(q.to(torch.bfloat16 if dtype == "bf16" else torch.float32), cache, i32(t), i32(lens),
                                 scale=1.0)
    assert torch.isnan(out).all()


def layered(first, second, seed=90):
    """8 sequences of 64 blocks of 32 slots, 4 KV heads of 64, whose kind
    changes every four blocks, so that each warp meets both kinds in turn:
    first, second = (score, size of the values); odd heads begin with the
    second.  Queries for a scale of 1."""
    B, H, d, blocks = 8, 4, 64, 64
    n = 32 * blocks
    rng = np.random.default_rng(seed)
    kind = (np.arange(n)[:, None] // 128 + np.arange(H)[None]) % 2
    k = rng.normal(size=(B, n, H, d)) * 0.25
    k[..., 0] = np.where(kind == 0, first[0], second[0])[None]
    v = rng.uniform(1, 2, size=(B, n, H, d)) * rng.choice([-1.0, 1.0], size=(B, n, H, 1))
    v *= np.where(kind == 0, first[1], second[1])[None, :, :, None]
    cache = new_cache(B * blocks, H, d, 32)
    t = rng.permutation(B * blocks).astype(np.int32).reshape(B, blocks)
    kt, vt = (torch.as_tensor(x.reshape(B * n, H, d), device=DEV).float() for x in (k, v))
    msa.cache_append(cache, kt, vt, i32(np.arange(B + 1) * n), i32(t), i32([n] * B), n)
    q = torch.randn((B, 1, 2 * H, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)) * 0.05
    q[..., 0] = 1.0
    return cache, t, [n] * B, q


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lead", [30.0, 44.0, 104.0, 288.0])
@pytest.mark.parametrize("big,small", [(1e30, 1e-30), (1e30, 1e10), (1e4, 1e-30)])
def test_a_leading_score_over_far_smaller_values(big, small, lead, dtype):
    """Blocks that lead by e^lead in weight and trail by up to 2^200 in value:
    the largest score and the largest weighted value are slots of their own."""
    check_in_fp32(*layered((0.0, big), (lead, small)), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [500, 9000])
@pytest.mark.parametrize("size", [1e-32, 1e-35, 1e-37, 1e-43])
def test_values_at_the_bottom_of_the_range(size, n, dtype):
    """Down to fp32's subnormals, with scales of 2^-126."""
    rng = np.random.default_rng(95)
    cache, t, lens = long_sequence(n, rng.normal(size=(n, 128)), rng.uniform(1, 2, size=(n, 128)) * size)
    check_in_fp32(cache, t, lens, torch.randn((1, 1, 8, 128), device=DEV), dtype, 1 / math.sqrt(128))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [1.0, 1e-8, 1e-12, 1e-30])
@pytest.mark.parametrize("lead", [0.0, 30.0, 208.0])
def test_blocks_of_zeros_beside_small_values(lead, value, dtype):
    """They take their share of the weight and none of the other values' bits."""
    check_in_fp32(*layered((lead, 0.0), (0.0, value)), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lead", [0.0, 30.0])
def test_a_scale_of_zero_over_any_codes(lead, dtype):
    """A slot is code * scale: 0 where the scale is, whatever the codes are."""
    cache, t, lens, q = layered((lead, 1.0), (0.0, 1e-3))
    cache.v_scale[cache.v_scale > 1e-4] = 0.0
    check_in_fp32(cache, t, lens, q, dtype)
    cache.v_scale.zero_()
    cache.k_scale.zero_()
    check_in_fp32(cache, t, lens, q, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_size,k_size", [(2.0 ** -83, 1.0), (1.0, 2.0 ** -90), (2.0 ** -60, 2.0 ** -30),
                                           (2.0 ** -70, 2.0 ** -70), (1.0, 1.0)])
def test_near_ties_of_tiny_scores(q_size, k_size, dtype):
    """Norms whose squares fall below fp32 still bound the scores' rounding:
    large parts that cancel, differences below fp32's rounding of them."""
    n, d, half = 2500, 64, 31
    rng = np.random.default_rng(n)
    means = np.zeros((n, 1, d))
    big = R.round_bf16(rng.normal(size=(n, half)) * 1000)
    means[:, 0, :half], means[:, 0, 32:63] = big, -big[:, rng.permutation(half)]   # cancels in the end
    means[:, 0, 63] = R.round_bf16(rng.integers(1, 256, n) * 2.0 ** -14)
    means *= k_size
    cache, t, lens = mean_cache(means)
    t = np.concatenate([t, [[n]]], axis=1)
    q = torch.full((1, 1, 2, d), q_size, device=DEV, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    pool = {"k_codes": np.zeros((1, 1, 32, d)), "k_mean": np.concatenate([means, means[:1]])}
    for top_k in (1, 17, n // 2):
        sel, cnt = msa.cache_block_select(q, cache, i32(t), i32(lens), 1, top_k)
        assert selected(sel, cnt) == R.select(pool, q.double().cpu().numpy(), t, lens, 1, top_k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_selection_is_attended_through_the_package(dtype):
    """What cache_block_select returns, attended, is cache_topk_attention; a
    caller's shorter lists, an empty one among them, are the reference's; and a
    call on another stream and from a graph gives the same."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    lens, d, window, top_k = [900, 130, 0], 128, 50, 5
    cache, pool, t, _ = filled(lens, 2, d, 64, seed=96)
    tt, tl = i32(t), i32(lens)
    q = torch.randn((3, 2, 8, d), device=DEV).to(dt)
    sel, cnt = msa.cache_block_select(q, cache, tt, tl, window, top_k)
    out, lse = msa.cache_select_attention(q, cache, tt, tl, window, sel, cnt)
    want = msa.cache_topk_attention(q, cache, tt, tl, window, top_k)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    cnt = torch.minimum(cnt, i32([[[0, 2], [1, 4]]] * 3))
    out, lse = msa.cache_select_attention(q, cache, tt, tl, window, sel, cnt, scale=0.1, out_dtype=torch.float32)
    ref = R.attention(pool, q.double().cpu().numpy(), t, lens, window, 0.1, sel=selected(sel.where(
        torch.arange(top_k, device=DEV) < cnt[..., None], -1), cnt))
    check_attention(out, lse, ref, d, dtype == "bf16", 6.0)
    assert binding().device_status() == 0
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    other = msa.cache_select_attention(q, cache, tt, tl, window, sel, cnt, 0.1, torch.float32, stream=side)
    side.synchronize()
    with torch.cuda.graph(graph):
        captured = msa.cache_select_attention(q, cache, tt, tl, window, sel, cnt, 0.1, torch.float32)
    graph.replay()
    torch.cuda.synchronize()
    for x in (other, captured):
        assert torch.equal(x[0], out) and torch.equal(x[1], lse)
    for error, bad in ((ValueError, (sel[0], cnt)), (ValueError, (sel[:, :1], cnt)), (ValueError, (sel, cnt[..., :1])),
                       (TypeError, (sel.long(), cnt)), (TypeError, (sel, cnt.long())), (ValueError, (sel, cnt.cpu())),
                       (msa.binding.MsaError, (sel[..., :0], cnt)),
                       (ValueError, (sel.transpose(0, 1).contiguous().transpose(0, 1), cnt))):
        with pytest.raises(error):
            msa.cache_select_attention(q, cache, tt, tl, window, *bad)


# -- sizes and layouts beyond the cases above --------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_scales_that_are_no_powers_of_two(d, dtype):
    """The attention takes any finite scale: a pool filled from elsewhere."""
    lens = [700, 65]
    cache, _, t, _ = filled(lens, 2, d, 64, seed=100)
    for scale in (cache.k_scale, cache.v_scale):
        scale.nan_to_num_(nan=1.0)
        scale *= 0.3 + torch.rand_like(scale)
    check_in_fp32(cache, t, lens, torch.randn((2, 1, 8, d), device=DEV), dtype, 0.1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,group,d", [(8, 8, 128), (9, 5, 64), (40, 3, 128), (130, 1, 64)])
def test_more_rows_than_a_tile(n_q, group, d, dtype):
    """Several 32-row tiles of a (sequence, KV head), the last one partly filled."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    lens = [700, 65, 20]
    cache, pool, t, _ = filled(lens, 2, d, 64, seed=101)
    q = torch.randn((3, n_q, 2 * group, d), device=DEV).to(dt)
    for window in (None, 33):
        ref = R.attention(pool, q.double().cpu().numpy(), t, lens, window or 1 << 30, 0.1)
        w = torch.zeros((3, 2, t.shape[1] * 64), device=DEV)
        out, lse = msa.cache_attention(q, cache, i32(t), i32(lens), window, scale=0.1, weights=w)
        check_attention(out, lse, ref, d, dtype == "bf16", 6.0)
        ds = (d + 4) * 2.0 ** -23 * ref[3].max()
        tol = ref[5] * (2 * ds + 2.0 ** -20 + max(lens) * 2.0 ** -23 + n_q * group * 2.0 ** -24) + 1e-30
        assert (np.abs(w.double().cpu().numpy() - ref[5]) <= tol).all()
    assert binding().device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,top", [(129, 70), (400, 300)])
def test_more_sequences_than_a_cta_has_threads(batch, top, dtype):
    """The list of sequences, or of query tokens, is scanned in rounds."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, top, batch).tolist()
    lens[0], lens[batch // 2], lens[-1] = 0, 0, top
    cache, pool, t, _ = filled(lens, 1, 64, 32, seed=batch)
    tt, tl = i32(t), i32(lens)
    q = torch.randn((batch, 2, 2, 64), device=DEV).to(dt)
    qn = q.double().cpu().numpy()
    w = torch.zeros((batch, 1, t.shape[1] * 32), device=DEV)
    out, lse = msa.cache_attention(q, cache, tt, tl, weights=w)
    ref = R.attention(pool, qn, t, lens, 1 << 30, 0.125)
    check_attention(out, lse, ref, 64, dtype == "bf16", 6.0)
    ds = (64 + 4) * 2.0 ** -23 * ref[3].max()
    tol = ref[5] * (2 * ds + 2.0 ** -20 + top * 2.0 ** -23 + 4 * 2.0 ** -24) + 1e-30
    assert (np.abs(w.double().cpu().numpy() - ref[5]) <= tol).all()
    sel, cnt = msa.cache_block_select(q, cache, tt, tl, 20, 2)
    want = R.select(pool, qn, t, lens, 20, 2)
    assert selected(sel, cnt) == want
    out, lse = msa.cache_topk_attention(q, cache, tt, tl, 20, 2)
    check_attention(out, lse, R.attention(pool, qn, t, lens, 20, 0.125, sel=want), 64, dtype == "bf16", 6.0)
    assert binding().device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_that_share_a_prefix(dtype):
    """Full pages in two tables: both attend them, appends and evictions of one
    leave the other's slots as they were."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cache, pool, t, free = filled([140, 40], 2, 64, 32, seed=102, extra=8, width=7)
    t[1, :6] = [*t[0, :4], *t[1, :2]]      # 128 shared slots, then 40 of its own
    t[1, 6] = free[0]
    lens = [140, 168]
    q = torch.randn((2, 1, 4, 64), device=DEV)
    check_in_fp32(cache, t, lens, q, dtype, 0.125)
    k = torch.randn((31, 2, 64), device=DEV).to(dt)
    lens = [141, 198]
    msa.cache_append(cache, k, k, i32([0, 1, 31]), i32(t), i32(lens), 30)
    kn = k.double().cpu().numpy()
    R.append(pool, kn, kn, [0, 1, 31], t, lens)
    same_pool(cache, pool)
    check_in_fp32(cache, t, lens, q, dtype, 0.125)
    w = torch.rand((2, 2, t.shape[1] * 32), device=DEV)
    check_evict(cache, pool, t, lens, w, free[1:7].reshape(2, 3), 90, 10)


def test_drafts_dropped_under_range_checks():
    """Shorter lengths after drafts, then other tokens in their slots (with
    windows and selections, beside the test of the lengths alone)."""
    cache, pool, t, free = filled([61, 30], 2, 64, 32, seed=103, extra=2, width=3)
    t[0, 2], t[1, 1] = free[:2]
    rng = np.random.default_rng(104)
    lens = [61, 30]
    for new, back in ((4, 3), (4, 4), (2, 0), (4, 1)):
        k, v, q = (torch.as_tensor(rng.normal(size=s), device=DEV).to(torch.bfloat16)
                   for s in ((2 * new, 2, 64), (2 * new, 2, 64), (2, 1, 4, 64)))
        lens, cu = [n + new for n in lens], [0, new, 2 * new]
        msa.cache_append(cache, k, v, i32(cu), i32(t), i32(lens), new)
        R.append(pool, k.double().cpu().numpy(), v.double().cpu().numpy(), cu, t, lens)
        same_pool(cache, pool)
        lens = [n - back for n in lens]
        qn = q.double().cpu().numpy()
        out, lse = msa.cache_attention(q, cache, i32(t), i32(lens), 20)
        check_attention(out, lse, R.attention(pool, qn, t, lens, 20, 1 / 8), 64, True, 6.0)
        out, lse = msa.cache_topk_attention(q, cache, i32(t), i32(lens), 5, 1)
        want = R.select(pool, qn, t, lens, 5, 1)
        check_attention(out, lse, R.attention(pool, qn, t, lens, 5, 1 / 8, sel=want), 64, True, 6.0)
    assert binding().device_status() == 0


@pytest.mark.parametrize("size", [2.0 ** 26, 1e30])
def test_evict_of_zeros_beside_far_larger_values(size):
    """Slots whose codes are all 0 in a block of large values join a block of
    small ones: they stay zeros."""
    rng = np.random.default_rng(105)
    k = rng.normal(size=(128, 1, 64)).astype(np.float32)
    k[:32] *= 1e-30 if size > 1e20 else 1.0
    k[32:64] = 0.0
    k[40, 0, 7] = size                   # dropped, with its scale
    t, dst = np.array([[0, 1, 2, 3]], dtype=np.int32), np.array([[6, 4]], dtype=np.int32)
    cache = new_cache(8, 1, 64, 32)
    kt = torch.as_tensor(k, device=DEV)
    msa.cache_append(cache, kt, kt, i32([0, 128]), i32(t), i32([128]), 128)
    w = torch.zeros((1, 1, 128), device=DEV)
    w[..., 10:39] = 1.0                  # 22 small slots and 7 of zeros in one block
    check_evict(cache, pool_of(cache), t, [128], w, dst, 40, 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [100, 9000])
def test_poisoned_values_leave_lse_and_weights(n, dtype):
    """The softmax does not know the values: a NaN among them makes the output
    NaN, the lse and the weights are those of the keys."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rng = np.random.default_rng(106)
    k, v = rng.normal(size=(2, n, 128))
    cache, t, lens = long_sequence(n, k, np.where(np.arange(n)[:, None] == 70, np.inf, v))
    clean, t2, _ = long_sequence(n, k, v)
    q = torch.randn((1, 1, 8, 128), device=DEV).to(dt)
    w = torch.zeros((1, 1, t.shape[1] * 64), device=DEV)
    out, lse = msa.cache_attention(q, cache, i32(t), i32(lens), weights=w)
    assert torch.isnan(out).all()
    ref = R.attention(pool_of(clean), q.double().cpu().numpy(), t2, lens, 1 << 30, 1 / math.sqrt(128))
    tol_l = bounds(ref, 128, dtype == "bf16", dt)[1]
    assert (np.abs(lse.double().cpu().numpy() - ref[1]) <= tol_l).all()
    ds = (128 + 4) * 2.0 ** -23 * ref[3].max()
    tol = ref[5] * (2 * ds + 2.0 ** -20 + n * 2.0 ** -23 + 8 * 2.0 ** -24) + 1e-30
    assert (np.abs(w.double().cpu().numpy() - ref[5]) <= tol).all()
