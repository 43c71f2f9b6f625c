"""The 4-bit KV cache, and reading either cache back, on the GPU against its
64-bit reference.

Codes, scales and values read back must be equal to the reference's; attention
is held to bounds derived from the arithmetic (see ``bounds``)."""
import threading

import numpy as np
import pytest
import torch

import long_context_sparse_landmark_gb300 as msa
from tests import cache4_ref as R
from tests.gpu_helpers import binding, check_guards, gempty, gfull

pytestmark = pytest.mark.gpu

DEV = "cuda"
NAMES = ("k_codes", "v_codes", "k_scale", "v_scale")


def new_cache(pages, hkv, d, block, fill=0xFF):
    """A pool in guarded memory, every byte of it `fill` (0xff: codes of -6, NaN scales)."""
    codes = [gfull((pages, hkv, block, d // 2), fill, torch.uint8) for _ in range(2)]
    scale = [gfull((pages, hkv, block, d // 32), fill, torch.uint8) for _ in range(2)]
    return msa.KVCache4(*codes, *scale)


def pool_of(cache):
    return {n: getattr(cache, n).cpu().numpy().copy() for n in NAMES}


def same_pool(cache, pool):
    for n in NAMES:
        np.testing.assert_array_equal(getattr(cache, n).cpu().numpy(), pool[n], err_msg=n)


def tables(lens, block, rng, extra=0, width=0):
    """Distinct pages in random order, -1 where a row has none."""
    need = [-(-n // block) for n in lens]
    pages = rng.permutation(sum(need) + extra)
    t = np.full((len(lens), max(1, width, max(need))), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = pages[at:at + k]
        at += k
    return t


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


def starts(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


def filled(lens, hkv, d, block, seed, extra=0, width=0, kscale=1.0, vscale=1.0):
    """A cache that holds random tokens, through cache_append, and its pool."""
    rng = np.random.default_rng(seed)
    t = tables(lens, block, rng, extra + 1, width)
    cache = new_cache(int(t.max(initial=0)) + extra + 2, hkv, d, block)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    k = torch.randn((sum(lens), hkv, d), generator=gen, device=DEV) * kscale
    k[..., :2] *= 6
    v = torch.randn((sum(lens), hkv, d), generator=gen, device=DEV) * vscale
    msa.cache_append(cache, k, v, i32(starts(lens)), i32(t), i32(lens), max(lens))
    torch.cuda.synchronize()
    assert binding().device_status() == 0
    return cache, pool_of(cache), t


def bounds(ref, d, bf16_in, out_dtype, apart=False):
    """How far out and lse may be off.

    Scores: sums of d exact products (fp32 queries as two halves: off by 2^-22 of
    each), each fp32 step off by at most 2^-23 of the absolute sum, the scalings
    and the two subtractions of the exponent by eight half steps more: ds = (d +
    8) 2^-23 S1 (+ 2^-22 S1), S1 the largest sum of |q k| scale.  Weights:
    relative error 2 ds, two exponentials (2^-22 each) and their arguments' other
    part (the value's exponent over the largest, up to 2^5 where it counts:
    2^-19), the sums' steps (one per slot at most, 2^-23 each), and the rounding
    to one half (2^-11) or two (2^-22).  A subnormal half is off by 2^-25 besides,
    a slot.  A half is the weight times the unit of its value, and the largest of
    them 2^9 or more when the output's unit was set (2^14 less five binades of
    room): a slot is off by 2^-34 of that weight times 6 units.  The unit is the
    scale of the largest value seen, four binades above it at most (2^4), and 2^12
    that of any value in it at most (codes of 4 or more: 1.5 * 2^12): 2^-33 of
    `unit`.  Where scales lie too far apart for a unit (`apart`: in every chunk) the
    halves hold their values' scales, and the largest is 2^14 when set: 2^-39 of the
    row's largest product, `top`, times 1.5.  Output: half a step of its type."""
    out, lse, absv, s1, count, top, unit = ref
    ds = ((d + 8) * 2.0 ** -23 + (0.0 if bf16_in else 2.0 ** -22)) * s1
    rel = 2 * ds + 2.0 ** -21 + 2.0 ** -19 + count * 2.0 ** -23 + (2.0 ** -11 if bf16_in else 2.0 ** -22)
    half = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -24
    tol_o = (absv * rel[..., None] + (count * (top * 2.0 ** -38 if apart else unit * 2.0 ** -33))[..., None]) * (1 + half) + np.abs(out) * half
    tol_l = (ds + 2.0 ** -20 + count * 2.0 ** -24).transpose(0, 2, 1)
    return tol_o, tol_l + np.abs(np.where(np.isfinite(lse), lse, 0.0)) * 2.0 ** -22


def check_attention(out, lse, ref, d, bf16_in, apart=False):
    tol_o, tol_l = bounds(ref, d, bf16_in, out.dtype, apart)
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


def rows_of(pool, t, lens, counts):
    """What cache_read gives: the last counts[b] slots of each sequence."""
    out = []
    for x in ("k", "v"):
        per = [np.stack([R.held(pool, x, t[b], h, n)[n - c:] for h in range(pool["k_codes"].shape[1])], axis=1)
               for b, (n, c) in enumerate(zip(lens, counts)) if c]
        out.append(np.concatenate(per))
    return out


# -- append ------------------------------------------------------------------

@pytest.mark.parametrize("hkv,d,block,dtype,before,new", [
    (1, 64, 32, "bf16", [0], [1]),
    (1, 128, 64, "bf16", [63], [1]),
    (2, 128, 64, "f32", [64], [1]),
    (3, 64, 32, "f32", [5, 0, 31], [40, 0, 1]),   # one sequence gets nothing
    (2, 128, 128, "bf16", [100, 7, 0], [300, 1, 128]),
    (1, 128, 256, "f32", [255, 0], [2, 513]),
    (8, 128, 64, "bf16", [1000, 999], [129, 64]),
    (5, 64, 64, "bf16", [3] * 40, list(range(40))),
])
def test_append_equals_the_definition(hkv, d, block, dtype, before, new):
    rng = np.random.default_rng(hkv * 1000 + block)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    lens = [a + b for a, b in zip(before, new)]
    t = tables(lens, block, rng, 2)
    cache = new_cache(int(t.max()) + 3, hkv, d, block)
    pool = pool_of(cache)
    at = [0] * len(lens)
    for part in (before, new):
        if not sum(part):
            continue
        at = [a + b for a, b in zip(at, part)]
        cu = starts(part)
        k = torch.as_tensor(rng.normal(size=(sum(part), hkv, d)) * np.exp(rng.normal(size=(sum(part), 1, 1))),
                            device=DEV).to(dt)
        v = torch.as_tensor(rng.normal(size=(sum(part), hkv, d)) * 1e-3, device=DEV).to(dt)
        msa.cache_append(cache, k, v, i32(cu), i32(t), i32(at), max(part))
        R.append(pool, k.double().cpu().numpy(), v.double().cpu().numpy(), cu, t, at)
        same_pool(cache, pool)   # slots past the lengths, and other slots, are left as they were
    msa.cache_append(cache, k, v, i32(cu), i32(t), i32(at), max(part))
    same_pool(cache, pool)
    assert binding().device_status() == 0


def special_rows(d):
    """Rows of d values where the format decides: ties, ends of binades, zeros of
    both signs, the smallest and the largest magnitudes, what no code stands for."""
    rows = []
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 7.0, 0.2500001, 0.7499999, -0.25, -5.0, 0.0, -0.0]
    for s in (1.0, 2.0 ** -30, 2.0 ** 40, 2.0 ** -120):
        rows.append([x * s for x in ties])
    rows.append([7.000001] + ties[:7])                     # the next exponent
    rows.append([2.0 ** -149, -2.0 ** -127, 2.0 ** -126, 3 * 2.0 ** -128])
    rows.append([1.75 * 2.0 ** 127, -2.0 ** 126, 2.0 ** 100])
    rows.append([0.0] * 4)
    rows.append([-0.0] * 4)
    for bad in (float("nan"), float("inf"), -float("inf"), 1.76 * 2.0 ** 127):
        rows.append([1.0, bad, 2.0])
    out = np.zeros((len(rows), d), dtype=np.float32)
    for i, r in enumerate(rows):
        out[i, 5:5 + len(r)] = r
        out[i, 40:40 + len(r)] = np.asarray(r[::-1], dtype=np.float32) * np.float32(1.0 if np.isnan(r).any() else 0.5)
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_append_of_special_values(d, dt):
    rows = torch.as_tensor(special_rows(d), device=DEV).to(dt)
    n = rows.shape[0]
    k, v = rows[:, None].contiguous(), rows.flip(0)[:, None].contiguous()
    cache = new_cache(2, 1, d, 32)
    pool = pool_of(cache)
    t = np.array([[1]], dtype=np.int32)
    msa.cache_append(cache, k, v, i32([0, n]), i32(t), i32([n]), n)
    with np.errstate(all="ignore"):
        R.append(pool, k.double().cpu().numpy(), v.double().cpu().numpy(), [0, n], t, [n])
    same_pool(cache, pool)
    for out_dt in (torch.float32, torch.bfloat16):
        got = msa.cache_read(cache, i32([0, n]), i32(t), i32([n]), n, n, dtype=out_dt)
        for x, want in zip(got, rows_of(pool, t, [n], [n])):
            np.testing.assert_array_equal(x.double().cpu().numpy(), want)   # NaN where the slot is
    assert binding().device_status() == 0


def test_tokens_one_by_one_are_those_appended_at_once():
    rng = np.random.default_rng(7)
    n, hkv, d, block = 150, 2, 128, 64
    t = tables([n], block, rng)
    a, b = new_cache(4, hkv, d, block), new_cache(4, hkv, d, block)
    k = torch.as_tensor(rng.normal(size=(n, hkv, d)) * np.exp2(np.arange(n) % 40 - 20)[:, None, None], device=DEV).float()
    v = torch.as_tensor(rng.normal(size=(n, hkv, d)), device=DEV).float()
    msa.cache_append(a, k, v, i32([0, n]), i32(t), i32([n]), n)
    for i in range(n):
        msa.cache_append(b, k[i:i + 1], v[i:i + 1], i32([0, 1]), i32(t), i32([i + 1]), 1)
    same_pool(b, pool_of(a))


def test_append_skips_what_cannot_be():
    cache = new_cache(3, 1, 64, 32)
    before = pool_of(cache)
    k = torch.ones((4, 1, 64), device=DEV)
    status = binding().device_status

    def call(cu, table, lens, most=4):
        msa.cache_append(cache, k, k, i32(cu), i32(table), i32(lens), most)
        torch.cuda.synchronize()

    call([0, 4], [[3]], [4])                 # no such page
    assert status() == 1
    call([0, 4], [[-1]], [4])
    assert status() == 1
    call([0, 4], [[0]], [33])                # longer than its table row
    assert status() == 1
    call([0, 4], [[0]], [3])                 # more rows than slots
    assert status() == 1
    call([0, 5], [[0]], [5])                 # rows past the last
    assert status() == 1
    call([0, 4], [[0]], [4], most=3)
    assert status() == 1
    call([2, 0], [[0]], [4])
    assert status() == 1
    same_pool(cache, before)
    call([0, 0], [[0]], [0])
    assert status() == 0
    same_pool(cache, before)


# -- attention ---------------------------------------------------------------

@pytest.fixture(params=["singles", "pairs"])
def either_form(request, monkeypatch):
    """Up to 8 rows in bf16 take a warp's chunks one by one or in pairs: pairs where
    there may be 96 chunks a CTA, as a table of many more columns allows."""
    if request.param == "singles":
        return
    call = msa.cache_attention

    def wide(q, cache, table, lens, **how):
        columns = -(-96 * 456 * 32 // (cache.block * cache.Hkv * q.shape[0]))
        more = torch.full((table.shape[0], max(0, columns - table.shape[1])), -1, dtype=torch.int32, device=DEV)
        return call(q, cache, torch.cat([table, more], dim=1), lens, **how)

    monkeypatch.setattr(msa, "cache_attention", wide)


def test_pairs_of_chunks_at_a_window():
    """Enough units for pairs although the window ends inside the long sequences."""
    hkv, d, window = 8, 128, 6000
    lens = [7001, 6010] + [0, 5, 70] * 10
    cache, pool, t = filled(lens, hkv, d, 64, seed=4)
    q = torch.randn((len(lens), 1, 16, d), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).bfloat16()
    ref = R.attention(pool, q.double().cpu().numpy(), t, lens, window, d ** -0.5)
    out, lse = msa.cache_attention(q, cache, i32(t), i32(lens), window=window)
    check_attention(out, lse, ref, d, True)


@pytest.mark.usefixtures("either_form")
@pytest.mark.parametrize("lens,T,hq,hkv,d,block,window,dtype", [
    ([1], 1, 1, 1, 64, 32, None, "bf16"),
    ([1], 1, 4, 1, 128, 32, None, "f32"),
    ([32], 1, 8, 1, 128, 32, None, "bf16"),
    ([33, 31], 1, 8, 2, 128, 32, None, "bf16"),
    ([257], 1, 5, 1, 64, 64, None, "bf16"),
    ([700, 3, 0, 128], 1, 8, 2, 128, 64, None, "bf16"),     # a padded batch
    ([700, 3, 0, 128], 1, 8, 2, 64, 128, None, "f32"),
    ([2047], 1, 4, 1, 64, 32, None, "f32"),
    ([3000], 1, 8, 1, 128, 64, None, "bf16"),
    ([3000], 1, 16, 1, 128, 256, None, "f32"),
    ([500, 41], 2, 16, 2, 128, 64, None, "bf16"),           # 16 rows
    ([500, 41], 4, 16, 2, 128, 64, None, "bf16"),           # 32 rows
    ([500, 41], 3, 24, 2, 128, 64, None, "bf16"),           # 36 rows: two tiles
    ([500, 41], 8, 16, 2, 64, 64, None, "f32"),             # 64 rows
    ([500, 41], 8, 40, 8, 64, 32, None, "bf16"),
    ([500, 2, 0], 4, 6, 3, 128, 32, None, "bf16"),          # rows before the first slot
    ([500, 2, 0], 4, 6, 3, 64, 32, None, "f32"),
    ([1000, 77], 1, 8, 2, 128, 64, 1, "bf16"),
    ([1000, 77], 1, 8, 2, 128, 64, 100, "bf16"),
    ([1000, 77], 4, 8, 2, 128, 64, 33, "bf16"),
    ([1000, 77], 5, 8, 2, 64, 256, 257, "f32"),
    ([1000, 77], 4, 8, 2, 128, 64, 5000, "f32"),
    ([7000, 6300, 12], 4, 8, 1, 128, 128, None, "bf16"),    # 32 rows together
    ([7000, 6300], 5, 8, 1, 64, 64, None, "bf16"),
    ([7000, 6300], 4, 8, 1, 128, 64, 6200, "bf16"),
])
def test_attention(lens, T, hq, hkv, d, block, window, dtype):
    cache, pool, t = filled(lens, hkv, d, block, seed=sum(lens) + T, extra=1, width=2)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn((len(lens), T, hq, d), generator=gen, device=DEV).to(dt)
    ref = R.attention(pool, q.double().cpu().numpy(), t, lens, window or 1 << 40, d ** -0.5)
    out, lse = msa.cache_attention(q, cache, i32(t), i32(lens), window=window)
    assert out.dtype == dt
    check_attention(out, lse, ref, d, dtype == "bf16")
    other = torch.float32 if dtype == "bf16" else torch.bfloat16
    out2, lse2 = msa.cache_attention(q, cache, i32(t), i32(lens), window=window, out_dtype=other)
    check_attention(out2, lse2, ref, d, dtype == "bf16")
    assert torch.equal(lse, lse2)
    same_pool(cache, pool)
    assert binding().device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_many_short_and_one_long_sequence(dtype):
    """More sequences than a CTA's threads, units cut anywhere."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, 200).tolist()
    lens[131] = 6000
    cache, pool, t = filled(lens, 1, 128, 32, seed=9)
    q = torch.as_tensor(rng.normal(size=(200, 1, 3, 128)), device=DEV).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    ref = R.attention(pool, q.double().cpu().numpy(), t, lens, 1 << 40, 0.3)
    out, lse = msa.cache_attention(q, cache, i32(t), i32(lens), scale=0.3)
    check_attention(out, lse, ref, 128, dtype == "bf16")


@pytest.mark.usefixtures("either_form")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_large_scores_and_queries_of_any_size(d, dtype):
    """Scores of some hundreds, queries from 2^-60 to 2^60."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cache, pool, t = filled([300, 65], 1, d, 64, seed=21, kscale=3.0)
    rng = np.random.default_rng(8)
    for size, scale in ((30.0, 1.0), (2.0 ** 60, 2.0 ** -58), (2.0 ** -60, 2.0 ** 61)):
        q = torch.as_tensor(rng.normal(size=(2, 1, 8, d)) * size, device=DEV).to(dt)
        ref = R.attention(pool, q.double().cpu().numpy(), t, [300, 65], 1 << 40, scale)
        out, lse = msa.cache_attention(q, cache, i32(t), i32([300, 65]), scale=scale, out_dtype=torch.float32)
        check_attention(out, lse, ref, d, dtype == "bf16")


@pytest.mark.usefixtures("either_form")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_far_apart_between_slots(dtype):
    """Slots whose values are 2^60 and more times others': where a large one draws
    no weight the small ones' sum stays, and keys of any size likewise."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n, d = 70, 64
    rng = np.random.default_rng(31)
    k = rng.normal(size=(n, 1, d)) * np.exp2(rng.integers(-40, 1, n))[:, None, None]
    v = rng.normal(size=(n, 1, d)) * np.exp2(rng.integers(-60, 60, n))[:, None, None]
    # slots 3 and 40: the largest values, and keys that are far off for query 0
    k[3], k[40] = -20.0, -20.0
    v[3], v[40] = 2.0 ** 80, -2.0 ** 70
    v[7] = 0.0
    cache = new_cache(4, 1, d, 32)
    t = np.array([[2, 0, 3]], dtype=np.int32)
    msa.cache_append(cache, torch.as_tensor(k, device=DEV).float(), torch.as_tensor(v, device=DEV).float(),
                     i32([0, n]), i32(t), i32([n]), n)
    pool = pool_of(cache)
    q = np.abs(rng.normal(size=(1, 1, 4, d)))
    q[0, 0, 1] *= -1
    q = torch.as_tensor(q, device=DEV).to(dt)
    for scale in (0.125, 0.01):
        ref = R.attention(pool, q.double().cpu().numpy(), t, [n], 1 << 40, scale)
        out, lse = msa.cache_attention(q, cache, i32(t), i32([n]), scale=scale, out_dtype=torch.float32)
        check_attention(out, lse, ref, d, dtype == "bf16")


@pytest.mark.usefixtures("either_form")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 3, 5])
def test_small_values_beside_zeros_of_large_slots(T, d, dtype):
    """Values of neighbouring slots 2^28 apart: a dim in which the large slots hold
    codes of 0 is the small ones' sum, to what their weights' halves leave."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n = 200
    rng = np.random.default_rng(T)
    k = rng.normal(size=(n, 1, d)) * 0.1
    v = rng.normal(size=(n, 1, d))
    v[::2] *= 2.0 ** 28
    t = np.array([[2, 0, 3, 1]], dtype=np.int32)
    cache = new_cache(4, 1, d, 64)
    msa.cache_append(cache, torch.as_tensor(k, device=DEV).float(), torch.as_tensor(v, device=DEV).float(),
                     i32([0, n]), i32(t), i32([n]), n)
    pool = pool_of(cache)
    q = torch.as_tensor(rng.normal(size=(1, T, 8, d)), device=DEV).to(dt)
    for window in (3, 8, 150):
        ref = R.attention(pool, q.double().cpu().numpy(), t, [n], window, 0.125)
        out, lse = msa.cache_attention(q, cache, i32(t), i32([n]), window=window, scale=0.125, out_dtype=torch.float32)
        check_attention(out, lse, ref, d, dtype == "bf16", apart=True)


@pytest.mark.usefixtures("either_form")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [4, 9, 14, 19, 22, 24, 26, 30])
def test_large_values_at_small_weights(dtype, shift):
    """Every third slot's values are 2^shift times the others', its weight 2^-shift:
    the sums of both are of one size, whatever a small weight's half holds."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n, d = 400, 128
    rng = np.random.default_rng(shift)
    k = rng.normal(size=(n, 1, d)) * 0.01
    k[:, 0, 0] = 0.0
    k[::3, 0, 0] = -4.0
    k[:, 0, 1] = rng.choice([0.0, 0.5, 1.0, 1.5, 2.0, 3.0], n)   # weights of many bits
    v = rng.normal(size=(n, 1, d))
    v[::3] *= 2.0 ** shift
    t = np.array([[3, 1, 6, 0, 4, 2, 5]], dtype=np.int32)
    cache = new_cache(7, 1, d, 64)
    msa.cache_append(cache, torch.as_tensor(k, device=DEV).float(), torch.as_tensor(v, device=DEV).float(),
                     i32([0, n]), i32(t), i32([n]), n)
    pool = pool_of(cache)
    q = rng.normal(size=(1, 1, 4, d)) * 0.01
    q[..., 0] = 1.0
    q[..., 1] = 0.1 + 0.01 * rng.normal(size=4)
    q = torch.as_tensor(q, device=DEV).to(dt)
    scale = shift * np.log(2.0) / 4
    for window in (1 << 40, 40):
        ref = R.attention(pool, q.double().cpu().numpy(), t, [n], window, scale)
        out, lse = msa.cache_attention(q, cache, i32(t), i32([n]), window=min(window, 10000), scale=scale, out_dtype=torch.float32)
        check_attention(out, lse, ref, d, dtype == "bf16")


@pytest.mark.usefixtures("either_form")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_groups_of_a_slot_far_apart(dtype):
    """Values of one group 2^22 times those of another, in every slot: the dims of
    the small one hold their own precision.  Keys likewise, the query's large dims
    against the small ones."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n, d = 200, 128
    rng = np.random.default_rng(12)
    apart = np.repeat([2.0 ** 20, 2.0 ** -2, 1.0, 2.0 ** 8], 32)
    k = rng.normal(size=(n, 1, d)) * apart / 2.0 ** 8
    v = rng.normal(size=(n, 1, d)) * apart
    cache = new_cache(8, 1, d, 32)
    t = rng.permutation(7)[None].astype(np.int32)
    msa.cache_append(cache, torch.as_tensor(k, device=DEV).float(), torch.as_tensor(v, device=DEV).float(),
                     i32([0, n]), i32(t), i32([n]), n)
    pool = pool_of(cache)
    q = torch.as_tensor(rng.normal(size=(1, 1, 4, d)) / apart, device=DEV).to(dt)
    ref = R.attention(pool, q.double().cpu().numpy(), t, [n], 1 << 40, 0.5)
    out, lse = msa.cache_attention(q, cache, i32(t), i32([n]), scale=0.5, out_dtype=torch.float32)
    check_attention(out, lse, ref, d, dtype == "bf16")


@pytest.mark.usefixtures("either_form")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_slots_reach_the_rows_that_attend_them_only(dtype):
    # rows that are not hit: values of a few units, out rounded to bf16 (2^-8) at
    # worst and weights to halves (2^-11); lse in fp32
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n, d, T = 80, 128, 4
    rng = np.random.default_rng(77)
    k, v = rng.normal(size=(2, n, 1, d)).astype(np.float32)
    q = torch.as_tensor(rng.normal(size=(1, T, 2, d)), device=DEV).to(dt)
    for where, at in (("k", 78), ("v", 78), ("v", 50), ("k", 10), ("v", 10)):
        kk, vv = k.copy(), v.copy()
        (kk if where == "k" else vv)[at, 0, 100] = np.nan
        cache = new_cache(4, 1, d, 32)
        t = np.array([[1, 3, 0]], dtype=np.int32)
        msa.cache_append(cache, torch.as_tensor(kk, device=DEV), torch.as_tensor(vv, device=DEV), i32([0, n]), i32(t),
                         i32([n]), n)
        pool = pool_of(cache)
        for window in (3, 40):
            out, lse = msa.cache_attention(q, cache, i32(t), i32([n]), window=window)
            o, l = out.float().cpu().numpy(), lse.cpu().numpy()
            with np.errstate(all="ignore"):
                ref = R.attention(pool, q.double().cpu().numpy(), t, [n], window, d ** -0.5)
            for row in range(T):
                p = n - T + row
                hit = p - window < at <= p
                if hit:
                    assert np.isnan(o[0, row]).all()
                    assert np.isnan(l[0, :, row]).all() == (where == "k")
                else:
                    assert np.abs(o[0, row] - ref[0][0, row]).max() < 0.02
                if not hit or where == "v":
                    assert np.abs(l[0, :, row] - ref[1][0, :, row]).max() < 1e-4


@pytest.mark.usefixtures("either_form")
def test_nan_slots_beside_the_largest_scales():
    """Scales next to NaN's byte, and slots that hold NaN among them."""
    n, d = 96, 64
    rng = np.random.default_rng(6)
    for kbig, vbig in ((True, False), (False, True)):
        k, v = rng.normal(size=(2, n, 1, d))
        (k if kbig else v)[:] *= 2.0 ** 123
        for where, at in (("k", 40), ("v", 70)):
            kk, vv = k.astype(np.float32), v.astype(np.float32)
            (kk if where == "k" else vv)[at, 0, 5] = np.inf
            cache = new_cache(4, 1, d, 32)
            t = np.array([[1, 3, 0]], dtype=np.int32)
            msa.cache_append(cache, torch.as_tensor(kk, device=DEV), torch.as_tensor(vv, device=DEV), i32([0, n]), i32(t),
                             i32([n]), n)
            q = torch.as_tensor(rng.normal(size=(1, 1, 2, d)) * (2.0 ** -123 if kbig else 1.0), device=DEV).float()
            out, lse = msa.cache_attention(q, cache, i32(t), i32([n]))
            assert torch.isnan(out).all()
            assert torch.isnan(lse).all() == (where == "k")
            short, _ = msa.cache_attention(q, cache, i32(t), i32([at]))
            assert torch.isfinite(short).all()


@pytest.mark.usefixtures("either_form")
def test_bad_pages_and_lengths():
    """A page that does not exist is not attended; a length that cannot be is clamped."""
    cache, pool, t = filled([100, 64], 1, 64, 32, seed=4, extra=2)
    q = torch.ones((2, 1, 2, 64), device=DEV)
    good = msa.cache_attention(q, cache, i32(t), i32([100, 64]))
    short = msa.cache_attention(q, cache, i32(t), i32([96, 64]))
    assert binding().device_status() == 0
    for page in (-1, cache.n_pages, 2 ** 31 - 1):
        bad = t.copy()
        bad[0, 3] = page     # holds the last four slots
        out, lse = msa.cache_attention(q, cache, i32(bad), i32([100, 64]))
        torch.cuda.synchronize()
        assert binding().device_status() == 1
        torch.testing.assert_close(lse, short[1], rtol=1e-6, atol=1e-6)
        torch.testing.assert_close(out[0], short[0][0], rtol=1e-5, atol=1e-5)
        torch.testing.assert_close(out[1], good[0][1], rtol=1e-5, atol=1e-5)
    for n in (-1, 129):
        out, lse = msa.cache_attention(q, cache, i32(t), i32([n, 64]))
        torch.cuda.synchronize()
        assert binding().device_status() == 1
        torch.testing.assert_close(out[1], good[0][1], rtol=1e-5, atol=1e-5)
    out, lse = msa.cache_attention(q, cache, i32(t), i32([0, 64]))
    assert not out[0].any() and torch.isneginf(lse[0]).all()


@pytest.mark.usefixtures("either_form")
def test_shared_prefix_pages():
    cache, pool, t = filled([128, 40], 2, 128, 64, seed=14, extra=2)
    t2 = np.array([[t[0, 0], t[0, 1]], [t[0, 0], t[1, 0]]], dtype=np.int32)
    lens = [128, 104]
    q = torch.randn((2, 2, 8, 128), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).bfloat16()
    ref = R.attention(pool, q.double().cpu().numpy(), t2, lens, 1 << 40, 0.1)
    out, lse = msa.cache_attention(q, cache, i32(t2), i32(lens), scale=0.1)
    check_attention(out, lse, ref, 128, True)


@pytest.mark.large
def test_codes_and_scales_past_32_bits():
    """Codes of K past 4 GB, scales past 2^31 values' worth of pages."""
    hkv, d, block = 8, 128, 256
    pages = 36000     # 131072 bytes of codes each
    cache = msa.KVCache4.empty(pages, hkv, d, block)
    assert cache.k_codes.numel() > 2 ** 32
    t = np.array([[pages - 1, 3, pages - 2], [17000, pages - 3, -1]], dtype=np.int32)
    lens = [700, 300]
    gen = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randn((1000, hkv, d), generator=gen, device=DEV).bfloat16()
    v = torch.randn((1000, hkv, d), generator=gen, device=DEV).bfloat16()
    cu = i32([0, 700, 1000])
    msa.cache_append(cache, k, v, cu, i32(t), i32(lens), 700)
    used = sorted(set(t.ravel().tolist()) - {-1})
    pool = {n: getattr(cache, n)[used].cpu().numpy() for n in NAMES}
    small = np.array([[used.index(p) if p >= 0 else -1 for p in row] for row in t], dtype=np.int32)
    want = rows_of(pool, small, lens, lens)
    ref_pool = {n: np.zeros_like(x) for n, x in pool.items()}
    R.append(ref_pool, k.double().cpu().numpy(), v.double().cpu().numpy(), [0, 700, 1000], small, lens)
    for x, got in zip(("k", "v"), msa.cache_read(cache, cu, i32(t), i32(lens), 1000, 700, dtype=torch.float32)):
        np.testing.assert_array_equal(got.double().cpu().numpy(), want["kv".index(x)])
    for b, n in enumerate(lens):
        for h in (0, hkv - 1):
            np.testing.assert_array_equal(R.held(pool, "k", small[b], h, n), R.held(ref_pool, "k", small[b], h, n))
    q = torch.randn((2, 1, 16, d), generator=gen, device=DEV).bfloat16()
    ref = R.attention(pool, q.double().cpu().numpy(), small, lens, 1 << 40, d ** -0.5)
    out, lse = msa.cache_attention(q, cache, i32(t), i32(lens))
    check_attention(out, lse, ref, d, True)


# -- reading back ------------------------------------------------------------

def eight_bit(lens, hkv, d, block, seed):
    """An 8-bit cache of random tokens; its table."""
    rng = np.random.default_rng(seed)
    t = tables(lens, block, rng, 1)
    cache = msa.KVCache.empty(int(t.max()) + 2, hkv, d, block)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    k = torch.randn((sum(lens), hkv, d), generator=gen, device=DEV)
    v = torch.randn((sum(lens), hkv, d), generator=gen, device=DEV) * 100
    msa.cache_append(cache, k, v, i32(starts(lens)), i32(t), i32(lens), max(lens))
    return cache, t


def eight_bit_rows(cache, t, lens, counts):
    out = []
    for codes, scale in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        val = codes.float().cpu().double().numpy() * scale.cpu().double().numpy()[..., None, None]
        per = []
        for b, (n, c) in enumerate(zip(lens, counts)):
            if c:
                pages = [t[b][j] for j in range(-(-n // cache.block))]
                per.append(val[pages].transpose(0, 2, 1, 3).reshape(-1, cache.Hkv, cache.d)[n - c:n])
        out.append(np.concatenate(per))
    return out


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lens,counts,hkv,d,block", [
    ([1], [1], 1, 64, 32),
    ([64], [1], 1, 128, 64),
    ([65, 0, 130], [65, 0, 130], 2, 128, 64),
    ([700, 33, 5], [300, 0, 5], 3, 64, 32),
    ([1000, 999], [999, 1], 8, 128, 256),
    ([17] * 50, list(range(17)) * 2 + [17] * 16, 5, 64, 128),
])
def test_read_gives_what_the_cache_stands_for(bits, lens, counts, hkv, d, block):
    if bits == 4:
        cache, pool, t = filled(lens, hkv, d, block, seed=sum(counts))
        want = rows_of(pool, t, lens, counts)
    else:
        cache, t = eight_bit(lens, hkv, d, block, seed=sum(counts))
        want = eight_bit_rows(cache, t, lens, counts)
    total, cu = sum(counts), starts(counts)
    for dt in (torch.float32, torch.bfloat16):
        got = msa.cache_read(cache, i32(cu), i32(t), i32(lens), total, max(counts), dtype=dt)
        for x, w in zip(got, want):
            assert x.shape == (total, hkv, d)
            # codes have few bits: bf16 holds them exactly, and fp32
            np.testing.assert_array_equal(x.double().cpu().numpy(), w)
    # rows of no sequence stay
    out = tuple(gfull((total + 9, hkv, d), 7.5) for _ in range(2))
    cu2 = cu + 4
    got = msa.cache_read(cache, i32(cu2), i32(t), i32(lens), total + 9, max(counts), dtype=torch.float32, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    for x, w in zip(out, want):
        y = x.double().cpu().numpy()
        assert (y[:4] == 7.5).all() and (y[4 + total:] == 7.5).all()
        np.testing.assert_array_equal(y[4:4 + total], w)
    assert binding().device_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
def test_read_of_bad_pages_and_sequences(bits):
    if bits == 4:
        cache, _, t = filled([100, 64], 2, 64, 32, seed=4)
    else:
        cache, t = eight_bit([100, 64], 2, 64, 32, seed=4)
    want = msa.cache_read(cache, i32([0, 100, 164]), i32(t), i32([100, 64]), 164, 100)
    bad = t.copy()
    bad[0, 1] = cache.n_pages
    got = msa.cache_read(cache, i32([0, 100, 164]), i32(bad), i32([100, 64]), 164, 100)
    torch.cuda.synchronize()
    assert binding().device_status() == 1
    for x, w in zip(got, want):
        assert not x[32:64].any()
        assert torch.equal(x[:32], w[:32]) and torch.equal(x[64:], w[64:])
    for cu, lens, most in (([0, 101, 164], [100, 64], 101), ([0, 100, 165], [100, 64], 100), ([0, 100, 164], [129, 64], 100),
                           ([0, 100, 164], [100, 64], 99), ([-1, 64, 164], [100, 64], 100)):
        out = tuple(gfull((164, 2, 64), 3.0) for _ in range(2))
        msa.cache_read(cache, i32(cu), i32(t), i32(lens), 164, most, dtype=torch.float32, out=out)
        torch.cuda.synchronize()
        assert binding().device_status() == 1
        check_guards()


def test_read_of_nothing():
    cache, _, t = filled([5], 1, 64, 32, seed=4)
    k, v = msa.cache_read(cache, i32([0, 0]), i32(t), i32([5]), 0, 0)
    assert k.shape == (0, 1, 64) and v.shape == (0, 1, 64)


def test_poisoned_blocks_of_the_8_bit_cache_read_as_nan():
    cache, t = eight_bit([32], 1, 64, 32, seed=3)
    bad = torch.full((1, 1, 64), float("inf"), device=DEV)
    msa.cache_append(cache, bad, torch.ones_like(bad), i32([0, 1]), i32(t), i32([32]), 1)
    k, v = msa.cache_read(cache, i32([0, 32]), i32(t), i32([32]), 32, 32)
    assert torch.isnan(k).all() and torch.isfinite(v).all()


# -- together, streams, graphs, threads, refusals ----------------------------

def test_a_cached_prefix_in_the_prefill():
    """A prefix written to the cache, read back and attended with what follows
    it: the same as the prefill over the values that the cache stands for."""
    n, hq, hkv, d = 512, 8, 2, 128
    gen = torch.Generator(device=DEV).manual_seed(5)
    q = torch.randn((n, hq, d), generator=gen, device=DEV).bfloat16()
    k = torch.randn((n, hkv, d), generator=gen, device=DEV).bfloat16()
    v = torch.randn((n, hkv, d), generator=gen, device=DEV).bfloat16()
    t = tables([n], 64, np.random.default_rng(1))
    cache = new_cache(9, hkv, d, 64)
    msa.cache_append(cache, k, v, i32([0, n]), i32(t), i32([n]), n)
    kr, vr = msa.cache_read(cache, i32([0, n]), i32(t), i32([n]), n, n)
    out, lse = msa.msa_attention(q, kr, vr, window=n, n_landmarks=0, out_dtype=torch.float32)
    want = [torch.as_tensor(x, device=DEV).bfloat16() for x in rows_of(pool_of(cache), t, [n], [n])]
    assert torch.equal(kr, want[0]) and torch.equal(vr, want[1])
    # the last token, attended over the cache itself
    o1, l1 = msa.cache_attention(q[None, -1:], cache, i32(t), i32([n]), out_dtype=torch.float32)
    # both round their weights to halves or bf16 (2^-9 of sums of |v| p <= max |v|)
    assert (o1[0, 0] - out[-1]).abs().max() <= 2 * 2.0 ** -9 * vr.abs().max()
    assert (l1[0, :, 0] - lse[:, -1]).abs().max() < 1e-3


def test_a_captured_step_replays_with_new_tokens_and_lengths():
    hkv, d, block, hq = 2, 128, 64, 8
    B = 3
    t = tables([200, 200, 200], block, np.random.default_rng(2))
    cache, eager = new_cache(15, hkv, d, block), new_cache(15, hkv, d, block)
    gen = torch.Generator(device=DEV).manual_seed(5)
    k0 = torch.randn((300, hkv, d), generator=gen, device=DEV).bfloat16()
    for c in (cache, eager):
        msa.cache_append(c, k0, k0 * 0.5, i32([0, 100, 200, 300]), i32(t), i32([100, 100, 100]), 100)
    k = torch.zeros((B, hkv, d), device=DEV, dtype=torch.bfloat16)
    v, q = torch.zeros_like(k), torch.zeros((B, 1, hq, d), device=DEV, dtype=torch.bfloat16)
    lens, cu, table = i32([101, 101, 101]), i32([0, 1, 2, 3]), i32(t)

    def step(c):
        msa.cache_append(c, k, v, cu, table, lens, 1)
        out = msa.cache_attention(q, c, table, lens)
        return (*out, *msa.cache_read(c, cu, table, lens, B, 1))

    step(eager)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(cache)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(cache)
    for i in range(40):
        k.normal_(generator=gen)
        v.normal_(generator=gen)
        q.normal_(generator=gen)
        lens.copy_(i32([101 + i, 102 + 2 * i, 101 if i < 20 else 0]))
        cu.copy_(i32([0, 1, 2, 3 if i < 20 else 2]))
        g.replay()
        want = step(eager)
        live = 3 if i < 20 else 2
        # (sequence 1 steps over slots that nothing wrote: NaN in both)
        for a, b in zip(outs[:2], want[:2]):
            assert torch.equal(a.nan_to_num(7.5), b.nan_to_num(7.5))
        for a, b in zip(outs[2:], want[2:]):
            assert torch.equal(a[:live], b[:live])
    same_pool(cache, pool_of(eager))


def test_calls_on_another_stream_see_its_tensors():
    hkv, d, block = 1, 64, 32
    s = torch.cuda.Stream()
    t = i32([[0, 1]])
    cache = new_cache(2, hkv, d, block)
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        k = torch.ones((40, hkv, d), device=DEV)
    lens, cu = i32([40]), i32([0, 40])
    q = torch.ones((1, 1, 1, d), device=DEV)
    torch.cuda.current_stream().synchronize()
    msa.cache_append(cache, k, k, cu, t, lens, 40, stream=s)
    out, lse = msa.cache_attention(q, cache, t, lens, stream=s)
    kr, vr = msa.cache_read(cache, cu, t, lens, 40, 40, dtype=torch.float32, stream=s)
    s.synchronize()
    assert (kr == 1).all() and (vr == 1).all()
    assert (out - 1).abs().max() < 1e-5


def test_two_host_threads():
    """Calls of two threads, each on its own stream and cache, do not fail or
    change each other's results."""
    lens = [300, 17]
    caches = [filled(lens, 2, 128, 64, seed=s) for s in (1, 2)]
    torch.cuda.synchronize()
    qs = [torch.randn((2, T, 8, 128), generator=torch.Generator(device=DEV).manual_seed(T), device=DEV).bfloat16()
          for T in (1, 4)]
    tl = [i32(c[2]) for c in caches]
    ln = i32(lens)
    cu = i32([0, 300, 317])
    want = [msa.cache_attention(q, c[0], t, ln) for q, c, t in zip(qs, caches, tl)]
    reads = [msa.cache_read(c[0], cu, t, ln, 317, 300) for c, t in zip(caches, tl)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(200):
                out, lse = msa.cache_attention(qs[i], caches[i][0], tl[i], ln, stream=s)
                k, v = msa.cache_read(caches[i][0], cu, tl[i], ln, 317, 300, stream=s)
                s.synchronize()
                if not (torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]) and torch.equal(k, reads[i][0])
                        and torch.equal(v, reads[i][1])):
                    bad.append((i, "differs"))
                    return
        except Exception as e:  # noqa: BLE001
            bad.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not bad, bad


def test_the_same_call_gives_the_same_bits():
    cache, _, t = filled([5000, 1200, 64], 2, 128, 64, seed=8)
    q = torch.randn((3, 4, 16, 128), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).bfloat16()
    first = msa.cache_attention(q, cache, i32(t), i32([5000, 1200, 64]))
    for _ in range(5):
        again = msa.cache_attention(q, cache, i32(t), i32([5000, 1200, 64]))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_output_buffers_are_not_overrun():
    cache, pool, t = filled([130], 1, 64, 32, seed=8)
    B = binding()
    for T, hq, dt in ((1, 1, torch.bfloat16), (3, 5, torch.bfloat16), (3, 5, torch.float32)):
        q = torch.ones((1, T, hq, 64), device=DEV, dtype=dt)
        out, lse = gempty((1, T, hq, 64), dt), gempty((1, hq, T))
        ws = gempty((B.cache4_attn_workspace_size(cache.ref, t.shape[1], 1, T, hq, dt),), torch.uint8)
        B.cache4_attn(cache.ref, q, i32(t), i32([130]), 1 << 30, 0.125, out, lse, ws)
        torch.cuda.synchronize()
        check_guards()


def test_refusals():
    cache, _, t = filled([40], 2, 64, 32, seed=8)
    eight, _ = eight_bit([40], 2, 64, 32, seed=8)
    table, lens = i32(t), i32([40])
    q = torch.ones((1, 1, 4, 64), device=DEV)
    w = torch.zeros((1, 2, 64), device=DEV)
    with pytest.raises(TypeError, match="KVCache"):
        msa.cache_attention(q, cache, table, lens, weights=w)
    with pytest.raises(TypeError, match="KVCache"):
        msa.cache_block_select(q, cache, table, lens, 8, 1)
    with pytest.raises(TypeError, match="KVCache"):
        msa.cache_topk_attention(q, cache, table, lens, 8, 1)
    with pytest.raises(TypeError, match="KVCache"):
        msa.cache_select_attention(q, cache, table, lens, 8, i32(np.zeros((1, 1, 2, 1))), i32(np.zeros((1, 1, 2))))
    with pytest.raises(TypeError, match="KVCache"):
        msa.cache_evict(cache, table, lens, w, i32([[1]]), 8, 2)
    with pytest.raises(ValueError):
        msa.cache_attention(q[..., :32].contiguous(), cache, table, lens)
    with pytest.raises(TypeError):
        msa.cache_attention(q.half(), cache, table, lens)
    with pytest.raises(ValueError):
        msa.cache_attention(q.cpu(), cache, table, lens)
    with pytest.raises(TypeError):
        msa.cache_attention(q, cache, table.long(), lens)
    with pytest.raises(binding().MsaError):
        msa.cache_attention(q, cache, table, lens, window=0)
    with pytest.raises(binding().MsaError):
        msa.cache_attention(q, cache, table, lens, scale=float("nan"))
    with pytest.raises(binding().MsaError):   # one head on two KV heads
        msa.cache_attention(q.transpose(1, 2), cache, table, lens)
    for c in (cache, eight):
        with pytest.raises(TypeError):
            msa.cache_read(c, i32([0, 40]), table, lens, 40, 40, dtype=torch.float16)
        with pytest.raises(ValueError):
            msa.cache_read(c, i32([0]), table, lens, 40, 40)
        with pytest.raises(binding().MsaError):
            msa.cache_read(c, i32([0, 40]), table, lens, 40, 41)
        out = torch.zeros((40, 2, 64), device=DEV)
        with pytest.raises(ValueError):
            msa.cache_read(c, i32([0, 40]), table, lens, 40, 40, dtype=torch.float32, out=(out, out))
        with pytest.raises(TypeError):
            msa.cache_read(c, i32([0, 40]), table, lens, 40, 40, out=(out, out.clone()))
        with pytest.raises(ValueError):
            msa.cache_read(c, i32([0, 40]), table, lens, 39, 39, dtype=torch.float32, out=(out, out.clone()))
    with pytest.raises(ValueError):
        msa.KVCache4(cache.k_codes, cache.v_codes, cache.k_scale[..., :1], cache.v_scale)
    with pytest.raises(TypeError):
        msa.KVCache4(cache.k_codes.view(torch.int8), cache.v_codes, cache.k_scale, cache.v_scale)
    with pytest.raises(ValueError):
        msa.KVCache4(cache.k_codes.transpose(0, 1), cache.v_codes.transpose(0, 1), cache.k_scale.transpose(0, 1),
                     cache.v_scale.transpose(0, 1))
    bad = msa.KVCache4(torch.zeros((2, 1, 48, 32), dtype=torch.uint8, device=DEV), torch.zeros((2, 1, 48, 32), dtype=torch.uint8, device=DEV),
                       torch.zeros((2, 1, 48, 2), dtype=torch.uint8, device=DEV), torch.zeros((2, 1, 48, 2), dtype=torch.uint8, device=DEV))
    with pytest.raises(binding().MsaError):
        msa.cache_attention(torch.ones((1, 1, 1, 64), device=DEV), bad, table, lens)


def test_a_read_refuses_outputs_that_overlap():
    n, hkv, d = 64, 2, 64
    cache, _, t = filled([n], hkv, d, 32, seed=3)
    buf = torch.zeros((2 * n * hkv * d,), device=DEV)

    def read(k, v):
        return msa.cache_read(cache, i32([0, n]), i32(t), i32([n]), n, n, dtype=torch.float32, out=(k, v))

    def at(i):
        return buf[i:i + n * hkv * d].view(n, hkv, d)

    for a, b in ((0, 0), (0, d), (d, 0), (0, n * hkv * d - 4), (n * hkv * d - 4, 0)):
        with pytest.raises(ValueError):
            read(at(a), at(b))
    k, v = msa.cache_read(cache, i32([0, n]), i32(t), i32([n]), n, n, dtype=torch.float32)
    read(at(n * hkv * d), at(0))   # side by side
    assert torch.equal(at(n * hkv * d), k) and torch.equal(at(0), v)


# -- long ranges a warp ------------------------------------------------------
# Lookups of pages are 32 of a warp's steps ahead; a stage of its ring is filled
# again after 2 to 8 steps.  The cases below give a warp 40 steps and more (the form
# that takes chunks one by one in bf16 has at most 24: from 96 chunks a CTA on it is
# the pairs').  CTAs: 3 an SM where a tile is 8 rows, or 16 in bf16, else 2.

def random_pool(pages, hkv, d, block, gen):
    """A pool of random codes: keys of 2^-6 to 2^-2 (scores of a third of a unit), values of
    2^-6 to 2^5, alike within a page and head.  Then, at random, one slot in 160: a key
    of 6 * 2^-1 in its first 32 dims, which queries of ones there weigh e^9; one in
    1500: zeros of a large scale, which move K's or V's references or fit none; one in
    2000: all zeros with the least scale, as appends write them, which fit none."""
    shape = (pages, hkv, block)
    codes = [torch.randint(0, 256, (*shape, d // 2), generator=gen, device=DEV, dtype=torch.uint8) for _ in range(2)]
    scale = [torch.randint(*span, (pages, hkv, 1, 1), generator=gen, device=DEV).expand(*shape, d // 32)
             .to(torch.uint8).contiguous() for span in ((121, 126), (121, 133))]

    def some(one_in):
        return torch.randint(0, one_in, shape, generator=gen, device=DEV) == 0

    heavy = some(160)
    codes[0][..., :16][heavy] = 0x77
    scale[0][..., 0][heavy] = 126
    for x, least in ((0, 143), (1, 130)):
        at = some(1500) & ~heavy
        codes[x][..., 16:32][at] = 0
        scale[x][..., 1][at] = torch.randint(least, least + 7, (int(at.sum()),), generator=gen, device=DEV).to(torch.uint8)
    at = some(2000) & ~heavy
    for x in range(2):
        codes[x][at] = 0
        scale[x][at] = 1
    return msa.KVCache4(*codes, *scale)


def dense_attention(cache, q, table, lens, window, scale):
    """R.attention's results (and the same besides) on the GPU, in 64 bits; slots of
    pages that do not exist are not attended."""
    steps = torch.as_tensor(np.concatenate([R.E2M1, -R.E2M1]), device=DEV)
    B, T, hq, d = q.shape
    hkv, block = cache.Hkv, cache.block
    g = hq // hkv
    out, absv = (torch.zeros((B, T, hq, d), dtype=torch.float64, device=DEV) for _ in range(2))
    lse = torch.full((B, hq, T), -np.inf, dtype=torch.float64, device=DEV)
    s1, count, top, unit = (torch.zeros((B, T, hq), dtype=torch.float64, device=DEV) for _ in range(4))
    q = q.double()

    def values(x, pages, h, n):
        c = getattr(cache, x + "_codes")[pages, h].reshape(-1, d // 2)[:n].int()
        e = getattr(cache, x + "_scale")[pages, h].reshape(-1, d // 32)[:n].double() - 127
        val = torch.stack([steps[c & 15], steps[c >> 4]], dim=-1).reshape(n, d)
        return val * torch.exp2(e).repeat_interleave(32, dim=-1)

    for b, n in enumerate(lens):
        if n == 0:
            continue
        pages = torch.as_tensor(table[b][:-(-n // block)].astype(np.int64), device=DEV)
        slot = torch.arange(n, device=DEV)
        there = (pages >= 0).repeat_interleave(block)[:n]
        for h in range(hkv):
            k, v = (values(x, pages.clamp(min=0), h, n) for x in ("k", "v"))
            size = v.abs().amax(dim=1)
            for t in range(T):
                p = n - T + t
                may = there & (slot <= p) & (slot > p - window)
                if not may.any():
                    continue
                rows = slice(h * g, (h + 1) * g)
                row = q[b, t, rows]
                s = torch.where(may, row @ k.T * scale, -np.inf)
                w = torch.softmax(s, dim=-1)
                out[b, t, rows], absv[b, t, rows] = w @ v, w @ v.abs()
                lse[b, rows, t] = torch.logsumexp(s, dim=-1)
                s1[b, t, rows] = torch.where(may, row.abs() @ k.abs().T * scale, 0.0).amax(dim=-1)
                count[b, t, rows] = may.sum()
                top[b, t, rows] = (w * size).amax(dim=-1)
                most = torch.where(may, size, 0.0).amax()
                unit[b, t, rows] = torch.minimum(2.0 ** 5 * w.amax(dim=-1) * most, 2.0 ** 13 * top[b, t, rows])
    return tuple(x.cpu().numpy() for x in (out, lse, absv, s1, count, top, unit))


def check_long(out, lse, ref, d, bf16_in, steps):
    """``bounds`` with the sums as they are made: a warp's chain of `steps` MMAs of 16
    slots (17 terms each, fp32), the lanes', warps' and parts' joins below 100 steps,
    not one step a slot; and the subnormal halves of slots whose scales lie apart."""
    out64, lse64, absv, s1, count, top, unit = ref
    ds = ((d + 8) * 2.0 ** -23 + (0.0 if bf16_in else 2.0 ** -22)) * s1
    chain = (17 * steps + 100) * 2.0 ** -23
    rel = 2 * ds + 2.0 ** -21 + 2.0 ** -19 + chain + (2.0 ** -11 if bf16_in else 2.0 ** -22)
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    small = (count * np.maximum(unit * 2.0 ** -33, top * 2.0 ** -38))[..., None]
    tol_o = (absv * rel[..., None] + small) * (1 + half) + np.abs(out64) * half
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(l), np.isneginf(lse64))
    fin = np.isfinite(lse64)
    err = np.abs(o - out64)
    assert (err <= tol_o).all(), f"out: worst {np.max(err / np.maximum(tol_o, 1e-300)):.3g} of the bound"
    tol_l = (ds + 2.0 ** -20 + chain).transpose(0, 2, 1) + np.abs(np.where(fin, lse64, 0)) * 2.0 ** -22
    err = np.abs(l - np.where(fin, lse64, 0))[fin]
    assert (err <= tol_l[fin]).all(), f"lse: worst {np.max(err / tol_l[fin]):.3g} of the bound"
    # of some 300 heavy slots one weighs more than the bounds let pass
    assert np.median(tol_l[fin]) < 2.0 ** -9


LONG = [
    # sequences, their length, T, query heads on 8, d, block, dtype, chunks a warp's step
    (9, 68000, 1, 64, 128, 64, "bf16", 2),     # 8 rows, pairs
    (9, 68000, 1, 40, 64, 32, "bf16", 2),
    (6, 26000, 1, 64, 128, 128, "bf16", 1),    # 8 rows, one by one
    (6, 26001, 1, 64, 64, 64, "bf16", 1),
    (7, 46000, 2, 64, 128, 64, "bf16", 1),     # 16 rows
    (7, 46000, 1, 128, 64, 256, "bf16", 1),
    (5, 46000, 4, 64, 128, 64, "bf16", 1),     # 32 rows
    (5, 46000, 3, 64, 64, 32, "bf16", 1),      # 24 rows of 32
    (7, 46000, 1, 64, 128, 32, "f32", 1),      # 8 rows of two halves
    (7, 46000, 1, 32, 64, 64, "f32", 1),
    (5, 46000, 2, 64, 128, 64, "f32", 1),      # 16 rows
    (5, 46000, 3, 64, 64, 128, "f32", 1),      # 24: two tiles
]


@pytest.mark.parametrize("missing", [False, True])
@pytest.mark.parametrize("batch,n,T,hq,d,block,dtype,pair", LONG)
def test_ranges_of_many_steps_a_warp(batch, n, T, hq, d, block, dtype, pair, missing):
    hkv = 8
    rng = np.random.default_rng(batch * n + T)
    gen = torch.Generator(device=DEV).manual_seed(n + T + d)
    lens = [n - int(x) for x in rng.integers(0, 2000, batch)]
    table = tables(lens, block, rng, 1)
    cache = random_pool(int(table.max()) + 2, hkv, d, block, gen)
    if missing:  # one page in 50, anywhere, and of one sequence a run of them
        table[rng.random(table.shape) < 0.02] = -1
        table[1, 100:100 + 4000 // block] = cache.n_pages + 7
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = torch.randn((batch, T, hq, d), generator=gen, device=DEV)
    q[..., :32] = 1 + 0.1 * q[..., :32]
    q = q.to(dt)
    scale = 9 / 96
    rows = T * hq // hkv
    tile = 8 if rows <= 8 else 16 if rows <= 16 or dtype == "f32" else 32
    ctas = 152 * (3 if tile == 8 or (tile == 16 and dtype == "bf16") else 2)
    chunks = sum(-(-x // 32) for x in lens) * hkv * -(-rows // tile)
    wide = batch * hkv * -(-rows // tile) * (table.shape[1] * block // 32)
    if tile == 8 and dtype == "bf16":
        assert (wide >= 96 * ctas) == (pair == 2)
    steps = chunks / ctas / 4 / pair
    assert steps >= (40 if (tile, dtype, pair) != (8, "bf16", 1) else 18)
    out, lse = msa.cache_attention(q, cache, i32(table), i32(lens), scale=scale, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert binding().device_status() == (1 if missing else 0)
    there = np.where(table < cache.n_pages, table, -1)
    ref = dense_attention(cache, q, there, lens, 1 << 40, scale)
    check_long(out, lse, ref, d, dtype == "bf16", 2 * pair * (steps + 2) * (1 if dtype == "bf16" else 2))


# -- pairs of chunks at windows ----------------------------------------------

@pytest.fixture
def padded_for_pairs(monkeypatch):
    """Calls with so many empty sequences behind their own that a window of few
    slots, too, has 96 chunks a CTA by what the launch knows."""
    call = msa.cache_attention

    def padded(q, cache, table, lens, window=None, **how):
        assert q.dtype == torch.bfloat16 and q.shape[1] * q.shape[2] <= 8 * cache.Hkv
        width = table.shape[1] * cache.block
        slots = min(width if window is None else window + q.shape[1], width)
        b = q.shape[0]
        more = -(-96 * 456 // (slots // 32 * cache.Hkv)) - b
        assert 0 < more + b <= 65535
        q = torch.cat([q, q.new_ones((more, *q.shape[1:]))])
        table = torch.cat([table, table.new_full((more, table.shape[1]), -1)])
        lens = torch.cat([lens, lens.new_zeros((more,))])
        out, lse = call(q, cache, table, lens, window=window, **how)
        assert not out[b:].any() and torch.isneginf(lse[b:]).all()
        return out[:b], lse[:b]

    monkeypatch.setattr(msa, "cache_attention", padded)


@pytest.mark.usefixtures("padded_for_pairs")
@pytest.mark.parametrize("lens,T,hq,hkv,d,block,window", [
    ([1000, 77], 1, 8, 2, 128, 64, 100),
    ([1000, 77], 2, 8, 2, 128, 64, 33),
    ([1000, 77], 4, 4, 2, 64, 256, 257),
    ([513, 0, 3, 64], 3, 4, 2, 128, 32, 31),
    ([513, 0, 3, 64], 8, 2, 2, 64, 32, 64),
])
def test_pairs_of_chunks_at_small_windows(lens, T, hq, hkv, d, block, window):
    cache, pool, t = filled(lens, hkv, d, block, seed=sum(lens) + T, extra=1, width=2)
    q = torch.randn((len(lens), T, hq, d), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).bfloat16()
    ref = R.attention(pool, q.double().cpu().numpy(), t, lens, window, d ** -0.5)
    out, lse = msa.cache_attention(q, cache, i32(t), i32(lens), window=window)
    check_attention(out, lse, ref, d, True)


@pytest.mark.usefixtures("padded_for_pairs")
@pytest.mark.parametrize("shift", [4, 14, 22, 24, 26, 30])
def test_pairs_with_large_values_at_small_weights(shift):
    test_large_values_at_small_weights("bf16", shift)


@pytest.mark.usefixtures("padded_for_pairs")
@pytest.mark.parametrize("window", [32, 40, 45, 64])
@pytest.mark.parametrize("where,at", [("k", 79), ("v", 78), ("v", 40), ("k", 39), ("v", 39), ("v", 35), ("k", 10), ("v", 10)])
def test_pairs_with_nan_slots_at_a_windows_edges(where, at, window):
    """A row is NaN if it attends the slot, and what it is without the slot if not
    (its softmax's references may be other ones: within the bounds)."""
    n, d, T = 80, 128, 4
    rng = np.random.default_rng(77)
    k, v = rng.normal(size=(2, n, 1, d)).astype(np.float32)
    q = torch.as_tensor(rng.normal(size=(1, T, 2, d)), device=DEV).bfloat16()
    t = np.array([[1, 3, 0]], dtype=np.int32)

    def pooled(x, y):
        cache = new_cache(4, 1, d, 32)
        msa.cache_append(cache, torch.as_tensor(x, device=DEV), torch.as_tensor(y, device=DEV), i32([0, n]), i32(t), i32([n]), n)
        return cache

    ref = R.attention(pool_of(pooled(k, v)), q.double().cpu().numpy(), t, [n], window, d ** -0.5)
    (k if where == "k" else v)[at, 0, 100] = np.nan
    out, lse = msa.cache_attention(q, pooled(k, v), i32(t), i32([n]), window=window)
    hit = [row for row in range(T) if n - T + row - window < at <= n - T + row]
    assert torch.isnan(out[0, hit]).all()
    assert torch.isnan(lse[0, :, hit]).all() if where == "k" else torch.isfinite(lse).all()
    rows = [row for row in range(T) if row not in hit]
    if rows:
        check_attention(out[:, rows], lse[:, :, rows], tuple(x[:, :, rows] if i == 1 else x[:, rows] for i, x in enumerate(ref)), d, True)
