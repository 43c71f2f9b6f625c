"""The 64-bit reference of the 8-bit KV cache against independent statements
of the same things (no GPU needed): torch's e4m3 conversion, a brute-force
softmax, one append against many."""
import math

import numpy as np
import pytest
import torch

from tests import cache_ref as R


def _pool(pages, hkv, block, d):
    return {"k_codes": np.zeros((pages, hkv, block, d)), "v_codes": np.zeros((pages, hkv, block, d)),
            "k_scale": np.zeros((pages, hkv)), "v_scale": np.zeros((pages, hkv)),
            "k_mean": np.zeros((pages, hkv, d))}


def test_rounding_is_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=5000) * 10.0 ** rng.uniform(-4, 2, 5000), R.E4M3, -R.E4M3,
                        (R.E4M3[1:] + R.E4M3[:-1]) / 2])  # every tie
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(R.round_e4m3(x.astype(np.float64)), want)


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (449.0, 1), (1.75, -8), (1.7500001, -7),
                                    (2.0 ** -140, -126), (3e38, 120)])
def test_scale_is_the_least_power_of_two(amax, e):
    assert R.scale_of_block(np.array([[amax, -amax / 3]])) == 2.0 ** e


def test_scale_of_zeros_and_of_what_is_not_finite():
    assert R.scale_of_block(np.zeros((4, 8))) == 0.0
    assert math.isnan(R.scale_of_block(np.array([1.0, np.inf])))
    assert math.isnan(R.scale_of_block(np.array([1.0, np.nan])))


def test_bf16_rounding_is_torchs():
    x = np.random.default_rng(1).normal(size=4000).astype(np.float32)
    x = np.concatenate([x, x * np.float32(2.0 ** -128), [0.0, 2.0 ** -138, 3e38]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    np.testing.assert_array_equal(R.round_bf16(x), want)


def test_append_one_by_one_is_append_at_once():
    """Power-of-two scales: the order of arrival leaves no trace while no code
    is subnormal."""
    rng = np.random.default_rng(2)
    k = rng.uniform(0.25, 4.0, size=(70, 2, 8)) * rng.choice([-1, 1], size=(70, 2, 8))
    once, step = _pool(4, 2, 32, 8), _pool(4, 2, 32, 8)
    table = [[3, 0, 2]]
    R.append(once, k, 2 * k, [0, 70], table, [70])
    for i in range(70):
        R.append(step, k[i:i + 1], 2 * k[i:i + 1], [0, 1], table, [i + 1])
    for name in once:
        np.testing.assert_array_equal(once[name], step[name], err_msg=name)


def test_attention_is_a_softmax_over_the_window():
    rng = np.random.default_rng(3)
    pool = _pool(3, 1, 32, 8)
    k, v = rng.normal(size=(2, 50, 1, 8))
    R.append(pool, k, v, [0, 50], [[2, 1]], [50])
    q = rng.normal(size=(1, 2, 2, 8))
    out, lse, *_ , w = R.attention(pool, q, [[2, 1]], [50], 10, 0.5)
    kk, vv = R.held(pool, "k", [2, 1], 0, 50), R.held(pool, "v", [2, 1], 0, 50)
    for t in range(2):
        at = slice(39 + t, 49 + t)
        for h in range(2):
            e = np.exp(kk[at] @ q[0, t, h] * 0.5)
            np.testing.assert_allclose(out[0, t, h], e @ vv[at] / e.sum(), rtol=1e-12)
            np.testing.assert_allclose(lse[0, h, t], np.log(e.sum()), rtol=1e-12)
    assert abs(w.sum() - 4) < 1e-12


def test_evict_keeps_the_heaviest_and_the_last():
    rng = np.random.default_rng(4)
    pool = _pool(6, 1, 32, 4)
    k = rng.normal(size=(60, 1, 4))
    R.append(pool, k, k, [0, 60], [[0, 1]], [60])
    w = np.zeros((1, 1, 64))
    w[0, 0, [5, 7, 30]] = [1.0, 3.0, 2.0]
    before = R.held(pool, "k", [0, 1], 0, 60).copy()
    lens, kept, kw = R.evict(pool, [[0, 1]], [60], w, [[4]], 8, 4)
    assert lens == [8] and kept[0][0].tolist() == [0, 5, 7, 30, 56, 57, 58, 59]
    got = R.held(pool, "k", [4], 0, 8)
    s = pool["k_scale"][4, 0]
    assert np.abs(got - before[kept[0][0]]).max() <= s * 2.0 ** -10  # half a subnormal step
