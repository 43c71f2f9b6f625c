"""Host-side checks of the 4-bit KV cache's, the read's and the norm and rotation's
C ABI (no GPU needed): bad arguments are refused with the documented status
before anything touches the GPU."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import long_context_sparse_landmark_gb300 as msa
from tests import cache4_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from long_context_sparse_landmark_gb300 import build
    path = build.build()
    from long_context_sparse_landmark_gb300 import _binding
    return _binding.load_library(path)


GOOD = 1 << 20        # never dereferenced: validation fails first
INVALID, UNSUPPORTED = 1, 2
FIELDS = ("k_codes", "v_codes", "k_scale", "v_scale", "k_mean", "n_pages", "Hkv", "d", "block")


def cache(bits, **kw):
    from long_context_sparse_landmark_gb300 import _binding
    a = dict(k_codes=GOOD, v_codes=GOOD, k_scale=GOOD, v_scale=GOOD, k_mean=GOOD, n_pages=10, Hkv=2, d=128, block=64)
    a.update(kw)
    s = _binding.KvCache4Struct if bits == 4 else _binding.KvCacheStruct
    return ctypes.byref(s(*[a[n] for n, _ in s._fields_]))


def split(kw, bits):
    c = {k: kw.pop(k) for k in list(kw) if k in FIELDS}
    return None if kw.pop("cache", 1) is None else cache(bits, **c)


def append(lib, **kw):
    c = split(kw, 4)
    a = dict(k=GOOD, v=GOOD, cu=GOOD, total=8, most=8, table=GOOD, nb=4, lens=GOOD, batch=1, dt=1)
    a.update(kw)
    return lib.msa_cache4_append(c, a["k"], a["v"], a["cu"], a["total"], a["most"], a["table"], a["nb"], a["lens"],
                                 a["batch"], a["dt"], None)


def attn(lib, **kw):
    c = split(kw, 4)
    a = dict(q=GOOD, table=GOOD, nb=4, lens=GOOD, batch=1, n_q=1, Hq=8, window=16, scale=0.1, out=GOOD, lse=GOOD,
             idt=1, odt=1, ws=GOOD, bytes=1 << 40)
    a.update(kw)
    return lib.msa_cache4_attn(c, a["q"], a["table"], a["nb"], a["lens"], a["batch"], a["n_q"], a["Hq"], a["window"],
                               a["scale"], a["out"], a["lse"], a["idt"], a["odt"], a["ws"], a["bytes"], None)


def read_of(bits):
    def read(lib, **kw):
        c = split(kw, bits)
        a = dict(k=GOOD, v=GOOD, cu=GOOD, total=8, most=8, table=GOOD, nb=4, lens=GOOD, batch=1, dt=1)
        a.update(kw)
        f = lib.msa_cache4_read if bits == 4 else lib.msa_cache_read
        return f(c, a["cu"], a["total"], a["most"], a["table"], a["nb"], a["lens"], a["batch"], a["k"], a["v"],
                 a["dt"], None)
    return read


COMMON = [
    (dict(cache=None), INVALID), (dict(k_codes=0), INVALID), (dict(v_scale=0), INVALID), (dict(v_codes=GOOD + 8), INVALID),
    (dict(k_scale=GOOD + 2), INVALID), (dict(n_pages=0), INVALID), (dict(n_pages=1 << 31), INVALID),
    (dict(Hkv=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(block=48), UNSUPPORTED), (dict(block=512), UNSUPPORTED),
    (dict(table=0), INVALID), (dict(table=GOOD + 1), INVALID), (dict(lens=0), INVALID), (dict(batch=0), INVALID),
    (dict(batch=65536), INVALID), (dict(nb=0), INVALID), (dict(nb=1 << 26), INVALID),
]


@pytest.mark.parametrize("call", [append, attn, read_of(4), read_of(8)])
def test_every_call_refuses_a_bad_cache_or_batch(lib, call):
    for kw, want in COMMON:
        assert call(lib, **dict(kw)) == want, kw
        assert lib.msa_last_error_string()
    if call in (append, attn):
        assert call(lib, v_scale=GOOD + 8) == INVALID
    assert call(lib, n_pages=1 << 25) == UNSUPPORTED     # 2^32 slots of 2 heads


@pytest.mark.parametrize("call", [append, read_of(4), read_of(8)])
def test_rows_refusals(lib, call):
    for kw in (dict(cu=0), dict(cu=GOOD + 2), dict(k=0), dict(v=GOOD + 4), dict(total=-1), dict(most=-1), dict(most=9),
               dict(total=1 << 31, most=1), dict(dt=7)):
        assert call(lib, **kw) == INVALID, kw
    assert call(lib, total=(1 << 31) - 1, most=(1 << 31) - 1, Hkv=16384) == UNSUPPORTED
    assert call(lib, most=0, k=0, v=0) == 0


def test_query_refusals(lib):
    for kw, want in [(dict(q=0), INVALID), (dict(q=GOOD + 8), INVALID), (dict(Hq=0), INVALID), (dict(Hq=5), INVALID),
                     (dict(n_q=0), INVALID), (dict(n_q=4096), UNSUPPORTED), (dict(window=0), INVALID),
                     (dict(idt=2), INVALID), (dict(odt=3), INVALID), (dict(ws=0), INVALID), (dict(ws=GOOD + 128), INVALID),
                     (dict(bytes=16), INVALID), (dict(out=0), INVALID), (dict(out=GOOD + 4), INVALID), (dict(lse=0), INVALID),
                     (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID)]:
        assert attn(lib, **dict(kw)) == want, kw


def test_workspace_sizes(lib):
    f = lib.msa_cache4_attn_workspace_size
    assert f(None, 4, 1, 1, 8, 1) == 0
    assert f(cache(4, d=96), 4, 1, 1, 8, 1) == 0
    assert f(cache(4), 4, 0, 1, 8, 1) == 0
    assert f(cache(4), 4, 1, 1, 7, 1) == 0
    assert 0 < f(cache(4), 1 << 14, 64, 8, 64, 1) <= 2 * 152 * 8 * 32 * (128 + 4) * 4 + 512
    g = lib.msa_qk_norm_rope_bwd_workspace_size
    assert g(-1, 1, 1, 128) == 0 and g(1, 0, 1, 128) == 0 and g(1, 1, 1, 96) == 0
    assert g(1 << 20, 64, 8, 128) >= 152 * 128 * 4


def rope(lib, **kw):
    a = dict(q=GOOD, qs=8 * 128, k=GOOD, ks=2 * 128, n=4, hq=8, hkv=2, d=128, pos=GOOD, f=GOOD, qw=GOOD, kw=GOOD, eps=1e-6,
             m=1.0, inter=0, qo=GOOD, ko=GOOD, dt=1, wdt=0)
    a.update(kw)
    return lib.msa_qk_norm_rope(a["q"], a["qs"], a["k"], a["ks"], a["n"], a["hq"], a["hkv"], a["d"], a["pos"], a["f"],
                                a["qw"], a["kw"], a["eps"], a["m"], a["inter"], a["qo"], a["ko"], a["dt"], a["wdt"], None)


def rope_bwd(lib, **kw):
    a = dict(gq=GOOD, gqs=8 * 128, gk=GOOD, gks=2 * 128, q=GOOD, qs=8 * 128, k=GOOD, ks=2 * 128, n=4, hq=8, hkv=2, d=128,
             pos=GOOD, f=GOOD, qw=GOOD, kw=GOOD, eps=1e-6, m=1.0, inter=0, qo=GOOD, ko=GOOD, dqw=GOOD, dkw=GOOD, dt=1, wdt=0,
             ws=GOOD, bytes=1 << 40)
    a.update(kw)
    return lib.msa_qk_norm_rope_bwd(a["gq"], a["gqs"], a["gk"], a["gks"], a["q"], a["qs"], a["k"], a["ks"], a["n"], a["hq"],
                                    a["hkv"], a["d"], a["pos"], a["f"], a["qw"], a["kw"], a["eps"], a["m"], a["inter"],
                                    a["qo"], a["ko"], a["dqw"], a["dkw"], a["dt"], a["wdt"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("call", [rope, rope_bwd])
def test_rope_refusals(lib, call):
    for kw, want in [(dict(q=0), INVALID), (dict(q=GOOD + 8), INVALID), (dict(k=0), INVALID), (dict(qs=8 * 128 - 8), INVALID),
                     (dict(ks=2 * 128 + 4), INVALID), (dict(dt=0, wdt=0, ks=2 * 128 + 2), INVALID), (dict(n=-1), INVALID),
                     (dict(n=1 << 31), INVALID), (dict(hq=0), INVALID), (dict(hkv=-1), INVALID), (dict(hq=1 << 15), INVALID),
                     (dict(d=96), UNSUPPORTED), (dict(pos=0), INVALID), (dict(pos=GOOD + 4), INVALID), (dict(f=0), INVALID),
                     (dict(qw=GOOD + 2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID),
                     (dict(m=float("nan")), INVALID), (dict(qo=0), INVALID), (dict(ko=GOOD + 4), INVALID), (dict(dt=5), INVALID),
                     (dict(wdt=5), INVALID)]:
        assert call(lib, **dict(kw)) == want, kw
    if call is rope:
        assert rope(lib, n=0, q=0, k=0, pos=0, f=0, qo=0, ko=0) == 0
    else:
        for kw in (dict(gq=0), dict(gk=GOOD + 8), dict(gqs=64), dict(dqw=0), dict(dkw=GOOD + 1), dict(ws=0), dict(bytes=100)):
            assert rope_bwd(lib, **kw) == INVALID, kw


def test_every_entry_point_opens_an_nvtx_range():
    csrc = os.path.join(ROOT, "long_context_sparse_landmark_gb300", "csrc")
    for header, source, n in (("msa_cache4.h", "msa_cache4_api.cu", 4), ("msa_rope.h", "msa_rope_api.cu", 2)):
        src = open(os.path.join(csrc, source)).read()
        declared = set(re.findall(r"^msa_status (msa_\w+)\(", open(os.path.join(ROOT, "include", header)).read(), re.M))
        assert len(declared) == n
        for name in sorted(declared):
            m = re.search(r"^msa_status " + name + r"\([^{]*\{\n(.*)\n", src, re.M)
            assert m and m.group(1).strip() == "MSA_NVTX_RANGE();", name


def test_python_calls_refuse_host_tensors():
    codes, scale = torch.zeros((2, 1, 32, 32), dtype=torch.uint8), torch.zeros((2, 1, 32, 2), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        msa.KVCache4(codes, codes, scale, scale)
    q = torch.zeros((2, 1, 64))
    with pytest.raises(ValueError, match="CUDA"):
        msa.qk_norm_rope(q, q, torch.zeros((2,), dtype=torch.int64), torch.zeros((32,), dtype=torch.int64))
    f = msa.rotary_frequencies(64, device="cpu")
    assert f.shape == (32,) and f[0].item() == round(2 ** 64 / (2 * 3.141592653589793))


def test_the_reference_of_the_format():
    assert R.code_of(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.9, -0.3, -0.0])).tolist() == [
        0, 2, 2, 4, 4, 6, 6, 7, 9, 8]
    assert R.exponent_of(7.0) == 0 and R.exponent_of(7.0001) == 1 and R.exponent_of(3.5) == -1
    assert R.exponent_of(0.0) == -126 and R.exponent_of(1.75 * 2.0 ** 127) == 125
    row = np.zeros(64)
    row[0], row[33] = 6.0, -2.0 ** -140
    codes, scale = R.pack(row)
    assert scale.tolist() == [127, 1] and codes[0] == 7 and codes[16] == 0x80
    np.testing.assert_array_equal(R.unpack(codes, scale)[:33], row[:33])
    row[5] = np.inf
    assert R.pack(row)[1].tolist() == [255, 255] and np.isnan(R.unpack(*R.pack(row))).all()
