"""Host-side checks of the 8-bit KV cache's C ABI and Python calls (no GPU
needed): bad arguments are refused with the documented status before anything
touches the GPU, and workspace sizes cover what the calls lay out."""
import ctypes
import os
import re

import pytest
import torch

import long_context_sparse_landmark_gb300 as msa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from long_context_sparse_landmark_gb300 import build
    path = build.build()
    from long_context_sparse_landmark_gb300 import _binding
    return _binding.load_library(path)


GOOD = 1 << 20        # never dereferenced: validation fails first
INVALID, UNSUPPORTED = 1, 2


def cache(**kw):
    from long_context_sparse_landmark_gb300 import _binding
    a = dict(k_codes=GOOD, v_codes=GOOD, k_scale=GOOD, v_scale=GOOD, k_mean=GOOD, n_pages=10, Hkv=2, d=128, block=64)
    a.update(kw)
    return ctypes.byref(_binding.KvCacheStruct(*[a[n] for n, _ in _binding.KvCacheStruct._fields_]))


# What is wrong with the cache or the batch, for every entry point.
COMMON = [
    (dict(cache=None), INVALID), (dict(k_codes=0), INVALID), (dict(k_mean=0), INVALID),
    (dict(v_codes=GOOD + 8), INVALID), (dict(k_scale=GOOD + 2), INVALID), (dict(n_pages=0), INVALID),
    (dict(n_pages=1 << 31), INVALID), (dict(Hkv=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(block=48), UNSUPPORTED), (dict(block=512), UNSUPPORTED), (dict(block=0), UNSUPPORTED),
    (dict(table=0), INVALID), (dict(table=GOOD + 1), INVALID), (dict(lens=0), INVALID),
    (dict(batch=0), INVALID), (dict(batch=65536), INVALID), (dict(nb=0), INVALID),
    (dict(nb=1 << 26), INVALID),
]
FIELDS = ("k_codes", "v_codes", "k_scale", "v_scale", "k_mean", "n_pages", "Hkv", "d", "block")


def split(kw):
    c = {k: kw.pop(k) for k in list(kw) if k in FIELDS}
    return None if kw.pop("cache", 1) is None else cache(**c)


def append(lib, **kw):
    c = split(kw)
    a = dict(k=GOOD, v=GOOD, cu=GOOD, total=8, most=8, table=GOOD, nb=4, lens=GOOD, batch=1, dt=1)
    a.update(kw)
    return lib.msa_cache_append(c, a["k"], a["v"], a["cu"], a["total"], a["most"], a["table"], a["nb"], a["lens"],
                                a["batch"], a["dt"], None)


def attn(lib, **kw):
    c = split(kw)
    a = dict(q=GOOD, table=GOOD, nb=4, lens=GOOD, batch=1, n_q=1, Hq=8, window=16, scale=0.1, out=GOOD, lse=GOOD,
             w=0, ld=0, idt=1, odt=1, ws=GOOD, bytes=1 << 40)
    a.update(kw)
    return lib.msa_cache_attn(c, a["q"], a["table"], a["nb"], a["lens"], a["batch"], a["n_q"], a["Hq"], a["window"],
                              a["scale"], a["out"], a["lse"], a["w"], a["ld"], a["idt"], a["odt"], a["ws"], a["bytes"],
                              None)


def select(lib, **kw):
    c = split(kw)
    a = dict(q=GOOD, table=GOOD, nb=4, lens=GOOD, batch=1, n_q=1, Hq=8, window=16, top_k=2, sel=GOOD, cnt=GOOD, idt=1,
             ws=GOOD, bytes=1 << 40)
    a.update(kw)
    return lib.msa_cache_select(c, a["q"], a["table"], a["nb"], a["lens"], a["batch"], a["n_q"], a["Hq"], a["window"],
                                a["top_k"], a["sel"], a["cnt"], a["idt"], a["ws"], a["bytes"], None)


def attn_select(lib, **kw):
    c = split(kw)
    a = dict(q=GOOD, table=GOOD, nb=4, lens=GOOD, batch=1, n_q=1, Hq=8, window=16, sel=GOOD, cnt=GOOD, top_k=2,
             scale=0.1, out=GOOD, lse=GOOD, idt=1, odt=1, ws=GOOD, bytes=1 << 40)
    a.update(kw)
    return lib.msa_cache_attn_select(c, a["q"], a["table"], a["nb"], a["lens"], a["batch"], a["n_q"], a["Hq"],
                                     a["window"], a["sel"], a["cnt"], a["top_k"], a["scale"], a["out"], a["lse"],
                                     a["idt"], a["odt"], a["ws"], a["bytes"], None)


def attn_topk(lib, **kw):
    c = split(kw)
    a = dict(q=GOOD, table=GOOD, nb=4, lens=GOOD, batch=1, n_q=1, Hq=8, window=16, top_k=2, scale=0.1, out=GOOD,
             lse=GOOD, idt=1, odt=1, ws=GOOD, bytes=1 << 40)
    a.update(kw)
    return lib.msa_cache_attn_topk(c, a["q"], a["table"], a["nb"], a["lens"], a["batch"], a["n_q"], a["Hq"],
                                   a["window"], a["top_k"], a["scale"], a["out"], a["lse"], a["idt"], a["odt"],
                                   a["ws"], a["bytes"], None)


def evict(lib, **kw):
    c = split(kw)
    a = dict(table=GOOD, nb=4, lens=GOOD, batch=1, w=GOOD, ld=256, budget=100, recent=10, dst=GOOD, db=2,
             new_lens=GOOD + 64, kept=GOOD, nw=GOOD + 64, nld=128)
    a.update(kw)
    return lib.msa_cache_evict(c, a["table"], a["nb"], a["lens"], a["batch"], a["w"], a["ld"], a["budget"],
                               a["recent"], a["dst"], a["db"], a["new_lens"], a["kept"], a["nw"], a["nld"], None)


@pytest.mark.parametrize("call", [append, attn, select, attn_select, attn_topk, evict])
def test_every_call_refuses_a_bad_cache_or_batch(lib, call):
    for kw, want in COMMON:
        assert call(lib, **dict(kw)) == want, kw
        assert lib.msa_last_error_string()


def test_append_refusals(lib):
    for kw in (dict(cu=0), dict(cu=GOOD + 2), dict(k=0), dict(v=GOOD + 4), dict(total=-1), dict(most=-1),
               dict(most=9), dict(total=1 << 31, most=1), dict(dt=7)):
        assert append(lib, **kw) == INVALID, kw
    assert append(lib, most=0, k=0, v=0) == 0     # nothing to append: nothing runs


QUERY = [(dict(q=0), INVALID), (dict(q=GOOD + 8), INVALID), (dict(Hq=0), INVALID), (dict(Hq=5), INVALID),
         (dict(n_q=0), INVALID), (dict(n_q=4096), UNSUPPORTED), (dict(window=0), INVALID), (dict(window=-1), INVALID),
         (dict(idt=2), INVALID), (dict(ws=0), INVALID), (dict(ws=GOOD + 128), INVALID), (dict(bytes=16), INVALID)]


@pytest.mark.parametrize("call", [attn, select, attn_select, attn_topk])
def test_query_refusals(lib, call):
    for kw, want in QUERY:
        assert call(lib, **dict(kw)) == want, kw
    if call is not select:
        for kw in (dict(out=0), dict(out=GOOD + 4), dict(lse=0), dict(lse=GOOD + 2), dict(odt=3), dict(scale=0.0),
                   dict(scale=float("nan")), dict(scale=-1.0), dict(scale=float("inf"))):
            assert call(lib, **kw) == INVALID, kw
    if call is not attn:
        for kw in (dict(top_k=0), dict(top_k=5)):
            assert call(lib, **kw) == INVALID, kw
    if call in (select, attn_select):
        for kw in (dict(sel=0), dict(cnt=0), dict(sel=GOOD + 2), dict(cnt=GOOD + 1)):
            assert call(lib, **kw) == INVALID, kw


def test_weights_refusals(lib):
    assert attn(lib, w=GOOD, ld=255) == INVALID
    assert attn(lib, w=GOOD + 2, ld=256) == INVALID
    assert attn(lib, w=GOOD, ld=256, batch=40000) == UNSUPPORTED


def test_evict_refusals(lib):
    for kw in (dict(w=0), dict(w=GOOD + 1), dict(ld=255), dict(budget=0), dict(budget=129), dict(recent=-1),
               dict(recent=101), dict(dst=0), dict(dst=GOOD + 2), dict(db=0), dict(new_lens=0), dict(new_lens=GOOD),
               dict(kept=0), dict(nw=0), dict(nw=GOOD), dict(nld=99)):
        assert evict(lib, **kw) == INVALID, kw
    assert evict(lib, Hkv=16384, batch=65535) == UNSUPPORTED


def test_workspace_sizes(lib):
    f = lib.msa_cache_attn_workspace_size
    assert f(None, 4, 1, 1, 8, 0, 1) == 0
    assert f(cache(d=96), 4, 1, 1, 8, 0, 1) == 0
    assert f(cache(), 4, 0, 1, 8, 0, 1) == 0
    assert f(cache(), 4, 1, 1, 7, 0, 1) == 0
    plain = f(cache(), 4, 3, 2, 8, 0, 1)
    assert plain > 0 and f(cache(), 4, 3, 2, 8, 1, 1) >= plain + 4 * 3 * 2 * 8 * 4 * 64
    # never more than two parts of 32 rows for each of 8 warps an SM
    assert f(cache(), 1 << 14, 64, 8, 64, 0, 1) <= 2 * 152 * 8 * 32 * (128 + 2) * 4 + 512
    s = lib.msa_cache_select_workspace_size
    assert s(cache(), 0, 1, 1) == 0
    assert s(cache(), 100, 3, 2) >= 16 * 3 * 2 * 2 * 100
    t = lib.msa_cache_attn_topk_workspace_size
    assert t(cache(), 4, 1, 1, 8, 5, 1) == 0
    assert t(cache(), 100, 3, 2, 8, 7, 1) >= s(cache(), 100, 3, 2) + lib.msa_cache_attn_select_workspace_size(
        cache(), 100, 3, 2, 8, 1) + 4 * 3 * 2 * 2 * 8


def test_every_entry_point_opens_an_nvtx_range():
    src = open(os.path.join(ROOT, "long_context_sparse_landmark_gb300", "csrc", "msa_cache_api.cu")).read()
    header = open(os.path.join(ROOT, "include", "msa_cache.h")).read()
    declared = set(re.findall(r"^msa_status (msa_\w+)\(", header, re.M))
    assert len(declared) == 6
    for name in sorted(declared):
        m = re.search(r"^msa_status " + name + r"\([^{]*\{\n(.*)\n", src, re.M)
        assert m and m.group(1).strip() == "MSA_NVTX_RANGE();", name


def test_python_calls_refuse_host_tensors():
    codes = torch.zeros((2, 1, 32, 64), dtype=torch.uint8)
    scale, mean = torch.zeros((2, 1)), torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        msa.KVCache(codes, codes, scale, scale, mean)
    with pytest.raises(ValueError):
        msa.KVCache(codes[0], codes, scale, scale, mean)
