"""Calls from two host threads at once, each with buffers and a stream of its
own and a size of its own: what a launch needs must not depend on what another
thread's call has set in between.  The C entry points are called through ctypes
with ready arguments: it lets go of Python's lock, and the threads spend most
of their time inside the library."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import long_context_sparse_landmark_gb300 as msa
from tests.gpu_helpers import binding, check_guards, gempty

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


def at_once(*calls, times=4000):
    """Each of calls(stream address) -> status, over and over on a thread."""
    torch.cuda.synchronize()
    failed = []
    start = threading.Barrier(len(calls))

    def work(call):
        stream = torch.cuda.Stream()
        start.wait()
        for i in range(times):
            st = call(stream.cuda_stream)
            if st != 0:
                failed.append((i, st, binding()._lib.msa_last_error_string().decode()))
                break
            if i % 256 == 255:
                stream.synchronize()
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    check_guards()


def evicting(blocks):
    """A call that keeps 32 of 64 * blocks slots of one list."""
    B = binding()
    cache = msa.KVCache.empty(blocks + 1, 1, 64, 64)
    k = torch.randn((blocks * 64, 1, 64), device=DEV)
    t, lens = i32([list(range(blocks))]), i32([blocks * 64])
    msa.cache_append(cache, k, k, i32([0, blocks * 64]), t, lens, blocks * 64)
    w = torch.rand((1, 1, blocks * 64), device=DEV)
    dst, new_lens = i32([[blocks]]), i32([0])
    kept, new_w = gempty((1, 1, 32), torch.int32), gempty((1, 1, 64))
    keep = (cache, t, lens, w, dst, new_lens, kept, new_w)
    p = [x.data_ptr() for x in keep[1:]]

    def call(stream, _keep=keep):
        return B._lib.msa_cache_evict(cache.ref, p[0], blocks, p[1], 1, p[2], blocks * 64, 32, 4, p[3], 1,
                                      p[4], p[5], p[6], 64, stream)
    return call


def selecting(n):
    """A call that chooses 8 of n blocks."""
    B = binding()
    cache = msa.KVCache.empty(n + 1, 1, 64, 32)
    cache.k_mean.normal_()
    t, lens = i32([list(range(n + 1))]), i32([n * 32 + 1])
    q = torch.randn((1, 1, 1, 64), device=DEV)
    sel, cnt = gempty((1, 1, 1, 8), torch.int32), gempty((1, 1, 1), torch.int32)
    ws = gempty((B.cache_select_workspace_size(cache.ref, n + 1, 1, 1),), torch.uint8)
    p = [x.data_ptr() for x in (q, t, lens, sel, cnt, ws)]

    def call(stream, _keep=(cache, q, t, lens, sel, cnt, ws)):
        return B._lib.msa_cache_select(cache.ref, p[0], p[1], n + 1, p[2], 1, 1, 1, 1, 8, p[3], p[4], 0, p[5],
                                       ws.nbytes, stream)
    return call


@pytest.mark.parametrize("blocks", [(2, 120), (1300, 5000)])
def test_evictions(blocks):
    at_once(*(evicting(n) for n in blocks), times=4000 if blocks[1] < 200 else 400)


@pytest.mark.parametrize("n", [(2100, 3900), (4200, 40000)])
def test_selections(n):
    at_once(*(selecting(x) for x in n), times=4000)


def merging(parts, heads):
    """A call that merges partial results; enough parts and heads take more
    than 48 KB of weights."""
    B = binding()
    o = [torch.randn((8, heads, 64), device=DEV) for _ in range(parts)]
    l = [torch.randn((heads, 8), device=DEV) for _ in range(parts)]
    out, lse = gempty((8, heads, 64)), gempty((heads, 8))
    po, pl = ((ctypes.c_void_p * parts)(*[t.data_ptr() for t in x]) for x in (o, l))
    want = (torch.stack(o).double() * torch.softmax(torch.stack(l).double(), 0).transpose(1, 2)[..., None]).sum(0)

    def call(stream, _keep=(o, l)):
        return B._lib.msa_lse_merge(po, pl, parts, out.data_ptr(), lse.data_ptr(), 8, heads, 64, 0, stream)
    return call, out, want


def test_merges():
    small, large = merging(64, 200), merging(64, 500)
    at_once(small[0], large[0])
    for _, out, want in (small, large):
        assert (out.double() - want).abs().max() < 1e-5


def choosing(G):
    """A call of the prefill's block selection with G key blocks."""
    B = binding()
    n = 1024
    q, lm = torch.randn((n, 1, 64), device=DEV), torch.randn((G, 1, 64), device=DEV)
    sel, cnt = gempty((n // 128, 1, 1), torch.int32), gempty((n // 128, 1), torch.int32)

    def call(stream, _keep=(q, lm, sel, cnt)):
        return B._lib.msa_block_select(q.data_ptr(), lm.data_ptr(), sel.data_ptr(), cnt.data_ptr(), n, 1, 1, 64, 32, G, 1,
                                       0, stream)
    return call


def test_prefill_selections():
    at_once(choosing(2), choosing(1024))
