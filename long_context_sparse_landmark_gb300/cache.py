"""The 8-bit and the 4-bit KV cache: the tokens generated after a long prefill.

A ``KVCache`` is a pool of pages, each one block of token slots of one
sequence (include/msa_cache.h has the format); a block table and the lengths say
which pages a batch of sequences uses.  ``cache_append`` quantises new keys
and values into it, ``cache_attention``, ``cache_topk_attention`` and
``cache_select_attention`` attend to it, ``cache_evict`` keeps the slots that
drew the most attention, ``cache_read`` reads it back as rows of keys and
values.  A ``KVCache4`` holds a token in half the bytes (include/msa_cache4.h);
``cache_append``, ``cache_attention`` and ``cache_read`` take either, the others
the 8-bit one.  As in ``api``, these only allocate outputs and marshal
arguments; they are not differentiable.

Every call runs on the device of its tensors and, unless ``stream`` says
otherwise, on that device's current stream; outputs and workspaces are
allocated for the stream the call runs on.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import _binding as B

_E4M3 = torch.float8_e4m3fn


_INT32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16
_CODES, _INPUTS = (_E4M3, torch.uint8), (_F32, _BF16)


def _want(t: torch.Tensor, what: str, dtypes, shape, dev: int):
    """Raise unless t has one of the dtypes, the shape and the device (that it
    is contiguous the binding checks)."""
    if t.dtype in dtypes and t.shape == shape and t.get_device() == dev:
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(x) for x in dtypes)}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{what} must be on cuda:{dev}, not {t.device}")


class KVCache:
    """Pages of 8-bit keys and values.

    k_codes, v_codes [n_pages, Hkv, block, d] float8_e4m3fn (or their bytes,
    uint8), k_scale, v_scale [n_pages, Hkv] fp32, k_mean [n_pages, Hkv, d]
    bf16; block 32, 64, 128 or 256, d 64 or 128.  ``KVCache.empty`` allocates
    them.
    """

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor, k_mean: torch.Tensor):
        if k_codes.dim() != 4 or not k_codes.is_cuda:
            raise ValueError("k_codes must be [n_pages, Hkv, block, d] on a CUDA device")
        shape = k_codes.shape
        n, h, block, d = shape
        dev = k_codes.get_device()
        _want(k_codes, "k_codes", _CODES, shape, dev)
        _want(v_codes, "v_codes", _CODES, shape, dev)
        _want(k_scale, "k_scale", (_F32,), (n, h), dev)
        _want(v_scale, "v_scale", (_F32,), (n, h), dev)
        _want(k_mean, "k_mean", (_BF16,), (n, h, d), dev)
        self._pool = (k_codes, v_codes, k_scale, v_scale, k_mean)
        self.n_pages, self.Hkv, self.block, self.d = n, h, block, d
        self.device = k_codes.device
        self.index = dev
        for t in (k_codes, v_codes, k_scale, v_scale, k_mean):
            if not t.is_contiguous():
                raise ValueError("the pool's tensors must be contiguous")
        self.struct = B.KvCacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(),
                                      v_scale.data_ptr(), k_mean.data_ptr(), n, h, d, block)
        self.ref = ctypes.byref(self.struct)

    # The kernels are given these tensors' addresses once: they can be written
    # to, not replaced.
    k_codes = property(lambda self: self._pool[0])
    v_codes = property(lambda self: self._pool[1])
    k_scale = property(lambda self: self._pool[2])
    v_scale = property(lambda self: self._pool[3])
    k_mean = property(lambda self: self._pool[4])

    @classmethod
    def empty(cls, n_pages: int, Hkv: int, d: int, block: int = 64, device="cuda") -> "KVCache":
        """A pool of n_pages pages; nothing in it needs a value before the
        first append."""
        codes = torch.empty((2, n_pages, Hkv, block, d), dtype=torch.uint8, device=device)
        scale = torch.empty((2, n_pages, Hkv), dtype=_F32, device=device)
        mean = torch.empty((n_pages, Hkv, d), dtype=torch.bfloat16, device=device)
        return cls(codes[0].view(_E4M3), codes[1].view(_E4M3), scale[0], scale[1], mean)


class KVCache4:
    """Pages of 4-bit keys and values (include/msa_cache4.h).

    k_codes, v_codes [n_pages, Hkv, block, d / 2] uint8, two e2m1 codes a byte,
    k_scale, v_scale [n_pages, Hkv, block, d / 32] uint8, the e8m0 scale of 32
    values; block 32, 64, 128 or 256, d 64 or 128.  ``KVCache4.empty``
    allocates them.
    """

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        if k_codes.dim() != 4 or not k_codes.is_cuda:
            raise ValueError("k_codes must be [n_pages, Hkv, block, d / 2] on a CUDA device")
        shape = k_codes.shape
        n, h, block, half = shape
        dev = k_codes.get_device()
        _want(k_codes, "k_codes", (torch.uint8,), shape, dev)
        _want(v_codes, "v_codes", (torch.uint8,), shape, dev)
        _want(k_scale, "k_scale", (torch.uint8,), (n, h, block, half // 16), dev)
        _want(v_scale, "v_scale", (torch.uint8,), (n, h, block, half // 16), dev)
        self._pool = (k_codes, v_codes, k_scale, v_scale)
        self.n_pages, self.Hkv, self.block, self.d = n, h, block, 2 * half
        self.device = k_codes.device
        self.index = dev
        for t in self._pool:
            if not t.is_contiguous():
                raise ValueError("the pool's tensors must be contiguous")
        self.struct = B.KvCache4Struct(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(),
                                       v_scale.data_ptr(), n, h, self.d, block)
        self.ref = ctypes.byref(self.struct)

    # As with KVCache: they can be written to, not replaced.
    k_codes = property(lambda self: self._pool[0])
    v_codes = property(lambda self: self._pool[1])
    k_scale = property(lambda self: self._pool[2])
    v_scale = property(lambda self: self._pool[3])

    @classmethod
    def empty(cls, n_pages: int, Hkv: int, d: int, block: int = 64, device="cuda") -> "KVCache4":
        """A pool of n_pages pages; nothing in it needs a value before the
        first append."""
        codes = torch.empty((2, n_pages, Hkv, block, d // 2), dtype=torch.uint8, device=device)
        scale = torch.empty((2, n_pages, Hkv, block, d // 32), dtype=torch.uint8, device=device)
        return cls(codes[0], codes[1], scale[0], scale[1])


def _eight_bit(cache, call: str):
    if isinstance(cache, KVCache4):
        raise TypeError(f"{call} takes a KVCache, not a KVCache4")


def _batch(cache: KVCache | KVCache4, table: torch.Tensor, lens: torch.Tensor):
    """Checks a batch's block table and lengths; returns their sizes."""
    shape = table.shape
    if len(shape) != 2:
        raise ValueError("block_table must be [batch, max_blocks]")
    _want(table, "block_table", (_INT32,), shape, cache.index)
    _want(lens, "lens", (_INT32,), shape[:1], cache.index)
    return shape


def _query(cache: KVCache, q: torch.Tensor, batch: int):
    """Checks query tokens; returns n_q and Hq."""
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [batch, n_q, Hq, d]")
    _want(q, "q", _INPUTS, (batch, shape[1], shape[2], cache.d), cache.index)
    return shape[1], shape[2]


def _run(cache: KVCache, stream, call):
    """call(stream address) with the cache's device current and allocations
    made for the stream that the kernels run on."""
    if stream is None:
        if torch._C._cuda_getDevice() == cache.index:  # (CUDA is up: there are tensors)
            return call(torch._C._cuda_getCurrentRawStream(cache.index))
        with torch.cuda.device(cache.index):
            return call(torch._C._cuda_getCurrentRawStream(cache.index))
    if stream.device.index != cache.index:
        raise ValueError("stream and cache are on different devices")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def cache_append(cache: KVCache | KVCache4, k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor,
                 block_table: torch.Tensor, lens: torch.Tensor, max_new: int,
                 stream=None) -> None:
    """Quantise new tokens into the cache (msa_cache_append, msa_cache4_append).

    k, v [total, Hkv, d] (bf16 or fp32): rows cu[b] .. cu[b+1] (cu
    [batch + 1] int32) are sequence b's last tokens; lens [batch] int32 are
    the lengths with them; no sequence has more than max_new of them.
    block_table [batch, max_blocks] int32 names the pages.
    """
    b, _ = _batch(cache, block_table, lens)
    if k.dim() != 3:
        raise ValueError("k must be [total, Hkv, d]")
    _want(k, "k", _INPUTS, (k.shape[0], cache.Hkv, cache.d), cache.index)
    _want(v, "v", (k.dtype,), k.shape, cache.index)
    _want(cu, "cu", (_INT32,), (b + 1,), cache.index)
    append = B.cache4_append if isinstance(cache, KVCache4) else B.cache_append
    max_new = int(max_new)
    _run(cache, stream, lambda s: append(cache.ref, k, v, cu, max_new, block_table, lens,
                                         stream=s))


def cache_read(cache: KVCache | KVCache4, cu: torch.Tensor, block_table: torch.Tensor,
               lens: torch.Tensor, total: int, max_rows: int,
               dtype: torch.dtype = torch.bfloat16, out=None, stream=None):
    """Read cached tokens back as rows of keys and values (msa_cache_read,
    msa_cache4_read), as the prefill's calls take them.

    Of each sequence b the last cu[b+1] - cu[b] of its lens[b] slots (at most
    max_rows; lower lens[b] for an earlier range) become the rows cu[b] ..
    cu[b+1] of k, v [total, Hkv, d] (``dtype``, bf16 or fp32).  ``out`` gives the
    two tensors to write; rows of no sequence are left as they were there, and
    hold anything in new ones.  Returns (k, v)."""
    b, _ = _batch(cache, block_table, lens)
    _want(cu, "cu", (_INT32,), (b + 1,), cache.index)
    shape = (int(total), cache.Hkv, cache.d)
    max_rows = int(max_rows)
    if dtype not in _INPUTS:
        raise TypeError(f"dtype must be float32 or bfloat16, not {dtype}")
    if out is not None:
        k, v = out
        _want(k, "out", (dtype,), shape, cache.index)
        _want(v, "out", (dtype,), shape, cache.index)
        if shape[0] and abs(k.data_ptr() - v.data_ptr()) < k.nbytes:
            raise ValueError("out: k and v must not share memory")

    def call(s):
        if out is not None:
            k, v = out
        else:
            k = torch.empty(shape, dtype=dtype, device=cache.device)
            v = torch.empty_like(k)
        B.cache_read(cache.ref, 4 if isinstance(cache, KVCache4) else 8, cu, max_rows,
                     block_table, lens, k, v, stream=s)
        return k, v

    return _run(cache, stream, call)


def cache_attention(q: torch.Tensor, cache: KVCache | KVCache4, block_table: torch.Tensor,
                    lens: torch.Tensor, window: int | None = None, scale: float | None = None,
                    weights: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                    stream=None):
    """Attention of the last n_q tokens of each sequence over its cached
    slots (msa_cache_attn, msa_cache4_attn): q [batch, n_q, Hq, d], causal
    among themselves, over the last ``window`` slots (None: all).  ``weights``
    [batch, Hkv, ld] fp32, ld >= max_blocks * block, is added the softmax weight
    each slot drew (8-bit cache).  Returns (out [batch, n_q, Hq, d], lse [batch, Hq, n_q] fp32)."""
    b, nb = _batch(cache, block_table, lens)
    n_q, Hq = _query(cache, q, b)
    d = cache.d
    window = nb * cache.block if window is None else int(window)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if isinstance(cache, KVCache4):
        if weights is not None:
            _eight_bit(cache, "cache_attention with weights")
        return _attention4(q, cache, block_table, lens, window, float(scale),
                           out_dtype or q.dtype, stream, nb)
    if weights is not None:
        if weights.dim() != 3:
            raise ValueError("weights must be [batch, Hkv, ld]")
        _want(weights, "weights", (_F32,), (b, cache.Hkv, weights.shape[2]), cache.index)

    def call(s):
        out = torch.empty((b, n_q, Hq, d), dtype=out_dtype or q.dtype, device=cache.device)
        lse = torch.empty((b, Hq, n_q), dtype=_F32, device=cache.device)
        ws = torch.empty((B.cache_attn_workspace_size(cache.ref, nb, b, n_q, Hq,
                                                      weights is not None, q.dtype),),
                         dtype=torch.uint8, device=cache.device)
        B.cache_attn(cache.ref, q, block_table, lens, window, scale, out, lse, weights, ws,
                     stream=s)
        return out, lse

    return _run(cache, stream, call)


@functools.lru_cache(4096)
def _attn4_bytes(n_pages: int, Hkv: int, d: int, block: int, *sizes) -> int:
    """Bytes of workspace of an attention over a 4-bit cache: they follow from the
    sizes, and are asked once for each."""
    pool = B.KvCache4Struct(None, None, None, None, n_pages, Hkv, d, block)
    return B.cache4_attn_workspace_size(ctypes.byref(pool), *sizes)


def _attention4(q, cache: KVCache4, block_table, lens, window: int, scale: float, out_dtype,
                stream, nb: int):
    b, n_q, Hq, d = q.shape
    nbytes = _attn4_bytes(cache.n_pages, cache.Hkv, d, cache.block, nb, b, n_q, Hq, q.dtype)

    def call(s):
        out = torch.empty(q.shape, dtype=out_dtype, device=cache.device)
        lse = torch.empty((b, Hq, n_q), dtype=_F32, device=cache.device)
        ws = torch.empty((nbytes,), dtype=torch.uint8, device=cache.device)
        B.cache4_attn(cache.ref, q, block_table, lens, window, scale, out, lse, ws, stream=s)
        return out, lse

    return _run(cache, stream, call)


def cache_block_select(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor,
                       lens: torch.Tensor, window: int, top_k: int, stream=None):
    """The top_k blocks before the window that each query token of q [batch,
    n_q, Hq, d] and KV head scores best by their mean keys
    (msa_cache_select).  Returns (sel [batch, n_q, Hkv, top_k] int32
    ascending, then -1; cnt [batch, n_q, Hkv] int32), as
    ``cache_select_attention`` takes them."""
    _eight_bit(cache, "cache_block_select")
    b, nb = _batch(cache, block_table, lens)
    n_q, _ = _query(cache, q, b)
    top_k = min(int(top_k), nb)

    def call(s):
        sel = torch.empty((b, n_q, cache.Hkv, top_k), dtype=_INT32, device=cache.device)
        cnt = torch.empty((b, n_q, cache.Hkv), dtype=_INT32, device=cache.device)
        ws = torch.empty((B.cache_select_workspace_size(cache.ref, nb, b, n_q),),
                         dtype=torch.uint8, device=cache.device)
        B.cache_select(cache.ref, q, block_table, lens, window, top_k, sel, cnt, ws, stream=s)
        return sel, cnt

    return _run(cache, stream, call)


def cache_topk_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor,
                         lens: torch.Tensor, window: int, top_k: int,
                         scale: float | None = None, out_dtype: torch.dtype | None = None,
                         stream=None):
    """``cache_attention`` over each query token's window and its own top_k
    blocks (msa_cache_attn_topk).  Returns (out, lse)."""
    _eight_bit(cache, "cache_topk_attention")
    b, nb = _batch(cache, block_table, lens)
    n_q, Hq = _query(cache, q, b)
    d = cache.d
    top_k = min(int(top_k), nb)
    scale = 1.0 / math.sqrt(d) if scale is None else scale

    def call(s):
        out = torch.empty((b, n_q, Hq, d), dtype=out_dtype or q.dtype, device=cache.device)
        lse = torch.empty((b, Hq, n_q), dtype=_F32, device=cache.device)
        ws = torch.empty((B.cache_attn_topk_workspace_size(cache.ref, nb, b, n_q, Hq, top_k,
                                                           q.dtype),),
                         dtype=torch.uint8, device=cache.device)
        B.cache_attn_topk(cache.ref, q, block_table, lens, window, top_k, scale, out, lse, ws,
                          stream=s)
        return out, lse

    return _run(cache, stream, call)


def cache_select_attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor,
                           lens: torch.Tensor, window: int, sel: torch.Tensor, cnt: torch.Tensor,
                           scale: float | None = None, out_dtype: torch.dtype | None = None,
                           stream=None):
    """``cache_attention`` over each query token's window and given blocks
    before it (msa_cache_attn_select): the first cnt [batch, n_q, Hkv] of sel
    [batch, n_q, Hkv, top_k], int32, as ``cache_block_select`` returned them for
    the same window or shorter lists without repeats.  Returns (out, lse)."""
    _eight_bit(cache, "cache_select_attention")
    b, nb = _batch(cache, block_table, lens)
    n_q, Hq = _query(cache, q, b)
    if sel.dim() != 4:
        raise ValueError("sel must be [batch, n_q, Hkv, top_k]")
    _want(sel, "sel", (_INT32,), (b, n_q, cache.Hkv, sel.shape[3]), cache.index)
    _want(cnt, "cnt", (_INT32,), (b, n_q, cache.Hkv), cache.index)
    d = cache.d
    scale = 1.0 / math.sqrt(d) if scale is None else scale

    def call(s):
        out = torch.empty((b, n_q, Hq, d), dtype=out_dtype or q.dtype, device=cache.device)
        lse = torch.empty((b, Hq, n_q), dtype=_F32, device=cache.device)
        ws = torch.empty((B.cache_attn_select_workspace_size(cache.ref, nb, b, n_q, Hq, q.dtype),),
                         dtype=torch.uint8, device=cache.device)
        B.cache_attn_select(cache.ref, q, block_table, lens, window, sel, cnt, scale, out, lse, ws,
                            stream=s)
        return out, lse

    return _run(cache, stream, call)


def cache_evict(cache: KVCache, block_table: torch.Tensor, lens: torch.Tensor,
                weights: torch.Tensor, dst_table: torch.Tensor, budget: int, recent: int,
                stream=None):
    """Keep at most ``budget`` slots of each sequence and KV head: the last
    ``recent`` and those of the greatest ``weights`` [batch, Hkv, ld]
    (msa_cache_evict).  They are written to the pages dst_table [batch,
    dst_blocks], which must not be among those in use.  Returns (new_lens
    [batch] int32, kept [batch, Hkv, budget] int32 slots ascending, then -1,
    new_weights [batch, Hkv, dst_blocks * block] fp32)."""
    _eight_bit(cache, "cache_evict")
    b, h = _batch(cache, block_table, lens)[0], cache.Hkv
    if weights.dim() != 3 or dst_table.dim() != 2:
        raise ValueError("weights must be [batch, Hkv, ld], dst_table [batch, dst_blocks]")
    _want(weights, "weights", (_F32,), (b, h, weights.shape[2]), cache.index)
    _want(dst_table, "dst_table", (_INT32,), (b, dst_table.shape[1]), cache.index)
    budget = int(budget)
    if budget < 1:
        raise ValueError("budget must be >= 1")

    def call(s):
        new_lens = torch.empty((b,), dtype=_INT32, device=cache.device)
        kept = torch.empty((b, h, budget), dtype=_INT32, device=cache.device)
        new_w = torch.empty((b, h, dst_table.shape[1] * cache.block), dtype=torch.float32,
                            device=cache.device)
        B.cache_evict(cache.ref, block_table, lens, weights, dst_table, budget, recent, new_lens,
                      kept, new_w, stream=s)
        return new_lens, kept, new_w

    return _run(cache, stream, call)
