"""Workloads of the 8-bit KV cache: append, attention over it, attention over
blocks that each query selects, and eviction by accumulated attention weight.

A case names an operator and its sizes.  ``prepare`` makes what a serving
program holds before the call (the page pool, block tables, lengths, the new
tokens or queries); ``run`` makes one pass, in plain torch operations where
``own`` is false and through the package's calls where it is true.

The pool: k_codes, v_codes [pages, Hkv, block, d] e4m3, k_scale, v_scale
[pages, Hkv] fp32 powers of two, k_mean [pages, Hkv, d] bf16 (mean of a full
block's dequantised keys).
"""
import math
import random

import numpy as np
import torch

own = False

_F8 = torch.float8_e4m3fn
_MAX_BYTES = 4_000_000_000  # of 8-bit K and V that a drawn case holds


def _append(batch, ctx, new, hkv, d, block, dtype):
    return {"op": "append", "batch": batch, "ctx": ctx, "new": new, "hkv": hkv, "d": d,
            "block": block, "dtype": dtype}


def _attend(batch, ctx, t, hq, hkv, d, block, window, weights, dtype):
    return {"op": "attend", "batch": batch, "ctx": ctx, "t": t, "hq": hq, "hkv": hkv, "d": d,
            "block": block, "window": window, "weights": weights, "dtype": dtype}


def _topk(batch, ctx, t, hq, hkv, d, block, window, top_k, dtype):
    return {"op": "topk", "batch": batch, "ctx": ctx, "t": t, "hq": hq, "hkv": hkv, "d": d,
            "block": block, "window": window, "top_k": top_k, "dtype": dtype}


def _evict(batch, ctx, budget, recent, hkv, d, block):
    return {"op": "evict", "batch": batch, "ctx": ctx, "budget": budget, "recent": recent, "hkv": hkv,
            "d": d, "block": block}


def listed():
    return [
        # the write of one generated token, one sequence: all latency
        dict(name="append 1 token", **_append(1, 32768, 1, 1, 128, 64, "bf16")),
        # prompts of odd lengths joining contexts that end inside a block, fp32 keys of the small layer's head size
        dict(name="append ragged prompts", **_append(24, 999, 501, 4, 64, 32, "fp32")),
        # the prefilled K and V of a 128K-token layer go into the cache
        dict(name="append 128K prefill", **_append(1, 0, 131072, 8, 128, 64, "bf16")),
        # the 2K-token fp32 layer, one token: the smallest attention
        dict(name="decode 2K fp32", **_attend(1, 2047, 1, 4, 1, 64, 32, 0, False, "fp32")),
        # one user at 32K tokens, 8 heads on one KV head
        dict(name="decode 32K", **_attend(1, 32768, 1, 8, 1, 128, 64, 0, False, "bf16")),
        # a serving batch of unequal lengths, 64 heads on 8
        dict(name="decode batch of 64", **_attend(64, 32768, 1, 64, 8, 128, 64, 0, False, "bf16")),
        # a million-token context, with the weights that an eviction goes by
        dict(name="decode 1M, weights", **_attend(1, 1048576, 1, 64, 8, 128, 64, 0, True, "bf16")),
        # four drafted tokens a sequence, over the 4096-token window
        dict(name="window, 4 drafts", **_attend(16, 131071, 4, 64, 8, 128, 128, 4096, False, "bf16")),
        # the top-k layer's sizes (512 blocks of 256, best 50, window 1024) for one generated token
        dict(name="top-k 128K", **_topk(1, 131072, 1, 64, 8, 128, 256, 1024, 50, "bf16")),
        # a batch with two drafted tokens each, finer blocks
        dict(name="top-k batch", **_topk(16, 65535, 2, 64, 8, 128, 64, 512, 32, "bf16")),
        # a step's eviction: one block over the budget
        dict(name="evict 64 of 4160", **_evict(8, 4160, 4096, 512, 8, 128, 64)),
        # a long prompt cut to an eighth after its prefill
        dict(name="evict 128K to 16K", **_evict(2, 131072, 16384, 4096, 8, 128, 64)),
    ]


def draw(rng):
    def logu(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))

    op = rng.choice(["append", "attend", "attend", "topk", "evict"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    block = rng.choice([32, 64, 64, 128, 256])
    batch = logu(1, 64)
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    most = _MAX_BYTES // (batch * hkv * d * 2)
    if op == "append":
        new = logu(1, max(1, min(131072, most // 8)))
        ctx = rng.choice([0, logu(1, 65536)])
        return _append(batch, min(ctx, max(0, most - new)), new, hkv, d, block, dtype)
    if op == "evict":
        ctx = logu(64, max(64, min(262144, most // 4)))
        budget = logu(16, ctx)
        recent = rng.choice([0, budget // 8, budget // 2])
        return _evict(batch, ctx, budget, recent, hkv, d, block)
    ctx = logu(1, max(1, min(1048576, most // (4 if dtype == "fp32" else 1))))
    group = rng.choice([1, 2, 4, 5, 8, 8, 16])
    t = min(rng.choice([1, 1, 1, 2, 3, 4, 8]), ctx)
    if op == "attend":
        window = rng.choice([0, 0, logu(1, 8192)])
        weights = rng.random() < 0.3
        return _attend(batch, ctx, t, hkv * group, hkv, d, block, window, weights, dtype)
    return _topk(batch, ctx, t, hkv * group, hkv, d, block, logu(1, 4096), logu(1, 128), dtype)


# -- sizes that follow from a case alone ------------------------------------

def _spread(case, top, least):
    """A length for each sequence, `top` the first, the others down to about half of it."""
    b = case["batch"]
    rng = random.Random(top * 31 + b)
    return [top] + [max(least, top - int(rng.random() * (top - top // 2))) for _ in range(b - 1)]


def _lens(case):
    """Lengths before the call (append) or with the query tokens (the others)."""
    if case["op"] == "append":
        return _spread(case, case["ctx"], 0)
    return _spread(case, case["ctx"], case.get("t", 1))


def _news(case):
    return _spread(case, case["new"], 0)


def _attended(case):
    """Slots that the rows of each sequence attend together, and the (row, slot) pairs."""
    slots = pairs = 0
    t, w = case["t"], case["window"] or (1 << 40)
    for n in _lens(case):
        slots += n - max(0, n - t - w + 1)
        pairs += sum(min(w, n - t + i + 1) for i in range(t))
    return slots, pairs


def work(case):
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "append":
        es = 2 if case["dtype"] == "bf16" else 4
        new, blk = sum(_news(case)), case["block"]
        full = sum((c + n) // blk - c // blk for c, n in zip(_lens(case), _news(case)))
        return {"bytes": new * hkv * d * 2 * (es + 1) + full * hkv * (2 * d + 8), "flops": new * hkv * d * 4}
    if case["op"] == "evict":
        byte = flop = 0
        for n in _lens(case):
            kept = min(n, case["budget"])
            byte += hkv * (4 * n + kept * (4 * d + 12)) + hkv * kept // case["block"] * (2 * d + 16)
            flop += hkv * (n + kept * d * 4)
        return {"bytes": byte, "flops": flop}
    hq, t = case["hq"], case["t"]
    es = 2 if case["dtype"] == "bf16" else 4
    rows = case["batch"] * t * hq * (2 * d * es + 4)
    if case["op"] == "attend":
        slots, pairs = _attended(case)
        more = slots * hkv * 8 if case["weights"] else 0
        return {"bytes": slots * hkv * (2 * d + 8 / case["block"]) + rows + more, "flops": pairs * hq * 4 * d}
    byte = flop = 0
    for n in _lens(case):
        # block means and the window once for all rows, each row's own blocks
        byte += (max(0, n - case["window"]) // case["block"] + min(n, case["window"] + t - 1)) * hkv * 2 * d
        for i in range(t):
            pos = n - t + i
            cand = max(0, pos - case["window"] + 1) // case["block"]
            far = min(case["top_k"], cand) * case["block"]
            byte += far * hkv * 2 * d
            flop += cand * hkv * 2 * d + (far + min(case["window"], pos + 1)) * hq * 4 * d
    return {"bytes": byte + rows, "flops": flop}


# -- inputs ------------------------------------------------------------------

def _pow2(e):
    """2^e as fp32, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _pool(case, gen, pages, dev):
    """Pages as an append of normal keys and values left them: a block's
    largest value takes a code near the top of the range."""
    hkv, block, d = case["hkv"], case["block"], case["d"]
    pool = {}
    for x, spread in (("k", 1.0), ("v", 0.5)):
        codes = torch.empty((pages, hkv, block, d), dtype=_F8, device=dev)
        scale = torch.empty((pages, hkv), dtype=torch.float32, device=dev)
        mean = torch.empty((pages, hkv, d), dtype=torch.bfloat16, device=dev)
        step = max(1, (1 << 26) // (hkv * block * d))
        for p in range(0, pages, step):
            q = min(pages, p + step)
            val = torch.randn((q - p, hkv, block, d), generator=gen, device=dev)
            # heads and blocks of unequal size, and a few channels that stand out
            val *= spread * torch.exp(0.5 * torch.randn((q - p, hkv, 1, 1), generator=gen, device=dev))
            if x == "k":
                val[..., :2] *= 4
                val += 0.7 * torch.randn((q - p, hkv, 1, d), generator=gen, device=dev)
            s, c = _quantise(val)
            codes[p:q], scale[p:q] = c, s
            mean[p:q] = ((c.to(torch.float32) * s[..., None, None]).double().mean(dim=2)).float().to(torch.bfloat16)
        pool[x + "_codes"], pool[x + "_scale"] = codes, scale
        if x == "k":
            pool["k_mean"] = mean
    return pool


def _quantise(val):
    """Scale 2^e of each [..., tokens, d] block, e the least with amax <= 448 * 2^e, and its codes."""
    amax = val.abs().amax(dim=(-1, -2))
    m, x = torch.frexp(amax)  # amax = m * 2^x, 0.5 <= m < 1
    e = (x - 9 + (m > 0.875).to(x.dtype)).clamp(min=-126)
    s = torch.where(amax > 0, _pow2(e), torch.zeros_like(amax))
    inv = torch.where(amax > 0, _pow2(-e), torch.zeros_like(amax))
    return s, (val * inv[..., None, None]).to(_F8)


def _table(lens, block, extra, gen, dev):
    """A page for each block of each sequence, in random order, -1 where a row has none."""
    most = max(1, max(-(-n // block) for n in lens))
    need = sum(-(-n // block) for n in lens)
    order = torch.randperm(need + extra, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    at = 0
    rows = order.cpu()
    for b, n in enumerate(lens):
        k = -(-n // block)
        table[b, :k] = rows[at:at + k]
        at += k
    return table.to(dev), need + extra, order[at:]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    block, hkv, d = case["block"], case["hkv"], case["d"]
    dt = torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32
    lens = _lens(case)
    st = {"case": case}
    if case["op"] == "append":
        new = _news(case)
        total = [a + b for a, b in zip(lens, new)]
        st["table"], pages, _ = _table(total, block, 1, gen, dev)
        st.update(_pool(case, gen, pages, dev))
        st["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=dev)
        st["lens"] = torch.tensor(total, dtype=torch.int32, device=dev)
        st["max_new"] = max(new)
        st["k"] = torch.randn((sum(new), hkv, d), generator=gen, device=dev).mul_(1.5).to(dt)
        st["v"] = torch.randn((sum(new), hkv, d), generator=gen, device=dev).to(dt)
        return st
    if case["op"] == "evict":
        budget = case["budget"]
        dst = -(-budget // block)
        st["table"], pages, free = _table(lens, block, dst * case["batch"], gen, dev)
        st.update(_pool(case, gen, pages, dev))
        st["dst"] = free.view(case["batch"], dst).contiguous()
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        w = torch.randn((case["batch"], hkv, st["table"].shape[1] * block), generator=gen, device=dev)
        w = torch.exp(2 * w)  # a few slots draw most of the weight
        w[torch.rand(w.shape, generator=gen, device=dev) < 0.05] = 0.0  # and some none at all
        st["weights"] = w
        return st
    st["table"], pages, _ = _table(lens, block, 1, gen, dev)
    st.update(_pool(case, gen, pages, dev))
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["q"] = torch.randn((case["batch"], case["t"], case["hq"], d), generator=gen, device=dev).to(dt)
    if case.get("weights"):
        # what a few earlier tokens have left there
        st["weights"] = torch.rand((case["batch"], hkv, st["table"].shape[1] * block), generator=gen, device=dev)
        st["weights"] *= 4 * case["t"] * (case["hq"] // hkv) / case["ctx"]
    return st


# -- one pass ----------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"append": _plain_append, "attend": _plain_attend, "topk": _plain_topk, "evict": _plain_evict}[case["op"]](case, state)


def _run_own(case, st):
    import long_context_sparse_landmark_gb300 as msa
    cache = msa.KVCache(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"], st["k_mean"])
    if case["op"] == "append":
        msa.cache_append(cache, st["k"], st["v"], st["cu"], st["table"], st["lens"], st["max_new"])
        return _pool_of(st)
    if case["op"] == "attend":
        out, lse = msa.cache_attention(st["q"], cache, st["table"], st["lens"], window=case["window"] or None,
                                       weights=st.get("weights"))
        return {"out": out, "lse": lse, "weights": st.get("weights")}
    if case["op"] == "topk":
        out, lse = msa.cache_topk_attention(st["q"], cache, st["table"], st["lens"], case["window"], case["top_k"])
        return {"out": out, "lse": lse}
    lens, kept, weights = msa.cache_evict(cache, st["table"], st["lens"], st["weights"], st["dst"], case["budget"],
                                          case["recent"])
    return {"lens": lens, "kept": kept, "weights": weights, **_pool_of(st)}


def _pool_of(st):
    return {k: st[k] for k in ("k_codes", "v_codes", "k_scale", "v_scale", "k_mean")}


def _store(st, x, pages, held, val, floor):
    """Blocks `val` [N, Hkv, block, d] go to `pages` [N]: slots where `held`
    [N, block] is true are written, and scales; `floor` [N, Hkv] is the least scale."""
    val = torch.where(held[:, None, :, None], val, torch.zeros_like(val))
    s, _ = _quantise(val)
    s = torch.maximum(s, floor)
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    codes = (val * inv[..., None, None]).to(_F8).view(torch.uint8)
    old = st[x + "_codes"].view(torch.uint8)
    old[pages] = torch.where(held[:, None, :, None], codes, old[pages])
    st[x + "_scale"][pages] = s
    if x == "k":
        full = held.all(dim=1)
        mean = (codes.view(_F8).to(torch.float32) * s[..., None, None]).double().mean(dim=2).float().to(torch.bfloat16)
        st["k_mean"][pages] = torch.where(full[:, None, None], mean, st["k_mean"][pages])


def _plain_append(case, st):
    block, table, lens, cu = case["block"], st["table"], st["lens"].long(), st["cu"].long()
    total = st["k"].shape[0]
    new = cu[1:] - cu[:-1]
    first = lens - new
    row = torch.arange(total, device=lens.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    slot = first[seq] + row - cu[seq]
    # every block that takes a token, once
    blocks = torch.zeros(table.shape, dtype=torch.bool, device=lens.device)
    blocks[seq, slot // block] = True
    b, j = torch.nonzero(blocks, as_tuple=True)
    pages = table[b, j].long()
    index = torch.full(table.shape, -1, dtype=torch.long, device=lens.device)
    index[b, j] = torch.arange(b.numel(), device=lens.device)
    at = torch.arange(block, device=lens.device)[None] + (j * block)[:, None]
    held, before = at < lens[b][:, None], at < first[b][:, None]
    for x in ("k", "v"):
        old = st[x + "_codes"].view(torch.uint8)[pages].view(_F8).to(torch.float32) * st[x + "_scale"][pages][..., None, None]
        val = torch.where(before[:, None, :, None], old, torch.zeros_like(old)).transpose(1, 2).contiguous()
        val[index[seq, slot // block], slot % block] = st[x].to(torch.float32)
        floor = st[x + "_scale"][pages] * before.any(dim=1)[:, None]
        _store(st, x, pages, held, val.transpose(1, 2), floor)
    return _pool_of(st)


def _gathered(case, st, x, dtype=torch.float32):
    """Dequantised [B, Hkv, slots, d] of a whole batch."""
    table = st["table"].long().clamp(min=0)
    codes = st[x + "_codes"].view(torch.uint8)[table].view(_F8).to(dtype)
    codes *= st[x + "_scale"][table][..., None, None].to(dtype)
    b, nb, h, block, d = codes.shape
    return codes.transpose(1, 2).reshape(b, h, nb * block, d)


def _attend_where(case, st, may):
    """Attention of q over the slots where `may` [B, T, Hkv or 1, slots] is true: out, lse, probabilities."""
    q = st["q"]
    b, t, hq, d = q.shape
    hkv = case["hkv"]
    k = _gathered(case, st, "k")
    qg = q.to(torch.float32).view(b, t, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4)  # [B, Hkv, T, g, d]
    s = torch.matmul(qg.reshape(b, hkv, -1, d), k.transpose(2, 3)).view(b, hkv, t, hq // hkv, -1) / math.sqrt(d)
    del k
    may = may.transpose(1, 2)[:, :, :, None]
    s = torch.where(may, s, torch.full_like(s, -math.inf))
    m = s.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - m)
    del s
    total = p.sum(dim=-1, keepdim=True)
    p = p / total.clamp(min=1e-37)
    v = _gathered(case, st, "v")
    out = torch.matmul(p.reshape(b, hkv, -1, p.shape[-1]), v).view(b, hkv, t, hq // hkv, d)
    lse = (m + torch.log(total))[..., 0]  # [B, Hkv, T, g]
    return out.permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(q.dtype), lse.permute(0, 1, 3, 2).reshape(b, hq, t).contiguous(), p


def _positions(case, st):
    """Position of each query row [B, T, 1, 1] and the slots [1, 1, 1, slots]."""
    t = case["t"]
    pos = st["lens"].long()[:, None] - t + torch.arange(t, device=st["lens"].device)[None]
    slot = torch.arange(st["table"].shape[1] * case["block"], device=st["lens"].device)
    return pos[:, :, None, None], slot[None, None, None]


def _plain_attend(case, st):
    pos, slot = _positions(case, st)
    may = slot <= pos
    if case["window"]:
        may = may & (slot > pos - case["window"])
    out, lse, p = _attend_where(case, st, may)
    if case["weights"]:
        st["weights"] += p.sum(dim=(2, 3))
    return {"out": out, "lse": lse, "weights": st.get("weights")}


def _plain_topk(case, st):
    """Scores in 64 bits: blocks next to each other in rank are told apart as the definition does."""
    q, block, top = st["q"], case["block"], case["top_k"]
    b, t, hq, d = q.shape
    hkv = case["hkv"]
    pos, slot = _positions(case, st)
    qs = q.double().view(b, t, hkv, hq // hkv, d).sum(dim=3).transpose(1, 2)  # [B, Hkv, T, d]
    mean = st["k_mean"][st["table"].long().clamp(min=0)].double().transpose(1, 2)  # [B, Hkv, blocks, d]
    score = torch.matmul(qs, mean.transpose(2, 3)).transpose(1, 2)  # [B, T, Hkv, blocks]
    nb = score.shape[-1]
    blocks = torch.arange(nb, device=q.device)
    cand = (blocks[None, None, None] + 1) * block <= pos - case["window"] + 1
    score = torch.where(cand, score, torch.full_like(score, -math.inf))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    chosen = torch.zeros(score.shape, dtype=torch.bool, device=q.device).scatter_(-1, order, True) & cand
    near = (slot <= pos) & (slot > pos - case["window"])
    out, lse, _ = _attend_where(case, st, near | chosen.repeat_interleave(block, dim=-1))
    return {"out": out, "lse": lse}


def _plain_evict(case, st):
    lens, w, block, budget = st["lens"].long(), st["weights"], case["block"], case["budget"]
    b, hkv, slots = w.shape
    slot = torch.arange(slots, device=w.device)[None, None]
    new = lens.clamp(max=budget)
    recent = torch.minimum(new, torch.full_like(new, case["recent"]))
    n = lens[:, None, None]
    # the last slots come first, then the others by weight, then what holds nothing
    key = torch.where(slot >= n - recent[:, None, None], torch.full_like(w, math.inf), w)
    key = torch.where(slot >= n, torch.full_like(w, -math.inf), key)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    if order.shape[-1] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]))
    rank = torch.arange(budget, device=w.device)[None, None]
    held = rank < new[:, None, None]
    kept = torch.sort(torch.where(held, order, torch.full_like(order, slots)), dim=-1).values
    src = torch.where(held, kept, torch.zeros_like(kept))
    out_w = torch.where(held, torch.gather(w, 2, src), torch.zeros((), device=w.device))
    nb = st["dst"].shape[1]
    pad = nb * block - budget
    src, full = torch.nn.functional.pad(src, (0, pad)), torch.nn.functional.pad(held, (0, pad))
    out_w = torch.nn.functional.pad(out_w, (0, pad))
    page = torch.gather(st["table"].long()[:, None].expand(-1, hkv, -1), 2, src // block).clamp(min=0)
    head = torch.arange(hkv, device=w.device)[None, :, None]
    used = (torch.arange(nb, device=w.device)[None] * block < new[:, None]).reshape(-1)
    dst = st["dst"].long().reshape(-1)[used]
    some = full[:, 0].reshape(b * nb, block)[used]
    for x in ("k", "v"):
        val = st[x + "_codes"].view(torch.uint8)[page, head, src % block].view(_F8).to(torch.float32)
        val = val * st[x + "_scale"][page, head][..., None]
        val = val.view(b, hkv, nb, block, -1).transpose(1, 2).reshape(b * nb, hkv, block, -1)[used]
        _store(st, x, dst, some, val, torch.zeros(val.shape[:2], device=w.device))
    return {"lens": new.to(torch.int32), "kept": torch.where(held, kept, torch.full_like(kept, -1)).to(torch.int32),
            "weights": out_w, **_pool_of(st)}


# -- the definition in 64 bits -----------------------------------------------

def _e4m3_values():
    """The 127 magnitudes of e4m3, ascending."""
    vals = [m * 2.0 ** -9 for m in range(8)]
    vals += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]
    return vals


def _round_to_code(x):
    """Nearest e4m3 value of each x (64 bits), ties to the even code."""
    vals = torch.tensor(_e4m3_values(), dtype=torch.float64, device=x.device)
    a = x.abs().contiguous()
    hi = torch.searchsorted(vals, a).clamp(max=vals.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = vals[hi] - a, a - vals[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(vals[code], x)


def _exact_block(val, least):
    """Scale and dequantised codes of one [tokens, d] block of 64-bit values."""
    amax = float(val.abs().max()) if val.numel() else 0.0
    s = 0.0
    if amax > 0:
        e = math.ceil(math.log2(amax / 448.0))
        while amax > 448.0 * 2.0 ** e:
            e += 1
        while amax <= 448.0 * 2.0 ** (e - 1):
            e -= 1
        s = 2.0 ** max(e, -126)
    s = max(s, least)
    return s, (_round_to_code(val / s) if s > 0 else torch.zeros_like(val))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "evict":
        return _exact_evict(case, st)
    return _exact_attend(case, st)


def _exact_write(st, pool, x, page, c, val, first, least, block):
    s, codes = _exact_block(val, least)
    pool[x + "_codes"][page, c, :val.shape[0]] = codes
    pool[x + "_scale"][page, c] = s
    if x == "k" and val.shape[0] == block:
        pool["k_mean"][page, c] = codes.mean(dim=0) * s


def _exact_pool(st):
    return {k: st[k].to(torch.float64) for k in ("k_codes", "v_codes", "k_scale", "v_scale", "k_mean")}


def _exact_append(case, st):
    block, hkv = case["block"], case["hkv"]
    cu, lens = st["cu"].tolist(), st["lens"].tolist()
    blocks = sum(-(-n // block) - (n - (y - x)) // block for n, x, y in zip(lens, cu, cu[1:]) if y > x)
    if blocks * hkv > 3000:
        return None
    pool = _exact_pool(st)
    for b, n in enumerate(lens):
        new = cu[b + 1] - cu[b]
        for j in range((n - new) // block, -(-n // block) if new else 0):
            page, lo, hi = int(st["table"][b, j]), j * block, min(n, (j + 1) * block)
            old = max(0, n - new - lo)
            for c in range(hkv):
                for x in ("k", "v"):
                    s = float(pool[x + "_scale"][page, c])
                    before = pool[x + "_codes"][page, c, :old] * s
                    fresh = st[x][cu[b] + lo + old - (n - new):cu[b] + hi - (n - new), c].to(torch.float64)
                    _exact_write(st, pool, x, page, c, torch.cat([before, fresh]), old, s if old else 0.0, block)
    return pool


def _exact_evict(case, st):
    block, hkv, budget = case["block"], case["hkv"], case["budget"]
    if -(-budget // block) * hkv * case["batch"] > 3000:
        return None
    pool = _exact_pool(st)
    weights = torch.zeros((case["batch"], hkv, st["dst"].shape[1] * block), dtype=torch.float64, device=st["lens"].device)
    for b, n in enumerate(st["lens"].tolist()):
        new = min(n, budget)
        recent = min(new, case["recent"])
        pages = st["table"][b].long()
        for c in range(hkv):
            w = st["weights"][b, c, :n].cpu().numpy().astype(np.float64)
            best = np.lexsort((np.arange(n - recent), -w[:n - recent]))[:new - recent]
            keep = torch.from_numpy(np.concatenate([np.sort(best), np.arange(n - recent, n)])).to(pages.device)
            weights[b, c, :new] = st["weights"][b, c, keep].to(torch.float64)
            for j in range(-(-new // block)):
                at = keep[j * block:(j + 1) * block]
                src, dst = pages[at // block], int(st["dst"][b, j])
                for x in ("k", "v"):
                    val = st[x + "_codes"].view(torch.uint8)[src, c, at % block].view(_F8).to(torch.float64)
                    val = val * st[x + "_scale"][src, c].to(torch.float64)[:, None]
                    _exact_write(st, pool, x, dst, c, val, 0, 0.0, block)
    return {"lens": None, "kept": None, "weights": weights, **pool}


def _exact_attend(case, st):
    """Row by row of the definition, a sequence and KV head at a time."""
    hkv, d, block, t = case["hkv"], case["d"], case["block"], case["t"]
    q = st["q"].to(torch.float64)
    group = q.shape[2] // hkv
    out = torch.zeros_like(q)
    lse = torch.full((q.shape[0], q.shape[2], t), -math.inf, dtype=torch.float64, device=q.device)
    weights = st["weights"].to(torch.float64) if "weights" in st else None
    for b, n in enumerate(st["lens"].tolist()):
        pages = st["table"][b, :-(-n // block)].long()
        for c in range(hkv):
            k, v = ((st[x + "_codes"].view(torch.uint8)[pages, c].view(_F8).to(torch.float64)
                     * st[x + "_scale"][pages, c].to(torch.float64)[:, None, None]).view(-1, d)[:n] for x in ("k", "v"))
            for i in range(t):
                pos = n - t + i
                rows = q[b, i, c * group:(c + 1) * group]
                lo = max(0, pos + 1 - case["window"]) if case["window"] else 0
                at = torch.arange(lo, pos + 1, device=q.device)
                if case["op"] == "topk" and lo >= block:
                    far = (st["k_mean"][pages[:lo // block], c].to(torch.float64) * rows.sum(dim=0)).sum(dim=1).cpu().numpy()
                    best = np.sort(np.lexsort((np.arange(far.size), -far))[:case["top_k"]])
                    best = torch.from_numpy(best).to(q.device)
                    at = torch.cat([(best[:, None] * block + torch.arange(block, device=q.device)).reshape(-1), at])
                s = (k[at] @ rows.T).T / math.sqrt(d)
                top = torch.logsumexp(s, dim=1)
                p = torch.exp(s - top[:, None])
                out[b, i, c * group:(c + 1) * group] = p @ v[at]
                lse[b, c * group:(c + 1) * group, i] = top
                if weights is not None:
                    weights[b, c, at] += p.sum(dim=0)
    return {"out": out, "lse": lse, "weights": weights}
