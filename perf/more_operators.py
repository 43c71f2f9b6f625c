"""Workloads of the 4-bit KV cache and of what stands before a cache: append,
attention over it, reading a cache back as rows of keys and values, and the
norms of queries and keys for each head with the position rotation, forward and
backward.

A case names an operator and its sizes.  ``prepare`` makes what a program holds
before the call (the page pool, block tables, lengths, the new tokens or
queries, positions and frequencies); ``run`` makes one pass, in plain torch
operations where ``own`` is false and through the package's calls where it is
true.

The 4-bit pool: k_codes, v_codes [pages, Hkv, block, d / 2] uint8, two e2m1
codes a byte, the even dim in the low half; k_scale, v_scale [pages, Hkv, block,
d / 32] uint8, x for 2^(x - 127).  The 8-bit pool: k_codes, v_codes [pages, Hkv,
block, d] e4m3, k_scale, v_scale [pages, Hkv] fp32, k_mean [pages, Hkv, d] bf16.
"""
import math
import random

import torch

own = False

_F8 = torch.float8_e4m3fn
_GROUP = 32
_MAX_BYTES = 2_000_000_000  # of 4-bit K and V that a drawn case holds


def _append(batch, ctx, new, hkv, d, block, dtype):
    return {"op": "append", "batch": batch, "ctx": ctx, "new": new, "hkv": hkv, "d": d, "block": block, "dtype": dtype}


def _attend(batch, ctx, t, hq, hkv, d, block, window, dtype):
    return {"op": "attend", "batch": batch, "ctx": ctx, "t": t, "hq": hq, "hkv": hkv, "d": d, "block": block,
            "window": window, "dtype": dtype}


def _read(batch, ctx, bits, hkv, d, block, dtype):
    return {"op": "read", "batch": batch, "ctx": ctx, "bits": bits, "hkv": hkv, "d": d, "block": block, "dtype": dtype}


def _rope(tokens, far, hq, hkv, d, norm, interleaved, backward, dtype):
    return {"op": "rope", "tokens": tokens, "far": far, "hq": hq, "hkv": hkv, "d": d, "norm": norm,
            "interleaved": interleaved, "backward": backward, "dtype": dtype}


def listed():
    return [
        # one generated token's keys and values, written and read as the next layers will see them: all latency
        dict(name="append 1 token", **_append(1, 32768, 1, 1, 128, 64, "bf16")),
        # prompts of odd lengths joining contexts that end inside a block, fp32 keys of the small layer's head size
        dict(name="append ragged prompts", **_append(24, 999, 501, 4, 64, 32, "fp32")),
        # the prefilled K and V of a 128K-token layer go into the cache
        dict(name="append 128K prefill", **_append(1, 0, 131072, 8, 128, 64, "bf16")),
        # the 2K-token fp32 layer, one token: the smallest attention
        dict(name="decode 2K fp32", **_attend(1, 2047, 1, 4, 1, 64, 32, 0, "fp32")),
        # one user at 32K tokens, 8 heads on one KV head
        dict(name="decode 32K", **_attend(1, 32768, 1, 8, 1, 128, 64, 0, "bf16")),
        # a serving batch of unequal lengths, 64 heads on 8
        dict(name="decode batch of 64", **_attend(64, 32768, 1, 64, 8, 128, 64, 0, "bf16")),
        # four drafted tokens a sequence, over the 4096-token window
        dict(name="window, 4 drafts", **_attend(16, 131071, 4, 64, 8, 128, 128, 4096, "bf16")),
        # a cached 128K-token prefix of one layer, for the prefill of what follows it
        dict(name="read 128K", **_read(1, 131072, 4, 8, 128, 64, "bf16")),
        # a batch of odd prefixes from the 8-bit cache, in fp32
        dict(name="read 8-bit ragged", **_read(24, 1501, 8, 4, 64, 32, "fp32")),
        # a decoding step of 64 sequences, positions up to a million
        dict(name="norm, rope: 64 tokens", **_rope(64, 1048576, 64, 8, 128, True, False, False, "bf16")),
        # a training step of the small fp32 layer, an odd number of tokens
        dict(name="norm, rope: train 2K fp32", **_rope(2047, 0, 4, 1, 64, True, True, True, "fp32")),
        # a training step over 32K tokens, 64 heads on 8
        dict(name="norm, rope: train 32K", **_rope(32768, 0, 64, 8, 128, True, False, True, "bf16")),
    ]


def draw(rng):
    def logu(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))

    op = rng.choice(["append", "attend", "attend", "read", "rope", "rope"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    block = rng.choice([32, 64, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "rope":
        hq = hkv * rng.choice([1, 2, 4, 5, 8])
        es = 2 if dtype == "bf16" else 4
        most = 32768 * 72 * 128 * 2 // ((hq + hkv) * d * es)
        far = rng.choice([0, logu(1, 1048576)])
        return _rope(logu(1, min(131072, most)), far, hq, hkv, d, rng.random() < 0.7, rng.random() < 0.4,
                     rng.random() < 0.5, dtype)
    batch = logu(1, 64)
    most = _MAX_BYTES // (batch * hkv * d)
    if op == "append":
        new = logu(1, max(1, min(131072, most // (20 if dtype == "fp32" else 10))))
        ctx = rng.choice([0, logu(1, 65536)])
        return _append(batch, min(ctx, max(0, most - new)), new, hkv, d, block, dtype)
    if op == "read":
        return _read(batch, logu(1, max(1, min(131072, most // 8))), rng.choice([4, 4, 8]), hkv, d, block, dtype)
    group = rng.choice([1, 2, 4, 5, 8, 8, 16])
    t = rng.choice([1, 1, 1, 2, 3, 4, 8])
    ctx = logu(1, max(1, min(1048576, most // max(1, group * t // 8) // (4 if dtype == "fp32" else 1))))
    t = min(t, ctx)
    return _attend(batch, ctx, t, hkv * group, hkv, d, block, rng.choice([0, 0, logu(1, 8192)]), dtype)


# -- sizes that follow from a case alone ------------------------------------

def _spread(case, top, least):
    """A length for each sequence, `top` the first, the others down to about half of it."""
    b = case["batch"]
    rng = random.Random(top * 31 + b)
    return [top] + [max(least, top - int(rng.random() * (top - top // 2))) for _ in range(b - 1)]


def _lens(case):
    """Lengths before the call (append) or with the query tokens."""
    return _spread(case, case["ctx"], 0 if case["op"] in ("append", "read") else case["t"])


def _news(case):
    return _spread(case, case["new"], 0)


def _es(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    d, hkv, es = case["d"], case["hkv"], _es(case)
    if case["op"] == "rope":
        values = case["tokens"] * (case["hq"] + hkv) * d
        passes = 2 + (3 if case["backward"] else 0)
        return {"bytes": values * es * passes + case["tokens"] * 8, "flops": values * (30 if case["backward"] else 10)}
    held = d / 2 + d / _GROUP  # of K, or of V: codes and scales of a slot
    if case["op"] == "append":  # in, into the cache, and the values that it stands for
        rows = sum(_news(case)) * hkv * 2
        return {"bytes": rows * (d * es * 2 + held), "flops": rows * d * 4}
    if case["op"] == "read":
        rows = sum(_lens(case)) * hkv * 2
        return {"bytes": rows * (d * es + (held if case["bits"] == 4 else d)), "flops": rows * d}
    slots = pairs = 0
    t, w = case["t"], case["window"] or (1 << 40)
    for n in _lens(case):
        slots += n - max(0, n - t - w + 1)
        pairs += sum(min(w, n - t + i + 1) for i in range(t))
    rows = case["batch"] * t * case["hq"] * (2 * d * es + 4)
    return {"bytes": slots * hkv * 2 * held + rows, "flops": pairs * case["hq"] * 4 * d}


# -- the 4-bit format --------------------------------------------------------

def _pow2(e):
    """2^e as fp32, from its bits (-126 <= e <= 127)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _pack(val):
    """Bytes of codes [..., d / 2] and scales [..., d / 32] of fp32 values [..., d]."""
    g = val.reshape(*val.shape[:-1], -1, _GROUP)
    m, x = torch.frexp(g.abs().amax(dim=-1))  # amax = m * 2^x, 0.5 <= m < 1
    e = (x - 3 + (m > 0.875).to(x.dtype)).clamp(min=-126)  # the least with amax <= 7 * 2^e
    y = g * _pow2(-e)[..., None]
    a = y.abs()
    code = (a > 0.25).to(torch.uint8)
    for most, tie in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= most) if tie else (a > most)
    code += torch.signbit(y).to(torch.uint8) * 8
    code = code.reshape(*val.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _unpack(codes, scale):
    """fp32 values [..., d] of codes and scales."""
    steps = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([steps, -steps])
    both = torch.stack([table.repeat(16), table.repeat_interleave(16)], dim=-1)  # of a byte
    val = both[codes.to(torch.int32)].reshape(*codes.shape[:-1], -1, _GROUP)
    val *= _pow2(scale.to(torch.int32) - 127)[..., None]
    return val.reshape(*codes.shape[:-1], -1)


# -- inputs ------------------------------------------------------------------

def _values(shape, x, gen, dev):
    """Keys or values [pages, Hkv, block, d] as a layer has them: heads and
    blocks of unequal size, and a few channels of the keys that stand out."""
    n, hkv, block, d = shape
    val = torch.randn(shape, generator=gen, device=dev)
    val *= (1.0 if x == "k" else 0.5) * torch.exp(0.5 * torch.randn((n, hkv, 1, 1), generator=gen, device=dev))
    if x == "k":
        val[..., :2] *= 4
        val += 0.7 * torch.randn((n, hkv, 1, d), generator=gen, device=dev)
    return val


def _pool(case, gen, pages, dev):
    """Pages as appends left them."""
    hkv, block, d = case["hkv"], case["block"], case["d"]
    four = case.get("bits", 4) == 4
    pool = {}
    step = max(1, (1 << 26) // (hkv * block * d))
    for x in ("k", "v"):
        if four:
            codes = torch.empty((pages, hkv, block, d // 2), dtype=torch.uint8, device=dev)
            scale = torch.empty((pages, hkv, block, d // _GROUP), dtype=torch.uint8, device=dev)
        else:
            codes = torch.empty((pages, hkv, block, d), dtype=_F8, device=dev)
            scale = torch.empty((pages, hkv), dtype=torch.float32, device=dev)
        for p in range(0, pages, step):
            q = min(pages, p + step)
            val = _values((q - p, hkv, block, d), x, gen, dev)
            if four:
                codes[p:q], scale[p:q] = _pack(val)
            else:
                m, e = torch.frexp(val.abs().amax(dim=(-1, -2)))
                e = e - 9 + (m > 0.875).to(e.dtype)  # amax <= 448 * 2^e
                codes[p:q], scale[p:q] = (val * _pow2(-e)[..., None, None]).to(_F8), _pow2(e)
        pool[x + "_codes"], pool[x + "_scale"] = codes, scale
    if not four:
        pool["k_mean"] = torch.zeros((pages, hkv, d), dtype=torch.bfloat16, device=dev)
    return pool


def _table(lens, block, gen, dev):
    """A page for each block of each sequence, in random order, -1 where a row has none."""
    most = max(1, max(-(-n // block) for n in lens))
    need = sum(-(-n // block) for n in lens)
    order = torch.randperm(need + 1, generator=gen, device=dev).to(torch.int32).cpu()
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // block)
        table[b, :k] = order[at:at + k]
        at += k
    return table.to(dev), need + 1


def _starts(counts, dev):
    """Row at which each sequence's rows start, and their number at the end."""
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    hkv, d = case["hkv"], case["d"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    st = {"case": case}
    if case["op"] == "rope":
        n, hq = case["tokens"], case["hq"]
        # the projections' output: q, k and v of a token side by side
        qkv = torch.randn((n, hq + 2 * hkv, d), generator=gen, device=dev)
        qkv *= torch.exp(0.5 * torch.randn((1, hq + 2 * hkv, 1), generator=gen, device=dev))
        qkv = qkv.to(dt)
        st["q"], st["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        if case["far"]:  # tokens of many sequences
            st["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device=dev)
        else:
            st["positions"] = torch.arange(n, device=dev)
        # angles a position, in radians; and in turns, 2^64 to the turn
        inv = [10000.0 ** (-2 * i / d) for i in range(d // 2)]
        turns = [int(f / (2 * math.pi) * 2 ** 64) for f in inv]
        st["inv_freq"] = torch.tensor(inv, dtype=torch.float64, device=dev)
        st["freqs"] = torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns], dtype=torch.int64, device=dev)
        for x in ("q", "k"):
            w = 1 + 0.2 * torch.randn((d,), generator=gen, device=dev)
            st[x + "_weight"] = w.to(dt) if case["norm"] else None
        if case["backward"]:
            st["dq"] = torch.randn((n, hq, d), generator=gen, device=dev).to(dt)
            st["dk"] = torch.randn((n, hkv, d), generator=gen, device=dev).to(dt)
        return st
    lens, block = _lens(case), case["block"]
    new = _news(case) if case["op"] == "append" else lens
    total = [a + b for a, b in zip(lens, new)] if case["op"] == "append" else lens
    st["table"], pages = _table(total, block, gen, dev)
    st.update(_pool(case, gen, pages, dev))
    st["lens"] = torch.tensor(total, dtype=torch.int32, device=dev)
    if case["op"] == "attend":
        st["q"] = torch.randn((case["batch"], case["t"], case["hq"], d), generator=gen, device=dev).to(dt)
        return st
    st["cu"], st["total"], st["most"] = _starts(new, dev), sum(new), max(new)
    if case["op"] == "append":
        st["k"] = torch.randn((sum(new), hkv, d), generator=gen, device=dev).mul_(1.5).to(dt)
        st["v"] = torch.randn((sum(new), hkv, d), generator=gen, device=dev).to(dt)
    return st


# -- one pass ----------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"append": _plain_append, "attend": _plain_attend, "read": _plain_read, "rope": _plain_rope}[case["op"]](case, state)


def _run_own(case, st):
    import long_context_sparse_landmark_gb300 as msa
    if case["op"] == "rope":
        how = dict(q_weight=st["q_weight"], k_weight=st["k_weight"], interleaved=case["interleaved"])
        q, k = msa.qk_norm_rope(st["q"], st["k"], st["positions"], st["freqs"], **how)
        if not case["backward"]:
            return {"q": q, "k": k}
        dq, dk, dqw, dkw = msa.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], st["positions"], st["freqs"], **how)
        return {"q": q, "k": k, "dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    if case.get("bits", 4) == 4:
        cache = msa.KVCache4(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"])
    else:
        cache = msa.KVCache(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"], st["k_mean"])
    if case["op"] == "attend":
        out, lse = msa.cache_attention(st["q"], cache, st["table"], st["lens"], window=case["window"] or None)
        return {"out": out, "lse": lse}
    if case["op"] == "append":
        msa.cache_append(cache, st["k"], st["v"], st["cu"], st["table"], st["lens"], st["most"])
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    k, v = msa.cache_read(cache, st["cu"], st["table"], st["lens"], st["total"], st["most"], dtype=dt)
    return {"k": k, "v": v}


def _places(case, st):
    """Page and slot in it of each row of st["cu"]."""
    cu, lens = st["cu"].long(), st["lens"].long()
    row = torch.arange(st["total"], device=lens.device)
    seq = torch.searchsorted(cu, row, right=True) - 1
    slot = lens[seq] - (cu[1:] - cu[:-1])[seq] + row - cu[seq]
    return st["table"][seq, slot // case["block"]].long(), slot % case["block"]


def _plain_append(case, st):
    page, at = _places(case, st)
    for x in ("k", "v"):
        st[x + "_codes"][page, :, at], st[x + "_scale"][page, :, at] = _pack(st[x].to(torch.float32))
    return _plain_read(case, st)


def _plain_read(case, st):
    page, at = _places(case, st)
    out = {}
    for x in ("k", "v"):
        if case.get("bits", 4) == 4:
            val = _unpack(st[x + "_codes"][page, :, at], st[x + "_scale"][page, :, at])
        else:
            val = st[x + "_codes"].view(torch.uint8)[page, :, at].view(_F8).to(torch.float32) * st[x + "_scale"][page][..., None]
        out[x] = val.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    return out


def _plain_attend(case, st):
    q, block, hkv = st["q"], case["block"], case["hkv"]
    b, t, hq, d = q.shape
    table = st["table"].long().clamp(min=0)

    def gathered(x):  # [B, Hkv, slots, d]
        val = _unpack(st[x + "_codes"][table], st[x + "_scale"][table])
        return val.transpose(1, 2).reshape(b, hkv, -1, d)

    pos = (st["lens"].long()[:, None] - t + torch.arange(t, device=q.device)[None])[:, None, :, None, None]
    slot = torch.arange(table.shape[1] * block, device=q.device)
    may = slot <= pos
    if case["window"]:
        may = may & (slot > pos - case["window"])
    k = gathered("k")
    qg = q.to(torch.float32).view(b, t, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4)  # [B, Hkv, T, g, d]
    s = torch.matmul(qg.reshape(b, hkv, -1, d), k.transpose(2, 3)).view(b, hkv, t, hq // hkv, -1) / math.sqrt(d)
    del k
    s = torch.where(may, s, torch.full_like(s, -math.inf))
    m = s.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - m)
    del s
    total = p.sum(dim=-1, keepdim=True)
    p = p / total.clamp(min=1e-37)
    out = torch.matmul(p.reshape(b, hkv, -1, p.shape[-1]), gathered("v")).view(b, hkv, t, hq // hkv, d)
    lse = (m + torch.log(total))[..., 0]  # [B, Hkv, T, g]
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(q.dtype),
            "lse": lse.permute(0, 1, 3, 2).reshape(b, hq, t).contiguous()}


def _turned(case, x, cos, sin):
    """Pairs of x [n, heads, d] turned by the angles of cos, sin [n, 1, d / 2]."""
    if case["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)


_EPS = 1e-6  # the default of the package's calls


def _plain_rope(case, st):
    angle = st["positions"].to(torch.float64)[:, None, None] * st["inv_freq"]  # far positions: in 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    out = {}
    for x in ("q", "k"):
        val = st[x].to(torch.float32)
        if case["norm"]:
            r = torch.rsqrt(val.square().mean(dim=-1, keepdim=True) + _EPS)
            w = st[x + "_weight"].to(torch.float32)
            out[x] = _turned(case, val * r * w, cos, sin).to(st[x].dtype)
        else:
            out[x] = _turned(case, val, cos, sin).to(st[x].dtype)
        if not case["backward"]:
            continue
        g = _turned(case, st["d" + x].to(torch.float32), cos, -sin)
        out["d" + x + "_weight"] = None
        if case["norm"]:
            # rows in two steps, so that no sum of 32 bits is long
            dw = (g * val * r).sum(dim=1)
            out["d" + x + "_weight"] = dw.to(torch.float64).sum(dim=0).to(st[x].dtype)
            u = g * w
            g = r * (u - val * (r * r) * (val * u).mean(dim=-1, keepdim=True))
        out["d" + x] = g.to(st[x].dtype)
    return out


# -- the definition in 64 bits -----------------------------------------------

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_value(case, st, x, page, c, slots):
    """Values that the cache holds in `slots` of `page`, KV head c, in 64 bits."""
    if case.get("bits", 4) == 8:
        codes = st[x + "_codes"].view(torch.uint8)[page, c, slots].view(_F8).to(torch.float64)
        return codes * st[x + "_scale"][page, c].to(torch.float64)[..., None]
    steps = torch.tensor(_E2M1 + [-s for s in _E2M1], dtype=torch.float64, device=st["table"].device)
    codes = st[x + "_codes"][page, c, slots].to(torch.int64)
    val = torch.empty((*codes.shape[:-1], case["d"]), dtype=torch.float64, device=codes.device)
    val[..., 0::2], val[..., 1::2] = steps[codes % 16], steps[codes // 16]
    e = st[x + "_scale"][page, c, slots].to(torch.float64) - 127
    return val * torch.exp2(e).repeat_interleave(_GROUP, dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "read": _exact_read, "rope": _exact_rope}[case["op"]](case, st)


def _exact_append(case, st):
    """Nearest value of the format, ties to the even code, at the least power of two that holds the group."""
    out = {}
    steps = torch.tensor(_E2M1, dtype=torch.float64, device=st["table"].device)
    for x in ("k", "v"):
        if st[x].numel() > 1 << 27:
            return None
        val = st[x].to(torch.float64).unflatten(-1, (-1, _GROUP))
        amax = val.abs().amax(dim=-1, keepdim=True)
        e = torch.ceil(torch.log2(amax / 7)).clamp(min=-126)
        e = torch.where(amax > 7 * torch.exp2(e), e + 1, e)
        e = torch.where((amax <= 7 * torch.exp2(e - 1)) & (e > -126), e - 1, e)
        a = val.abs() / torch.exp2(e)
        hi = torch.searchsorted(steps, a.contiguous()).clamp(max=7)
        lo = (hi - 1).clamp(min=0)
        up, down = steps[hi] - a, a - steps[lo]
        code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        out[x] = (torch.copysign(steps[code], val) * torch.exp2(e)).flatten(-2)
    return out


def _exact_read(case, st):
    if st["total"] * case["hkv"] * case["d"] > 1 << 28:
        return None
    out = {x: torch.empty((st["total"], case["hkv"], case["d"]), dtype=torch.float64, device=st["table"].device) for x in ("k", "v")}
    cu = st["cu"].tolist()
    for b, n in enumerate(st["lens"].tolist()):
        slot = torch.arange(n - (cu[b + 1] - cu[b]), n, device=st["table"].device)
        page = st["table"][b].long()[slot // case["block"]]
        for c in range(case["hkv"]):
            for x in ("k", "v"):
                out[x][cu[b]:cu[b + 1], c] = _exact_value(case, st, x, page, c, slot % case["block"])
    return out


def _exact_attend(case, st):
    """Row by row of the definition, a sequence and KV head at a time."""
    hkv, d, block, t = case["hkv"], case["d"], case["block"], case["t"]
    q = st["q"].to(torch.float64)
    group = q.shape[2] // hkv
    out = torch.zeros_like(q)
    lse = torch.full((q.shape[0], q.shape[2], t), -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(st["lens"].tolist()):
        first = max(0, n - t - case["window"] + 1) if case["window"] else 0
        slot = torch.arange(first, n, device=q.device)
        page = st["table"][b].long()[slot // block]
        for c in range(hkv):
            k, v = (_exact_value(case, st, x, page, c, slot % block) for x in ("k", "v"))
            for i in range(t):
                p = n - t + i
                lo = max(0, p - case["window"] + 1) if case["window"] else 0
                at = slice(lo - first, p + 1 - first)
                rows = slice(c * group, (c + 1) * group)
                s = q[b, i, rows] @ k[at].T / math.sqrt(d)
                lse[b, rows, i] = torch.logsumexp(s, dim=-1)
                out[b, i, rows] = torch.softmax(s, dim=-1) @ v[at]
    return {"out": out, "lse": lse}


def _exact_rope(case, st):
    if st["q"].numel() > 1 << 29:
        return None
    d = case["d"]
    i = torch.arange(d // 2, dtype=torch.float64, device=st["q"].device)
    angle = st["positions"].to(torch.float64)[:, None, None] * torch.exp(-2 * i / d * math.log(10000.0))
    turn = torch.polar(torch.ones_like(angle), angle)
    # pairs as complex numbers, turned by a product
    halves = (lambda x: torch.complex(x[..., 0::2], x[..., 1::2])) if case["interleaved"] else (lambda x: torch.complex(x[..., :d // 2], x[..., d // 2:]))
    whole = (lambda z: torch.view_as_real(z).flatten(-2)) if case["interleaved"] else (lambda z: torch.cat([z.real, z.imag], dim=-1))
    out = {}
    for x in ("q", "k"):
        val = st[x].to(torch.float64)
        norm = (val.square().mean(dim=-1, keepdim=True) + _EPS).sqrt() if case["norm"] else torch.ones((), dtype=torch.float64, device=val.device)
        w = st[x + "_weight"].to(torch.float64) if case["norm"] else torch.ones((d,), dtype=torch.float64, device=val.device)
        unit = val / norm
        out[x] = whole(halves(unit * w) * turn)
        if case["backward"]:
            g = whole(halves(st["d" + x].to(torch.float64)) * turn.conj())
            out["d" + x + "_weight"] = (g * unit).sum(dim=(0, 1)) if case["norm"] else None
            g = g * w
            out["d" + x] = (g - unit * (g * unit).mean(dim=-1, keepdim=True)) / norm if case["norm"] else g
    return out
