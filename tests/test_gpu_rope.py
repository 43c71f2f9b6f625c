"""Norms of queries and keys with the rotation, forward and backward, on the GPU
against the formulas in 64 bits.

Bounds (half steps u = 2^-24 of fp32).  Forward: the sum of 128 squares (16
products in a lane, 4 joins: 20 u, half of it in the root), the root (4 u), two
products, cos and sin (an argument off by 2^-26 of a half turn, two ulps of the
result: 8 u of 1), the scale, and the turn's products and sum (3 u): below 32 u =
2^-19 of |a| + |b|, a pair's members, and half a step of the output's type.
Backward: g likewise, and dx = r (u - x r^2 mean(x u)) two sums and a few
products more: 2^-18 of r (|u| + |x| r^2 mean |x u|).  Weights' gradients: a sum
of N terms in any order is off by N u of the sum of their magnitudes, and each
term by 2^-18."""
import math

import numpy as np
import pytest
import torch

import long_context_sparse_landmark_gb300 as msa
from tests.gpu_helpers import binding, check_guards, gempty, gfull

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().double().cpu().numpy()


def pairs(x, interleaved):
    d = x.shape[-1]
    return (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :d // 2], x[..., d // 2:])


def joined(a, b, interleaved):
    if not interleaved:
        return np.concatenate([a, b], axis=-1)
    return np.stack([a, b], axis=-1).reshape(*a.shape[:-1], 2 * a.shape[-1])


def angles(positions, freqs):
    """Position times frequency, less whole turns, in integers of 2^-64 of a turn."""
    freqs = [int(f) for f in freqs]
    return np.array([[[int(p) * f % 2 ** 64 / 2.0 ** 64 * 2 * math.pi for f in freqs]] for p in positions])


def turned(x, ang, interleaved, back=False):
    a, b = pairs(x, interleaved)
    c, s = np.cos(ang), np.sin(ang) * (-1 if back else 1)
    return joined(a * c - b * s, a * s + b * c, interleaved)


def forward(x, w, ang, eps, interleaved, mscale):
    z = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    a, b = pairs(z, interleaved)
    size = joined(np.abs(a) + np.abs(b), np.abs(a) + np.abs(b), interleaved)
    return mscale * turned(z, ang, interleaved), abs(mscale) * size * 2.0 ** -19


def backward(dy, x, w, ang, eps, interleaved, mscale):
    g = mscale * turned(dy, ang, interleaved, back=True)
    a, b = pairs(dy, interleaved)
    size = abs(mscale) * joined(np.abs(a) + np.abs(b), np.abs(a) + np.abs(b), interleaved)
    if w is None:
        return g, size * 2.0 ** -19, None, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = g * w
    dx = r * (u - x * r * r * (x * u).mean(-1, keepdims=True))
    su = size * np.abs(w)
    tol = 2.0 ** -18 * r * (su + np.abs(x) * r * r * (np.abs(x) * su).mean(-1, keepdims=True))
    n = x.shape[0] * x.shape[1]
    dw = (g * x * r).sum((0, 1))
    return dx, tol, dw, (size * np.abs(x) * r).sum((0, 1)) * (2.0 ** -18 + n * 2.0 ** -24)


def close(got, want, tol, what):
    x = f64(got)
    assert x.shape == want.shape
    if not x.size:
        return
    err = np.abs(x - want)
    most = tol * (1 + HALF[got.dtype]) + np.abs(want) * HALF[got.dtype] + 2.0 ** -133
    assert np.isfinite(x).all() and (err <= most).all(), f"{what}: {np.max(err / most):.3g} of the bound"


def inputs(n, hq, hkv, d, dt, seed=1, fused=True, far=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if fused:  # slices of a common tensor
        qkv = (torch.randn((n, hq + 2 * hkv, d), generator=gen, device=DEV) * 2).to(dt)
        q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    else:
        q = torch.randn((n, hq, d), generator=gen, device=DEV).to(dt)
        k = torch.randn((n, hkv, d), generator=gen, device=DEV).to(dt)
    if far:
        pos = torch.randint(-far, far, (n,), generator=gen, device=DEV)
    else:
        pos = torch.arange(n, device=DEV)
    return q, k, pos


CASES = [
    # n, hq, hkv, d, dtype, weight dtype (None: no norm), interleaved, fused, far
    (1, 1, 1, 64, "f32", "f32", False, False, 0),
    (1, 64, 8, 128, "bf16", "bf16", False, True, 1 << 20),
    (3, 5, 1, 128, "bf16", "f32", True, True, 1 << 20),
    (7, 3, 2, 64, "f32", "bf16", True, True, 1 << 30),
    (130, 8, 2, 128, "f32", "f32", False, True, 0),
    (257, 2, 1, 64, "bf16", "bf16", False, True, 1 << 20),
    (600, 1, 1, 64, "f32", "f32", True, False, 1 << 20),
    (33, 16, 4, 128, "bf16", None, False, True, 1 << 40),
    (33, 7, 3, 64, "f32", None, True, True, 1 << 60),
    (2000, 4, 1, 128, "bf16", "f32", False, True, 0),
    (41, 4, 0, 128, "bf16", "bf16", True, False, 1 << 20),   # queries alone
]


def weights(d, w_dt, seed=9):
    if w_dt is None:
        return None, None
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = torch.float32 if w_dt == "f32" else torch.bfloat16
    return tuple((1 + 0.3 * torch.randn((d,), generator=gen, device=DEV)).to(dt) for _ in range(2))


@pytest.mark.parametrize("n,hq,hkv,d,dtype,w_dt,inter,fused,far", CASES)
def test_against_the_formulas(n, hq, hkv, d, dtype, w_dt, inter, fused, far):
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    q, k, pos = inputs(n, hq, hkv, d, dt, fused=fused, far=far)
    qw, kw = weights(d, w_dt)
    inv = [500000.0 ** (-2 * i / d) for i in range(d // 2)]
    freqs = msa.rotary_frequencies(d, inv_freq=inv)
    ang = angles(pos.tolist(), freqs.tolist())
    eps, mscale = 1e-5, 1.25
    how = dict(q_weight=qw, k_weight=kw, eps=eps, interleaved=inter, mscale=mscale)
    outs = msa.qk_norm_rope(q, k, pos, freqs, **how)
    gen = torch.Generator(device=DEV).manual_seed(4)
    dys = [torch.randn(x.shape, generator=gen, device=DEV).to(dt) for x in (q, k)]
    grads = msa.qk_norm_rope_backward(*dys, q, k, pos, freqs, **how)
    for i, (x, w) in enumerate(((q, qw), (k, kw))):
        w64 = None if w is None else f64(w)
        want, tol = forward(f64(x), w64, ang, eps, inter, mscale)
        assert outs[i].shape == x.shape and outs[i].dtype == dt and outs[i].is_contiguous()
        close(outs[i], want, tol, "qk"[i])
        dx, tol, dw, tol_w = backward(f64(dys[i]), f64(x), w64, ang, eps, inter, mscale)
        close(grads[i], dx, tol, "d" + "qk"[i])
        if w is None:
            assert grads[2 + i] is None
        else:
            assert grads[2 + i].dtype == w.dtype
            close(grads[2 + i], dw, tol_w, "dw of " + "qk"[i])
    again = msa.qk_norm_rope_backward(*dys, q, k, pos, freqs, **how)
    for a, b in zip(grads, again):
        assert a is None or torch.equal(a, b)


def test_one_side_alone_has_a_norm():
    d = 64
    q, k, pos = inputs(50, 4, 2, d, torch.float32)
    freqs = msa.rotary_frequencies(d)
    ang = angles(range(50), freqs.tolist())
    w = weights(d, "f32")[0]
    dys = [torch.randn(x.shape, device=DEV) for x in (q, k)]
    for qw, kw in ((w, None), (None, w)):
        outs = msa.qk_norm_rope(q, k, pos, freqs, qw, kw)
        grads = msa.qk_norm_rope_backward(*dys, q, k, pos, freqs, qw, kw)
        for i, (x, ww) in enumerate(((q, qw), (k, kw))):
            w64 = None if ww is None else f64(ww)
            close(outs[i], *forward(f64(x), w64, ang, 1e-6, False, 1.0), "out")
            dx, tol, dw, tol_w = backward(f64(dys[i]), f64(x), w64, ang, 1e-6, False, 1.0)
            close(grads[i], dx, tol, "dx")
            assert (grads[2 + i] is None) == (ww is None)
            if ww is not None:
                close(grads[2 + i], dw, tol_w, "dw")


def test_gradients_against_differences():
    """The kernel's gradients against central differences of the formula in 64
    bits: error h^2 times third derivatives (of order one to ten here) and 2^-53 / h."""
    d, n, hq, hkv = 64, 3, 2, 1
    q, k, pos = inputs(n, hq, hkv, d, torch.float32, seed=5)
    ang = angles(range(n), msa.rotary_frequencies(d).tolist())
    qw, kw = weights(d, "f32")
    dys = [torch.randn(x.shape, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV) for x in (q, k)]
    grads = msa.qk_norm_rope_backward(*dys, q, k, pos, msa.rotary_frequencies(d), qw, kw)
    rng = np.random.default_rng(1)
    h = 1e-4
    for i, (x, w) in enumerate(((q, qw), (k, kw))):
        x64, w64, dy = f64(x), f64(w), f64(dys[i])

        def loss(a, b):
            return (forward(a, b, ang, 1e-6, False, 1.0)[0] * dy).sum()

        for _ in range(20):
            at = tuple(rng.integers(0, s) for s in x64.shape)
            e = np.zeros_like(x64)
            e[at] = h
            diff = (loss(x64 + e, w64) - loss(x64 - e, w64)) / (2 * h)
            assert abs(f64(grads[i])[at] - diff) <= 1e-5 * max(1.0, abs(diff))
            j = rng.integers(0, d)
            e = np.zeros(d)
            e[j] = h
            diff = (loss(x64, w64 + e) - loss(x64, w64 - e)) / (2 * h)
            assert abs(f64(grads[2 + i])[j] - diff) <= 1e-5 * max(1.0, abs(diff))


def test_far_positions_keep_their_angles():
    """Positions of a million and of 2^62: the angle is that of exact integers."""
    d = 128
    pos = torch.tensor([0, 1, -1, 999_999, 1_048_575, 2 ** 40 + 1, -(2 ** 40), 2 ** 62 + 12345, -(2 ** 63)],
                       device=DEV)
    n = pos.numel()
    q = torch.zeros((n, 1, d), device=DEV)
    q[..., :d // 2] = 1.0
    freqs = msa.rotary_frequencies(d)
    out, _ = msa.qk_norm_rope(q, q, pos, freqs)
    for i, p in enumerate(pos.tolist()):
        for j, f in enumerate(freqs.tolist()):
            turn = (p * f) % 2 ** 64 / 2 ** 64
            assert abs(float(out[i, 0, j]) - math.cos(2 * math.pi * turn)) < 2.0 ** -21
            assert abs(float(out[i, 0, d // 2 + j]) - math.sin(2 * math.pi * turn)) < 2.0 ** -21


def test_frequencies():
    f = msa.rotary_frequencies(128, base=10000.0)
    assert f.dtype == torch.int64 and f.shape == (64,) and f.is_cuda
    for i in (0, 1, 63):
        want = 10000.0 ** (-2 * i / 128) / (2 * math.pi)
        assert abs((f[i].item() % 2 ** 64) / 2 ** 64 - want) <= want * 2.0 ** -50 + 2.0 ** -64
    # a frequency of several turns, and a negative one, count within a turn
    g = msa.rotary_frequencies(4, inv_freq=torch.tensor([2 * math.pi * 3.25, -2 * math.pi * 0.25]))
    assert g.tolist() == pytest.approx([2 ** 62, -(2 ** 62)], rel=1e-6)
    for bad in (dict(d=3), dict(d=0), dict(d=4, inv_freq=[1.0]), dict(d=4, inv_freq=[1.0, float("nan")]), dict(d=4, base=0.0)):
        with pytest.raises(ValueError):
            msa.rotary_frequencies(**bad)


def test_extreme_values():
    """Rows of zeros, of tiny and of large values; a NaN stays in its row."""
    d = 64
    q = torch.zeros((6, 1, d), device=DEV)
    q[1] = 1e-30
    q[2] = 1e15
    q[3, 0, 7] = float("nan")
    q[4, 0, 7] = float("inf")
    q[5] = 1.0
    pos = torch.arange(6, device=DEV)
    w = torch.ones((d,), device=DEV)
    out, _ = msa.qk_norm_rope(q, q, pos, msa.rotary_frequencies(d), w, w)
    assert not out[0].any()
    assert (out[1].abs() < 1e-20).all()
    assert torch.isfinite(out[2]).all() and out[2].abs().max() < 1.5
    assert torch.isnan(out[3]).all() and torch.isnan(out[4]).any()
    assert torch.isfinite(out[5]).all()
    grads = msa.qk_norm_rope_backward(torch.ones_like(q[:3]), torch.ones_like(q[:3]), q[:3], q[:3], pos[:3],
                                      msa.rotary_frequencies(d), w, w)
    assert all(torch.isfinite(g).all() for g in grads)


def test_nothing_to_do():
    d = 128
    q = torch.zeros((0, 4, d), device=DEV)
    k = torch.zeros((0, 2, d), device=DEV)
    pos = torch.zeros((0,), dtype=torch.int64, device=DEV)
    f = msa.rotary_frequencies(d)
    w = torch.ones((d,), device=DEV)
    a, b = msa.qk_norm_rope(q, k, pos, f, w, w)
    assert a.shape == q.shape and b.shape == k.shape
    dq, dk, dqw, dkw = msa.qk_norm_rope_backward(q, k, q, k, pos, f, w, w)
    assert dq.shape == q.shape and not dqw.any() and not dkw.any()


def test_only_the_outputs_are_written():
    for d, n, hq, hkv in ((64, 3, 1, 1), (128, 70, 5, 2)):
        q, k, pos = inputs(n, hq, hkv, d, torch.float32)
        f = msa.rotary_frequencies(d)
        w = torch.ones((d,), device=DEV)
        B = binding()
        outs = [gempty(x.shape) for x in (q, k, q, k)] + [gempty((d,)), gempty((d,))]
        ws = gfull((B.qk_norm_rope_bwd_workspace_size(n, hq, hkv, d),), 0xFF, torch.uint8)
        B.qk_norm_rope(q, k, pos, f, w, w, 1e-6, 1.0, False, outs[0], outs[1])
        B.qk_norm_rope_bwd(outs[0], outs[1], q, k, pos, f, w, w, 1e-6, 1.0, False, *outs[2:], ws)
        torch.cuda.synchronize()
        check_guards()
        assert all(torch.isfinite(o).all() for o in outs)   # a workspace of NaN is not read


def test_trainable_and_module():
    """Gradients through the rotation, the norms and the attention: those of the
    two steps one after the other."""
    n, hq, hkv, d = 256, 4, 2, 128
    layer = msa.SparseLandmarkAttention(window=64, num_global=8, qk_norm=True, head_dim=d,
                                        rotary=msa.rotary_frequencies(d)).to(DEV)
    with torch.no_grad():
        for w, s in ((layer.q_weight, 1), (layer.k_weight, 2)):
            w.copy_(1 + 0.2 * torch.randn((d,), generator=torch.Generator(device=DEV).manual_seed(s), device=DEV))
    q0, k0, _ = inputs(n, hq, hkv, d, torch.bfloat16, fused=False)
    v0 = torch.randn((n, hkv, d), device=DEV).bfloat16()
    leaves = [x.clone().requires_grad_() for x in (q0, k0, v0)]
    out = layer(*leaves)
    do = torch.randn_like(out)
    out.backward(do)
    pos = torch.arange(n, device=DEV)
    f = layer.rotary
    qn, kn = msa.qk_norm_rope(q0, k0, pos, f, layer.q_weight, layer.k_weight)
    o2, lse = msa.msa_attention(qn, kn, v0, 64, 8)
    assert torch.equal(out, o2)
    dq, dk, dv = msa.msa_attention_backward(qn, kn, v0, o2, lse, do, 64, 8)
    want = msa.qk_norm_rope_backward(dq, dk, q0, k0, pos, f, layer.q_weight, layer.k_weight)
    assert torch.equal(leaves[2].grad, dv)
    for got, w in zip((leaves[0].grad, leaves[1].grad, layer.q_weight.grad, layer.k_weight.grad), want):
        assert torch.equal(got, w)
    # a batch, other positions, without gradients
    with torch.no_grad():
        both = layer(torch.stack([q0, q0]), torch.stack([k0, k0]), torch.stack([v0, v0]),
                     positions=torch.stack([pos, pos + 1000]))
    assert torch.equal(both[0], o2)
    assert (both[1] - both[0]).abs().max() > 0   # rounded anew: relative angles are the same, bits are not


def test_gradients_reach_the_common_projection():
    """q and k as slices of one leaf, broadcast gradients: the leaf's gradient holds
    both, and zeros where the values are."""
    n, hq, hkv, d = 21, 4, 2, 64
    q, k, pos = inputs(n, hq, hkv, d, torch.float32)
    leaf = torch.cat([q, k, k], dim=1).requires_grad_()
    f = msa.rotary_frequencies(d)
    ws = [w.requires_grad_() for w in weights(d, "f32")]
    a, b = msa.qk_norm_rope_trainable(leaf[:, :hq], leaf[:, hq:hq + hkv], pos, f, *ws)
    (a.sum() + 2 * b.sum()).backward()
    want = msa.qk_norm_rope_backward(torch.ones_like(a), 2 * torch.ones_like(b), q.contiguous(), k.contiguous(), pos, f,
                                     *(w.detach() for w in ws))
    assert torch.equal(leaf.grad[:, :hq], want[0]) and torch.equal(leaf.grad[:, hq:hq + hkv], want[1])
    assert not leaf.grad[:, hq + hkv:].any()
    assert torch.equal(ws[0].grad, want[2]) and torch.equal(ws[1].grad, want[3])
    # one output alone
    b, = torch.autograd.grad(msa.qk_norm_rope_trainable(q, leaf[:, hq:hq + hkv], pos, f)[1].sum(), leaf)
    assert torch.equal(b[:, hq:hq + hkv], msa.qk_norm_rope_backward(torch.zeros_like(q).contiguous(), torch.ones_like(k).contiguous(),
                                                                   q.contiguous(), k.contiguous(), pos, f)[1])


def test_module_in_another_type_and_its_state():
    d = 128
    layer = msa.SparseLandmarkAttention(window=16, num_global=4, rotary=msa.rotary_frequencies(d), qk_norm=True, head_dim=d)
    layer = layer.to(DEV).to(torch.bfloat16)
    assert layer.q_weight.dtype == torch.bfloat16 and layer.rotary.dtype == torch.int64
    assert sorted(layer.state_dict()) == ["k_weight", "q_weight"]
    q, k, pos = inputs(64, 4, 2, d, torch.bfloat16)
    with torch.no_grad():
        out = layer(q, k, k.contiguous())
        qn, kn = msa.qk_norm_rope(q, k, torch.arange(64, device=DEV), layer.rotary, layer.q_weight, layer.k_weight)
    assert torch.equal(out, msa.msa_attention(qn, kn, k.contiguous(), 16, 4)[0])
    assert not list(msa.SparseLandmarkAttention(window=16, num_global=4).state_dict())


def test_second_derivatives_are_refused():
    d = 64
    q, k, pos = inputs(5, 2, 1, d, torch.float32, fused=False)
    q.requires_grad_()
    w = torch.ones((d,), device=DEV, requires_grad=True)
    out, _ = msa.qk_norm_rope_trainable(q, k, pos, msa.rotary_frequencies(d), w, w)
    g, = torch.autograd.grad((out * out).sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        (g.sum() + q.sum()).backward()


def test_a_captured_training_step_replays():
    """Forward and backward of the differentiable form in a CUDA graph; nothing of
    the first step, outside of it, is still held."""
    d = 128
    q, k, pos = inputs(70, 4, 2, d, torch.bfloat16, fused=False)
    f = msa.rotary_frequencies(d)
    ws = weights(d, "f32")
    dys = [torch.randn(x.shape, device=DEV).bfloat16() for x in (q, k)]
    leaves = [x.detach().requires_grad_() for x in (q, k, *ws)]

    def step():
        out = msa.qk_norm_rope_trainable(*leaves[:2], pos, f, *leaves[2:])
        return torch.autograd.grad(out, leaves, dys)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        grads = step()
    for i in range(3):
        with torch.no_grad():
            for x in (q, k, *dys):
                x.copy_(torch.randn(x.shape, device=DEV))
        g.replay()
        for a, b in zip(grads, msa.qk_norm_rope_backward(*dys, q, k, pos, f, *ws)):
            assert torch.equal(a, b)


def test_a_captured_backward_replays():
    d = 128
    q, k, pos = inputs(100, 4, 2, d, torch.bfloat16)
    qw, kw = weights(d, "bf16")
    f = msa.rotary_frequencies(d)
    dys = [torch.randn(x.shape, device=DEV).bfloat16() for x in (q, k)]

    def step():
        return (*msa.qk_norm_rope(q, k, pos, f, qw, kw), *msa.qk_norm_rope_backward(*dys, q, k, pos, f, qw, kw))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(3):
        for x in (q, k, *dys):
            x.copy_(torch.randn(x.shape, device=DEV))
        pos.add_(1000)
        g.replay()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)


def test_another_stream():
    d = 64
    s = torch.cuda.Stream()
    f = msa.rotary_frequencies(d)
    pos = torch.zeros((500,), dtype=torch.int64, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        q = torch.ones((500, 2, d), device=DEV)
    a, b = msa.qk_norm_rope(q, q, pos, f, stream=s)
    g = msa.qk_norm_rope_backward(a, b, q, q, pos, f, stream=s)
    s.synchronize()
    assert (a == 1).all() and (b == 1).all() and (g[0] == 1).all()


def test_refusals():
    d = 128
    q, k, pos = inputs(4, 2, 1, d, torch.bfloat16, fused=False)
    f = msa.rotary_frequencies(d)
    w = torch.ones((d,), device=DEV)
    E = binding().MsaError
    for kw, err in ((dict(q=q.half(), k=k.half()), TypeError), (dict(k=k.float()), TypeError),
                    (dict(pos=pos.int()), TypeError), (dict(pos=pos[:3]), ValueError), (dict(f=f[:10]), ValueError),
                    (dict(f=f.float()), TypeError), (dict(k=k[:3]), ValueError), (dict(q=q[0]), ValueError),
                    (dict(q=q.transpose(0, 1)), ValueError), (dict(w=w[:64]), ValueError), (dict(w=w.half()), TypeError),
                    (dict(w=w.cpu()), ValueError), (dict(pos=pos.cpu()), ValueError),
                    (dict(eps=-1.0), E), (dict(eps=float("nan")), E), (dict(mscale=float("inf")), E),
                    (dict(q=q.flip(2)[..., :64].contiguous(), k=k[..., :64].contiguous()), ValueError)):
        a = dict(q=q, k=k, pos=pos, f=f, w=w, eps=1e-6, mscale=1.0)
        a.update(kw)
        with pytest.raises(err):
            msa.qk_norm_rope(a["q"], a["k"], a["pos"], a["f"], a["w"], None, eps=a["eps"], mscale=a["mscale"])
    with pytest.raises(TypeError):
        msa.qk_norm_rope(q, k, pos, f, w, w.bfloat16())
    with pytest.raises(E):   # heads of 96
        msa.qk_norm_rope(q[..., :96].contiguous(), k[..., :96].contiguous(), pos, msa.rotary_frequencies(96))
    wide = torch.zeros((4, 3 * d + 1), device=DEV)
    with pytest.raises(E):   # tokens not 16 bytes apart
        msa.qk_norm_rope(wide[:, :2 * d].unflatten(1, (2, d)), torch.zeros((4, 1, d), device=DEV), pos, f)
    with pytest.raises(E):   # not 16-byte aligned
        msa.qk_norm_rope(wide.reshape(-1)[1:1 + 4 * 3 * d].view(4, 3, d), torch.zeros((4, 1, d), device=DEV), pos, f)
    with pytest.raises(ValueError):
        msa.qk_norm_rope_backward(q[:3], k, q, k, pos, f)
    with pytest.raises(TypeError):
        msa.qk_norm_rope_backward(q.float(), k, q, k, pos, f)
    with pytest.raises(ValueError):
        msa.qk_norm_rope(q.cpu(), k.cpu(), pos.cpu(), f.cpu())
    with pytest.raises(ValueError):
        msa.SparseLandmarkAttention(window=4, num_global=0, qk_norm=True)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv", [(1, 9000), (16, 16384), (16384, 16)])
def test_sides_of_unequal_numbers_of_heads(hq, hkv, dt):
    """Both sides are written, however few of the rows are one's."""
    n, d = 8, 64
    q, k, pos = inputs(n, hq, hkv, d, dt, fused=False)
    f, (qw, kw) = msa.rotary_frequencies(d), weights(d, "f32")
    ang = angles(range(n), f.tolist())
    dys = [torch.randn(x.shape, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV).to(dt) for x in (q, k)]
    B = binding()
    nan = float("nan")
    outs = [gfull(x.shape, nan, dt) for x in (q, k)]
    grads = [gfull(x.shape, nan, dt) for x in (q, k)] + [gfull((d,), nan) for _ in range(2)]
    ws = gfull((B.qk_norm_rope_bwd_workspace_size(n, hq, hkv, d),), 0xFF, torch.uint8)
    B.qk_norm_rope(q, k, pos, f, qw, kw, 1e-6, 1.0, False, *outs)
    B.qk_norm_rope_bwd(*dys, q, k, pos, f, qw, kw, 1e-6, 1.0, False, *grads, ws)
    for i, (x, w) in enumerate(((q, qw), (k, kw))):
        close(outs[i], *forward(f64(x), f64(w), ang, 1e-6, False, 1.0), "qk"[i])
        dx, tol, dw, tol_w = backward(f64(dys[i]), f64(x), f64(w), ang, 1e-6, False, 1.0)
        close(grads[i], dx, tol, "d" + "qk"[i])
        close(grads[2 + i], dw, tol_w, "dw of " + "qk"[i])


@pytest.mark.parametrize("d,dt", [(64, torch.float32), (128, torch.bfloat16)])
def test_gradients_of_tiny_rows_without_eps(d, dt):
    """Rows of 2^-64: r is 2^64, its square past fp32's range.  Squares are
    subnormal, 2^-21 of themselves apart: r is off by 2^-22 more, within the bound's
    room."""
    q, k, pos = inputs(20, 2, 1, d, torch.float32, fused=False)
    q, k = (torch.where(x.abs() < 0.25, 0.25, x).mul(2.0 ** -64).to(dt) for x in (q, k))
    f, (qw, kw) = msa.rotary_frequencies(d), weights(d, "f32")
    ang = angles(range(20), f.tolist())
    gen = torch.Generator(device=DEV).manual_seed(4)
    dys = [torch.randn(x.shape, generator=gen, device=DEV).to(dt) for x in (q, k)]
    outs = msa.qk_norm_rope(q, k, pos, f, qw, kw, eps=0.0)
    grads = msa.qk_norm_rope_backward(*dys, q, k, pos, f, qw, kw, eps=0.0)
    for i, (x, w) in enumerate(((q, qw), (k, kw))):
        close(outs[i], *forward(f64(x), f64(w), ang, 0.0, False, 1.0), "qk"[i])
        dx, tol, dw, tol_w = backward(f64(dys[i]), f64(x), f64(w), ang, 0.0, False, 1.0)
        close(grads[i], dx, tol, "d" + "qk"[i])
        close(grads[2 + i], dw, tol_w, "dw of " + "qk"[i])


@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "bf16")])
def test_long_sums_of_the_weights_gradients(d, dtype):
    """Equal terms 1 + 2^-17 - 2^-23, some 216 passes a thread: a sum of 32 bits
    beyond 128 drops 2^-17 of each.  Where no fp32 sum is longer than a group of 8
    passes and 8 lanes (11 half steps), a term has 4 half steps (its product, and
    two ulps of rsqrtf twice over) and the result one: 2^-20 of it."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    n = 304 * 216 * (4096 // d)
    m = 1 + 2.0 ** -17 - 2.0 ** -23
    x = torch.ones((n, 1, d), dtype=dt, device=DEV)
    pos = torch.zeros((n,), dtype=torch.int64, device=DEV)
    w = torch.ones((d,), device=DEV)
    for hkv in (0, 1):
        k = x[:, :hkv]
        g = msa.qk_norm_rope_backward(x, k, x, k, pos, msa.rotary_frequencies(d), w, w, eps=0.0, mscale=m)
        for i in range(1 + hkv):
            off = (g[2 + i].double() / (n * m) - 1).abs().max().item()
            assert off <= 2.0 ** -20, off * 2.0 ** 24


def test_infinite_sums_of_the_weights_gradients():
    """Terms past fp32's range give infinities, not NaN; a NaN among them a NaN."""
    d, n = 64, 40000
    x = torch.ones((n, 1, d), device=DEV)
    dy = torch.ones((n, 1, d), device=DEV)
    dy[100:200, 0, 3] = 2e38
    dy[30000:, 0, 4] = -2e38
    dy[7, 0, 5] = float("inf")
    dy[9, 0, 6] = float("nan")
    w = torch.ones((d,), device=DEV)
    pos = torch.zeros((n,), dtype=torch.int64, device=DEV)
    g = msa.qk_norm_rope_backward(dy, x[:, :0], x, x[:, :0], pos, msa.rotary_frequencies(d), w, None, eps=0.0)[2]
    # (dims 3 .. 5 are the first of their pairs: a zero sine times an infinity is a NaN in the others')
    assert g[3] == math.inf and g[4] == -math.inf and g[5] == math.inf and torch.isnan(g[6])
    keep = [i for i in range(d) if i % 32 not in (3, 4, 5, 6)]
    assert (g[keep] == n).all()


def test_positions_of_a_batch_in_the_module():
    """One sequence's positions [n] serve every sequence of a batch."""
    n, d = 64, 128
    layer = msa.SparseLandmarkAttention(window=16, num_global=4, rotary=msa.rotary_frequencies(d))
    layer = layer.to(DEV)
    q, k, _ = inputs(n, 4, 2, d, torch.bfloat16, fused=False)
    pos = torch.arange(n, device=DEV) * 3 + 1000
    with torch.no_grad():
        one = layer(q, k, k, positions=pos)
        both = layer(torch.stack([q, q]), torch.stack([k, k]), torch.stack([k, k]), positions=pos)
    assert torch.equal(both[0], one) and torch.equal(both[1], one)
    with pytest.raises(ValueError):
        layer(torch.stack([q, q]), torch.stack([k, k]), torch.stack([k, k]), positions=pos[:5])
    with pytest.raises(ValueError):
        layer(torch.stack([q, q]), torch.stack([k, k]), torch.stack([k, k]), positions=torch.stack([pos] * 3))


# Sizes of 20 passes a CTA and more, forward (608 CTAs) and backward (304), both
# sides: several groups of 8 passes, and a ring that wraps.  Of hq + hkv heads, 32
# (d = 128) or 64 rows a pass.
LONG = [
    # hq, hkv, d, dtype, interleaved, norm
    (5, 3, 128, "bf16", False, True),
    (5, 3, 128, "f32", True, True),
    (24, 8, 128, "bf16", True, True),
    (24, 8, 128, "f32", False, True),
    (4, 1, 128, "bf16", False, False),
    (7, 2, 64, "bf16", False, True),
    (7, 2, 64, "f32", True, True),
    (1, 1, 64, "bf16", True, True),    # groups of one pass
    (1, 1, 64, "f32", False, False),
]


def long_tokens(hq, hkv, d, ctas):
    return (32 * ctas * (4096 // d) * 4 // 3) // (hq + hkv) | 1


@pytest.mark.parametrize("hq,hkv,d,dtype,inter,norm", LONG)
def test_many_passes_give_what_one_gives(hq, hkv, d, dtype, inter, norm):
    """Rows of a long call equal those of calls so short that each CTA has one
    pass, which the other tests hold to the formulas: a row's arithmetic is the
    same wherever it lies."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    n = long_tokens(hq, hkv, d, 608)
    q, k, pos = inputs(n, hq, hkv, d, dt, far=1 << 40)
    qw, kw = weights(d, "f32" if norm else None)
    gen = torch.Generator(device=DEV).manual_seed(4)
    dys = [torch.randn(x.shape, generator=gen, device=DEV).to(dt) for x in (q, k)]
    f = msa.rotary_frequencies(d)
    how = dict(q_weight=qw, k_weight=kw, interleaved=inter, mscale=0.75)
    outs = msa.qk_norm_rope(q, k, pos, f, **how)
    grads = msa.qk_norm_rope_backward(*dys, q, k, pos, f, **how)
    step = 300 * (4096 // d) // (hq + hkv)
    for at in range(0, n, step):
        s = slice(at, at + step)
        few = msa.qk_norm_rope(q[s], k[s], pos[s], f, **how)
        few_g = msa.qk_norm_rope_backward(*(x[s] for x in dys), q[s], k[s], pos[s], f, **how)
        for a, b in zip((*outs, *grads[:2]), (*few, *few_g[:2])):
            assert torch.equal(a[s], b), f"tokens {at} on"


@pytest.mark.parametrize("hq,hkv,d,dtype,inter,norm", [c for c in LONG if c[-1]])
def test_every_row_counts_in_the_weights_gradients(hq, hkv, d, dtype, inter, norm):
    """Values of +-1, no angle, no eps: r is 1 (rsqrtf: two ulps, 2^-22), each term
    an odd integer and every partial sum an integer below 2^24: exact but for r,
    2^-22 of the sum of their magnitudes (2 on average), below the 1 that a row
    adds at least."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    n = long_tokens(hq, hkv, d, 304)
    gen = torch.Generator(device=DEV).manual_seed(6)
    x = [(torch.randint(0, 2, (n, h, d), generator=gen, device=DEV) * 2 - 1).to(dt) for h in (hq, hkv)]
    dy = [(torch.randint(0, 4, (n, h, d), generator=gen, device=DEV) * 2 - 3).to(dt) for h in (hq, hkv)]
    pos = torch.zeros((n,), dtype=torch.int64, device=DEV)
    w = weights(d, "f32")
    grads = msa.qk_norm_rope_backward(*dy, *x, pos, msa.rotary_frequencies(d), *w, eps=0.0, interleaved=inter)
    for i in range(2):
        terms = x[i].double() * dy[i].double()
        want, tol = terms.sum((0, 1)), terms.abs().sum((0, 1)) * 2.0 ** -22
        assert tol.max() < 0.5
        assert ((grads[2 + i].double() - want).abs() <= tol).all()
