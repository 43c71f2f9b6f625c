"""Norms of queries and keys for each head, with the rotary position embedding
in the same pass (include/msa_rope.h): what stands between a layer's projections
and its attention or its cache.

``qk_norm_rope`` and ``qk_norm_rope_backward`` run the kernels,
``qk_norm_rope_trainable`` is the differentiable form.  As in ``cache``, every
call runs on the device of its tensors and, unless ``stream`` says otherwise, on
that device's current stream.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import _binding as B

_INPUTS = (torch.float32, torch.bfloat16)


def rotary_frequencies(d: int, base: float = 10000.0, inv_freq=None,
                       device="cuda") -> torch.Tensor:
    """Frequencies [d / 2] int64 that ``qk_norm_rope`` takes: turns a position,
    2^64 to the turn.

    ``inv_freq`` are d / 2 angles a position in radians (any sequence of numbers,
    or a tensor), as an extension of the context scales them; by default
    base^(-2 i / d)."""
    if d < 2 or d % 2:
        raise ValueError("d must be even and >= 2")
    if inv_freq is None:
        if not base > 0:
            raise ValueError("base must be > 0")
        inv_freq = [base ** (-2.0 * i / d) for i in range(d // 2)]
    elif isinstance(inv_freq, torch.Tensor):
        inv_freq = inv_freq.detach().to("cpu", torch.float64).reshape(-1).tolist()
    inv_freq = [float(f) for f in inv_freq]
    if len(inv_freq) != d // 2 or not all(math.isfinite(f) for f in inv_freq):
        raise ValueError(f"inv_freq must be {d // 2} finite numbers")
    turns = []
    for f in inv_freq:
        t = round(math.fmod(f / (2 * math.pi), 1.0) * 2 ** 64) % 2 ** 64
        turns.append(t - 2 ** 64 if t >= 2 ** 63 else t)
    return torch.tensor(turns, dtype=torch.int64).to(device)


def _check(q, k, positions, freqs, q_weight, k_weight, grads=()):
    """Checks the tensors' types, shapes and devices; returns the device's index."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [n, Hq, d] and k [n, Hkv, d]")
    n, _, d = q.shape
    dev = q.get_device()
    dt = q.dtype
    if dt not in _INPUTS:
        raise TypeError(f"q must be float32 or bfloat16, not {dt}")
    _want(k, "k", dt, (n, k.shape[1], d), dev)
    _want(positions, "positions", torch.int64, (n,), dev)
    _want(freqs, "freqs", torch.int64, (d // 2,), dev)
    w_dt = None
    for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            if w.dtype not in _INPUTS or w_dt not in (None, w.dtype):
                raise TypeError("the weights must be both float32 or both bfloat16")
            w_dt = w.dtype
            _want(w, what, w_dt, (d,), dev)
    for g, x, what in grads:
        _want(g, what, dt, x.shape, dev)
    return dev


def _want(t, what: str, dtype, shape, dev: int):
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        return
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{what} must be on device {dev}, not {t.device}")


def _run(dev: int, stream, call):
    """call(stream address) with the device current and allocations made for
    the stream that the kernels run on."""
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("stream and tensors are on different devices")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)
    if torch._C._cuda_getDevice() == dev:
        return call(torch._C._cuda_getCurrentRawStream(dev))
    with torch.cuda.device(dev):
        return call(torch._C._cuda_getCurrentRawStream(dev))


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                 eps: float = 1e-6, interleaved: bool = False, mscale: float = 1.0, stream=None):
    """Root-mean-square norm of each head of q [n, Hq, d] and k [n, Hkv, d] (bf16
    or fp32) with its weight [d] (None: no norm of that side), then the rotation
    by positions [n] int64 and freqs (``rotary_frequencies``): pairs of dims (i, i
    + d/2), or (2i, 2i + 1) if ``interleaved``, times ``mscale``.  q and k may be
    slices of one tensor [n, heads, d].  Returns (q, k), new tensors
    (msa_qk_norm_rope)."""
    dev = _check(q, k, positions, freqs, q_weight, k_weight)
    like = dict(dtype=q.dtype, device=q.device)

    def call(s):
        q_out, k_out = torch.empty(q.shape, **like), torch.empty(k.shape, **like)
        B.qk_norm_rope(q, k, positions, freqs, q_weight, k_weight, eps, mscale, interleaved,
                       q_out, k_out, stream=s)
        return q_out, k_out

    return _run(dev, stream, call)


def qk_norm_rope_backward(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor,
                          k: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor,
                          q_weight: torch.Tensor | None = None,
                          k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                          interleaved: bool = False, mscale: float = 1.0, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight; None where there is no weight) of
    sum <dq_out, q_out> + sum <dk_out, k_out> for ``qk_norm_rope``
    (msa_qk_norm_rope_bwd)."""
    dev = _check(q, k, positions, freqs, q_weight, k_weight,
                 ((dq_out, q, "dq_out"), (dk_out, k, "dk_out")))
    n, Hq, d = q.shape
    like = dict(dtype=q.dtype, device=q.device)

    def call(s):
        dq, dk = torch.empty(q.shape, **like), torch.empty(k.shape, **like)
        dqw = None if q_weight is None else torch.empty_like(q_weight)
        dkw = None if k_weight is None else torch.empty_like(k_weight)
        ws = None
        if dqw is not None or dkw is not None:
            ws = torch.empty((B.qk_norm_rope_bwd_workspace_size(n, Hq, k.shape[1], d),),
                             dtype=torch.uint8, device=q.device)
        B.qk_norm_rope_bwd(dq_out, dk_out, q, k, positions, freqs, q_weight, k_weight, eps,
                           mscale, interleaved, dq, dk, dqw, dkw, ws, stream=s)
        return dq, dk, dqw, dkw

    return _run(dev, stream, call)


class _NormRope(torch.autograd.Function):
    """``qk_norm_rope`` as a differentiable op."""

    @staticmethod
    def forward(ctx, q, k, positions, freqs, q_weight, k_weight, eps, interleaved, mscale):
        ctx.save_for_backward(q, k, positions, freqs, q_weight, k_weight)
        ctx.cfg = (eps, interleaved, mscale)
        return qk_norm_rope(q, k, positions, freqs, q_weight, k_weight, eps, interleaved, mscale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, positions, freqs, q_weight, k_weight = ctx.saved_tensors
        dq, dk, dqw, dkw = qk_norm_rope_backward(
            dq_out.to(q.dtype).contiguous(), dk_out.to(q.dtype).contiguous(), q, k, positions,
            freqs, q_weight, k_weight, *ctx.cfg)
        return dq, dk, None, None, dqw, dkw, None, None, None


def qk_norm_rope_trainable(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor,
                           freqs: torch.Tensor, q_weight: torch.Tensor | None = None,
                           k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                           interleaved: bool = False, mscale: float = 1.0):
    """Differentiable ``qk_norm_rope``, in q, k and the weights, once: a gradient of
    the gradients raises.

    A backward pass may be captured into a CUDA graph if its forward is in the
    capture and no earlier graph of the same leaves is still held (PyTorch ties a
    leaf's accumulation to the stream of the first one)."""
    return _NormRope.apply(q, k, positions, freqs, q_weight, k_weight, eps, interleaved, mscale)
