"""RMS norm and rotation of query and key heads over libkda.so (include/kda.h).

    q, k = kda.qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, 1e-6, "BSND")

Per token and head, r = 1 / sqrt(mean(x^2) + eps) and n = x r weight; the pair i of the first
2 * len(inv_freq) channels then turns by position * inv_freq[i].  The outputs are dense in the
layout, as flash_kda and decode take them.  ``qk_norm_rope`` is differentiable with respect to q, k
and the weights (once, in reverse mode: inputs with a forward-mode tangent are refused);
``qk_norm_rope_backward`` is its backward pass as a call of its own.  Neither can be recorded by
torch.jit.trace or make_fx, nor batched by vmap.

Single tokens (a decode batch) are the TND layout with one token per sequence: q [B, Nq, D],
positions [B].
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import KdaError, KdaQkShape, check
from ._views import (address, dense_like, dtype_code, expect, expect_dense, launch_on, needs_grad,
                     negated, no_tangents, not_recorded, readable, results, used_on, view, written)
from .api import LAYOUTS


_LIMIT = 1 << 31
_workspace_bytes = {}


def _check(q, k, positions, inv_freq, q_weight, k_weight, eps, layout, interleaved) -> KdaQkShape:
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("qk_norm_rope runs on a CUDA device only")
    if layout not in LAYOUTS:
        raise KdaError(2, f"layout {layout!r}")
    if q.dim() != (3 if layout == "TND" else 4) or k.dim() != q.dim():
        raise KdaError(3, f"q and k have {q.dim()} and {k.dim()} dimensions under {layout}")
    code = dtype_code(q, "q")
    if layout == "TND":
        (S, Nq, D), B, Nk = q.shape, 1, k.shape[1]
        k_shape, tokens = (S, Nk, D), (S,)
    elif layout == "BSND":
        (B, S, Nq, D), Nk = q.shape, k.shape[2]
        k_shape, tokens = (B, S, Nk, D), (B, S)
    else:
        (B, Nq, S, D), Nk = q.shape, k.shape[1]
        k_shape, tokens = (B, Nk, S, D), (B, S)
    if B >= _LIMIT or S >= _LIMIT or Nq >= _LIMIT or Nk >= _LIMIT or D >= _LIMIT:
        raise KdaError(3, "a size of q or k does not fit 32 bits")
    if q.is_neg():
        negated("q")
    expect(k, "k", q.dtype, dev, k_shape)
    if positions is not None:
        expect_dense(positions, "positions", torch.int32, dev, tokens)
    turned = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise KdaError(3, "inv_freq must be a vector")
        turned = 2 * inv_freq.shape[0]
        expect_dense(inv_freq, "inv_freq", torch.float32, dev, inv_freq.shape)
    if q_weight is not None:
        expect_dense(q_weight, "q_weight", torch.float32, dev, (D,))
    if k_weight is not None:
        expect_dense(k_weight, "k_weight", torch.float32, dev, (D,))
    return KdaQkShape(LAYOUTS[layout], B, Nq, Nk, S, D, code, turned, int(bool(interleaved)), eps)


def _forward(q, k, positions, inv_freq, q_weight, k_weight, eps, layout, interleaved, q_out, k_out,
             stream):
    shape = _check(q, k, positions, inv_freq, q_weight, k_weight, eps, layout, interleaved)
    dev = q.device
    results(q_out, k_out)
    given = q_out, k_out
    if q_out is not None:
        expect_dense(q_out, "q_out", q.dtype, dev, q.shape)
    if k_out is not None:
        expect_dense(k_out, "k_out", q.dtype, dev, k.shape)
    ctx, handle = launch_on(dev, stream)
    if stream is not None:
        used_on(stream, q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out)
    with ctx:
        if q_out is None:
            q_out = dense_like(q)
        if k_out is None:
            k_out = dense_like(k)
        check(_lib.load().kda_qk_norm_rope(
            ctypes.byref(shape), ctypes.byref(view(q, "q", layout)),
            ctypes.byref(view(k, "k", layout)), address(positions), address(inv_freq), address(q_weight),
            address(k_weight), q_out.data_ptr(), k_out.data_ptr(), handle), "kda_qk_norm_rope")
    written(*given)
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, q_weight, k_weight,
                          eps: float, layout: str, interleaved: bool = False,
                          dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None):
    """Gradients (dq, dk, dq_weight, dk_weight) of qk_norm_rope at its inputs.

    dq_out, dk_out: the outputs' gradients, like q and k (strides allowed).  dq and dk may be given
    (dq_out and dk_out themselves where those are dense).  A weight's gradient is None when the
    weight is.
    """
    calls = _lib.calls()
    if dq is None and dk is None and stream is None and calls is not None:
        res = calls.qk_backward(q, k, positions, inv_freq, q_weight, k_weight, eps, layout,
                                interleaved, dq_out, dk_out)
        if res is not None:
            return res if res.__class__ is tuple else check(res, "kda_qk_norm_rope_backward")
    not_recorded("qk_norm_rope_backward")
    no_tangents("qk_norm_rope_backward", dq_out, dk_out, q, k, inv_freq, q_weight, k_weight)
    shape = _check(q, k, positions, inv_freq, q_weight, k_weight, eps, layout, interleaved)
    dev = q.device
    expect(dq_out, "dq_out", q.dtype, dev, q.shape)
    expect(dk_out, "dk_out", q.dtype, dev, k.shape)
    results(dq, dk)
    given = dq, dk
    for t, name, like in ((dq, "dq", q), (dk, "dk", k)):
        if t is not None:
            expect_dense(t, name, q.dtype, dev, like.shape)
    L = _lib.load()
    ws_bytes = _workspace_bytes.get(shape.D)  # it goes by the head dim alone
    if ws_bytes is None:
        size = ctypes.c_size_t(0)
        check(L.kda_qk_norm_rope_workspace_size(ctypes.byref(shape), ctypes.byref(size)),
              "kda_qk_norm_rope_workspace_size")
        ws_bytes = _workspace_bytes[shape.D] = size.value
    ctx, handle = launch_on(dev, stream)
    if stream is not None:
        used_on(stream, dq_out, dk_out, q, k, positions, inv_freq, q_weight, k_weight, dq, dk)
    with ctx:
        if dq is None:
            dq = dense_like(q)
        if dk is None:
            dk = dense_like(k)
        dqw = torch.empty_like(q_weight) if q_weight is not None else None
        dkw = torch.empty_like(k_weight) if k_weight is not None else None
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        check(L.kda_qk_norm_rope_backward(
            ctypes.byref(shape), ctypes.byref(view(dq_out, "dq_out", layout)),
            ctypes.byref(view(dk_out, "dk_out", layout)), ctypes.byref(view(q, "q", layout)),
            ctypes.byref(view(k, "k", layout)), address(positions), address(inv_freq), address(q_weight),
            address(k_weight), ws.data_ptr(), ws_bytes, dq.data_ptr(), dk.data_ptr(),
            address(dqw), address(dkw), handle), "kda_qk_norm_rope_backward")
    written(*given)
    return dq, dk, dqw, dkw


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, q_weight, k_weight, eps, layout, interleaved):
        ctx.save_for_backward(q, k, positions, inv_freq, q_weight, k_weight)
        ctx.call = eps, layout, interleaved
        # no gradient is wanted in here, so this takes the short way
        return qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, layout, interleaved)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        dq_out, dk_out = readable(dq_out), readable(dk_out)
        q, k, positions, inv_freq, q_weight, k_weight = ctx.saved_tensors
        dq, dk, dqw, dkw = qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq,
                                                 q_weight, k_weight, *ctx.call)
        return dq, dk, None, None, dqw, dkw, None, None, None


def qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps: float, layout: str,
                 interleaved: bool = False, q_out: torch.Tensor | None = None,
                 k_out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Norm and rotation of q and k in one pass.  Returns (q_out, k_out), dense in the layout.

    q, k: bf16, fp16 or fp32, head dim 128 or 64, any numbers of heads (any strides over slots,
    heads and tokens; channels contiguous and 16-byte aligned, so slices of a fused projection are
    taken as they lie).  positions: int32 [B, S] ([T] under TND) or None for 0..S-1; a negative one
    marks padding (zeros out, no part in the gradients).  inv_freq: fp32, radians per position, up
    to D/2 of them in multiples of 8, or None for no rotation.  q_weight, k_weight: fp32 [D] or
    None.  Pairs are (i, i + len(inv_freq)), or (2i, 2i + 1) when ``interleaved``.  q_out and k_out
    may be q and k themselves where those are dense.

    Differentiable when q, k or a weight requires a gradient; then q_out, k_out and stream cannot
    be given (choose the stream with torch.cuda.stream).  Supplied results may not require a
    gradient, and autograd notices that they are written.  A call on a given stream does not wait for
    the streams that made its inputs.
    """
    calls = _lib.calls()
    if q_out is None and k_out is None and stream is None and calls is not None:
        res = calls.qk_forward(q, k, positions, inv_freq, q_weight, k_weight, eps, layout, interleaved)
        if res is not None:
            return res if res.__class__ is tuple else check(res, "kda_qk_norm_rope")
    not_recorded("qk_norm_rope")
    if inv_freq is not None and needs_grad(inv_freq):
        raise ValueError("inv_freq has no gradient here")
    if needs_grad(q, k, q_weight, k_weight):
        if q_out is not None or k_out is not None or stream is not None:
            raise ValueError("q_out, k_out and stream cannot be combined with inputs that require "
                             "a gradient")
        return _QkNormRope.apply(q, k, positions, inv_freq, q_weight, k_weight, eps, layout,
                                 interleaved)
    return _forward(q, k, positions, inv_freq, q_weight, k_weight, eps, layout, interleaved, q_out,
                    k_out, stream)
