"""The gated recurrence over libkda.so: the vector form of the KDA state (include/kda.h).

    plan = kda.recurrence_plan(x, "BSND", cu_seqlens=None)
    out, final_state = kda.gated_recurrence(x, g, beta, initial_state, A_log, dt_bias, -5.0,
                                            "BSND", plan)

Per sequence, head n and channel d, with flash_kda's activations of the gate and the write logit:

    a_t = exp(lower_bound * sigmoid(exp(A_log[n]) * (g_t + dt_bias[n, d])))
    h_t = a_t h_{t-1} + sigmoid(beta_t[n]) x_t,        out_t = h_t

``gated_recurrence`` is differentiable with respect to x, g, beta, initial_state, A_log and
dt_bias (once, in reverse mode: inputs with a forward-mode tangent are refused).
``gated_recurrence_backward`` is its backward pass as a call of its own, and
``gated_recurrence_step`` one token for each sequence, from the state that a prefill returned.
None of them can be recorded by torch.jit.trace or make_fx, nor batched by vmap.

Every call can be captured in a CUDA graph; the plan is made before.  When a training step is
captured, torch's rule holds: no eager autograd graph of the same leaves may be alive then, since
their gradients would be accumulated on that graph's stream (``torch.autograd.grad`` does not).
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, fields

import numpy as np
import torch

from . import _lib
from ._lib import KdaError, KdaRecurrenceShape, check
from ._views import (DTYPES, address, dense_like, dtype_code, expect, expect_dense, launch_on,
                     needs_grad, no_tangents, not_recorded, readable, results, used_on, view, written)
from .api import LAYOUTS

_F32 = torch.float32
_STATUS_BYTES = 256  # a workspace that holds the device status alone
_P_I32 = ctypes.POINTER(ctypes.c_int32)


@dataclass
class KdaRecurrencePlan:
    """Host and device copies of the schedule, and the sizes that it asks for."""
    shape: KdaRecurrenceShape
    layout: str
    host: np.ndarray
    dev: torch.Tensor
    workspace_bytes: int
    backward_workspace_bytes: int
    states_shape: tuple
    cu_seqlens: np.ndarray | None

    def __post_init__(self):
        sh = self.shape
        self._host_ptr = self.host.ctypes.data_as(_P_I32)
        self._rows = torch.Size({"BNSD": (sh.B, sh.N, sh.S), "BSND": (sh.B, sh.S, sh.N),
                                 "TND": (sh.S, sh.N)}[self.layout])
        self._x = self._rows + torch.Size((sh.D,))
        self._state = torch.Size((sh.B, sh.N, sh.D))
        self._heads = torch.Size((sh.N,))
        self._params = torch.Size((sh.N, sh.D))
        self._index = self.dev.get_device()
        calls = _lib.calls()
        self._handle = calls and calls.plan(
            sh.layout, sh.B, sh.N, sh.S, sh.D, self.host.ctypes.data, self.host.size, self.host,
            self.dev, self.workspace_bytes, self.backward_workspace_bytes, self.states_shape[0])
        self._shapes = {}

    # copies and pickles hold the fields; the addresses and the compiled calls' handle are made anew
    def __getstate__(self):
        return {f.name: getattr(self, f.name) for f in fields(self)}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self.__post_init__()

    def _shape_for(self, dtype: int) -> KdaRecurrenceShape:
        """The shape with a call's element type (the schedule does not depend on it)."""
        s = self._shapes.get(dtype)
        if s is None:
            sh = self.shape
            s = self._shapes[dtype] = KdaRecurrenceShape(sh.layout, sh.B, sh.N, sh.S, sh.D, dtype)
        return s

    @property
    def tiles(self) -> int:
        """Tiles that hold valid tokens."""
        return int(self.host[10])


def recurrence_plan(x: torch.Tensor, layout: str, cu_seqlens=None) -> KdaRecurrencePlan:
    """Shape, layout and valid lengths of x -> schedule (host work and one small device copy).

    x: [B, N, S, D] (BNSD), [B, S, N, D] (BSND) or [T, N, D] (TND).  ``cu_seqlens`` as for
    ``plan``: prefix sums of the valid lengths, required for TND.
    """
    if layout not in LAYOUTS:
        raise KdaError(2, f"layout {layout!r}")
    if x.dim() != (3 if layout == "TND" else 4):
        raise KdaError(3, f"x has {x.dim()} dimensions under {layout}")
    if isinstance(cu_seqlens, torch.Tensor):
        cu_seqlens = cu_seqlens.detach().to("cpu").numpy()
    cu = cu_ptr = None
    if cu_seqlens is not None:
        cu = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int64))
        if cu.ndim != 1 or cu.size < 2 or cu.min() < 0 or cu.max() >= 1 << 31:
            raise KdaError(7, "cu_seqlens must be a vector of at least two int32 prefix sums")
        cu = cu.astype(np.int32)
        cu_ptr = cu.ctypes.data_as(_P_I32)
    if layout == "TND":
        if cu is None:
            raise KdaError(7, "TND layout needs cu_seqlens")
        S, N, D = x.shape
        B = cu.size - 1
    else:
        B = x.shape[0]
        N, S = (x.shape[1], x.shape[2]) if layout == "BNSD" else (x.shape[2], x.shape[1])
        D = x.shape[3]
        if cu is not None and cu.size != B + 1:
            raise KdaError(7, f"cu_seqlens has {cu.size} entries for {B} sequences")
    if max(B, N, S, D) >= 1 << 31:
        raise KdaError(3, "a size of x does not fit 32 bits")
    shape = KdaRecurrenceShape(LAYOUTS[layout], B, N, S, D, dtype_code(x, "x"))
    L = _lib.load()
    n = ctypes.c_size_t(0)
    check(L.kda_recurrence_plan_size(ctypes.byref(shape), cu_ptr, ctypes.byref(n)),
          "kda_recurrence_plan_size")
    host = np.zeros(n.value, dtype=np.int32)
    hp = host.ctypes.data_as(_P_I32)
    check(L.kda_recurrence_plan(ctypes.byref(shape), cu_ptr, hp, host.size), "kda_recurrence_plan")
    sizes = []
    for backward in (0, 1):
        ws = ctypes.c_size_t(0)
        check(L.kda_recurrence_workspace_size(hp, host.size, backward, ctypes.byref(ws)),
              "kda_recurrence_workspace_size")
        sizes.append(int(ws.value))
    states = ctypes.c_size_t(0)
    check(L.kda_recurrence_states_size(hp, host.size, ctypes.byref(states)),
          "kda_recurrence_states_size")
    dev = torch.from_numpy(host.copy()).to(x.device)
    return KdaRecurrencePlan(shape, layout, host, dev, sizes[0], sizes[1],
                             (int(states.value) // (N * D), N, D), cu)


def _check(plan, layout, dev, x, g, beta, initial_state, A_log, dt_bias):
    """Types, devices and shapes of the inputs against the plan; the element type's code."""
    kind, index, shape = x.dtype, plan._index, plan._x
    code = DTYPES.get(kind)
    # all of it at once (half the time of the checks below, which name what is wrong)
    if (index >= 0 and x.get_device() == g.get_device() == beta.get_device() == A_log.get_device()
            == dt_bias.get_device() == index and plan.layout == layout and code is not None
            and g.dtype is kind and beta.dtype is kind and A_log.dtype is dt_bias.dtype is _F32
            and x.shape == g.shape == shape and beta.shape == plan._rows
            and A_log.shape == plan._heads and dt_bias.shape == plan._params
            and A_log.is_contiguous() and dt_bias.is_contiguous()
            and not (x.is_neg() or g.is_neg() or beta.is_neg() or A_log.is_neg() or dt_bias.is_neg())
            and (initial_state is None
                 or (initial_state.get_device() == index and initial_state.dtype is _F32
                     and initial_state.shape == plan._state and initial_state.is_contiguous()
                     and not initial_state.is_neg()))):
        return code
    if dev.type != "cuda":
        raise ValueError("the gated recurrence runs on a CUDA device only")
    if plan.layout != layout:
        raise KdaError(8, "plan was built for another layout")
    if plan.dev.device != dev:
        raise ValueError(f"the plan's device copy is on {plan.dev.device}, the tensors on {dev}")
    code = dtype_code(x, "x")
    expect(x, "x", x.dtype, dev, plan._x)
    expect(g, "g", x.dtype, dev, plan._x)
    expect(beta, "beta", x.dtype, dev, plan._rows)
    N, D = plan.shape.N, plan.shape.D
    expect_dense(A_log, "A_log", torch.float32, dev, (N,))
    expect_dense(dt_bias, "dt_bias", torch.float32, dev, (N, D))
    if initial_state is not None:
        expect_dense(initial_state, "initial_state", torch.float32, dev, plan._state)
    return code


def _workspace(workspace, nbytes, dev):
    # a call's own scratch by default: calls on other streams and captured graphs share nothing
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    return workspace, workspace.numel() * workspace.element_size()


def _forward(x, g, beta, initial_state, A_log, dt_bias, lower_bound, layout, plan, out,
             final_state, want_states, workspace, stream):
    dev = x.device
    code = _check(plan, layout, dev, x, g, beta, initial_state, A_log, dt_bias)
    results(out, final_state)
    given = out, final_state
    if out is not None:
        expect_dense(out, "out", x.dtype, dev, plan._x)
    if final_state is not None:
        expect_dense(final_state, "final_state", torch.float32, dev, plan._state)
    ctx, handle = launch_on(dev, stream)
    if stream is not None:
        used_on(stream, x, g, beta, initial_state, A_log, dt_bias, plan.dev, out, final_state,
                workspace)
    with ctx:
        if out is None:
            out = dense_like(x)
        if final_state is None:
            final_state = (torch.empty_like(initial_state) if initial_state is not None else
                           torch.empty(plan._state, dtype=torch.float32, device=dev))
        states = A_log.new_empty(plan.states_shape) if want_states else None
        if workspace is None and plan.workspace_bytes == _STATUS_BYTES:
            ws_ptr, ws_bytes = None, 0  # nobody could read the status
        else:
            workspace, ws_bytes = _workspace(workspace, plan.workspace_bytes, dev)
            ws_ptr = workspace.data_ptr()
        check(_lib.load().kda_recurrence_forward(
            ctypes.byref(plan._shape_for(code)), plan._host_ptr, plan.dev.data_ptr(),
            plan.host.size, ctypes.byref(view(x, "x", layout)), ctypes.byref(view(g, "g", layout)),
            ctypes.byref(view(beta, "beta", layout, channels=False)), address(initial_state),
            A_log.data_ptr(), dt_bias.data_ptr(), float(lower_bound), address(states), ws_ptr,
            ws_bytes, out.data_ptr(), final_state.data_ptr(), handle), "kda_recurrence_forward")
    written(*given)
    return out, final_state, states


def gated_recurrence_backward(dout, dfinal_state, x, g, beta, initial_state, A_log, dt_bias,
                              lower_bound: float, layout: str, plan: KdaRecurrencePlan,
                              states: torch.Tensor, workspace: torch.Tensor | None = None,
                              stream: torch.cuda.Stream | None = None):
    """Gradients (dx, dg, dbeta, dinitial_state, dA_log, ddt_bias) of gated_recurrence.

    ``dout`` and ``dfinal_state`` are the gradients of its outputs (None: zeros), ``states`` what
    ``gated_recurrence(..., return_states=True)`` returned for the same inputs and plan.
    dinitial_state is None when initial_state is.
    """
    if workspace is None and stream is None and plan._handle is not None:
        res = _lib.calls().recurrence_backward(plan._handle, layout, x, g, beta, initial_state, A_log,
                                               dt_bias, lower_bound, states, dout, dfinal_state)
        if res is not None:
            return res if res.__class__ is tuple else check(res, "kda_recurrence_backward")
    not_recorded("gated_recurrence_backward")
    no_tangents("gated_recurrence_backward", dout, dfinal_state, x, g, beta, initial_state, A_log,
                dt_bias, states)
    dev = x.device
    code = _check(plan, layout, dev, x, g, beta, initial_state, A_log, dt_bias)
    if dout is not None:
        expect(dout, "dout", x.dtype, dev, plan._x)
    if dfinal_state is not None:
        expect_dense(dfinal_state, "dfinal_state", torch.float32, dev, plan._state)
    expect_dense(states, "states", torch.float32, dev, plan.states_shape)
    ctx, handle = launch_on(dev, stream)
    if stream is not None:
        used_on(stream, dout, dfinal_state, x, g, beta, A_log, dt_bias, states, plan.dev, workspace)
    with ctx:
        dx, dg, dbeta = dense_like(x), dense_like(x), dense_like(beta)
        dh0 = torch.empty_like(initial_state) if initial_state is not None else None
        dA_log = torch.empty_like(A_log)
        ddt_bias = torch.empty_like(dt_bias)
        ws, ws_bytes = _workspace(workspace, plan.backward_workspace_bytes, dev)
        check(_lib.load().kda_recurrence_backward(
            ctypes.byref(plan._shape_for(code)), plan._host_ptr, plan.dev.data_ptr(),
            plan.host.size,
            ctypes.byref(view(dout, "dout", layout)) if dout is not None else None,
            address(dfinal_state), ctypes.byref(view(x, "x", layout)),
            ctypes.byref(view(g, "g", layout)),
            ctypes.byref(view(beta, "beta", layout, channels=False)), A_log.data_ptr(),
            dt_bias.data_ptr(), float(lower_bound), states.data_ptr(),
            ws.data_ptr(), ws_bytes, dx.data_ptr(), dg.data_ptr(), dbeta.data_ptr(), address(dh0),
            dA_log.data_ptr(), ddt_bias.data_ptr(), handle), "kda_recurrence_backward")
    return dx, dg, dbeta, dh0, dA_log, ddt_bias


class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, beta, initial_state, A_log, dt_bias, lower_bound, layout, plan):
        # no gradient is wanted in here, so this takes the short way
        out, final_state, states = gated_recurrence(x, g, beta, initial_state, A_log, dt_bias,
                                                    lower_bound, layout, plan, return_states=True)
        ctx.save_for_backward(x, g, beta, initial_state, A_log, dt_bias, states)
        ctx.call = lower_bound, layout, plan
        ctx.set_materialize_grads(False)
        return out, final_state

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dfinal_state):
        if dout is None and dfinal_state is None:
            return (None,) * 9
        x, g, beta, initial_state, A_log, dt_bias, states = ctx.saved_tensors
        if dout is not None:
            dout = readable(dout)
        if dfinal_state is not None:
            dfinal_state = readable(dfinal_state.contiguous())
        grads = gated_recurrence_backward(dout, dfinal_state, x, g, beta, initial_state, A_log,
                                          dt_bias, *ctx.call, states)
        return grads + (None,) * 3


def gated_recurrence(x, g, beta, initial_state, A_log, dt_bias, lower_bound: float, layout: str,
                     plan: KdaRecurrencePlan, out: torch.Tensor | None = None,
                     final_state: torch.Tensor | None = None, return_states: bool = False,
                     workspace: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None):
    """The recurrence over whole sequences.  Returns (out, final_state).

    x, g: bf16, fp16 or fp32 in the plan's layout, beta the same without channels (any strides over
    slots, heads and tokens; channels contiguous and 16-byte aligned); initial_state: fp32
    [B, N, D] or None (zeros); A_log: fp32 [N]; dt_bias: fp32 [N, D].  out: dense, x's shape and
    type; rows past a valid length are zeros.  final_state: fp32 [B, N, D].

    Differentiable when an input requires a gradient; then out, final_state, return_states,
    workspace and stream cannot be given (choose the stream with torch.cuda.stream).  A call on a
    given stream does not wait for the streams that made its inputs.
    Supplied results may not require a gradient, and autograd notices that they are written.
    ``return_states=True`` adds the states that gated_recurrence_backward needs.  ``workspace``
    (plan.workspace_bytes) keeps the call's device status for device_status; by default every call
    has a scratch of its own.
    """
    if (out is None and final_state is None and workspace is None and stream is None
            and plan._handle is not None):
        res = _lib.calls().recurrence_forward(plan._handle, layout, x, g, beta, initial_state, A_log,
                                              dt_bias, lower_bound, return_states)
        if res is not None:
            return res if res.__class__ is tuple else check(res, "kda_recurrence_forward")
    not_recorded("gated_recurrence")
    if needs_grad(x, g, beta, initial_state, A_log, dt_bias):
        if (out is not None or final_state is not None or return_states or workspace is not None
                or stream is not None):
            raise ValueError("out, final_state, return_states, workspace and stream cannot be "
                             "combined with inputs that require a gradient")
        return _GatedRecurrence.apply(x, g, beta, initial_state, A_log, dt_bias, lower_bound,
                                      layout, plan)
    res = _forward(x, g, beta, initial_state, A_log, dt_bias, lower_bound, layout, plan, out,
                   final_state, return_states, workspace, stream)
    return res if return_states else res[:2]


def gated_recurrence_step(x, g, beta, state, A_log, dt_bias, lower_bound: float,
                          out: torch.Tensor | None = None, state_out: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None):
    """One token of the recurrence for each sequence.  Returns (out, state_out).

    x, g: [B, N, D] in bf16, fp16 or fp32, beta: [B, N], all dense; state: fp32 [B, N, D] or None
    (zeros); pass ``state_out=state`` to update it in place.  Not differentiable.  Supplied results
    may not require a gradient, and autograd notices that they are written.
    """
    calls = _lib.calls()
    if stream is None and calls is not None:
        res = calls.recurrence_step(x, g, beta, state, A_log, dt_bias, lower_bound, out, state_out)
        if res is not None:
            return res if res.__class__ is tuple else check(res, "kda_recurrence_step")
    not_recorded("gated_recurrence_step")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("gated_recurrence_step runs on a CUDA device only")
    if needs_grad(x, g, beta, state, A_log, dt_bias):
        raise ValueError("gated_recurrence_step is not differentiable: use gated_recurrence, or "
                         "torch.no_grad()")
    code = dtype_code(x, "x")
    if x.dim() != 3:
        raise KdaError(3, "gated_recurrence_step expects x [B, N, D]")
    shape, kind, index = x.shape, x.dtype, dev.index
    B, N, D = shape
    # all of it at once, then what is wrong
    if not (g.get_device() == beta.get_device() == A_log.get_device() == dt_bias.get_device() == index
            and g.dtype is kind and beta.dtype is kind and A_log.dtype is dt_bias.dtype is _F32
            and g.shape == shape and beta.shape == (B, N) and A_log.shape == (N,)
            and dt_bias.shape == (N, D) and x.is_contiguous() and g.is_contiguous()
            and beta.is_contiguous() and A_log.is_contiguous() and dt_bias.is_contiguous()
            and not (x.is_neg() or g.is_neg() or beta.is_neg() or A_log.is_neg() or dt_bias.is_neg())):
        expect_dense(x, "x", kind, dev, shape)
        expect_dense(g, "g", kind, dev, shape)
        expect_dense(beta, "beta", kind, dev, shape[:2])
        expect_dense(A_log, "A_log", _F32, dev, shape[1:2])
        expect_dense(dt_bias, "dt_bias", _F32, dev, shape[1:])
    if state is not None:
        expect_dense(state, "state", _F32, dev, shape)
    results(out, state_out)
    given = out, state_out
    if out is not None:
        expect_dense(out, "out", x.dtype, dev, shape)
    if state_out is not None:
        expect_dense(state_out, "state_out", torch.float32, dev, shape)
    ctx, handle = launch_on(dev, stream)
    if stream is not None:
        used_on(stream, x, g, beta, state, A_log, dt_bias, out, state_out)
    with ctx:
        if out is None:
            out = torch.empty_like(x)
        if state_out is None:
            state_out = (torch.empty_like(state) if state is not None else
                         torch.empty(shape, dtype=torch.float32, device=dev))
        check(_lib.load().kda_recurrence_step(
            B, N, D, code, x.data_ptr(), g.data_ptr(), beta.data_ptr(), address(state),
            A_log.data_ptr(), dt_bias.data_ptr(), float(lower_bound), out.data_ptr(),
            state_out.data_ptr(), handle), "kda_recurrence_step")
    written(*given)
    return out, state_out
