"""What the operators around the prefill share in the binding: element types, strided tensor
arguments, the launch stream and the device of a call."""
from __future__ import annotations

import contextlib
import sys

import torch
from torch.autograd import forward_ad

from ._lib import KdaError, KdaView

# kda_dtype_t
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


_included = torch._C._dispatch_tls_is_dispatch_key_included
_PRE_DISPATCH = torch._C.DispatchKey.PreDispatch


def dtype_code(t: torch.Tensor, name: str) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bf16, fp16 or fp32, got {t.dtype}")
    return code


def negated(name: str) -> None:
    raise ValueError(f"{name} is marked as negated but not rewritten: pass {name}.resolve_neg()")


def address(t: torch.Tensor | None) -> int | None:
    """Of an argument that may be left out (None)."""
    if t is None:
        return None
    p = t.data_ptr()
    if not p and t.numel():  # a null address would mean that it was left out
        raise ValueError("an argument has no memory of its own")
    return p


def expect(t, name: str, dtype, device, shape) -> None:
    """A tensor of exactly this type, device and shape; its strides are the caller's business."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.shape != shape:
        raise KdaError(3, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_neg():
        negated(name)


def expect_dense(t, name: str, dtype, device, shape) -> None:
    expect(t, name, dtype, device, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def view(t: torch.Tensor, name: str, layout: str, channels: bool = True) -> KdaView:
    """kda_view_t of a tensor in a layout (the library checks alignment and ranges)."""
    st = t.stride()
    if channels and st[-1] != 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    if layout == "BNSD":
        return KdaView(address(t), st[0], st[1], st[2])
    if layout == "BSND":
        return KdaView(address(t), st[0], st[2], st[1])
    return KdaView(address(t), 0, st[1], st[0])


def viewable(t: torch.Tensor) -> bool:
    """Whether view() and the library's alignment rule take a tensor with channels as it lies."""
    size = t.element_size()
    return (t.stride(-1) == 1 and t.data_ptr() % 16 == 0
            and all(n == 1 or s * size % 16 == 0 for n, s in zip(t.shape[:-1], t.stride()[:-1])))


def readable(t: torch.Tensor) -> torch.Tensor:
    """A gradient as view() and the alignment rule take it: itself, or a dense copy (contiguous() would
    keep a dense slice that starts at an odd address).  A lazy negation is carried out."""
    t = t.resolve_neg()
    return t if viewable(t) else t.clone(memory_format=torch.contiguous_format)


@contextlib.contextmanager
def _on(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


_here = contextlib.nullcontext()


def launch_on(device: torch.device, stream):
    """(context, cuda stream handle): inside the context the call's device is the current one, and
    what is allocated belongs to the stream that the kernels run on."""
    index = device.index
    if stream is None and index == torch._C._cuda_getDevice():
        # the handle alone: a Stream object would cost a call 2 us
        return _here, torch._C._cuda_getCurrentRawStream(index)
    s = stream if stream is not None else torch.cuda.current_stream(device)
    if s.device != device:
        raise ValueError(f"stream is on {s.device}, the tensors on {device}")
    return _on(device, s), s.cuda_stream


def used_on(stream, *tensors) -> None:
    """Memory of tensors that a call on a stream of the caller's choice uses is not handed out again
    before that stream has come past the call."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def has_tangent(*tensors) -> bool:
    """Whether one carries a forward-mode derivative (which requires_grad does not say)."""
    if getattr(forward_ad, "_current_level", 0) < 0:  # none can: asking each costs half a microsecond
        return False
    return any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def needs_grad(*tensors) -> bool:
    for t in tensors:
        if t is not None and t.requires_grad:
            if torch.is_grad_enabled():
                return True
            break
    return has_tangent(*tensors)


def results(*tensors) -> None:
    """Checks the results that a caller supplies: a call writes to their memory, which autograd does not
    follow."""
    for t in tensors:
        if t is not None and needs_grad(t):
            raise ValueError("results that require a gradient cannot be written to; use "
                             "torch.no_grad()")


def written(*tensors) -> None:
    """Tells autograd that supplied results have new values, for graphs that saved the old ones."""
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def not_recorded(what: str) -> None:
    """Refuses a call while torch.jit.trace or make_fx records: they see no operation of torch here and
    would keep the results as constants."""
    if torch.compiler.is_compiling():  # it takes none of these calls into its graphs
        return
    recorded = torch._C._is_tracing()
    if not recorded and (torch._C._len_torch_dispatch_stack() > 0 or _included(_PRE_DISPATCH)):
        # a mode is on; without this module it is not make_fx's
        proxies = sys.modules.get("torch.fx.experimental.proxy_tensor")
        recorded = proxies is not None and proxies.get_proxy_mode() is not None
    if recorded:
        raise RuntimeError(f"{what} cannot be recorded by torch.jit.trace or make_fx: its results "
                           "would be constants of the recording")


def no_tangents(what: str, *tensors) -> None:
    if has_tangent(*tensors):
        raise ValueError(f"{what} has no forward-mode derivative")


def dense_like(t: torch.Tensor) -> torch.Tensor:
    """An empty dense tensor of t's shape, type and device (less than half the time of empty())."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)
