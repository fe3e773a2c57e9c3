"""What the binding of the operators around the prefill sees of a call, without a GPU."""
import copy
import ctypes
import pickle

import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

import chunked_kda_prefill_b200 as kda
from chunked_kda_prefill_b200 import _views, build
from test_abi import gpu_visible
from test_layer_abi import rec_call, rec_plan, rec_shape


def test_tangents_count_as_wanted_gradients():
    t, leaf = torch.ones(3), torch.ones(3, requires_grad=True)
    assert not _views.needs_grad(t, None) and _views.needs_grad(None, t, leaf)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(t, t)
        for grad in (torch.enable_grad, torch.no_grad):
            with grad():
                assert _views.needs_grad(None, dual) and _views.needs_grad(leaf, dual)
                assert not _views.has_tangent(t, leaf, None)
    with torch.no_grad():
        assert not _views.needs_grad(leaf, t)


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda p: pickle.loads(pickle.dumps(p))])
def test_plans_are_copied_and_pickled(again):
    plan = kda.recurrence_plan(torch.zeros(9, 2, 64), "TND", cu_seqlens=[0, 4, 9])
    twin = again(plan)
    assert twin.layout == "TND" and twin.tiles == plan.tiles and twin._shape_for(1).dtype == 1
    assert np.array_equal(twin.host, plan.host) and torch.equal(twin.dev, plan.dev)
    assert (twin.workspace_bytes, twin.backward_workspace_bytes, twin.states_shape) == (
        plan.workspace_bytes, plan.backward_workspace_bytes, plan.states_shape)
    assert (twin._handle is None) == (plan._handle is None)
    # its address is that of its own words
    assert ctypes_address(twin._host_ptr) == twin.host.ctypes.data


def ctypes_address(p):
    return ctypes.cast(p, ctypes.c_void_p).value


def test_gradients_are_taken_from_any_address():
    whole = torch.arange(3 + 4 * 2 * 64.)
    odd = whole[3:].view(4, 2, 64)
    assert odd.is_contiguous() and odd.data_ptr() % 16 and not _views.viewable(odd)
    even = _views.readable(odd)
    assert _views.viewable(even) and even.is_contiguous() and torch.equal(even, odd)
    for kept in (even, even[:, :1], even[::2]):
        assert _views.readable(kept) is kept
    for copied in (torch.ones(()).expand(4, 2, 64), odd.transpose(1, 2)):
        assert _views.readable(copied).is_contiguous() and torch.equal(_views.readable(copied), copied)


def test_marked_negations_are_not_read_as_they_lie():
    t = torch.arange(1, 9 * 64 + 1.).view(9, 64)
    minus = torch._neg_view(t)
    assert minus.is_neg() and minus.data_ptr() == t.data_ptr() and minus.is_contiguous()
    _views.expect(t, "t", t.dtype, t.device, t.shape)
    for check in (_views.expect, _views.expect_dense):
        with pytest.raises(ValueError, match="negat"):
            check(minus, "t", t.dtype, t.device, t.shape)
    got = _views.readable(minus)
    assert not got.is_neg() and torch.equal(got, -t)


def test_tensors_without_memory_have_no_address():
    t = torch.zeros(3, 64)

    def check(a):
        with pytest.raises((RuntimeError, ValueError)):
            _views.address(a)
        return a * 1

    torch.func.functionalize(check)(t)
    torch.vmap(check)(t)
    assert _views.address(None) is None and _views.address(t) == t.data_ptr()
    assert _views.address(torch.zeros(0)) == 0


@pytest.mark.parametrize("backward", [False, True])
def test_a_workspace_over_an_input_is_refused(backward):
    L, shape = kda.load(), rec_shape(B=1, S=9000, N=1)
    st, p = rec_plan(L, shape)
    assert st == 0 and p[12] > 0  # cut: the workspace holds maps, and the gradients' parts
    ok = (11, 13)  # no device
    names = {"x": 0x10000000, "g": 0x20000000, "beta": 0x30000000, "A": 0x50000000, "bias": 0x51000000,
             "plan_dev": 0x52000000}
    names |= ({"dout": 0x38000000, "states": 0x60000000, "dfinal": 0x41000000} if backward
              else {"h0": 0x40000000})
    for name, address in names.items():
        assert rec_call(L, p, shape, backward, ws=address) == 9, name
    if not gpu_visible():
        assert rec_call(L, p, shape, backward) in ok
        # behind the last byte
        assert rec_call(L, p, shape, backward, ws=0x50000100) in ok


def test_compiled_calls_that_no_longer_fit_are_removed(tmp_path, monkeypatch):
    """Without a compiler that works, the file of an earlier build does not stay beside a newer library."""
    calls = tmp_path / "_calls.so"
    calls.write_bytes(b"of an earlier header")
    monkeypatch.setattr(build, "CALLS", str(calls))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError):
        build.build_calls()
    assert not calls.exists()
    monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))
    calls.write_bytes(b"of an earlier header")
    with pytest.raises(OSError):
        build.build_calls()
    assert not calls.exists()


def test_recordings_are_told_from_other_modes():
    from torch.fx.experimental.proxy_tensor import make_fx
    from torch.utils._python_dispatch import TorchDispatchMode
    t = torch.ones(3)

    def call(x):
        _views.not_recorded("call")
        return x * 2

    for pre_dispatch in (False, True):
        for mode in ("real", "fake", "symbolic"):
            with pytest.raises(RuntimeError, match="recorded"):
                make_fx(call, pre_dispatch=pre_dispatch, tracing_mode=mode)(t)
    with pytest.raises(RuntimeError, match="recorded"):
        torch.jit.trace(call, (t,))

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            return func(*args, **(kwargs or {}))

    with Watch():
        assert torch.equal(call(t), 2 * t)
    assert torch.equal(torch.compile(call, backend="eager")(t), 2 * t)
