"""The gated recurrence and the q/k norm with rotation on the host (no GPU): the tile planner, sizes
and argument checks of the C calls, and the binding's checks.  Placeholder device addresses are
never dereferenced: every check named here comes before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

import chunked_kda_prefill_b200 as kda
from chunked_kda_prefill_b200 import _views
from chunked_kda_prefill_b200._lib import KdaQkShape, KdaRecurrenceShape, KdaView
from test_abi import gpu_visible

P_I32 = ctypes.POINTER(ctypes.c_int32)
NULL, LAYOUT, SHAPE, HEADS, DIM, BOUND, SEQLENS, PLAN, ALIAS, WORKSPACE = 1, 2, 3, 4, 5, 6, 7, 8, 9, 10
ALIGN, DTYPE = 14, 16


@pytest.fixture(scope="module")
def L():
    return kda.load()


def rec_shape(layout=1, B=2, N=3, S=300, D=128, dtype=0):
    return KdaRecurrenceShape(layout, B, N, S, D, dtype)


def rec_plan(L, shape, cu=None):
    p = None if cu is None else np.asarray(cu, dtype=np.int32).ctypes.data_as(P_I32)
    keep = None if cu is None else np.asarray(cu, dtype=np.int32)
    p = None if keep is None else keep.ctypes.data_as(P_I32)
    n = ctypes.c_size_t(0)
    st = L.kda_recurrence_plan_size(ctypes.byref(shape), p, ctypes.byref(n))
    if st:
        return st, None
    buf = np.zeros(n.value, dtype=np.int32)
    return L.kda_recurrence_plan(ctypes.byref(shape), p, buf.ctypes.data_as(P_I32), buf.size), buf


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), DIM), (dict(B=0), SHAPE), (dict(S=0), SHAPE), (dict(N=0), HEADS),
    (dict(layout=3), LAYOUT), (dict(dtype=3), DTYPE), (dict(dtype=-1), DTYPE),
    (dict(B=1 << 30, N=4), SHAPE), (dict(B=1 << 30, N=1, S=1 << 30), SHAPE),
    (dict(layout=2), SEQLENS)])
def test_recurrence_shapes(L, kw, code):
    assert rec_plan(L, rec_shape(**kw))[0] == code


@pytest.mark.parametrize("layout,B,S,cu,code", [
    (2, 2, 100, [1, 50, 100], SEQLENS), (2, 2, 100, [0, 50, 99], SEQLENS),
    (2, 2, 100, [0, 100, 100], SEQLENS), (2, 2, 100, [0, 120, 100], SEQLENS),
    (1, 2, 100, [0, 0, 50], SEQLENS), (1, 2, 100, [0, 101, 150], SEQLENS),
    (0, 2, 100, [0, 60, 161], SEQLENS), (0, 2, 100, [0, 60, 160], 0), (2, 2, 100, [0, 1, 100], 0)])
def test_recurrence_lengths(L, layout, B, S, cu, code):
    assert rec_plan(L, rec_shape(layout=layout, B=B, S=S), cu)[0] == code


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("N", [1, 3, 32])
@pytest.mark.parametrize("layout,S,lengths", [
    (2, None, [1]), (2, None, [130, 1, 700, 64, 65, 63]), (1, 300, [300, 1, 128]), (0, 129, [129, 64]),
    (0, 8192, [8192]), (2, None, [65536]), (1, 4000, [4000, 2777]), (2, None, [9000] + [3] * 400), (2, None, [2, 3, 1] * 100), (1, 40, [39, 40] * 1300)])
def test_plan_records(L, D, N, layout, S, lengths):
    """The segments, longest first, cover every sequence in order, in whole tiles but the last; their
    tiles, parts and maps lie side by side."""
    cu = np.concatenate([[0], np.cumsum(lengths)])
    S = S or int(cu[-1])
    st, p = rec_plan(L, rec_shape(layout=layout, B=len(lengths), S=S, D=D, N=N), cu)
    assert st == 0
    R, rec = 1024 // D, p[24:].reshape(-1, 8).tolist()
    tiles = lambda n: -(-n // R)  # noqa: E731
    assert int(p[11]) == len(rec) and int(p[9]) == R
    assert [r[2] for r in rec] == sorted((r[2] for r in rec), reverse=True)
    solo = tiles(max(lengths)) * 148 * 16 <= sum(map(tiles, lengths)) * N
    assert int(p[17]) == solo
    tile = part = 0
    for r in rec:
        assert r[3:5] == [tile, part]
        tile, part = tile + tiles(r[2]), part + min(1 if solo else 16, tiles(r[2]))
    assert (int(p[10]), int(p[13]), int(p[14])) == (tile, part, tiles(rec[0][2]))
    maps = 0
    for b, n in enumerate(lengths):
        mine = sorted((r for r in rec if r[0] == b), key=lambda r: r[5])
        at = int(cu[b]) if layout == 2 else 0
        for k, (_, start, length, _, _, index, count, first) in enumerate(mine):
            assert (start, index, count, first) == (at, k, len(mine), maps)
            assert length % R == 0 or k + 1 == len(mine)
            at += length
        assert at == (int(cu[b]) if layout == 2 else 0) + n
        lens = [tiles(r[2]) for r in mine]
        assert max(lens) - min(lens) <= 1
        maps += len(mine) if len(mine) > 1 else 0
    assert int(p[12]) == maps
    assert int(p[15]) == (layout != 2 and min(lengths) < S)
    if maps:  # a cut pays only where it fills the machine
        assert len(rec) * N <= 8 * 148
    floats = ctypes.c_size_t(0)
    assert L.kda_recurrence_states_size(p.ctypes.data_as(P_I32), p.size, ctypes.byref(floats)) == 0
    assert floats.value == tile * N * D
    sizes = []
    for backward in (0, 1):
        n = ctypes.c_size_t(0)
        assert L.kda_recurrence_workspace_size(p.ctypes.data_as(P_I32), p.size, backward,
                                               ctypes.byref(n)) == 0
        sizes.append(n.value)
    assert sizes[0] == 256 + maps * N * 2 * D * 4
    assert sizes[1] == sizes[0] + part * N * (D + 1) * 4


def test_recurrence_plan_capacity_and_corruption(L):
    st, p = rec_plan(L, rec_shape())
    assert st == 0
    n = ctypes.c_size_t(0)
    ok = lambda a, k=None: L.kda_recurrence_workspace_size(  # noqa: E731
        a.ctypes.data_as(P_I32), a.size if k is None else k, 0, ctypes.byref(n))
    assert ok(p) == 0 and n.value >= 256
    assert ok(p, p.size - 1) == PLAN and ok(p, 3) == PLAN
    for word in (0, 4, 5, 10, 11, 12, 13, 14, 15, 16, 17, 23):
        bad = p.copy()
        bad[word] += 1
        assert ok(bad) == PLAN, word
    assert L.kda_recurrence_plan(ctypes.byref(rec_shape()), None, p.ctypes.data_as(P_I32),
                                 p.size - 1) == PLAN


def views(**kw):
    return {n: KdaView(*kw.get(n, d)) for n, d in {
        "x": (0x10000000, 0, 0, 0), "g": (0x20000000, 0, 0, 0), "beta": (0x30000000, 0, 0, 0),
        "dout": (0x38000000, 0, 0, 0)}.items()}


def dense_strides(layout, N, S, D):
    return (N * S * D, S * D, D) if layout == 0 else (S * N * D, D, N * D)


def rec_call(L, p, shape, backward=False, **over):
    N, S, D = shape.N, shape.S, shape.D
    st = dense_strides(shape.layout, N, S, D)
    bt = dense_strides(shape.layout, N, S, 1)
    a = dict(x=(0x10000000, *st), g=(0x20000000, *st), beta=(0x30000000, *bt),
             dout=(0x38000000, *st), h0=0x40000000, A=0x50000000, bias=0x51000000, lb=-5.0,
             states=0x60000000, ws=0x70000000, ws_bytes=1 << 40, out=0x180000000, fs=0x190000000,
             plan_dev=0x52000000, dx=0x180000000, dg=0x1A0000000, dbeta=0x1B0000000,
             dh0=0x1C0000000, dA=0x1D0000000, dbias=0x1E0000000, dfinal=0x41000000)
    a.update(over)
    v = {n: (ctypes.byref(KdaView(*a[n])) if a[n] is not None else None)
         for n in ("x", "g", "beta", "dout")}
    head = (ctypes.byref(shape), p.ctypes.data_as(P_I32), a["plan_dev"], p.size)
    if backward:
        return L.kda_recurrence_backward(
            *head, v["dout"], a["dfinal"], v["x"], v["g"], v["beta"], a["A"], a["bias"], a["lb"],
            a["states"], a["ws"], a["ws_bytes"], a["dx"], a["dg"], a["dbeta"], a["dh0"],
            a["dA"], a["dbias"], None)
    return L.kda_recurrence_forward(
        *head, v["x"], v["g"], v["beta"], a["h0"], a["A"], a["bias"], a["lb"], a["states"], a["ws"],
        a["ws_bytes"], a["out"], a["fs"], None)


def test_recurrence_argument_checks(L):
    shape = rec_shape()
    st, p = rec_plan(L, shape)
    row = dense_strides(1, 3, 300, 128)
    nbytes = 2 * 300 * 3 * 128 * 2
    for backward in (False, True):
        c = lambda **kw: rec_call(L, p, shape, backward, **kw)  # noqa: E731
        for name in ("x", "g", "beta"):
            assert c(**{name: None}) == NULL
            assert c(**{name: (None, *row)}) == NULL
        for name in ("A", "bias", "plan_dev") + (("dx", "dg", "dbeta", "dA", "dbias", "states")
                                                 if backward else ("out", "fs")):
            assert c(**{name: None}) == NULL, name
        assert c(lb=0.5) == BOUND and c(lb=-6.0) == BOUND and c(lb=float("nan")) == BOUND
        assert c(ws=0x70000010) == WORKSPACE and c(ws_bytes=8) == WORKSPACE
        # without a workspace there is no place for more than the status
        assert c(ws=None) == (NULL if backward else c())
        assert c(x=(0x10000008, *row)) == ALIGN
        assert c(g=(0x20000000, row[0], row[1], row[2] + 4)) == ALIGN   # rows off 16 bytes
        assert c(x=(0x10000000, -row[0], row[1], row[2])) == SHAPE      # negative stride
        assert c(x=(0x10000000, 1 << 60, row[1], row[2])) == SHAPE
        assert c(beta=(0x30000001, 900, 1, 3)) == ALIGN
        assert backward or c(h0=0x40000004) == ALIGN
        name = "dx" if backward else "out"
        assert c(**{name: 0x10000000 + 256}) == ALIAS                    # an input
        assert c(**{name: 0x10000000 - nbytes + 16}) == ALIAS
        assert c(**{name: 0x70000000}) == ALIAS                          # the workspace
        # strides reach over the output although the first rows do not
        assert c(x=(0x180000000 - 2 * (300 * row[2] - 128), 0, row[1], row[2])) == ALIAS
        other = rec_shape(S=301)
        assert rec_call(L, p, other, backward) == PLAN
        assert rec_call(L, p, rec_shape(dtype=7), backward) == DTYPE
        if not gpu_visible():
            assert c() in (11, 13) and c(h0=None) in (11, 13) and c(x=(0x10000000, 0, 0, 0)) in (11, 13)
    assert rec_call(L, p, shape, fs=0x40000000 + 16) == ALIAS            # partly initial_state
    assert rec_call(L, p, shape, fs=0x60000000) == ALIAS                 # the states
    assert rec_call(L, p, shape, True, dg=0x180000000) == ALIAS          # dx
    assert rec_call(L, p, shape, True, dx=0x38000000) == ALIAS           # dout
    assert rec_call(L, p, shape, True, dh0=0x41000000) == ALIAS          # dfinal
    if not gpu_visible():
        assert rec_call(L, p, shape, fs=0x40000000) in (11, 13)          # in place
        assert rec_call(L, p, shape, states=None) in (11, 13)
        assert rec_call(L, p, shape, True, dout=None, dfinal=None, dh0=None) in (11, 13)


def test_step_argument_checks(L):
    def c(B=2, N=3, D=128, dtype=0, x=0x10000000, g=0x11000000, beta=0x12000000, s0=0x13000000,
          A=0x14000000, bias=0x15000000, lb=-5.0, out=0x16000000, s1=0x17000000):
        return L.kda_recurrence_step(B, N, D, dtype, x, g, beta, s0, A, bias, lb, out, s1, None)
    assert c(D=32) == DIM and c(B=0) == SHAPE and c(N=0) == HEADS and c(dtype=9) == DTYPE
    assert c(x=None) == NULL and c(s1=None) == NULL and c(lb=1.0) == BOUND
    assert c(x=0x10000002) == ALIGN and c(s1=0x17000008) == ALIGN and c(beta=0x12000001) == ALIGN
    assert c(out=0x10000000) == ALIAS and c(s1=0x13000010) == ALIAS and c(out=0x17000000) == ALIAS
    if not gpu_visible():
        assert c(s1=0x13000000) in (11, 13) and c(s0=None) in (11, 13)


def qk_call(L, backward=False, **over):
    a = dict(layout=1, B=2, Nq=4, Nk=2, S=50, D=128, dtype=0, rot=128, inter=0, eps=1e-6,
             q=0x10000000, k=0x20000000, dqo=0x90000000, dko=0xA0000000, pos=0x30000000,
             inv=0x31000000, qw=0x32000000, kw=0x33000000, qo=0x40000000, ko=0x50000000,
             ws=0x60000000, ws_bytes=1 << 30, dqw=0x70000000, dkw=0x71000000, q_strides=None)
    a.update(over)
    sh = KdaQkShape(a["layout"], a["B"], a["Nq"], a["Nk"], a["S"], a["D"], a["dtype"], a["rot"],
                    a["inter"], a["eps"])
    qs = a["q_strides"] or dense_strides(a["layout"], a["Nq"], a["S"], a["D"])
    ks = dense_strides(a["layout"], a["Nk"], a["S"], a["D"])
    q, k = ctypes.byref(KdaView(a["q"], *qs)), ctypes.byref(KdaView(a["k"], *ks))
    if not backward:
        return L.kda_qk_norm_rope(ctypes.byref(sh), q, k, a["pos"], a["inv"], a["qw"], a["kw"],
                                  a["qo"], a["ko"], None)
    dense = dense_strides(a["layout"], a["Nq"], a["S"], a["D"])
    return L.kda_qk_norm_rope_backward(
        ctypes.byref(sh), ctypes.byref(KdaView(a["dqo"], *dense)),
        ctypes.byref(KdaView(a["dko"], *ks)), q, k, a["pos"], a["inv"], a["qw"], a["kw"], a["ws"],
        a["ws_bytes"], a["qo"], a["ko"], a["dqw"], a["dkw"], None)


@pytest.mark.parametrize("backward", [False, True])
def test_qk_argument_checks(L, backward):
    c = lambda **kw: qk_call(L, backward, **kw)  # noqa: E731
    assert c(D=96) == DIM and c(rot=8) == DIM and c(rot=144) == DIM and c(rot=-16) == DIM
    assert c(layout=5) == LAYOUT and c(dtype=3) == DTYPE and c(Nq=0) == HEADS and c(Nk=0) == HEADS
    assert c(S=0) == SHAPE and c(B=0) == SHAPE and c(inter=2) == SHAPE
    assert c(eps=-1e-6) == SHAPE and c(eps=float("inf")) == SHAPE and c(eps=float("nan")) == SHAPE
    assert c(Nq=70000) == SHAPE
    assert c(q=None) == NULL and c(k=None) == NULL and c(qo=None) == NULL and c(inv=None) == NULL
    assert c(q=0x10000008) == ALIGN and c(qo=0x40000008) == ALIGN and c(pos=0x30000002) == ALIGN
    assert c(q_strides=(4 * 50 * 128, 128, 4 * 128 + 4)) == ALIGN
    assert c(q_strides=(4 * 50 * 128, -128, 4 * 128)) == SHAPE
    assert c(qo=0x20000000) == ALIAS and c(ko=0x40000000) == ALIAS and c(qo=0x10000100) == ALIAS
    assert c(qo=0x32000000) == ALIAS and c(ko=0x30000000) == ALIAS
    # in place needs the very same tensor: a view with other strides is not it
    assert c(**{"qo": 0x10000000, "q_strides": (8 * 50 * 128, 128, 8 * 128)}) == ALIAS
    if backward:
        assert c(ws=None) == NULL and c(ws_bytes=16) == WORKSPACE and c(ws=0x60000010) == WORKSPACE
        assert c(dqw=0x71000000) == ALIAS and c(dqw=0x10000000) == ALIAS
        assert c(qo=0x10000000) == ALIAS                   # dq over q
        assert c(qo=0xA0000000) == ALIAS                   # dq over dk_out
    if not gpu_visible():
        assert c() in (11, 13) and c(pos=None) in (11, 13) and c(rot=0, inv=None) in (11, 13)
        assert c(layout=2, B=0) in (11, 13) and c(qw=None, kw=None) in (11, 13)
        if backward:
            assert c(qo=0x90000000, ko=0xA0000000) in (11, 13) and c(dqw=None) in (11, 13)
        else:
            assert c(qo=0x10000000, ko=0x20000000) in (11, 13)


def test_binding_refuses_before_the_library():
    cpu = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    with pytest.raises(ValueError):
        kda.qk_norm_rope(cpu, cpu, None, None, w, w, 1e-6, "TND")
    with pytest.raises(ValueError):
        kda.gated_recurrence_step(cpu, cpu, cpu[..., 0], None, w[:2], torch.zeros(2, 64), -1.0)
    plan = kda.recurrence_plan(cpu, "TND", cu_seqlens=[0, 4])
    with pytest.raises(ValueError):
        kda.gated_recurrence(cpu, cpu, cpu[..., 0], None, w[:2], torch.zeros(2, 64), -1.0, "TND",
                             plan)
    with pytest.raises(TypeError):
        kda.recurrence_plan(cpu.double(), "TND", cu_seqlens=[0, 4])
    for cu in (None, [0], [0, 3], [0, -1, 4], [0, 1 << 40], [[0, 4]]):
        with pytest.raises(kda.KdaError):
            kda.recurrence_plan(cpu, "TND", cu_seqlens=cu)
    with pytest.raises(kda.KdaError):
        kda.recurrence_plan(cpu[None], "BSND", cu_seqlens=[0, 2, 4])   # two sequences, one slot
    with pytest.raises(kda.KdaError):
        kda.recurrence_plan(cpu, "BSND")
    with pytest.raises(kda.KdaError):
        kda.recurrence_plan(cpu, "NTD", cu_seqlens=[0, 4])


def test_views_of_tensors():
    t = torch.zeros(2, 5, 3, 64, dtype=torch.bfloat16)
    v = _views.view(t, "t", "BSND")
    assert (v.stride_b, v.stride_n, v.stride_s) == (5 * 3 * 64, 64, 3 * 64)
    v = _views.view(t, "t", "BNSD")
    assert (v.stride_b, v.stride_n, v.stride_s) == (5 * 3 * 64, 3 * 64, 64)
    v = _views.view(t[0], "t", "TND")
    assert (v.stride_b, v.stride_n, v.stride_s) == (0, 64, 3 * 64)
    v = _views.view(t[..., 0], "t", "BSND", channels=False)
    assert (v.stride_b, v.stride_n, v.stride_s) == (5 * 3 * 64, 64, 3 * 64)
    with pytest.raises(ValueError):
        _views.view(t.transpose(-1, -2), "t", "BSND")
    assert _views.viewable(t) and _views.viewable(t[..., :8])
    assert not _views.viewable(t[..., 1:]) and not _views.viewable(t.transpose(-1, -2))
    assert not _views.viewable(torch.ones((), dtype=torch.bfloat16).expand(2, 64))
    odd = torch.zeros(4, 68, dtype=torch.bfloat16)
    assert not _views.viewable(odd[:, :64]) and _views.viewable(odd[:1, :64])


def test_compiled_calls_leave_to_python_what_does_not_fit():
    """The compiled calls are built here, answer None to what is not theirs to take, and never raise
    or run for it."""
    import torch

    import chunked_kda_prefill_b200 as kda
    from chunked_kda_prefill_b200 import _lib
    m = _lib.calls()
    assert m is not None and m.torch_version == torch.__version__
    x = torch.zeros(4, 2, 64)
    beta, A, bias, state = x[..., 0].contiguous(), torch.zeros(2), torch.zeros(2, 64), x[:1]
    plan = kda.recurrence_plan(x, "TND", cu_seqlens=[0, 4])
    rec = [plan._handle, "TND", x, x, beta, state, A, bias, -1.0]
    assert m.recurrence_forward(*rec, False) is None                    # not on a CUDA device
    assert m.recurrence_backward(*rec, x, None, None) is None
    assert m.recurrence_step(x, x, beta, None, A, bias, -1.0, None, None) is None
    assert m.qk_forward(x, x, None, None, None, None, 1e-6, "TND", False) is None
    assert m.qk_backward(x, x, None, None, None, None, 1e-6, "TND", False, x, x) is None
    for call, n in ((m.recurrence_forward, 10), (m.recurrence_backward, 12), (m.recurrence_step, 9),
                    (m.qk_forward, 9), (m.qk_backward, 11)):
        assert call(*[None] * n) is None and call(*["TND"] * n) is None and call() is None
    for bad in ((), (1, 2), (0,) * 6, ("a",) * 6):
        with pytest.raises((TypeError, ValueError)):
            m.bind(*bad)
    with pytest.raises(TypeError):
        m.plan(*range(12))
