"""The gated recurrence and the q/k norm with rotation where a call could go wrong without a sign:
broken and infinite parameters, padding inside a tile, what autograd, forward-mode derivatives and
tracing see of a call, results written in place, plans that are copied, gradients at odd addresses."""
import pytest
import torch

import chunked_kda_prefill_b200 as kda
from chunked_kda_prefill_b200 import _lib
from test_gpu_recurrence import BF, FP, args, make

pytestmark = pytest.mark.gpu

NAMES = ("dx", "dg", "dbeta", "dh0", "dA_log", "ddt_bias")
# whole (a ring of warps to a sequence; tiles of 8 rows of 128 channels: the first length ends inside a
# tile, the second with one), cut into segments, and a warp to each of many short ones
FORMS = {"whole": [150, 144] + [1] * 100, "cut": [4001, 8], "many": [1 + (7 * i) % 40 for i in range(1300)]}


def form(name, D=128, seed=0, kind=BF):
    d = make("TND", FORMS[name], 4 if name == "many" else 2, D, kind, seed=seed)
    host = d["plan"].host
    assert (host[12] > 0, host[17] == 1) == (name == "cut", name == "many")
    return d, FORMS[name]


def both(d, lb=-2.0):
    a = args(d, lb, "TND")
    out, final, states = kda.gated_recurrence(*a, return_states=True)
    grads = kda.gated_recurrence_backward(d["dout"], d["dfinal"], *a, states)
    return {"out": out, "final": final} | dict(zip(NAMES, grads))


def single(d, lb=-2.0, **kw):
    n = d["h0"].shape[0]
    x, g, beta = (d[name][:n].contiguous() for name in ("x", "g", "beta"))
    return kda.gated_recurrence_step(x, g, beta, kw.pop("state", d["h0"]), d["A_log"], d["dt_bias"], lb, **kw)


@pytest.fixture(params=["compiled", "python"])
def way(request, monkeypatch, cuda_ok):
    """Both ways of a call: the compiled one and the one through ctypes."""
    if request.param == "python":
        monkeypatch.setattr(_lib, "_calls", None)
    else:
        assert _lib.calls() is not None
    return request.param


@pytest.mark.parametrize("name", list(FORMS))
def test_nan_in_a_log_spoils_its_head_alone(name, cuda_ok):
    """A broken A_log gives NaN wherever its gate has a part, and the other heads keep their bits."""
    d, lengths = form(name, seed=1)
    clean, step = both(d), single(d)
    d["A_log"] = d["A_log"].clone()
    d["A_log"][1] = float("nan")
    got, bad = both(d), single(d)
    keep = [n for n in range(d["A_log"].numel()) if n != 1]
    for t in (got["out"], got["final"], got["dg"], got["dh0"], *bad):
        assert torch.isnan(t[:, 1]).all()
    assert torch.isnan(got["dA_log"][1]) and torch.isnan(got["ddt_bias"][1]).all()
    for n in ("out", "final", "dx", "dg", "dbeta", "dh0"):
        assert torch.equal(got[n][:, keep], clean[n][:, keep]), n
    for n in ("dA_log", "ddt_bias"):
        assert torch.equal(got[n][keep], clean[n][keep]), n
    assert all(torch.equal(p[:, keep], q[:, keep]) for p, q in zip(bad, step))


def last_tokens(lengths):
    return torch.tensor(lengths).cumsum(0).sub(1).cuda()


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("name", list(FORMS))
def test_infinite_bias_is_a_gate_held_open(name, D, cuda_ok):
    """dt_bias = inf makes the sigmoid one, as a bias of 1e30 does, and so does every result that has a
    value: dA_log is 0 * inf by its formula and left out."""
    d, lengths = form(name, D, seed=2)
    d["dt_bias"] = d["dt_bias"].clone()
    d["dt_bias"][1, 5] = 1e30
    want, step = both(d), single(d)
    d["dt_bias"][1, 5] = float("inf")
    got, open_step = both(d), single(d)
    for n in got:
        if n == "dA_log":
            assert torch.equal(got[n][:1], want[n][:1])
        else:
            assert torch.isfinite(got[n]).all() and torch.equal(got[n], want[n]), n
    assert all(torch.equal(p, q) for p, q in zip(open_step, step))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("name", list(FORMS))
def test_last_token_does_not_reach_the_parameters(name, bad, cuda_ok):
    """No gradient but dbeta contains the last token's value: an infinite or broken one leaves the
    bits of all others, wherever in a tile the sequence ends."""
    d, lengths = form(name, seed=3)
    clean = both(d)
    d["x"] = d["x"].clone()
    last = last_tokens(lengths)
    d["x"][last, 1, 5] = bad
    got = both(d)
    assert not torch.isfinite(got["final"][:, 1, 5]).any()
    for n in ("dx", "dg", "dh0", "dA_log", "ddt_bias"):
        assert torch.equal(got[n], clean[n]), n
    others = torch.ones_like(clean["dbeta"], dtype=torch.bool)
    others[last, 1] = False
    assert torch.equal(got["dbeta"][others], clean["dbeta"][others])


@pytest.mark.parametrize("param", ["A_log", "dt_bias"])
@pytest.mark.parametrize("name", list(FORMS))
def test_broken_parameter_leaves_the_last_gradient(name, param, cuda_ok):
    """No decay lies behind a sequence's last token: its dx and dbeta are those of whole parameters."""
    d, lengths = form(name, seed=4)
    clean = both(d)
    d[param] = d[param].clone()
    d[param][1] = float("nan")
    got, last = both(d), last_tokens(lengths)
    for n in ("dx", "dbeta"):
        assert torch.equal(got[n][last], clean[n][last]), n
        assert torch.equal(got[n][:, 0], clean[n][:, 0]), n
    assert torch.isnan(got["dg"][:, 1]).all() and torch.isnan(got["out"][:, 1]).all()


def qk_inputs(kind=FP, S=40):
    gen = torch.Generator().manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    return {"q": rnd(S, 3, 64).to(kind), "k": rnd(S, 2, 64).to(kind), "positions": None,
            "inv_freq": rnd(16).abs(), "q_weight": rnd(64), "k_weight": rnd(64), "eps": 1e-6,
            "layout": "TND"}


def test_forward_mode_derivatives_are_refused(way):
    """An input with a tangent: there is no forward-mode formula, and no call drops the tangent."""
    from torch.autograd import forward_ad as fa
    d = make("TND", [30, 9], 2, 64, FP, seed=5)
    if way == "python":
        d["plan"]._handle = None
    plain = args(d, -1.0, "TND")
    states = kda.gated_recurrence(*plain, return_states=True)[2]
    qk = qk_inputs()
    calls = 0
    for grad in (torch.enable_grad, torch.no_grad):
        with grad(), fa.dual_level():
            dual = lambda t: fa.make_dual(t, torch.ones_like(t))  # noqa: E731
            refused = (NotImplementedError, ValueError, RuntimeError)
            for i in range(6):
                a = list(plain)
                a[i] = dual(a[i])
                with pytest.raises(refused):
                    kda.gated_recurrence(*a)
                with pytest.raises(refused):
                    kda.gated_recurrence_backward(d["dout"], None, *a, states)
                calls += 1
            for name in ("dout", "dfinal"):
                g = {"dout": d["dout"], "dfinal": d["dfinal"]}
                g[name] = dual(g[name])
                with pytest.raises(refused):
                    kda.gated_recurrence_backward(g["dout"], g["dfinal"], *plain, states)
            for name in ("x", "g", "beta", "h0", "A_log", "dt_bias"):
                with pytest.raises(refused):
                    single(dict(d, **{name: dual(d[name])}))
            for name in ("q", "k", "inv_freq", "q_weight", "k_weight"):
                c = dict(qk, **{name: dual(qk[name])})
                with pytest.raises(refused):
                    kda.qk_norm_rope(**c)
                with pytest.raises(refused):
                    kda.qk_norm_rope_backward(qk["q"], qk["k"], **c)
            for i in range(2):
                g = [qk["q"], qk["k"]]
                g[i] = dual(g[i])
                with pytest.raises(refused):
                    kda.qk_norm_rope_backward(*g, **qk)
            # inputs without a tangent are taken at a dual level as anywhere
            assert kda.gated_recurrence(*plain)[0].isfinite().all()
            assert kda.qk_norm_rope(**qk)[0].isfinite().all() and single(d)[0].isfinite().all()
    assert calls == 12


def test_recording_a_call_is_refused(way):
    """torch.jit.trace and make_fx would keep the results of the traced call as constants."""
    from torch.fx.experimental.proxy_tensor import make_fx
    d = make("TND", [30, 9], 2, 64, FP, seed=6)
    if way == "python":
        d["plan"]._handle = None
    a = args(d, -1.0, "TND")
    states = kda.gated_recurrence(*a, return_states=True)[2]
    qk = qk_inputs()
    rest = {n: v for n, v in qk.items() if n != "q"}
    runs = [lambda x: kda.gated_recurrence(x, *a[1:])[0],
            lambda x: kda.gated_recurrence_backward(x, None, *a, states)[0],
            lambda x: single(dict(d, x=x))[0]]
    for f, t in [(f, d["x"]) for f in runs] + [
            (lambda q: kda.qk_norm_rope(q=q, **rest)[0], qk["q"]),
            (lambda q: kda.qk_norm_rope_backward(q, qk["k"], **qk)[0], qk["q"])]:
        for want in (False, True):
            t = t.clone().requires_grad_(want)
            with pytest.raises(RuntimeError, match="recorded"):
                torch.jit.trace(f, (t,), check_trace=False)
            with pytest.raises(RuntimeError, match="recorded"):
                make_fx(f)(t)
        # modes that only watch are no recording
        from torch.utils._python_dispatch import TorchDispatchMode

        class Watch(TorchDispatchMode):
            def __torch_dispatch__(self, func, types, args=(), kwargs=None):
                return func(*args, **(kwargs or {}))
        with Watch(), torch.no_grad():
            watched = f(t)
        with torch.no_grad():
            assert torch.equal(watched, f(t))


def test_results_in_place_are_seen_by_autograd(way):
    """A tensor that a graph has saved and a call then writes to: the graph's backward pass says so."""
    def saved(t):
        leaf = torch.ones_like(t, requires_grad=True)
        return (leaf * t).sum()

    d = make("TND", [30, 9], 2, 64, FP, seed=7)
    if way == "python":
        d["plan"]._handle = None
    a = args(d, -1.0, "TND")
    qk = qk_inputs()
    empty = {n: torch.empty_like(d[n]) for n in ("x", "h0")}
    one = torch.empty_like(d["x"][:2])
    dense = lambda n: qk[n].clone()  # noqa: E731
    grads = {"dq": dense("q"), "dk": dense("k")}
    turned = {"q_out": dense("q"), "k_out": dense("k")}
    cases = [
        (d["h0"], lambda: single(d, state_out=d["h0"])),
        (empty["h0"], lambda: single(d, state_out=empty["h0"])),
        (one, lambda: single(d, out=one)),
        (d["h0"], lambda: kda.gated_recurrence(*a, final_state=d["h0"])),
        (empty["x"], lambda: kda.gated_recurrence(*a, out=empty["x"])),
        (qk["q"], lambda: kda.qk_norm_rope(**qk, q_out=qk["q"])),
        (turned["k_out"], lambda: kda.qk_norm_rope(**qk, **turned)),
        (grads["dq"], lambda: kda.qk_norm_rope_backward(grads["dq"], grads["dk"], **qk, **grads)),
        (grads["dk"], lambda: kda.qk_norm_rope_backward(grads["dq"], grads["dk"], **qk, **grads))]
    for i, (t, call) in enumerate(cases):
        loss = saved(t)
        with torch.no_grad():
            call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        # a call that is refused changes nothing, and a view tells its base
        before = t._version
        base = torch.zeros(2, *t.shape, device="cuda", dtype=t.dtype)
        with pytest.raises((kda.KdaError, ValueError)):
            single(d, lb=-7.0, state_out=d["h0"])
        assert t._version == before, i
        base[0].copy_(t)
        loss = saved(base)
        with torch.no_grad():
            single(d, state_out=base.flatten()[:d["h0"].numel()].view_as(d["h0"]))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():
        state = d["h0"].clone()
    single(d, state_out=state)  # no counter to move


def test_results_that_want_a_gradient_are_refused(way):
    d = make("TND", [30, 9], 2, 64, FP, seed=8)
    if way == "python":
        d["plan"]._handle = None
    a = args(d, -1.0, "TND")
    qk = qk_inputs()
    leaf = lambda t: torch.empty_like(t).requires_grad_()  # noqa: E731
    calls = [lambda: single(d, out=leaf(d["x"][:2])), lambda: single(d, state_out=leaf(d["h0"])),
             lambda: kda.gated_recurrence(*a, out=leaf(d["x"])),
             lambda: kda.gated_recurrence(*a, final_state=leaf(d["h0"])),
             lambda: kda.qk_norm_rope(**qk, q_out=leaf(qk["q"])),
             lambda: kda.qk_norm_rope(**qk, k_out=leaf(qk["k"])),
             lambda: kda.qk_norm_rope_backward(qk["q"], qk["k"], **qk, dq=leaf(qk["q"])),
             lambda: kda.qk_norm_rope_backward(qk["q"], qk["k"], **qk, dk=leaf(qk["k"]))]
    for call in calls:
        with pytest.raises(ValueError):
            call()
        with torch.no_grad():
            call()


def test_copies_of_a_plan(cuda_ok):
    """A plan that went through copy and pickle, as a module that keeps one does."""
    import copy
    import pickle
    d = make("TND", [700, 31], 2, 64, BF, seed=9)
    want = both(d)
    for again in (copy.copy, copy.deepcopy, lambda p: pickle.loads(pickle.dumps(p))):
        plan = again(d["plan"])
        assert plan._handle is not None
        got = both(dict(d, plan=plan))
        assert all(torch.equal(got[n], want[n]) for n in want)
        del plan
    assert all(torch.equal(p, want[n]) for n, p in both(d).items())


def after_an_odd_number(t):
    """t behind three values of another tensor: its gradient is a dense slice that starts 12 (fp32) or
    6 (bf16) bytes off any alignment."""
    return torch.cat([torch.zeros(3, dtype=t.dtype, device=t.device), t.flatten()])


@pytest.mark.parametrize("kind", [BF, FP])
def test_gradients_at_odd_addresses(kind, cuda_ok):
    d = make("TND", [70, 33], 2, 64, kind, seed=10)
    gen = torch.Generator().manual_seed(3)
    leaves = lambda: [d[n].clone().requires_grad_() for n in  # noqa: E731
                      ("x", "g", "beta", "h0", "A_log", "dt_bias")]

    def grads(ts, results, ups, spread):
        pieces = [spread(t) for t in results]
        ups = [spread(u) for u in ups]
        return torch.autograd.grad(pieces, ts, ups)

    ups = [torch.randn(d["x"].shape, generator=gen).cuda().to(kind), d["dfinal"]]
    got = []
    for spread in (after_an_odd_number, lambda t: t):
        ts = leaves()
        got.append(grads(ts, kda.gated_recurrence(*ts, -1.0, "TND", d["plan"]), ups, spread))
    assert all(torch.equal(p, q) for p, q in zip(*got))
    qk = qk_inputs(kind)
    names = ("q", "k", "q_weight", "k_weight")
    ups = [torch.randn(qk[n].shape, generator=gen).cuda().to(kind) for n in ("q", "k")]
    got = []
    for spread in (after_an_odd_number, lambda t: t):
        ts = {n: qk[n].clone().requires_grad_() for n in names}
        got.append(grads(list(ts.values()), kda.qk_norm_rope(**dict(qk, **ts)), ups, spread))
    assert all(torch.equal(p, q) for p, q in zip(*got))


def test_lazily_negated_tensors(way):
    """Values that torch has marked as negated but not rewritten are refused, and as gradients taken
    for what they stand for."""
    d = make("TND", [30, 9], 2, 64, FP, seed=11)
    if way == "python":
        d["plan"]._handle = None
    a = args(d, -1.0, "TND")
    names = ("x", "g", "beta", "h0", "A_log", "dt_bias")
    for i, name in enumerate(names):
        mine = list(a)
        mine[i] = torch._neg_view(a[i])
        assert mine[i].is_neg() and mine[i].is_contiguous()
        with pytest.raises(ValueError, match="negat"):
            kda.gated_recurrence(*mine)
        with pytest.raises(ValueError, match="negat"):
            kda.gated_recurrence(*mine[:6], *a[6:], final_state=torch.empty_like(d["h0"]))
    one = [d[n][:2].contiguous() for n in names[:3]] + [d[n] for n in names[3:]]
    for i in range(6):
        mine = one[:i] + [torch._neg_view(one[i])] + one[i + 1:]
        with pytest.raises(ValueError, match="negat"):
            kda.gated_recurrence_step(*mine, -1.0)
    for kw in ({"out": torch._neg_view(torch.empty_like(one[0]))},
               {"state_out": torch._neg_view(torch.empty_like(one[3]))}):
        with pytest.raises(ValueError, match="negat"):
            kda.gated_recurrence_step(*one, -1.0, **kw)
    states = kda.gated_recurrence(*a, return_states=True)[2]
    for g in ((torch._neg_view(d["dout"]), None), (None, torch._neg_view(d["dfinal"]))):
        with pytest.raises(ValueError, match="negat"):
            kda.gated_recurrence_backward(*g, *a, states)
    qk = qk_inputs()
    for name in ("q", "k", "inv_freq", "q_weight", "k_weight"):
        c = dict(qk, **{name: torch._neg_view(qk[name])})
        with pytest.raises(ValueError, match="negat"):
            kda.qk_norm_rope(**c)
        with pytest.raises(ValueError, match="negat"):
            kda.qk_norm_rope_backward(qk["q"], qk["k"], **c)
    # a gradient that arrives like this
    ts = [d[n].clone().requires_grad_() for n in ("x", "g", "beta", "h0", "A_log", "dt_bias")]
    out, final = kda.gated_recurrence(*ts, -1.0, "TND", d["plan"])
    got = torch.autograd.grad([out, final], ts, [torch._neg_view(d["dout"]), torch._neg_view(d["dfinal"])])
    want = kda.gated_recurrence_backward(-d["dout"], -d["dfinal"], *a, states)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    q, k = (qk[n].clone().requires_grad_() for n in ("q", "k"))
    both_out = kda.qk_norm_rope(**dict(qk, q=q, k=k))
    got = torch.autograd.grad(both_out, [q, k], [torch._neg_view(qk["q"]), torch._neg_view(qk["k"])])
    want = kda.qk_norm_rope_backward(-qk["q"], -qk["k"], **qk)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_tensors_without_memory_of_their_own(way):
    """Batched (vmap) and functional tensors have no address to pass on: every call says so, also where
    the argument could be left out."""
    d = make("TND", [30, 9], 2, 64, FP, seed=12)
    if way == "python":
        d["plan"]._handle = None
    a = args(d, -1.0, "TND")
    names = ("x", "g", "beta", "h0", "A_log", "dt_bias")
    one = [d[n][:2].contiguous() for n in names[:3]] + [d[n] for n in names[3:]]
    states = kda.gated_recurrence(*a, return_states=True)[2]
    qk = qk_inputs()
    qk["positions"] = torch.arange(40, dtype=torch.int32, device="cuda")
    put = lambda ts, i, t: (*ts[:i], t, *ts[i + 1:])  # noqa: E731
    cases = [(a[i], lambda t, i=i: kda.gated_recurrence(*put(a, i, t))[0]) for i in range(6)]
    cases += [(a[i], lambda t, i=i: kda.gated_recurrence_backward(d["dout"], None, *put(a, i, t), states)[0])
              for i in range(6)]
    cases += [(one[i], lambda t, i=i: kda.gated_recurrence_step(*put(one, i, t), -1.0)[0]) for i in range(6)]
    cases += [(t, lambda t, i=i: kda.gated_recurrence_backward(
        *put((d["dout"], d["dfinal"]), i, t), *a, states)[0]) for i, t in ((0, d["dout"]), (1, d["dfinal"]))]
    for name in ("q", "k", "positions", "inv_freq", "q_weight", "k_weight"):
        cases += [(qk[name], lambda t, n=name: kda.qk_norm_rope(**dict(qk, **{n: t}))[0]),
                  (qk[name], lambda t, n=name: kda.qk_norm_rope_backward(
                      qk["q"], qk["k"], **dict(qk, **{n: t}))[0])]
    for i, (t, call) in enumerate(cases):
        with pytest.raises((RuntimeError, ValueError)):
            torch.vmap(call)(torch.stack([t, t]))
        with pytest.raises((RuntimeError, ValueError)):
            torch.func.functionalize(call)(t)
        assert call(t) is not None, i


def test_calls_in_a_compiled_function(way):
    """torch.compile takes no call into its graphs, and runs it between them as it stands."""
    d = make("TND", [30, 9], 2, 64, FP, seed=13)
    if way == "python":
        d["plan"]._handle = None
    a, qk, out = args(d, -1.0, "TND"), qk_inputs(), torch.empty_like(d["x"])
    rest = {n: v for n, v in qk.items() if n != "q"}
    for f, t in ((lambda x: kda.gated_recurrence(x * 2, *a[1:])[0] * 3, d["x"]),
                 (lambda x: kda.gated_recurrence(x * 2, *a[1:], out=out)[0] * 3, d["x"]),
                 (lambda q: kda.qk_norm_rope(q=q * 2, **rest)[0] * 3, qk["q"])):
        torch._dynamo.reset()
        assert torch.equal(torch.compile(f, backend="eager")(t), f(t))
    torch._dynamo.reset()
    t, u = (d["x"].clone().requires_grad_() for _ in range(2))
    f = lambda x: kda.gated_recurrence(x * 2, *a[1:])[0].sum()  # noqa: E731
    torch.compile(f, backend="eager")(t).backward()
    f(u).backward()
    assert torch.equal(t.grad, u.grad)
