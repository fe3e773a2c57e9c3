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
