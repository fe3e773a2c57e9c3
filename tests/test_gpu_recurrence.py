"""The gated recurrence on the GPU against its definition in fp64 (tests/layer_refs.py, which
derives the tolerances): layouts, head dims, types, lengths around the tiles, padding, strides,
start and end states, gates at their ends, single tokens, streams, graphs and autograd."""
import pytest
import torch

import chunked_kda_prefill_b200 as kda
import layer_refs as R

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def make(layout, lengths, N, D, kind, S=None, seed=0, pad=float("nan")):
    """Inputs on the GPU; rows past a valid length are filled with `pad`."""
    gen = torch.Generator().manual_seed(seed)
    S = sum(lengths) if layout == "TND" else (S or max(lengths))
    B = len(lengths)
    shape = {"BNSD": (B, N, S, D), "BSND": (B, S, N, D), "TND": (S, N, D)}[layout]
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = {"x": rnd(*shape).to(kind), "g": rnd(*shape).to(kind), "beta": rnd(*shape[:-1]).to(kind),
         "h0": rnd(B, N, D), "A_log": rnd(N), "dt_bias": rnd(N, D)}
    d["dout"], d["dfinal"] = rnd(*shape).to(kind), rnd(B, N, D)
    if layout != "TND":
        for b, n in enumerate(lengths):
            for name in ("x", "g", "beta", "dout"):
                t = d[name]
                (t[b, :, n:] if layout == "BNSD" else t[b, n:]).fill_(pad)
    d = {k: v.cuda() for k, v in d.items()}
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    d["plan"] = kda.recurrence_plan(d["x"], layout, cu_seqlens=cu)
    return d


def args(d, lb, layout, h0=True):
    return (d["x"], d["g"], d["beta"], d["h0"] if h0 else None, d["A_log"], d["dt_bias"], lb,
            layout, d["plan"])


def clean(d, layout, lengths):
    """The inputs with zeros in the padding, for the reference."""
    c = dict(d)
    if layout != "TND":
        for name in ("x", "g", "beta", "dout"):
            t = c[name].clone()
            for b, n in enumerate(lengths):
                (t[b, :, n:] if layout == "BNSD" else t[b, n:]).zero_()
            c[name] = t
    return c


def run_both(d, lb, layout, lengths, h0=True, dout=True, dfinal=True):
    a = args(d, lb, layout, h0)
    out, final, states = kda.gated_recurrence(*a, return_states=True)
    grads = kda.gated_recurrence_backward(d["dout"] if dout else None,
                                          d["dfinal"] if dfinal else None, *a, states)
    names = ("dx", "dg", "dbeta", "dh0", "dA_log", "ddt_bias")
    got = {"out": out, "final": final} | dict(zip(names, grads))
    c = clean(d, layout, lengths)
    want = R.recurrence(c["x"], c["g"], c["beta"], c["h0"] if h0 else None, c["A_log"],
                        c["dt_bias"], lb, layout, lengths, c["dout"] if dout else None,
                        c["dfinal"] if dfinal else None)
    if not h0:
        assert got.pop("dh0") is None
    return got, want


def check_all(got, want):
    for name, t in got.items():
        R.check(t, want[name], name)


@pytest.mark.parametrize("layout", ["BNSD", "BSND", "TND"])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("lengths", [[1], [2, 1], [63, 64, 65], [127, 129, 1, 128], [300, 7, 516]])
def test_matches_definition(layout, D, lengths, cuda_ok):
    d = make(layout, lengths, 3, D, BF, seed=len(lengths) + D)
    check_all(*run_both(d, -5.0, layout, lengths))


@pytest.mark.parametrize("kind", [BF, HF, FP])
@pytest.mark.parametrize("lb", [-5.0, -0.25, 0.0])
def test_types_and_bounds(kind, lb, cuda_ok):
    lengths = [5, 200, 131]
    d = make("BSND", lengths, 2, 128, kind, S=333, seed=3)  # slots longer than any sequence
    check_all(*run_both(d, lb, "BSND", lengths))


@pytest.mark.parametrize("h0,dout,dfinal", [(False, True, True), (True, False, True),
                                            (True, True, False), (False, True, False)])
def test_absent_states_and_gradients(h0, dout, dfinal, cuda_ok):
    lengths = [1, 150]
    d = make("BNSD", lengths, 2, 64, FP, seed=4)
    check_all(*run_both(d, -2.0, "BNSD", lengths, h0, dout, dfinal))


@pytest.mark.parametrize("D", [128, 64])
def test_long_sequence_and_slow_decay(D, cuda_ok):
    """Many tiles in a row, with a carry that matters over all of them."""
    lengths = [6000, 33]
    d = make("TND", lengths, 1, D, FP, seed=5)
    d["A_log"].fill_(1.0)
    d["dt_bias"].fill_(-1.5)  # decays near one
    check_all(*run_both(d, -0.5, "TND", lengths))


@pytest.mark.parametrize("layout", ["BNSD", "TND"])
def test_many_short_sequences(layout, cuda_ok):
    lengths = [1 + (7 * i) % 11 for i in range(300)]
    d = make(layout, lengths, 2, 64, BF, seed=6)
    check_all(*run_both(d, -1.0, layout, lengths))


def test_padding_far_past_the_tokens(cuda_ok):
    """Slots of 1000 rows that hold 1 and 64 tokens: NaN behind them is never read, and every
    output row there is zero."""
    lengths = [1, 64]
    for layout in ("BNSD", "BSND"):
        d = make(layout, lengths, 2, 128, BF, S=1000, seed=7)
        got, want = run_both(d, -5.0, layout, lengths)
        check_all(got, want)
        for name in ("out", "dx", "dg", "dbeta"):
            for b, n in enumerate(lengths):
                tail = got[name][b, :, n:] if layout == "BNSD" else got[name][b, n:]
                assert torch.count_nonzero(tail) == 0, name


def test_gates_at_their_ends(cuda_ok):
    """Raw gates so large that the exponential overflows or vanishes: the sigmoid is 0 or 1."""
    lengths = [100]
    d = make("TND", lengths, 2, 128, BF, seed=8)
    d["g"][::3] = -3e38
    d["g"][1::3] = 3e38
    d["beta"][::2] = 300.0
    d["beta"][1::4] = -300.0
    check_all(*run_both(d, -5.0, "TND", lengths))


@pytest.mark.parametrize("layout", ["BNSD", "BSND", "TND"])
def test_strided_and_broadcast_inputs(layout, cuda_ok):
    """x and g as slices of one projection, beta as every second value, one gate for all heads."""
    lengths, N, D = [70, 33], 3, 64
    d = make(layout, lengths, N, D, BF, seed=9, pad=0.0)
    both = torch.cat([d["x"], d["g"], d["x"]], -1)
    d["x"], wide = both[..., :D], both[..., D:2 * D]
    beta = torch.stack([d["beta"], d["beta"] * 0 + float("nan")], -1).flatten(-2)
    d["beta"] = beta[..., ::2]
    head = 1 if layout != "BSND" else 2
    d["g"] = wide.narrow(head, 0, 1).expand(wide.shape)
    wide_dout = torch.cat([d["dout"], d["dout"] * 0 + 7], -1)
    d["dout"] = wide_dout[..., :D]
    assert not d["x"].is_contiguous() and not d["beta"].is_contiguous()
    got, want = run_both(d, -2.0, layout, lengths)
    check_all(got, want)
    dense = dict(d, **{n: d[n].contiguous() for n in ("x", "g", "beta", "dout")})
    same, _ = run_both(dense, -2.0, layout, lengths)
    for name in got:
        assert torch.equal(got[name], same[name]), name


def test_same_bits_on_every_run(cuda_ok):
    lengths = [3000, 2000, 999]
    d = make("TND", lengths, 2, 128, BF, seed=10)
    a = args(d, -1.0, "TND")
    runs = []
    for _ in range(5):
        out, final, states = kda.gated_recurrence(*a, return_states=True)
        runs.append((out, final) + kda.gated_recurrence_backward(d["dout"], d["dfinal"], *a, states))
    for r in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(runs[0], r))


def test_split_sequence_carries_its_state(cuda_ok):
    """Two calls, the second from the first one's final state, equal one call over the whole."""
    d = make("BSND", [500], 2, 128, FP, seed=11)
    out, final = kda.gated_recurrence(*args(d, -1.0, "BSND"))
    state, parts = d["h0"], []
    for lo, hi in ((0, 1), (1, 130), (130, 500)):
        x, g, beta = (d[n][:, lo:hi] for n in ("x", "g", "beta"))
        plan = kda.recurrence_plan(x, "BSND")
        o, state = kda.gated_recurrence(x, g, beta, state, d["A_log"], d["dt_bias"], -1.0, "BSND",
                                        plan)
        parts.append(o)
    want = R.recurrence(d["x"], d["g"], d["beta"], d["h0"], d["A_log"], d["dt_bias"], -1.0, "BSND",
                        [500])
    R.check(torch.cat(parts, 1), want["out"], "parts")
    R.check(state, want["final"], "state")
    R.check(out, want["out"], "whole")


@pytest.mark.parametrize("kind", [BF, HF, FP])
@pytest.mark.parametrize("B,N,D", [(1, 1, 64), (3, 5, 128), (257, 2, 64), (64, 32, 128)])
def test_step(kind, B, N, D, cuda_ok):
    d = make("BSND", [1] * B, N, D, kind, seed=B)
    x, g, beta = d["x"][:, 0], d["g"][:, 0], d["beta"][:, 0]
    want = R.recurrence(d["x"], d["g"], d["beta"], d["h0"], d["A_log"], d["dt_bias"], -5.0, "BSND",
                        [1] * B)
    call = (x.contiguous(), g.contiguous(), beta.contiguous())
    out, state = kda.gated_recurrence_step(*call, d["h0"], d["A_log"], d["dt_bias"], -5.0)
    R.check(out[:, None], want["out"], "out")
    R.check(state, want["final"], "state")
    mine = d["h0"].clone()
    out2, state2 = kda.gated_recurrence_step(*call, mine, d["A_log"], d["dt_bias"], -5.0,
                                             state_out=mine)
    assert state2.data_ptr() == mine.data_ptr()
    assert torch.equal(out, out2) and torch.equal(state, state2)
    none = kda.gated_recurrence_step(*call, None, d["A_log"], d["dt_bias"], -5.0)
    zero = kda.gated_recurrence_step(*call, torch.zeros_like(mine), d["A_log"], d["dt_bias"], -5.0)
    assert torch.equal(none[0], zero[0]) and torch.equal(none[1], zero[1])


def test_final_state_in_place(cuda_ok):
    lengths = [1, 400]
    d = make("TND", lengths, 3, 128, BF, seed=12)
    out, final = kda.gated_recurrence(*args(d, -1.0, "TND"))
    state = d["h0"].clone()
    a = list(args(d, -1.0, "TND"))
    a[3] = state
    out2, final2 = kda.gated_recurrence(*a, final_state=state)
    assert final2.data_ptr() == state.data_ptr()
    assert torch.equal(out, out2) and torch.equal(final, final2)


def test_guard_bands(cuda_ok):
    """out and final_state between bytes that must survive; the workspace's status says OK."""
    lengths = [130, 1, 64]
    d = make("BNSD", lengths, 2, 64, BF, S=200, seed=13)
    n, m = d["x"].numel(), d["h0"].numel()
    buf = torch.full((n + 8192,), 3.0, dtype=BF, device="cuda")
    sbuf = torch.full((m + 4096,), 3.0, device="cuda")
    ws = torch.full((d["plan"].workspace_bytes + 4096,), 7, dtype=torch.uint8, device="cuda")
    out = buf[4096:4096 + n].view(d["x"].shape)
    fs = sbuf[2048:2048 + m].view(d["h0"].shape)
    work = ws[:d["plan"].workspace_bytes]
    kda.gated_recurrence(*args(d, -5.0, "BNSD"), out=out, final_state=fs, workspace=work)
    kda.device_status(work)
    want, wfs = kda.gated_recurrence(*args(d, -5.0, "BNSD"))
    assert torch.equal(out, want) and torch.equal(fs, wfs)
    assert (buf[:4096] == 3).all() and (buf[4096 + n:] == 3).all()
    assert (sbuf[:2048] == 3).all() and (sbuf[2048 + m:] == 3).all()
    assert (ws[d["plan"].workspace_bytes:] == 7).all()


def test_another_plan_on_the_device_is_reported(cuda_ok):
    """A device copy that is not the host plan's: nothing is computed and the status says so."""
    d = make("TND", [100, 30], 2, 64, BF, seed=14)
    plan = d["plan"]
    plan.dev[23] += 1
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    kda.gated_recurrence(*args(d, -5.0, "TND"), workspace=ws)
    with pytest.raises(kda.KdaError) as e:
        kda.device_status(ws)
    assert e.value.code == 8


def test_streams_side_by_side(cuda_ok):
    """One plan, two streams at once: every call has a scratch of its own."""
    lengths = [4000, 100]
    d = [make("TND", lengths, 4, 128, BF, seed=s) for s in (15, 16)]
    d[1]["plan"] = d[0]["plan"]
    alone = [kda.gated_recurrence(*args(v, -1.0, "TND")) for v in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for v, s in zip(d, streams):
            got.append(kda.gated_recurrence(*args(v, -1.0, "TND"), stream=s))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(alone[i % 2], r))


def test_captured_graphs(cuda_ok):
    """Forward and backward in two graphs over one plan, replayed side by side with new inputs."""
    lengths = [700, 90]
    d = make("TND", lengths, 2, 128, BF, seed=17)

    def step():
        a = args(d, -1.0, "TND")
        out, final, states = kda.gated_recurrence(*a, return_states=True)
        return (out, final) + kda.gated_recurrence_backward(d["dout"], d["dfinal"], *a, states)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    graphs, results = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(step())
        graphs.append(graph)
    new = make("TND", lengths, 2, 128, BF, seed=18)
    for name in ("x", "g", "beta", "h0", "dout", "dfinal"):
        d[name].copy_(new[name])
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for r in results:
        assert all(torch.equal(p, q) for p, q in zip(want, r))


def leaves(d):
    return [d[n].detach().clone().requires_grad_() for n in
            ("x", "g", "beta", "h0", "A_log", "dt_bias")]


def test_autograd(cuda_ok):
    """Through torch.autograd: dense and broadcast gradients, unused outputs, frozen inputs."""
    lengths, layout = [90, 41], "BSND"
    d = make(layout, lengths, 2, 64, FP, seed=19, pad=0.0)
    got, _ = run_both(d, -2.0, layout, lengths)
    ts = leaves(d)
    out, final = kda.gated_recurrence(*ts, -2.0, layout, d["plan"])
    torch.autograd.backward([out, final], [d["dout"], d["dfinal"]])
    for t, name in zip(ts, ("dx", "dg", "dbeta", "dh0", "dA_log", "ddt_bias")):
        assert torch.equal(t.grad, got[name]), name
    # sum() hands over a gradient of ones with stride 0; final_state is not used
    ts = leaves(d)
    kda.gated_recurrence(*ts, -2.0, layout, d["plan"])[0].sum().backward()
    ones = dict(d, dout=torch.ones_like(d["dout"]))
    only, _ = run_both(ones, -2.0, layout, lengths, dfinal=False)
    for t, name in zip(ts, ("dx", "dg", "dbeta", "dh0", "dA_log", "ddt_bias")):
        assert torch.equal(t.grad, only[name]), name
    # the final state alone, parameters frozen, no initial state
    x, g = (d[n].clone().requires_grad_() for n in ("x", "g"))
    _, final = kda.gated_recurrence(x, g, d["beta"], None, d["A_log"], d["dt_bias"], -2.0, layout,
                                    d["plan"])
    final.backward(d["dfinal"])
    only, _ = run_both(d, -2.0, layout, lengths, h0=False, dout=False)
    assert torch.equal(x.grad, only["dx"]) and torch.equal(g.grad, only["dg"])
    # a broadcast start state gets the sum over the sequences
    h0 = d["h0"][:1].clone().requires_grad_()
    out, _ = kda.gated_recurrence(d["x"], d["g"], d["beta"], h0.expand(2, -1, -1).contiguous(),
                                  d["A_log"], d["dt_bias"], -2.0, layout, d["plan"])
    out.backward(d["dout"])
    assert h0.grad.shape == h0.shape and torch.isfinite(h0.grad).all()


def test_gradients_against_differences(cuda_ok):
    """The kernel's gradients along a direction, against central differences of the definition in
    fp64: the step 1e-4 leaves 1e-8 relative from the third derivative and 1e-11 from rounding, both
    far below the kernel's own bound."""
    lengths, layout, lb = [40, 75], "TND", -3.0
    d = make(layout, lengths, 2, 64, FP, seed=20)
    got, want = run_both(d, lb, layout, lengths)
    names = ("x", "g", "beta", "h0", "A_log", "dt_bias")
    gen = torch.Generator().manual_seed(1)
    for name, grad in zip(names, ("dx", "dg", "dbeta", "dh0", "dA_log", "ddt_bias")):
        v = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
        loss = []
        for e in (1e-4, -1e-4):
            c = {n: d[n].double().cpu() for n in names}
            c[name] = c[name] + e * v
            R.HALF.setdefault(torch.float64, 0.0)
            r = R.recurrence(*(c[n] for n in names), lb, layout, lengths)
            loss.append((r["out"][0] * d["dout"].double().cpu()).sum()
                        + (r["final"][0] * d["dfinal"].double().cpu()).sum())
        diff = float(loss[0] - loss[1]) / 2e-4
        mine = float((got[grad].double().cpu() * v).sum())
        bound = float((want[grad][1] * v.abs()).sum())
        scale = float((want[grad][0] * v).abs().sum())
        assert abs(mine - diff) <= bound + 1e-7 * scale, (name, mine, diff, bound)


@pytest.mark.parametrize("bad", ["x_type", "g_type", "shape", "channels", "device", "layout",
                                 "align", "alias", "step_grad", "out_grad", "plan", "lower_bound"])
def test_refusals(bad, cuda_ok):
    d = make("BSND", [40, 7], 2, 64, BF, seed=21, pad=0.0)
    a = list(args(d, -1.0, "BSND"))
    kw = {}
    if bad == "x_type":
        a[0] = a[0].double()
    elif bad == "g_type":
        a[1] = a[1].half()
    elif bad == "shape":
        a[2] = a[2][:, :-1]
    elif bad == "channels":
        a[0] = a[0].transpose(-1, -2).contiguous().transpose(-1, -2)
    elif bad == "device":
        a[1] = a[1].cpu()
    elif bad == "layout":
        a[7] = "BNSD"
    elif bad == "align":
        a[0] = torch.zeros(a[0].numel() + 1, dtype=BF, device="cuda")[1:].view(a[0].shape)
    elif bad == "alias":
        kw["out"] = a[0]
    elif bad == "out_grad":
        a[0] = a[0].clone().requires_grad_()
        kw["out"] = torch.empty_like(a[1])
    elif bad == "lower_bound":
        a[6] = -5.5
    elif bad == "plan":
        a[8] = kda.recurrence_plan(d["x"][:, :20], "BSND")
    with pytest.raises((TypeError, ValueError, kda.KdaError)):
        if bad == "step_grad":
            x = d["x"][:, 0].clone().requires_grad_()
            kda.gated_recurrence_step(x, d["g"][:, 0].contiguous(), d["beta"][:, 0].contiguous(),
                                      None, d["A_log"], d["dt_bias"], -1.0)
        else:
            kda.gated_recurrence(*a, **kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("layout", ["BNSD", "BSND", "TND"])
@pytest.mark.parametrize("kind,D", [(BF, 128), (HF, 64), (FP, 128), (FP, 64)])
def test_cut_sequences(layout, kind, D, cuda_ok):
    """Long sequences of few heads, which the plan cuts: segments that start from joined maps, next
    to a sequence that stays whole."""
    lengths = [2500, 1, 700]
    d = make(layout, lengths, 2, D, kind, S=None if layout == "TND" else 2600, seed=22)
    d["A_log"].fill_(1.0)
    d["dt_bias"].fill_(-1.5)  # slow decays: a segment's start matters far into it
    assert d["plan"].host[12] > 0 and d["plan"].host[11] > len(lengths)
    check_all(*run_both(d, -0.5, layout, lengths))
    check_all(*run_both(d, -0.5, layout, lengths, h0=False, dout=False))
    check_all(*run_both(d, -0.5, layout, lengths, dfinal=False))


def test_cut_sequence_in_place(cuda_ok):
    """The end of a cut sequence replaces its start while other segments are still at work."""
    d = make("BNSD", [6000, 4000], 1, 128, BF, S=6000, seed=23)
    assert d["plan"].host[12] > 0
    a = list(args(d, -0.25, "BNSD"))
    out, final = kda.gated_recurrence(*a)
    for _ in range(3):
        a[3] = d["h0"].clone()
        out2, final2 = kda.gated_recurrence(*a, final_state=a[3])
        assert final2.data_ptr() == a[3].data_ptr()
        assert torch.equal(out, out2) and torch.equal(final, final2)


def test_nan_stays_in_its_channel_and_after_its_token(cuda_ok):
    """A NaN gate or value spoils its own channel from its token on (dbeta, a sum over channels, from
    nowhere else), and a NaN gradient its channel up to its token; everything else keeps its bits."""
    lengths, t, c = [150], 77, 5
    d = make("TND", lengths, 2, 64, BF, seed=24)
    clean, _ = run_both(d, -1.0, "TND", lengths)
    for name in ("x", "g"):
        bad = dict(d, **{name: d[name].clone()})
        bad[name][t, 1, c] = float("nan")
        got, _ = run_both(bad, -1.0, "TND", lengths)
        spoilt = torch.zeros(150, 2, 64, dtype=torch.bool, device="cuda")
        spoilt[t:, 1, c] = True
        assert torch.isnan(got["out"][spoilt]).all()
        assert torch.equal(got["out"][~spoilt], clean["out"][~spoilt])
        assert torch.isnan(got["final"][0, 1, c]) and torch.isnan(got["final"]).sum() == 1
    bad = dict(d, dout=d["dout"].clone())
    bad["dout"][t, 1, c] = float("nan")
    got, _ = run_both(bad, -1.0, "TND", lengths)
    spoilt = torch.zeros(150, 2, 64, dtype=torch.bool, device="cuda")
    spoilt[:t + 1, 1, c] = True
    for name in ("dx", "dg"):
        assert torch.isnan(got[name][spoilt]).all()
        assert torch.equal(got[name][~spoilt], clean[name][~spoilt]), name
    assert torch.isnan(got["dbeta"][:t + 1, 1]).all()
    assert torch.equal(got["dbeta"][t + 1:], clean["dbeta"][t + 1:])
    assert torch.equal(got["dbeta"][:, 0], clean["dbeta"][:, 0])
    assert torch.equal(got["out"], clean["out"])


def test_offsets_past_32_bits(cuda_ok):
    """Inputs whose heads lie 2^31 elements apart, and outputs of more than 2^31 elements: every head
    of equal inputs and parameters gives the same bits, the last as the first."""
    D, S = 128, 96
    far = torch.empty((1 << 31) + S * D, dtype=BF, device="cuda")
    d = make("BNSD", [S], 2, D, BF, seed=25)
    near, _ = run_both(d, -1.0, "BNSD", [S])
    wide = torch.as_strided(far, (1, 2, S, D), (0, 1 << 31, D, 1))
    for name in ("x", "g", "dout"):
        wide.copy_(d[name])
        got, _ = run_both(dict(d, **{name: wide}), -1.0, "BNSD", [S])
        assert all(torch.equal(got[n], near[n]) for n in got), name
    del far, wide
    N, S = 130, 131072
    one = make("BNSD", [S], 1, D, BF, seed=26)
    every = {n: one[n].expand(1, N, *one[n].shape[2:]) for n in ("x", "g", "beta", "dout")}
    every |= {n: one[n].expand(1, N, D).contiguous() for n in ("h0", "dfinal")}
    every |= {"A_log": one["A_log"].expand(N).contiguous(),
              "dt_bias": one["dt_bias"].expand(N, D).contiguous()}
    every["plan"] = kda.recurrence_plan(every["x"], "BNSD")
    a = args(every, -1.0, "BNSD")
    out, final, states = kda.gated_recurrence(*a, return_states=True)
    assert out.numel() > 1 << 31
    grads = kda.gated_recurrence_backward(every["dout"], every["dfinal"], *a, states)
    for t in (out, final) + grads[:4]:
        assert torch.equal(t[:, :1], t[:, -1:]) and torch.equal(t[:, :1], t[:, 64:65])
    assert torch.equal(grads[4][:1], grads[4][-1:]) and torch.equal(grads[5][:1], grads[5][-1:])
    few = kda.gated_recurrence(*args(one, -1.0, "BNSD"))[0]  # cut, so not the same bits
    diff = (few[0, 0].float() - out[0, -1].float()).abs()
    # each is within half a step of bf16 of what its own fp32 error leaves, far below another half
    assert (diff <= 2 * 2.0 ** -8 * few[0, 0].float().abs() + 1e-5).all()


def test_captured_training_step(cuda_ok):
    """Forward and backward through torch.autograd in one graph, replayed with new data."""
    lengths = [300, 45]
    d = make("TND", lengths, 2, 64, FP, seed=27)
    ts = leaves(d)

    def step():
        out, final = kda.gated_recurrence(*ts, -1.0, "TND", d["plan"])
        return torch.autograd.grad([out, final], ts, [d["dout"], d["dfinal"]])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    new = make("TND", lengths, 2, 64, FP, seed=28)
    with torch.no_grad():
        for t, name in zip(ts, ("x", "g", "beta", "h0", "A_log", "dt_bias")):
            t.copy_(new[name])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, step()))


def test_calls_from_two_threads(cuda_ok):
    """One plan, a thread and a stream each, first calls of a kernel included."""
    from concurrent.futures import ThreadPoolExecutor
    lengths = [900, 70]
    d = make("TND", lengths, 3, 64, HF, seed=29)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def work(s):
        with torch.cuda.stream(s):
            a = args(d, -1.0, "TND")
            res = None
            for _ in range(5):
                out, final, states = kda.gated_recurrence(*a, return_states=True)
                res = (out, final) + kda.gated_recurrence_backward(d["dout"], d["dfinal"], *a, states)
            s.synchronize()
            return res

    with ThreadPoolExecutor(2) as pool:
        got = list(pool.map(work, streams))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    check_all(*run_both(d, -1.0, "TND", lengths))


@pytest.mark.parametrize("lengths,cut", [([150], False), ([4000], True)])
def test_infinite_values_stay_infinite(lengths, cut, cuda_ok):
    """An infinite value makes its channel's state infinite for good, however small the decays that
    follow multiply to, and touches nothing else."""
    d = make("TND", lengths, 2, 64, BF, seed=30)
    if not cut:
        lengths = [150] + [1] * 100  # enough units to leave every sequence whole
        d = make("TND", lengths, 2, 64, BF, seed=30)
    assert (d["plan"].host[12] > 0) == cut
    clean, _ = kda.gated_recurrence(*args(d, -5.0, "TND"))
    d["x"] = d["x"].clone()
    d["x"][77, 1, 5] = float("inf")
    out, final = kda.gated_recurrence(*args(d, -5.0, "TND"))
    spoilt = torch.zeros(clean.shape, dtype=torch.bool, device="cuda")
    spoilt[77:lengths[0], 1, 5] = True
    assert (out[spoilt] == float("inf")).all() and final[0, 1, 5] == float("inf")
    assert torch.equal(out[~spoilt], clean[~spoilt])


def test_long_padding_behind_few_sequences(cuda_ok):
    """Two heads, slots of 20000 rows: the zeros come from every block, in all layouts' strides."""
    lengths = [3, 20000, 900]
    for layout in ("BNSD", "BSND"):
        d = make(layout, lengths, 2, 64, HF, S=20000, seed=31)
        for name in ("out", "dx", "dg"):
            torch.full(d["x"].shape, 7.0, dtype=HF, device="cuda")  # what the results' memory may hold
        a = args(d, -5.0, layout)
        out, final, states = kda.gated_recurrence(*a, return_states=True)
        grads = kda.gated_recurrence_backward(d["dout"], d["dfinal"], *a, states)
        for t in (out,) + grads[:3]:
            for b, n in enumerate(lengths):
                slot = t[b] if layout == "BSND" else t[b].transpose(0, 1)
                assert torch.count_nonzero(slot[n:]) == 0
                assert torch.isfinite(slot[:n]).all() and torch.count_nonzero(slot[:n]) > 0


@pytest.mark.parametrize("layout,kind,D", [("TND", BF, 128), ("BNSD", HF, 64), ("BSND", FP, 128)])
def test_more_sequences_than_warps(layout, kind, D, cuda_ok):
    """So many short sequences that every warp walks its own, several one after another."""
    lengths = [1 + (7 * i) % 40 for i in range(1300)]
    d = make(layout, lengths, 4, D, kind, seed=32)
    assert d["plan"].host[17] == 1
    check_all(*run_both(d, -1.0, layout, lengths))
    check_all(*run_both(d, -1.0, layout, lengths, h0=False, dout=False))


def test_inputs_may_go_while_another_stream_uses_them(cuda_ok):
    """Inputs and the plan are dropped right after a call on another stream, and their memory is asked
    for again; a long wait on that stream comes first."""
    lengths = [600, 30]
    d = make("TND", lengths, 2, 64, BF, seed=33)
    want = kda.gated_recurrence(*args(d, -1.0, "TND"))
    q = d["x"].contiguous()
    inv = torch.ones(32, device="cuda")
    turned = kda.qk_norm_rope(q, q.clone(), None, inv, None, None, 1e-6, "TND")
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(50_000_000)
    mine = {n: t.clone() for n, t in d.items() if n != "plan"}
    mine["plan"] = kda.recurrence_plan(mine["x"], "TND", cu_seqlens=[0, 600, 630])
    k, f = q.clone(), inv.clone()
    torch.cuda.current_stream().synchronize()
    got = kda.gated_recurrence(*args(mine, -1.0, "TND"), stream=other)
    rot = kda.qk_norm_rope(mine["x"], k, None, f, None, None, 1e-6, "TND", stream=other)
    sizes = [t.numel() for t in mine.values() if isinstance(t, torch.Tensor)] + [k.numel()]
    del mine, k, f
    junk = [torch.full((n,), float("nan"), dtype=t, device="cuda") for n in sizes for t in (BF, FP)]
    torch.cuda.synchronize()
    assert junk and all(torch.equal(a, b) for a, b in zip(got + rot, want + turned))


def test_compiled_and_python_calls_agree(cuda_ok, monkeypatch):
    """The compiled calls are there, and give what the Python functions give by way of ctypes: results,
    their shapes and types, statuses and refusals."""
    from chunked_kda_prefill_b200 import _lib
    assert _lib.calls() is not None
    for layout, lengths, kind, lb in (("BNSD", [200, 3], BF, -5), ("BSND", [70, 90], HF, -1.0),
                                      ("TND", [3000, 5], FP, -0.5)):
        d = make(layout, lengths, 2, 64, kind, S=None if layout == "TND" else 210, seed=34)
        one = [d[n].movedim(2, 1)[:, 0] if layout == "BNSD" else d[n][:, 0] if layout == "BSND" else
               d[n][:2] for n in ("x", "g", "beta")]
        one = [t.contiguous() for t in one]
        inv = torch.rand(16, device="cuda")
        w = torch.rand(64, device="cuda")

        def everything():
            res = []
            for h0 in (True, False):
                a = args(d, lb, layout, h0)
                out, final, states = kda.gated_recurrence(*a, return_states=True)
                res += [*kda.gated_recurrence(*a), out, final]
                res += kda.gated_recurrence(*a, return_states=1)
                for dout in (d["dout"], None):
                    for dfinal in (d["dfinal"], None):
                        res += kda.gated_recurrence_backward(dout, dfinal, *a, states)
                state = d["h0"].clone()
                res += kda.gated_recurrence_step(*one, state if h0 else None, d["A_log"],
                                                 d["dt_bias"], lb)
                res += kda.gated_recurrence_step(*one, state, d["A_log"], d["dt_bias"], lb,
                                                 state_out=state)
                assert res[-1] is state
            for pos, f, qw in ((None, inv, None), (None, None, w)):
                c = (d["x"], d["g"], pos, f, qw, w, 1e-6, layout)
                res += kda.qk_norm_rope(*c, interleaved=True)
                res += kda.qk_norm_rope_backward(d["dout"], d["x"], *c, interleaved=True)
            bad = list(args(d, lb, layout))
            for i, v in ((6, -7.0), (2, d["beta"][:1]), (4, d["A_log"].double()), (7, "NBD")):
                with pytest.raises((TypeError, ValueError, kda.KdaError)) as e:
                    kda.gated_recurrence(*bad[:i], v, *bad[i + 1:])
                res.append(str(e.value))
            with pytest.raises(kda.KdaError) as e:
                kda.qk_norm_rope(d["x"], d["x"], None, None, None, None, -1.0, layout)
            return res + [str(e.value)]

        fast = everything()
        with monkeypatch.context() as m:
            m.setattr(_lib, "_calls", None)
            m.setattr(d["plan"], "_handle", None)
            slow = everything()
        assert len(fast) == len(slow)
        for a, b in zip(fast, slow):
            if isinstance(a, torch.Tensor):
                assert a.dtype == b.dtype and a.is_contiguous() and a.shape == b.shape
                assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
            else:
                assert a == b


def test_compiled_calls_follow_stream_grad_mode_and_capture(cuda_ok):
    """The current stream is the one that results are made on; inputs that want a gradient, and results
    under no_grad and inference mode, are told apart."""
    lengths = [500]
    d = make("TND", lengths, 2, 64, BF, seed=35)
    want, _ = kda.gated_recurrence(*args(d, -1.0, "TND"))
    out = None
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        # the stream's own memory first: asking the device for some may wait for all of its work
        for _ in range(2):
            del out
            out, _ = kda.gated_recurrence(*args(d, -1.0, "TND"))
        s.synchronize()
        torch.cuda._sleep(400_000_000)
        del out
        out, _ = kda.gated_recurrence(*args(d, -1.0, "TND"))
        done = torch.cuda.Event()
        done.record()
    assert not done.query()
    s.synchronize()
    assert torch.equal(out, want)
    ts = leaves(d)
    assert kda.gated_recurrence(*ts, -1.0, "TND", d["plan"])[0].grad_fn is not None
    with torch.no_grad():
        assert not kda.gated_recurrence(*ts, -1.0, "TND", d["plan"])[0].requires_grad
    with torch.inference_mode():
        out, _ = kda.gated_recurrence(*ts, -1.0, "TND", d["plan"])
        assert torch.equal(out, want) and out.is_inference()


@pytest.mark.parametrize("lengths,N,S", [([4000, 9], 2, 4100), ([1 + i % 30 for i in range(900)], 8, 31),
                                         ([70, 500, 3], 3, 500)])
def test_workspace_and_results_between_guards(lengths, N, S, cuda_ok):
    """Cut sequences, a warp for each of many short ones, and a ring: the workspaces of both passes and
    the forward's results end where they say, and the status is left in them."""
    d = make("BSND", lengths, N, 64, HF, S=S, seed=36)
    plan, a = d["plan"], args(d, -1.0, "BSND")

    def guarded(n, dtype, fill):
        buf = torch.full((n + 8192,), fill, dtype=dtype, device="cuda")
        return buf, buf[4096:4096 + n]

    want = kda.gated_recurrence(*a, return_states=True)
    want_grads = kda.gated_recurrence_backward(d["dout"], d["dfinal"], *a, want[2])
    ob, out = guarded(d["x"].numel(), HF, 3.0)
    fb, final = guarded(d["h0"].numel(), FP, 3.0)
    wb, ws = guarded(plan.workspace_bytes, torch.uint8, 7)
    got = kda.gated_recurrence(*a, out=out.view(d["x"].shape), final_state=final.view(d["h0"].shape),
                               workspace=ws, return_states=True)
    kda.device_status(ws)
    bb, bws = guarded(plan.backward_workspace_bytes, torch.uint8, 7)
    grads = kda.gated_recurrence_backward(d["dout"], d["dfinal"], *a, got[2], workspace=bws)
    kda.device_status(bws)
    assert all(torch.equal(p, q) for p, q in zip(got + grads, want + want_grads))
    for buf, fill in ((ob, 3), (fb, 3), (wb, 7), (bb, 7)):
        assert (buf[:4096] == fill).all() and (buf[-4096:] == fill).all()
    short = torch.empty(plan.backward_workspace_bytes - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(kda.KdaError):
        kda.gated_recurrence_backward(d["dout"], d["dfinal"], *a, got[2], workspace=short)


def test_broadcast_writes_and_gates(cuda_ok):
    """One write logit for all heads and tokens, one gate for all tokens, one gradient for all: strides
    of zero in every place, the gradients of every copy apart."""
    lengths, layout = [700, 41], "BSND"
    d = make(layout, lengths, 3, 64, FP, S=700, seed=37, pad=0.0)
    d["beta"] = d["beta"][:1, :1, :1].expand(2, 700, 3)
    d["g"] = d["g"][:, :1].expand(2, 700, 3, 64)
    d["dout"] = d["dout"][:1, :1, :1].expand(2, 700, 3, 64)
    check_all(*run_both(d, -2.0, layout, lengths))
