"""Norm and rotation of query and key heads on the GPU against the definition in fp64
(tests/layer_refs.py, which derives the tolerances): layouts, head dims, types, head counts, both
pairings, partial and no rotation, far positions, padding, strides, in place, graphs, autograd."""
import pytest
import torch

import chunked_kda_prefill_b200 as kda
import layer_refs as R

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def make(layout, B, Nq, Nk, S, D, kind, turned=None, seed=0, far=1 << 20):
    gen = torch.Generator().manual_seed(seed)
    shape = {"BNSD": lambda n: (B, n, S, D), "BSND": lambda n: (B, S, n, D),
             "TND": lambda n: (S, n, D)}[layout]
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    half = (D if turned is None else turned) // 2
    d = {"q": rnd(*shape(Nq)).to(kind), "k": rnd(*shape(Nk)).to(kind),
         "dq": rnd(*shape(Nq)).to(kind), "dk": rnd(*shape(Nk)).to(kind),
         "pos": torch.randint(0, far, (S,) if layout == "TND" else (B, S), generator=gen,
                              dtype=torch.int32),
         "inv": (10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float(),
         "qw": 1 + 0.3 * rnd(D), "kw": 1 + 0.3 * rnd(D)}
    return {n: t.cuda() for n, t in d.items()}


def inputs(d):
    return d["q"], d["k"], d["pos"], d["inv"], d["qw"], d["kw"]


def run_both(d, layout, interleaved=False, eps=EPS):
    q, k = kda.qk_norm_rope(*inputs(d), eps, layout, interleaved=interleaved)
    dq, dk, dqw, dkw = kda.qk_norm_rope_backward(d["dq"], d["dk"], *inputs(d), eps, layout,
                                                 interleaved=interleaved)
    got = {"q": q, "k": k, "dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    want = {}
    for n in ("q", "k"):
        r = R.qk_side(d[n], d[n + "w"], d["pos"], d["inv"], eps, layout, interleaved, d["d" + n])
        want |= {n: r["out"], "d" + n: r["dx"], f"d{n}w": r["dw"]}
    return got, want


def check_all(got, want):
    for name, t in got.items():
        if t is not None:
            R.check(t, want[name], name)


@pytest.mark.parametrize("layout", ["BNSD", "BSND", "TND"])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("B,Nq,Nk,S", [(1, 1, 1, 1), (3, 5, 2, 17), (2, 4, 4, 131), (2, 33, 3, 9)])
def test_matches_definition(layout, D, B, Nq, Nk, S, cuda_ok):
    d = make(layout, B, Nq, Nk, S, D, BF, seed=S + D)
    for interleaved in (False, True):
        check_all(*run_both(d, layout, interleaved))


@pytest.mark.parametrize("kind", [BF, HF, FP])
@pytest.mark.parametrize("D,turned", [(128, 0), (128, 16), (128, 48), (128, 112), (64, 32), (64, 64)])
def test_types_and_partial_rotation(kind, D, turned, cuda_ok):
    d = make("BSND", 2, 3, 2, 40, D, kind, turned=turned, seed=turned + 1)
    for interleaved in (False, True):
        check_all(*run_both(d, "BSND", interleaved))


def test_absent_arguments(cuda_ok):
    """No positions (0..S-1 in every slot), no weights, no frequencies."""
    for layout in ("BNSD", "TND"):
        d = make(layout, 3, 2, 1, 50, 64, FP, seed=2)
        d |= {"pos": None, "qw": None, "kw": None}
        check_all(*run_both(d, layout))
        d["inv"] = None
        check_all(*run_both(d, layout))


def test_far_positions(cuda_ok):
    """Positions up to the end of int32: the phase does not lose its place."""
    d = make("TND", 1, 2, 2, 64, 128, FP, seed=3, far=(1 << 31) - 1)
    d["pos"][0], d["pos"][1] = (1 << 31) - 1, 0
    check_all(*run_both(d, "TND"))


@pytest.mark.parametrize("layout", ["BNSD", "BSND", "TND"])
def test_padding(layout, cuda_ok):
    """Rows at negative positions: NaN there is not read, outputs are zeros, and the weights'
    gradients do not see them; a batch of nothing but padding has zero gradients."""
    for eps in (EPS, 0.0):
        d = make(layout, 2, 3, 2, 37, 64, BF, seed=4)
        dead = torch.zeros_like(d["pos"], dtype=torch.bool)
        dead[..., 30:] = True
        dead[..., 3] = True
        d["pos"][dead] = -1
        clean = dict(d)
        mask = dead[:, None, :, None] if layout == "BNSD" else dead[..., None, None]
        for n in ("q", "k", "dq", "dk"):
            d[n] = torch.where(mask, torch.full_like(d[n], float("nan")), d[n])
            clean[n] = torch.where(mask, torch.zeros_like(d[n]), d[n])
        got, _ = run_both(d, layout, eps=eps)
        _, want = run_both(clean, layout, eps=max(eps, 1e-30))
        check_all(got, want)
        for n in ("q", "k", "dq", "dk"):
            assert torch.count_nonzero(torch.where(mask, got[n], torch.zeros_like(got[n]))) == 0
        d["pos"].fill_(-5)
        got, _ = run_both(d, layout, eps=eps)
        assert all(torch.count_nonzero(t) == 0 for t in got.values())


def test_rows_of_zeros_and_of_large_values(cuda_ok):
    d = make("BSND", 1, 2, 2, 20, 128, BF, seed=5)
    d["q"][:, 3] = 0
    d["k"][:, 4] = 3e4
    d["k"][:, 5] = 1e-20
    check_all(*run_both(d, "BSND"))


@pytest.mark.parametrize("layout", ["BSND", "TND"])
def test_slices_of_a_fused_projection(layout, cuda_ok):
    D, Nq, Nk, S = 128, 6, 2, 50
    d = make(layout, 2, Nq, Nk, S, D, BF, seed=6)
    qkv = torch.cat([d["q"], d["k"], d["k"]], -2)
    d["q"], d["k"] = qkv[..., :Nq, :], qkv[..., Nq:Nq + Nk, :]
    dqkv = torch.cat([d["dk"], d["dq"], d["dk"]], -2)
    d["dq"], d["dk"] = dqkv[..., Nk:Nk + Nq, :], dqkv[..., Nk + Nq:, :]
    got, want = run_both(d, layout)
    check_all(got, want)
    dense = {n: t.contiguous() for n, t in d.items()}
    same, _ = run_both(dense, layout)
    assert all(torch.equal(got[n], same[n]) for n in got)
    assert got["q"].is_contiguous() and got["k"].is_contiguous()
    # one key head read by all: a broadcast input
    d["k"] = d["k"][..., :1, :].expand(d["k"].shape)
    check_all(*run_both(d, layout))


def test_in_place(cuda_ok):
    d = make("TND", 1, 4, 2, 70, 64, BF, seed=7)
    got, _ = run_both(d, "TND")
    q, k, dq, dk = (d[n].clone() for n in ("q", "k", "dq", "dk"))
    a = (d["pos"], d["inv"], d["qw"], d["kw"], EPS, "TND")
    back = kda.qk_norm_rope_backward(dq, dk, q, k, *a, dq=dq, dk=dk)
    assert torch.equal(dq, got["dq"]) and torch.equal(dk, got["dk"])
    assert torch.equal(back[2], got["dqw"]) and torch.equal(back[3], got["dkw"])
    o = kda.qk_norm_rope(q, k, *a, q_out=q, k_out=k)
    assert o[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, got["q"]) and torch.equal(k, got["k"])


def test_many_tokens(cuda_ok):
    """More tokens than the backward pass has blocks for: every block takes several."""
    d = make("TND", 1, 2, 1, 20011, 64, FP, seed=8)
    check_all(*run_both(d, "TND"))


def test_same_bits_on_every_run(cuda_ok):
    d = make("BNSD", 2, 8, 2, 700, 128, BF, seed=9)
    runs = [run_both(d, "BNSD")[0] for _ in range(2)]
    assert all(torch.equal(runs[0][n], runs[1][n]) for n in runs[0])


def test_streams_and_graphs(cuda_ok):
    """Two captured passes replayed side by side, after new inputs were copied in."""
    d = make("BSND", 2, 4, 2, 300, 128, BF, seed=10)

    def step():
        a = inputs(d) + (EPS, "BSND")
        return kda.qk_norm_rope(*a) + kda.qk_norm_rope_backward(d["dq"], d["dk"], *a)

    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    q, k = kda.qk_norm_rope(*inputs(d), EPS, "BSND", stream=other)
    other.synchronize()
    eager = step()
    assert torch.equal(q, eager[0]) and torch.equal(k, eager[1])
    graphs, results = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(step())
        graphs.append(graph)
    new = make("BSND", 2, 4, 2, 300, 128, BF, seed=11)
    for n in ("q", "k", "dq", "dk", "pos"):
        d[n].copy_(new[n])
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    for graph, s in zip(graphs, (other, torch.cuda.Stream())):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(want, r))


def test_autograd(cuda_ok):
    d = make("BSND", 2, 3, 2, 30, 64, FP, seed=12)
    got, _ = run_both(d, "BSND", True)
    ts = [d[n].clone().requires_grad_() for n in ("q", "k", "qw", "kw")]
    q, k = kda.qk_norm_rope(ts[0], ts[1], d["pos"], d["inv"], ts[2], ts[3], EPS, "BSND",
                            interleaved=True)
    torch.autograd.backward([q, k], [d["dq"], d["dk"]])
    for t, n in zip(ts, ("dq", "dk", "dqw", "dkw")):
        assert torch.equal(t.grad, got[n]), n
    # k unused, a gradient of stride 0, slices of one leaf
    qkv = torch.cat([d["q"], d["k"]], -2).requires_grad_()
    q, _ = kda.qk_norm_rope(qkv[..., :3, :], qkv[..., 3:, :], d["pos"], d["inv"], None, None, EPS,
                            "BSND")
    q.sum().backward()
    want = R.qk_side(d["q"], None, d["pos"], d["inv"], EPS, "BSND", False,
                     torch.ones_like(d["q"]))
    R.check(qkv.grad[..., :3, :], want["dx"], "dq")
    assert torch.count_nonzero(qkv.grad[..., 3:, :]) == 0


def test_gradients_against_differences(cuda_ok):
    """Along a direction, against central differences of the definition in fp64: the step 1e-4 is off
    by 1e-8 relative, far below the kernel's own bound."""
    d = make("TND", 1, 2, 2, 25, 64, FP, seed=13)
    got, want = run_both(d, "TND")
    gen = torch.Generator().manual_seed(2)
    for side in ("q", "k"):
        for name, grad in ((side, "d" + side), (side + "w", f"d{side}w")):
            v = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
            loss = []
            for e in (1e-4, -1e-4):
                c = dict(d, **{side: d[side].double(), side + "w": d[side + "w"].double()})
                c[name] = c[name] + e * v.cuda()
                R.HALF.setdefault(torch.float64, 0.0)
                r = R.qk_side(c[side], c[side + "w"], d["pos"], d["inv"], EPS, "TND", False)
                loss.append(float((r["out"][0] * d["d" + side].double().cpu()).sum()))
            diff = (loss[0] - loss[1]) / 2e-4
            mine = float((got[grad].double().cpu() * v).sum())
            bound = float((want[grad][1] * v.abs()).sum())
            scale = float((want[grad][0] * v).abs().sum())
            assert abs(mine - diff) <= bound + 1e-6 * scale, (name, mine, diff, bound)


@pytest.mark.parametrize("bad", ["type", "k_type", "k_shape", "positions", "inv_freq", "weight",
                                 "align", "alias", "overlap", "out_grad", "eps", "layout", "channels"])
def test_refusals(bad, cuda_ok):
    d = make("BSND", 1, 2, 2, 9, 64, BF, seed=14)
    a, layout, eps, kw = list(inputs(d)), "BSND", EPS, {}
    if bad == "type":
        a[0], a[1] = a[0].double(), a[1].double()
    elif bad == "k_type":
        a[1] = a[1].half()
    elif bad == "k_shape":
        a[1] = a[1][:, :-1]
    elif bad == "positions":
        a[2] = a[2].long()
    elif bad == "inv_freq":
        a[3] = a[3][:-1]
    elif bad == "weight":
        a[4] = a[4].bfloat16()
    elif bad == "align":
        a[0] = torch.zeros(a[0].numel() + 1, dtype=BF, device="cuda")[1:].view(a[0].shape)
    elif bad == "alias":
        kw["q_out"] = a[1]
    elif bad == "overlap":
        kw["q_out"] = kw["k_out"] = torch.empty_like(a[0])
    elif bad == "out_grad":
        a[0] = a[0].clone().requires_grad_()
        kw["q_out"] = torch.empty_like(d["q"])
    elif bad == "eps":
        eps = -1.0
    elif bad == "layout":
        layout = "NBSD"
    elif bad == "channels":
        a[0] = a[0].transpose(-1, -2).contiguous().transpose(-1, -2)
    with pytest.raises((TypeError, ValueError, kda.KdaError)):
        kda.qk_norm_rope(*a, eps, layout, **kw)
    torch.cuda.synchronize()


def test_offsets_past_32_bits(cuda_ok):
    """Heads 2^31 elements apart, and outputs of more than 2^31 elements: equal heads give equal bits."""
    D, S = 128, 40
    d = make("BNSD", 1, 2, 2, S, D, BF, seed=15)
    near, _ = run_both(d, "BNSD")
    far = torch.empty((1 << 31) + S * D, dtype=BF, device="cuda")
    wide = torch.as_strided(far, (1, 2, S, D), (0, 1 << 31, D, 1))
    for n in ("q", "k", "dq", "dk"):
        wide.copy_(d[n])
        got, _ = run_both(dict(d, **{n: wide}), "BNSD")
        assert all(torch.equal(got[m], near[m]) for m in got), n
    del far, wide
    d = make("BSND", 1, 1, 1, 131072, D, BF, seed=16)
    q, dq = (d[n].expand(1, 131072, 130, D) for n in ("q", "dq"))
    a = (q, d["k"], d["pos"], d["inv"], d["qw"], d["kw"], EPS, "BSND")
    out, _ = kda.qk_norm_rope(*a)
    assert out.numel() > 1 << 31
    assert torch.equal(out[:, :, :1], out[:, :, -1:])
    grad = kda.qk_norm_rope_backward(dq, d["dk"], *a)[0]
    assert torch.equal(grad[:, :, :1], grad[:, :, -1:])
    one = kda.qk_norm_rope(d["q"], *a[1:])[0]
    assert torch.equal(one, out[:, :, :1])


def test_nan_stays_in_its_row(cuda_ok):
    """A NaN in a row spoils that row (and the weights' gradients of its side), nothing else."""
    d = make("TND", 1, 3, 2, 21, 64, BF, seed=17)
    clean, _ = run_both(d, "TND")
    bad = dict(d, q=d["q"].clone())
    bad["q"][7, 1, 3] = float("nan")
    got, _ = run_both(bad, "TND")
    row = torch.zeros(21, 3, 1, dtype=torch.bool, device="cuda")
    row[7, 1] = True
    for n in ("q", "dq"):
        assert torch.isnan(torch.where(row, got[n], float("nan"))).all()
        assert torch.equal(torch.where(row, 0, got[n]), torch.where(row, 0, clean[n]))
    assert all(torch.equal(got[n], clean[n]) for n in ("k", "dk", "dkw"))


def test_captured_training_step(cuda_ok):
    d = make("TND", 1, 4, 2, 90, 128, FP, seed=18)
    ts = [d[n].clone().requires_grad_() for n in ("q", "k", "qw", "kw")]

    def step():
        out = kda.qk_norm_rope(ts[0], ts[1], d["pos"], d["inv"], ts[2], ts[3], EPS, "TND")
        return torch.autograd.grad(out, ts, [d["dq"], d["dk"]])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    new = make("TND", 1, 4, 2, 90, 128, FP, seed=19)
    with torch.no_grad():
        for t, n in zip(ts, ("q", "k", "qw", "kw")):
            t.copy_(new[n])
        for n in ("dq", "dk", "pos"):
            d[n].copy_(new[n])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, step()))


def test_frequencies_of_every_size(cuda_ok):
    """Very slow and very fast rotations, negative ones and none; a frequency that is not a number
    spoils its own pair alone.  Positions below 2^20 and frequencies below 7: the reference's angle, a
    product in fp64, is off by at most 2^-53 of 7e6, 1e-9, far below the bound."""
    d = make("TND", 1, 2, 1, 48, 64, FP, seed=20)
    d["pos"][:8] = torch.arange(8, dtype=torch.int32)
    d["inv"] = torch.tensor([1e-12, 1e-7, 3.0, 6.2831855, 0.7, -2.5, 0.0, 1.5707964] * 4, device="cuda")
    for interleaved in (False, True):
        check_all(*run_both(d, "TND", interleaved))
    # a turn of 1e-7 keeps its own relative accuracy: x alone, one position
    one = dict(d, q=torch.zeros(1, 1, 64, device="cuda"), pos=torch.ones(1, dtype=torch.int32).cuda())
    one["q"][0, 0, 2] = 8.0
    q, _ = kda.qk_norm_rope(one["q"], one["q"], one["pos"], d["inv"], None, None, 0.0, "TND",
                            interleaved=True)
    assert abs(q[0, 0, 3].item() / (8.0 * 1e-7) - 1) < 1e-6
    d["inv"][5] = float("nan")
    q, _ = kda.qk_norm_rope(*inputs(d), EPS, "TND")
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[5] = bad[37] = True
    assert torch.isnan(q[..., bad]).all() and torch.isfinite(q[..., ~bad]).all()


@pytest.mark.parametrize("layout,B,S", [("TND", 1, 20011), ("BNSD", 3, 6007), ("BSND", 2, 9001)])
def test_in_place_over_many_turns(layout, B, S, cuda_ok):
    """Every block takes several tokens, with the next ones' rows under way while it writes."""
    d = make(layout, B, 3, 2, S, 64, BF, seed=21)
    a = (d["pos"], d["inv"], d["qw"], d["kw"], EPS, layout)
    want = kda.qk_norm_rope(d["q"], d["k"], *a)
    back = kda.qk_norm_rope_backward(d["dq"], d["dk"], d["q"], d["k"], *a)
    dq, dk = d["dq"].clone(), d["dk"].clone()
    mine = kda.qk_norm_rope_backward(dq, dk, d["q"], d["k"], *a, dq=dq, dk=dk)
    assert mine[0].data_ptr() == dq.data_ptr() and mine[1].data_ptr() == dk.data_ptr()
    assert all(torch.equal(p, q) for p, q in zip(mine, back))
    q, k = d["q"].clone(), d["k"].clone()
    kda.qk_norm_rope(q, k, *a, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
