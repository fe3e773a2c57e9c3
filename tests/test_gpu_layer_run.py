"""The operators as a layer runs them: a gated moving average on the values, norm and rotation of
queries and keys, then the KDA prefill; then single tokens through the step forms and the decode
step.  Also a training step of the differentiable part."""
import numpy as np
import pytest
import torch

import chunked_kda_prefill_b200 as kda
import layer_refs as R
import oracle
from kda_gpu import compare

pytestmark = pytest.mark.gpu

B, NQK, NV, D, LB, EPS = 2, 2, 4, 128, -5.0, 1e-6
SCALE = D ** -0.5


def params(seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    half = D // 2
    return {"A1": rnd(NV), "b1": rnd(NV, D), "A2": rnd(NV), "b2": rnd(NV, D),
            "qw": 1 + 0.1 * rnd(D), "kw": 1 + 0.1 * rnd(D),
            "inv": (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()}


def tokens(S, seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen).bfloat16().cuda()  # noqa: E731
    return {"q": rnd(B, S, NQK, D), "k": rnd(B, S, NQK, D), "v": rnd(B, S, NV, D),
            "g1": rnd(B, S, NV, D), "w1": rnd(B, S, NV), "g2": rnd(B, S, NV, D),
            "w2": rnd(B, S, NV)}


def prefill(t, p, h0, S0, start=0):
    S = t["q"].shape[1]
    pos = (start + torch.arange(S, dtype=torch.int32, device="cuda")).expand(B, S).contiguous()
    v, h = kda.gated_recurrence(t["v"], t["g1"], t["w1"], h0, p["A1"], p["b1"], LB, "BSND",
                                kda.recurrence_plan(t["v"], "BSND"))
    q, k = kda.qk_norm_rope(t["q"], t["k"], pos, p["inv"], p["qw"], p["kw"], EPS, "BSND")
    o, state = kda.flash_kda(q, k, v, t["g2"], t["w2"], SCALE, S0, p["A2"], p["b2"], LB, "BSND",
                             kda.plan(q, v, S0, "BSND"))
    return o, h, state, (q, k, v)


def test_prefill_then_tokens(cuda_ok):
    """A prefill over L tokens and T steps give what a prefill over L + T tokens gives, and both
    match the oracle on the operators' own outputs."""
    L, T = 150, 4
    p, t = params(1), tokens(L + T, 2)
    h0 = torch.randn(B, NV, D, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    whole, h_whole, s_whole, (q, k, v) = prefill(t, p, h0, None)
    o, h, state, _ = prefill({n: x[:, :L].contiguous() for n, x in t.items()}, p, h0, None)
    outs = []
    for i in range(L, L + T):
        one = {n: x[:, i].contiguous() for n, x in t.items()}
        v1, h = kda.gated_recurrence_step(one["v"], one["g1"], one["w1"], h, p["A1"], p["b1"], LB,
                                          state_out=h)
        pos = torch.full((B,), i, dtype=torch.int32, device="cuda")
        q1, k1 = kda.qk_norm_rope(one["q"], one["k"], pos, p["inv"], p["qw"], p["kw"], EPS, "TND")
        o1, state = kda.decode(q1, k1, v1, one["g2"], one["w2"], SCALE, state, p["A2"], p["b2"], LB,
                               state_out=state)
        outs.append(o1)
    torch.cuda.synchronize()
    got = torch.cat([o, torch.stack(outs, 1)], 1)
    compare(got.float().cpu().numpy(), whole.float().cpu().numpy(), "out")
    compare(state.cpu().numpy(), s_whole.cpu().numpy(), "state")
    want = R.recurrence(t["v"], t["g1"], t["w1"], h0, p["A1"], p["b1"], LB, "BSND", [L + T] * B)
    R.check(h, want["final"], "recurrence state after steps")
    R.check(h_whole, want["final"], "recurrence state")
    bits = lambda x: x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    inp = {"q": bits(q), "k": bits(k), "v": bits(v), "g": bits(t["g2"]), "beta": bits(t["w2"]),
           "A_log": p["A2"].cpu().numpy(), "dt_bias": p["b2"].cpu().numpy(),
           "initial_state": np.zeros((B, NV, D, D), np.float32)}
    ref, ref_state, _ = oracle.flash_kda(inp, "BSND", B, NQK, NV, L + T, D, SCALE, LB, None)
    compare(whole.float().cpu().numpy(), ref, "out against the oracle")
    compare(s_whole.cpu().numpy(), ref_state, "state against the oracle")


def test_training_step(cuda_ok):
    """Gradients of a loss on the recurrence and on the rotated heads, packed with a fused
    projection's slices as leaves; a second step on updated weights runs on the same plan."""
    lengths = [37, 1, 90]
    S = sum(lengths)
    gen = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    fused = rnd(S, 2 * NQK + 2 * NV, D).requires_grad_()
    beta = rnd(S, NV).requires_grad_()
    p = params(5)
    weights = [p[n].requires_grad_() for n in ("A1", "b1", "qw", "kw")]
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lengths]).cuda()
    plan = None
    cu = np.concatenate([[0], np.cumsum(lengths)])
    for _ in range(2):
        q, k, x, g = fused.split([NQK, NQK, NV, NV], 1)
        plan = plan or kda.recurrence_plan(x, "TND", cu_seqlens=cu)
        out, final = kda.gated_recurrence(x, g, beta, None, weights[0], weights[1], LB, "TND", plan)
        qo, ko = kda.qk_norm_rope(q, k, pos, p["inv"], weights[2], weights[3], EPS, "TND")
        loss = (out ** 2).sum() + final.sum() + (qo * ko).sum()
        grads = torch.autograd.grad(loss, [fused, beta] + weights)
        want = R.recurrence(x, g, beta, None, weights[0], weights[1], LB, "TND", lengths,
                            2 * out.detach(), torch.ones_like(final))
        R.check(grads[0][:, 2 * NQK:2 * NQK + NV], want["dx"], "dx")
        R.check(grads[0][:, 2 * NQK + NV:], want["dg"], "dg")
        R.check(grads[1], want["dbeta"], "dbeta")
        R.check(grads[2], want["dA_log"], "dA_log")
        R.check(grads[3], want["ddt_bias"], "ddt_bias")
        for i, (a, b, w, name) in enumerate(((q, ko, weights[2], "q"), (k, qo, weights[3], "k"))):
            side = R.qk_side(a, w, pos, p["inv"], EPS, "TND", False, b)
            R.check(grads[0][:, i * NQK:(i + 1) * NQK], side["dx"], "d" + name)
            R.check(grads[4 + i], side["dw"], f"d{name}w")
        with torch.no_grad():
            for w, gr in zip([fused, beta] + weights, grads):
                w -= 1e-3 * gr
