"""fp64 references of the gated recurrence and of the q/k norm with rotation, token by token and
head by head from the definitions, each with a bound on what fp32 arithmetic may add.

The bounds are first-order running error bounds in units of u = 2^-24, half a step of fp32.  A
result that is rounded to its type adds half a step of that type, eps/2 of the value.

Recurrence.  In h_t = a_t h_{t-1} + b_t x_t the decay a = 2^(l sigmoid(z)) comes out with a relative
error of at most (8 |lower_bound| + 6) u: z comes out with 8 u relatively (4 u of exp(A_log) and
four roundings), which moves sigmoid(z) by at most 8 u |z| sigmoid'(z) <= 2 u absolutely, the power
of two inside it is off by 4 u and the reciprocal by 2 u, which bounds the sigmoid's error by 8 u; the exponent multiplies that by |lower_bound|; its own power of
two adds 4 u and the scaling 2 u.  b = sigmoid(beta) is off by at most 4 u, the product b x and the
sum by 1 u each, and joining a tile's part to what came before it repeats the product and the sum
(4 u).  So with C = 8 |lower_bound| + 16 and the magnitude M_t = a_t M_{t-1} + b_t |x_t|, the error
obeys E_t = a_t E_{t-1} + C u M_t.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}


def rows(t, layout, b, lo, n):
    """[n, N, ...] of sequence b: tokens lo.. of its slot, or of the packed rows."""
    if layout == "TND":
        return t[lo:lo + n]
    return t[b, lo:lo + n] if layout == "BSND" else t[b, :, lo:lo + n].transpose(0, 1)


def spans(layout, lengths):
    at = 0
    for b, n in enumerate(lengths):
        yield b, (at if layout == "TND" else 0), n
        at += n


def _sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def recurrence(x, g, beta, h0, A_log, dt_bias, lb, layout, lengths, dout=None, dfinal=None):
    """Forward, and backward when dout or dfinal is given: {name: (value, bound of the fp32 error)}
    in fp64 on the CPU; rows past a valid length are zeros with bound zero."""
    cpu = lambda t: None if t is None else t.detach().double().cpu()  # noqa: E731
    kind = x.dtype
    x, g, beta, h0, A_log, dt_bias, dout, dfinal = map(
        cpu, (x, g, beta, h0, A_log, dt_bias, dout, dfinal))
    B, (N, D), C = len(lengths), dt_bias.shape, 8 * abs(lb) + 16
    backward = dout is not None or dfinal is not None
    zero = lambda t: (torch.zeros_like(t), torch.zeros_like(t))  # noqa: E731
    res = {"out": zero(x), "final": (torch.zeros(B, N, D, dtype=torch.float64),
                                     torch.zeros(B, N, D, dtype=torch.float64))}
    if backward:
        res |= {"dx": zero(x), "dg": zero(g), "dbeta": zero(beta), "dA_log": zero(A_log),
                "ddt_bias": zero(dt_bias),
                "dh0": (torch.zeros(B, N, D, dtype=torch.float64),
                        torch.zeros(B, N, D, dtype=torch.float64))}
    ea = torch.exp(A_log)[:, None]
    for b, lo, n in spans(layout, lengths):
        pick = lambda t: rows(t, layout, b, lo, n)  # noqa: E731
        xs, raw, w = pick(x), pick(g) + dt_bias, _sigmoid(pick(beta))[..., None]
        s = _sigmoid(ea * raw)
        a = torch.exp(lb * s)
        h = h0[b] if h0 is not None else torch.zeros(N, D, dtype=torch.float64)
        M, E = h.abs(), torch.zeros_like(h)
        hs, Es = [h], [E]
        for t in range(n):
            h = a[t] * h + w[t] * xs[t]
            M = a[t] * M + w[t] * xs[t].abs()
            E = a[t] * E + C * U * M
            hs.append(h)
            Es.append(E)
        pick(res["out"][0])[:] = torch.stack(hs[1:])
        pick(res["out"][1])[:] = torch.stack(Es[1:])
        res["final"][0][b], res["final"][1][b] = h, E
        if not backward:
            continue
        lam = torch.zeros(n, N, D, dtype=torch.float64) if dout is None else pick(dout).clone()
        M = lam.abs()  # of the terms: a map's product and sum round each before they may cancel
        if dfinal is not None:
            lam[n - 1] += dfinal[b]
            M[n - 1] += dfinal[b].abs()
        E = torch.zeros_like(lam)
        E[n - 1] = U * M[n - 1]
        for t in range(n - 2, -1, -1):
            lam[t] += a[t + 1] * lam[t + 1]
            M[t] += a[t + 1] * M[t + 1]
            E[t] = a[t + 1] * E[t + 1] + C * U * M[t]
        H, EH = torch.stack(hs[:-1]), torch.stack(Es[:-1])
        pick(res["dx"][0])[:] = w * lam
        pick(res["dx"][1])[:] = w * (E + 6 * U * lam.abs())
        slope = w * _sigmoid(-pick(beta))[..., None]  # 1 - w would cancel
        pick(res["dbeta"][0])[:] = ((lam * xs).sum(-1, keepdim=True) * slope)[..., 0]
        # D products are summed: at most D roundings on top of the terms' own, and the slope's 10
        pick(res["dbeta"][1])[:] = (((E + (D + 10) * U * lam.abs()) * xs.abs()).sum(-1, keepdim=True)
                                    * slope)[..., 0]
        f = a * abs(lb) * s * _sigmoid(-ea * raw) * ea
        dg = -lam * H * f if lb else torch.zeros_like(lam)
        # the factor: a (C u), exp(A_log) (4 u), the products (6 u), and sigmoid (1 - sigmoid): 8 u for
        # each of the two and, since its logarithm's slope in z is 1 - 2 sigmoid, at most one, the
        # 8 u |z| by which z is off (for |z| = 30 more than everything else)
        Eg = (f * (E * H.abs() + lam.abs() * EH)
              + (C + 26 + 8 * (ea * raw).abs()) * U * dg.abs())
        pick(res["dg"][0])[:] = dg
        pick(res["dg"][1])[:] = Eg
        # sums over tokens: the terms' bounds, and the roundings on a term's way: 16 tokens in order
        # at the most, one for each tile of at least 8 tokens, 4 channels and 32 lanes
        K = 64 + n // 8
        res["ddt_bias"][0].add_(dg.sum(0))
        res["ddt_bias"][1].add_((Eg + K * U * dg.abs()).sum(0))
        res["dA_log"][0].add_((dg * raw).sum((0, 2)))
        res["dA_log"][1].add_(((Eg + (K + 2) * U * dg.abs()) * raw.abs()).sum((0, 2)))
        res["dh0"][0][b] = a[0] * lam[0]
        res["dh0"][1][b] = a[0] * (E[0] + C * U * M[0])
    for name in ("out", "dx", "dg", "dbeta"):
        if name in res:
            v, e = res[name]
            res[name] = (v, e + HALF[kind] * v.abs() + tiny(kind))
    for name in ("final", "dh0", "ddt_bias", "dA_log"):
        if name in res:
            v, e = res[name]
            res[name] = (v, e + U * v.abs() + tiny(torch.float32))
    return res


def tiny(kind):
    """Half a step below the normal range (fp16 gets there; the approximate powers flush)."""
    return torch.finfo(kind).smallest_normal * (1 if kind == torch.float32 else torch.finfo(kind).eps)


def qk_side(x, w, positions, inv_freq, eps, layout, interleaved, dy=None):
    """One side (queries or keys): {name: (value, bound)}.

    fp32: the sum of squares is off by at most (D + 2) u relatively, half of which enters r, with 2 u
    for the reciprocal root; the two products of n add 2 u, the cosine and sine are off by 4 u of 1
    (phase and evaluation) and the turn adds 2 u: (D/2 + 16) u of the pair's magnitude.
    """
    kind = x.dtype
    x, dy = x.detach().double().cpu(), None if dy is None else dy.detach().double().cpu()
    D = x.shape[-1]
    w = torch.ones(D, dtype=torch.float64) if w is None else w.detach().double().cpu()
    if positions is None:
        S = x.shape[2] if layout == "BNSD" else x.shape[-3]
        shape = (S,) if layout == "TND" else (x.shape[0], S)
        positions = torch.arange(S).expand(shape)
    positions = positions.detach().cpu()
    half = 0 if inv_freq is None else inv_freq.numel()
    angle = positions.double()[..., None] * (
        torch.zeros(0, dtype=torch.float64) if half == 0 else inv_freq.detach().double().cpu())
    heads = 1 if layout == "BNSD" else -2
    cos, sin = angle.cos().unsqueeze(heads), angle.sin().unsqueeze(heads)
    live = (positions >= 0)[..., None].unsqueeze(heads)
    i = torch.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)

    def rotate(n, sign):
        o = n.clone()
        o[..., one] = n[..., one] * cos - sign * n[..., two] * sin
        o[..., two] = sign * n[..., one] * sin + n[..., two] * cos
        return o

    def reach(n):  # the magnitude that a channel's pair can turn into it
        o = n.abs().clone()
        o[..., one] = o[..., two] = (n[..., one] ** 2 + n[..., two] ** 2).sqrt() * 2 ** 0.5
        return o

    x = torch.where(live, x, torch.zeros((), dtype=torch.float64))
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r * w
    K = (D / 2 + 16) * U
    zero = torch.zeros((), dtype=torch.float64)
    out = torch.where(live, rotate(n, 1), zero)
    res = {"out": (out, K * reach(n) + HALF[kind] * out.abs() + tiny(kind))}
    if dy is not None:
        dy = torch.where(live, dy, zero)
        dn = rotate(dy, -1)
        xh = x * r
        e = dn * w
        m = (e * xh).mean(-1, keepdim=True)
        dx = torch.where(live, r * (e - xh * m), zero)
        size = reach(dy) * w.abs()
        mm = (size * xh.abs()).mean(-1, keepdim=True)
        # as above for each factor, and D + 4 roundings in the mean of the products
        bound = r * (2 * K * size + (2 * D + 32) * U * xh.abs() * mm)
        res["dx"] = (dx, torch.where(live, bound, zero) + HALF[kind] * dx.abs() + tiny(kind))
        terms = torch.where(live, dn * xh, zero).flatten(0, -2)
        sizes = torch.where(live, reach(dy) * xh.abs(), zero).flatten(0, -2)
        # rows are summed a few hundred in order at most, then block by block
        count = min(terms.shape[0], 1024) + 64
        dw = terms.sum(0)
        res["dw"] = (dw, (2 * K + count * U) * sizes.sum(0) + U * dw.abs())
    return res


def check(got, want, what):
    """|got - value| <= bound, everywhere."""
    value, bound = want
    got = got.detach().double().cpu()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    over = (got - value).abs() - bound
    worst = over.max().item() if over.numel() else 0.0
    at = int(over.argmax()) if over.numel() else 0
    assert worst <= 0, (f"{what}: {float(got.flatten()[at])} against {float(value.flatten()[at])}, "
                        f"bound {float(bound.flatten()[at])}, {int((over > 0).sum())} of "
                        f"{over.numel()} outside")
