"""What surrounds the chunked KDA prefill and its decode step in a layer: the gated linear recurrence
(the vector form of the KDA state, on the same gate and write logits) and the norm and rotation of
queries and keys, each as plain torch operations and as this package's kernels.

Gated recurrence, for every sequence, head n and channel d (h_0 is the initial state):

    a_t = exp(lower_bound * sigmoid(exp(A_log[n]) * (g_t + dt_bias[n, d])))
    h_t = a_t * h_{t-1} + sigmoid(beta_t[n]) * x_t

Queries and keys, for every token and head, with r = 1 / sqrt(mean(x^2) + eps):

    n = x * r * weight,    out = rotation of n's first 2 * len(inv_freq) channels by position * inv_freq

A token whose position is negative is padding: its row of the output is zero and it takes no part.
"""
import math

import numpy as np
import torch

own = False

KINDS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------------------------
# cases

def listed():
    packed = "10599,7936,6369,3362,3836,512,938,206,2183,10132,8091,11372"
    short = "1,2,63,64,65,127,128,129,3,700,1,31,33,257,900,16,255,1330"
    return [
        # one long prompt through three heads: few rows to spread over the machine
        _scan("scan_single_bnsd_1x3x8192", "BNSD", "8192", 3, 8192, 128, "bf16", -5.0, False),
        # two slots of unequal length in the token-major layout, a start state: a ragged prefill
        _scan("scan_tail_bsnd_2x16x4000", "BSND", "4000,2777", 16, 4000, 128, "bf16", -2.0, False),
        # the largest prefill: four prompts of 16384 tokens, 32 heads
        _scan("scan_large_bnsd_4x32x16384", "BNSD", ",".join(["16384"] * 4), 32, 16384, 128, "bf16", -5.0, False),
        # a training step on a packed batch of twelve documents
        _scan("scan_train_packed_tnd_65536x32", "TND", packed, 32, 65536, 128, "bf16", -5.0, True),
        # a training step at head dim 64 in half precision, full slots
        _scan("scan_train_headdim64_bnsd_8x32x4096", "BNSD", ",".join(["4096"] * 8), 32, 4096, 64, "fp16", -5.0, True),
        # a training step in 32 bits on many short documents of odd lengths, an odd number of heads
        _scan("scan_train_short_tnd_fp32", "TND", short, 5, sum(int(v) for v in short.split(",")), 128, "fp32", -0.5, True),
        # one token for each of 256 sequences: a decode batch; and for a single sequence: latency
        {"name": "step_256x32x128", "op": "step", "B": 256, "N": 32, "D": 128, "type": "bf16", "bound": -5.0},
        {"name": "step_1x32x128", "op": "step", "B": 1, "N": 32, "D": 128, "type": "bf16", "bound": -5.0},
        # queries and keys of the largest prefill
        _qk("qk_large_bnsd_4x32x16384", "BNSD", 4, 32, 32, 16384, 128, 128, "bf16", False, False, 0, False),
        # a training step on slices of a fused projection, packed documents, shared key heads
        _qk("qk_train_fused_tnd_65536x32x8", "TND", 1, 32, 8, 65536, 128, 128, "bf16", True, False, 0, True),
        # a training step in half precision, head dim 64, half of the channels turned, pairs side by side, padded slots
        _qk("qk_train_odd_bsnd_3x1777", "BSND", 3, 6, 3, 1777, 64, 32, "fp16", True, True, 200, True),
        # one token for each of 64 sequences, far into their contexts, from a fused projection: a decode batch
        _qk("qk_step_tnd_64x32x8", "TND", 1, 32, 8, 64, 128, 128, "bf16", True, False, 0, False),
    ]


def _scan(name, layout, lengths, N, S, D, kind, bound, train):
    c = {"op": "scan", "layout": layout, "lengths": lengths, "N": N, "S": S, "D": D, "type": kind, "bound": bound, "train": train}
    return {"name": name, **c} if name else c


def _qk(name, layout, B, Nq, Nk, S, D, turned, kind, fused, interleaved, padded, train):
    c = {"op": "qk", "layout": layout, "B": B, "Nq": Nq, "Nk": Nk, "S": S, "D": D, "turned": turned, "type": kind, "fused": fused,
         "interleaved": interleaved, "padded": padded, "train": train}
    return {"name": name, **c} if name else c


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], evenly over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.5 / hi))))


def draw(rng):
    op = rng.choice(("scan", "scan", "scan", "step", "qk", "qk"))
    D, kind = rng.choice((64, 128)), rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op == "step":
        return {"op": op, "B": _spread(rng, 1, 256), "N": _spread(rng, 1, 64), "D": D, "type": kind, "bound": rng.choice((-5.0, -2.0, -0.25))}
    layout, train = rng.choice(("BNSD", "BSND", "TND")), rng.random() < 0.5
    most = (1 << 27) if kind != "fp32" or not train else (1 << 26)  # values of one tensor
    if op == "scan":
        N = _spread(rng, 1, 32)
        total = _spread(rng, 1, max(1, min(65536, most // (N * D))))
        parts = _spread(rng, 1, min(total, 64))
        if layout == "TND":
            cuts = sorted(rng.sample(range(1, total), parts - 1)) if parts > 1 else []
            lengths = [b - a for a, b in zip([0] + cuts, cuts + [total])]
            S = total
        else:
            parts = min(parts, 8)
            S = min(16384, -(-total // parts))
            lengths = [S if rng.random() < 0.5 else _spread(rng, 1, S) for _ in range(parts)]
        return _scan(None, layout, ",".join(str(v) for v in lengths), N, S, D, kind, rng.choice((-5.0, -2.0, -0.25)), train)
    B = 1 if layout == "TND" else _spread(rng, 1, 8)
    Nk = _spread(rng, 1, 16)
    Nq = Nk * rng.choice((1, 2, 4))
    S = _spread(rng, 1, max(1, min(65536, most // (B * (Nq + Nk) * D))))
    turned = rng.choice((D, D, D // 2, D // 4, 0))
    fused = layout != "BNSD" and rng.random() < 0.5
    padded = rng.choice((0, 0, _spread(rng, 1, S)))
    return _qk(None, layout, B, Nq, Nk, S, D, turned, kind, fused, rng.random() < 0.4, padded if padded < S else 0, train)


# ---------------------------------------------------------------------------------------------
# inputs

def _lengths(case):
    return [int(v) for v in case["lengths"].split(",")]


def _shapes(case):
    """(x's shape, beta's shape) of a scan case."""
    B, N, S, D = len(_lengths(case)), case["N"], case["S"], case["D"]
    x = {"BNSD": (B, N, S, D), "BSND": (B, S, N, D), "TND": (S, N, D)}[case["layout"]]
    return x, x[:-1]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    kind = KINDS[case["type"]]

    def normal(shape, dtype=torch.float32, std=1.0):
        t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return (t if std == 1.0 else t.mul_(std)).to(dtype)

    if case["op"] == "qk":
        return _prepare_qk(case, kind, normal, gen)
    if case["op"] == "step":
        B, N, D = case["B"], case["N"], case["D"]
        return {"case": case, "x": normal((B, N, D), kind), "g": normal((B, N, D), kind), "beta": normal((B, N), kind), "h0": normal((B, N, D)),
                "A_log": normal((N,)), "dt_bias": normal((N, D))}
    shape, heads = _shapes(case)
    B, N, D = len(_lengths(case)), case["N"], case["D"]
    s = {"case": case, "x": normal(shape, kind), "g": normal(shape, kind), "beta": normal(heads, kind), "h0": normal((B, N, D)),
         "A_log": normal((N,)), "dt_bias": normal((N, D)), "lengths": torch.tensor(_lengths(case), device="cuda")}
    if case["train"]:
        s["dout"], s["dfinal"] = normal(shape, kind), normal((B, N, D))
    if own:
        import chunked_kda_prefill_b200 as kda
        cu = np.concatenate([[0], np.cumsum(_lengths(case))]).astype(np.int32)
        s["plan"] = kda.recurrence_plan(s["x"], case["layout"], cu_seqlens=cu)
    return s


def _prepare_qk(case, kind, normal, gen):
    layout, B, Nq, Nk, S, D = (case[k] for k in ("layout", "B", "Nq", "Nk", "S", "D"))
    if case["fused"]:  # q and k are slices of one projection's output that also holds the values
        lead = (S,) if layout == "TND" else (B, S)
        qkv = normal(lead + ((Nq + 2 * Nk) * D,), kind)
        q = qkv[..., :Nq * D].unflatten(-1, (Nq, D))
        k = qkv[..., Nq * D:(Nq + Nk) * D].unflatten(-1, (Nk, D))
    else:
        of = {"BNSD": lambda n: (B, n, S, D), "BSND": lambda n: (B, S, n, D), "TND": lambda n: (S, n, D)}[layout]
        q, k = normal(of(Nq), kind), normal(of(Nk), kind)
    tokens = (S,) if layout == "TND" else (B, S)
    # every row's tokens follow one another from a start somewhere in a long context
    start = torch.randint(0, 1 << 17, tokens[:-1] + (1,), generator=gen, device="cuda", dtype=torch.int32)
    if layout == "TND" and S <= 256:  # single tokens of as many sequences
        positions = torch.randint(0, 1 << 17, tokens, generator=gen, device="cuda", dtype=torch.int32)
    else:
        positions = (start + torch.arange(S, device="cuda", dtype=torch.int32)).expand(tokens).contiguous()
    if case["padded"]:
        positions[..., S - case["padded"]:] = -1
    half = case["turned"] // 2
    inv_freq = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(half, 1))).float()
    s = {"case": case, "q": q, "k": k, "positions": positions, "inv_freq": inv_freq, "qw": 1 + normal((D,), std=0.1), "kw": 1 + normal((D,), std=0.1)}
    if case["train"]:
        s["dq"], s["dk"] = normal(q.shape, kind), normal(k.shape, kind)
    return s


# ---------------------------------------------------------------------------------------------
# one pass

def run(s):
    case = s["case"]
    if case["op"] == "step":
        return _own_step(s) if own else _plain_step(s)
    if case["op"] == "scan":
        return _own_scan(s) if own else _plain_scan(s)
    return _own_qk(s) if own else _plain_qk(s)


def _own_step(s):
    import chunked_kda_prefill_b200 as kda
    out, state = kda.gated_recurrence_step(s["x"], s["g"], s["beta"], s["h0"], s["A_log"], s["dt_bias"], s["case"]["bound"])
    return {"out": out, "state": state}


def _own_scan(s):
    import chunked_kda_prefill_b200 as kda
    c = s["case"]
    inputs = (s["x"], s["g"], s["beta"], s["h0"], s["A_log"], s["dt_bias"], c["bound"], c["layout"], s["plan"])
    if not c["train"]:
        out, final = kda.gated_recurrence(*inputs)
        return {"out": out, "final": final}
    out, final, states = kda.gated_recurrence(*inputs, return_states=True)
    dx, dg, dbeta, dh0, dA_log, ddt_bias = kda.gated_recurrence_backward(s["dout"], s["dfinal"], *inputs, states)
    return {"out": out, "final": final, "dx": dx, "dg": dg, "dbeta": dbeta, "dh0": dh0, "dA_log": dA_log, "ddt_bias": ddt_bias}


def _own_qk(s):
    import chunked_kda_prefill_b200 as kda
    c = s["case"]
    inputs = (s["q"], s["k"], s["positions"], s["inv_freq"], s["qw"], s["kw"], EPS, c["layout"])
    q, k = kda.qk_norm_rope(*inputs, interleaved=c["interleaved"])
    if not c["train"]:
        return {"q": q, "k": k}
    dq, dk, dqw, dkw = kda.qk_norm_rope_backward(s["dq"], s["dk"], *inputs, interleaved=c["interleaved"])
    return {"q": q, "k": k, "dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}


# ---------------------------------------------------------------------------------------------
# the plain forms

def _gate(s, g):
    """(z / exp(A_log), sigmoid(z), a) of raw gates in token-major order [..., N, D]."""
    raw = g.float() + s["dt_bias"]
    sig = torch.sigmoid(torch.exp(s["A_log"])[:, None] * raw)
    return raw, sig, torch.exp(s["case"]["bound"] * sig)


def _plain_step(s):
    _, _, a = _gate(s, s["g"])
    h = a * s["h0"] + torch.sigmoid(s["beta"].float())[..., None] * s["x"].float()
    return {"out": h.to(s["x"].dtype), "state": h}


def _running(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1, from zero: by doubling the reach of every element."""
    reach, T = 1, a.shape[1]
    while reach < T:
        u = torch.cat([u[:, :reach], torch.addcmul(u[:, reach:], a[:, reach:], u[:, :-reach])], 1)
        a = torch.cat([a[:, :reach], a[:, reach:] * a[:, :-reach]], 1)
        reach *= 2
    return u


def _plain_scan(s):
    c = s["case"]
    kind, tnd, bound = s["x"].dtype, c["layout"] == "TND", c["bound"]
    major = {"BNSD": lambda t: t.transpose(1, 2), "BSND": lambda t: t, "TND": lambda t: t[None]}[c["layout"]]
    back = {"BNSD": lambda t: t.transpose(1, 2).contiguous(), "BSND": lambda t: t, "TND": lambda t: t[0]}[c["layout"]]
    L = s["lengths"]
    T = c["S"]
    # the storage row (slot, row) of each sequence's first and last token, and the rows in use
    if tnd:
        ends = torch.cumsum(L, 0)
        first, last, slot = ends - L, ends - 1, torch.zeros_like(L)
        valid = torch.ones((1, T), dtype=torch.bool, device=L.device)
    else:
        first, last, slot = torch.zeros_like(L), L - 1, torch.arange(len(L), device=L.device)
        valid = torch.arange(T, device=L.device) < L[:, None]
    mask = valid[..., None, None]
    x = torch.where(mask, major(s["x"]), 0).float()
    b = torch.sigmoid(torch.where(valid[..., None], major(s["beta"]), 0).float())[..., None]
    raw, sig, a = _gate(s, torch.where(mask, major(s["g"]), 0))
    u = b * x * mask
    a_first = a[slot, first]
    u[slot, first] += a_first * s["h0"]
    keep = a.clone()
    keep[slot, first] = 0  # nothing flows from one sequence into the next
    h = _running(keep, u)
    res = {"out": back((h * mask).to(kind)), "final": h[slot, last]}
    if not c["train"]:
        return res
    # backwards: lam_t = dout_t + a_{t+1} lam_{t+1}
    lam = torch.where(mask, major(s["dout"]), 0).float()
    lam[slot, last] += s["dfinal"]
    ahead = torch.cat([keep[:, 1:], torch.zeros_like(keep[:, :1])], 1)
    lam = _running(ahead.flip(1), lam.flip(1)).flip(1) * mask
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    before[slot, first] = s["h0"]
    dz = lam * before * a * (bound * sig * (1 - sig))
    dg = dz * torch.exp(s["A_log"])[:, None] * mask
    res |= {"dx": back((lam * b).to(kind)), "dg": back(dg.to(kind)), "dbeta": back(((lam * x).sum(-1) * (b * (1 - b))[..., 0]).to(kind)),
            "dh0": lam[slot, first] * a_first, "dA_log": (dg * raw).sum((0, 1, 3), dtype=torch.float64).float(),
            "ddt_bias": dg.sum((0, 1), dtype=torch.float64).float()}
    return res


def _turn(n, cos, sin, interleaved):
    """n's first 2 * cos.shape[-1] channels turned by the angles."""
    half = cos.shape[-1]
    part, rest = n[..., :2 * half], n[..., 2 * half:]
    x, y = part.unflatten(-1, (half, 2)).unbind(-1) if interleaved else (part[..., :half], part[..., half:])
    p, q = x * cos - y * sin, x * sin + y * cos
    part = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([part, rest], -1)


def _plain_qk(s):
    c = s["case"]
    # [B, S] -> one entry for each token, next to the heads
    spread = (lambda t: t[:, None]) if c["layout"] == "BNSD" else (lambda t: t[..., None, :])
    angle = s["positions"].double()[..., None] * s["inv_freq"].double()
    cos, sin = spread(torch.cos(angle).float()), spread(torch.sin(angle).float())
    real = spread((s["positions"] >= 0)[..., None])
    res = {}
    sides = {"q": (s["q"], s["qw"], s.get("dq")), "k": (s["k"], s["kw"], s.get("dk"))}
    res |= {n: _plain_forward(x, w, cos, sin, real, c["interleaved"]) for n, (x, w, _) in sides.items()}
    if c["train"]:
        both = {n: _plain_backward(x, w, dy, cos, sin, real, c["interleaved"]) for n, (x, w, dy) in sides.items()}
        res |= {"dq": both["q"][0], "dqw": both["q"][1], "dk": both["k"][0], "dkw": both["k"][1]}
    return res


def _plain_forward(x, w, cos, sin, real, interleaved):
    f = x.float()
    n = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * w
    return torch.where(real, _turn(n, cos, sin, interleaved), 0).to(x.dtype)


def _plain_backward(x, w, dy, cos, sin, real, interleaved):
    f = x.float()
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    hat = f * r
    dn = torch.where(real, _turn(dy.float(), cos, -sin, interleaved), 0)  # a rotation's gradient turns back
    dhat = dn * w
    dx = r * (dhat - hat * (dhat * hat).mean(-1, keepdim=True))
    dw = torch.where(real, dn * hat, 0).flatten(0, -2).sum(0, dtype=torch.float64)
    return torch.where(real, dx, 0).to(x.dtype), dw.float()


# ---------------------------------------------------------------------------------------------
# the bytes and operations that a pass cannot do without

def work(case):
    size = KINDS[case["type"]].itemsize
    if case["op"] == "step":
        rows, D = case["B"] * case["N"], case["D"]
        return {"bytes": rows * (D * (3 * size + 8) + size) + case["N"] * (D + 1) * 4, "flops": rows * D * 10}
    if case["op"] == "scan":
        L, N, D = _lengths(case), case["N"], case["D"]
        valid = sum(L) * N
        stored = valid if case["layout"] == "TND" else len(L) * case["S"] * N
        state, params = len(L) * N * D * 4, N * (D + 1) * 4
        got = valid * (2 * D + 1) * size + state + params + stored * D * size + state
        if case["train"]:
            got += valid * D * size + 2 * state + stored * (2 * D + 1) * size + params
        return {"bytes": got, "flops": valid * D * (30 if case["train"] else 10)}
    tokens, heads, D = case["B"] * case["S"], case["Nq"] + case["Nk"], case["D"]
    real = case["B"] * (case["S"] - case["padded"])
    got = (real + tokens) * heads * D * size + tokens * 4 + 2 * D * 4
    if case["train"]:
        got += (real + tokens) * heads * D * size + 2 * D * 4
    return {"bytes": got, "flops": real * heads * D * (25 if case["train"] else 8)}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk":
        return _exact_qk(case, s)
    A, bias, low = s["A_log"].double().exp()[:, None], s["dt_bias"].double(), case["bound"]
    if case["op"] == "step":
        decay = torch.exp(low / (1 + torch.exp(-A * (s["g"].double() + bias))))
        h = decay * s["h0"].double() + s["x"].double() / (1 + torch.exp(-s["beta"].double()))[..., None]
        return {"out": h, "state": h}
    shape, heads = _shapes(case)
    names = ["out"] + (["dx", "dg"] if case["train"] else [])
    res = {n: torch.zeros(shape, dtype=torch.float64, device="cuda") for n in names}
    finals = torch.zeros_like(s["h0"], dtype=torch.float64)
    res["final"] = finals
    if case["train"]:
        res["dbeta"] = torch.zeros(heads, dtype=torch.float64, device="cuda")
        res["dh0"] = torch.zeros_like(finals)
        res["dA_log"], res["ddt_bias"] = torch.zeros_like(A[:, 0]), torch.zeros_like(bias)
    begin = 0
    for i, n in enumerate(_lengths(case)):
        # one sequence, token by token: row(t) is its [n, N, ...] part of a tensor
        if case["layout"] == "TND":
            row = lambda t: t[begin:begin + n]
        elif case["layout"] == "BSND":
            row = lambda t: t[i, :n]
        else:
            row = lambda t: t[i, :, :n].transpose(0, 1)
        x, raw = row(s["x"]).double(), row(s["g"]).double() + bias
        write = 1 / (1 + torch.exp(-row(s["beta"]).double()))[..., None]
        sg = 1 / (1 + torch.exp(-A * raw))
        decay = torch.exp(low * sg)
        put = write * x
        h = torch.empty((n + 1,) + tuple(x.shape[1:]), dtype=torch.float64, device="cuda")
        h[0] = s["h0"][i]
        for t in range(n):
            torch.addcmul(put[t], decay[t], h[t], out=h[t + 1])
        row(res["out"]).copy_(h[1:])
        finals[i] = h[n]
        if case["train"]:
            lam = row(s["dout"]).double()
            lam[n - 1] += s["dfinal"][i]
            for t in range(n - 2, -1, -1):
                lam[t].addcmul_(decay[t + 1], lam[t + 1])
            row(res["dx"]).copy_(write * lam)
            row(res["dbeta"]).copy_(((lam * x).sum(-1, keepdim=True) * write * (1 - write))[..., 0])
            dz = lam * h[:-1] * decay * low * sg * (1 - sg)
            row(res["dg"]).copy_(dz * A)
            res["dA_log"] += (dz * A * raw).sum((0, 2))
            res["ddt_bias"] += (dz * A).sum(0)
            res["dh0"][i] = decay[0] * lam[0]
        begin += n
    return res


def _exact_qk(case, s):
    D, half = case["D"], case["turned"] // 2
    # the whole turn as one matrix for each token: [.., D, D] acts on pairs (i, j)
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    angle = s["positions"].double().unsqueeze(-1) * s["inv_freq"].double()
    cos = torch.ones(angle.shape[:-1] + (D,), dtype=torch.float64, device="cuda")
    sin = torch.zeros_like(cos)
    cos[..., first], cos[..., second] = angle.cos(), angle.cos()
    sin[..., first], sin[..., second] = -angle.sin(), angle.sin()
    other = torch.arange(D, device="cuda")
    other[first], other[second] = second, first
    heads = 1 if case["layout"] == "BNSD" else -2
    cos, sin = cos.unsqueeze(heads), sin.unsqueeze(heads)
    live = (s["positions"] >= 0).unsqueeze(-1).unsqueeze(heads)
    res = {}
    for name, x, w in (("q", s["q"], s["qw"]), ("k", s["k"], s["kw"])):
        x, w = x.double(), w.double()
        r = (x.square().sum(-1, keepdim=True) / D + EPS) ** -0.5
        n = x * r * w
        res[name] = torch.where(live, n * cos + n[..., other] * sin, 0.0)
        if case["train"]:
            dy = s["d" + name].double()
            dn = torch.where(live, dy * cos + (dy * sin)[..., other], 0.0)
            res["d%sw" % name] = (dn * x * r).flatten(0, -2).sum(0)
            e = dn * w
            res["d" + name] = torch.where(live, r * e - x * r ** 3 * (e * x).sum(-1, keepdim=True) / D, 0.0)
    return res
