"""The operators around the quantised MoE layer, as cases to measure: the RMS norm with residual and
int8 output, SwiGLU with int8 output, the int8 product with scales per token and channel, and the
selection of experts with groups.

Sizes: hidden 6144, 2048 and 7168, FFN 2048, 256 and 64 experts with top-8 are this repository's
layer shapes; the dense FFN is 12288 wide (two hidden widths), the token counts run from one decode
step to a prefill of 4096 (its two prompt halves and odd remainders among them).
"""
import math

import torch

own = False

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6
DTYPES = {"f32": F32, "bf16": BF16}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _norm(name, T, H, x, res, codes, pad=0):
    return {"name": name, "op": "norm", "T": T, "H": H, "x": x, "res": res, "codes": codes, "pad": pad}


def _swiglu(name, T, F, x, pad=0):
    return {"name": name, "op": "swiglu", "T": T, "F": F, "x": x, "pad": pad}


def _linear(name, T, N, K, out, bias, pad=0):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "out": out, "bias": bias, "pad": pad}


def _route(name, T, E, k, score, groups, keep, best, bias, renorm, x):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "groups": groups,
            "keep": keep, "best": best, "bias": bias, "renorm": renorm, "x": x}


def listed():
    return [
        # one decoded token in front of an MoE layer: the new residual and the layer's bf16 input
        _norm("norm_moe_1x6144", 1, 6144, "bf16", "bf16", False),
        # a prefill of 4096 tokens in front of an int8 product: the new residual, codes and scales
        _norm("norm_codes_4096x6144", 4096, 6144, "bf16", "bf16", True),
        # an odd remainder of a prompt after an MoE layer with fp32 output, fp32 residual stream, rows of
        # an odd width inside wider ones
        _norm("norm_codes_333x7001_f32", 333, 7001, "f32", "f32", True, 3),
        # one decoded token between the products of a dense FFN
        _swiglu("swiglu_1x12288", 1, 12288, "bf16"),
        # the same for a prefill of 4096 tokens
        _swiglu("swiglu_4096x12288", 4096, 12288, "bf16"),
        # one decoded token, a square projection: a stream of weights
        _linear("linear_1x6144x6144", 1, 6144, 6144, "bf16", False),
        # a batch of 24 decoding sequences, gate and up of the dense FFN in one product
        _linear("linear_24x24576x6144", 24, 24576, 6144, "bf16", False),
        # an odd remainder of a prompt through an odd-sized head with bias, fp32 output
        _linear("linear_333x5003x2048_f32", 333, 5003, 2048, "f32", True),
        # a prefill of 4096 tokens, gate and up of the dense FFN in one product
        _linear("linear_4096x24576x6144", 4096, 24576, 6144, "bf16", False),
        # a batch of 16 decoding sequences: sigmoid, bias, 8 groups of which 4 stay, renormalised
        _route("route_groups_16x256", 16, 256, 8, "sigmoid", 8, 4, 2, True, True, "f32"),
        # a prefill of 4096 tokens, the same routing
        _route("route_groups_4096x256", 4096, 256, 8, "sigmoid", 8, 4, 2, True, True, "f32"),
        # a prefill of 1000 tokens through a softmax router of 64 experts on bf16 logits, with their many
        # equal values, the probabilities as they are
        _route("route_softmax_1000x64_bf16", 1000, 64, 8, "softmax", 1, 1, 1, False, False, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Half of the widths are multiples of 64, a quarter of 8, a quarter any number (3072, which no
    layer here has, is left out)."""
    n = _log(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    n = max(lo, n - n % step)
    return n if n != 3072 else n + step


def draw(rng):
    op = rng.choice(("norm", "swiglu", "linear", "linear", "route"))
    if op == "norm":
        H = _width(rng, 256, 12288)
        T = min(_log(rng, 1, 8192), 4096 * 6144 // H)
        return {"op": op, "T": T, "H": H, "x": rng.choice(("bf16", "f32")), "res": rng.choice(("bf16", "f32", "none")),
                "codes": rng.random() < 0.5, "pad": rng.choice((0, 0, 8, 3))}
    if op == "swiglu":
        F = _width(rng, 256, 18432)
        T = min(_log(rng, 1, 8192), 4096 * 12288 // F)
        return {"op": op, "T": T, "F": F, "x": rng.choice(("bf16", "bf16", "f32")), "pad": rng.choice((0, 0, 8, 3))}
    if op == "linear":
        N, K = _width(rng, 64, 24576), _width(rng, 64, 12288)
        T = max(1, min(_log(rng, 1, 4096), 4096 * 24576 * 6144 // (N * K)))
        return {"op": op, "T": T, "N": N, "K": K, "out": rng.choice(("bf16", "f32")), "bias": rng.random() < 0.3,
                "pad": rng.choice((0, 0, 16, 3))}
    groups = rng.choice((1, 1, 2, 4, 5, 8))
    E = groups * max(4, _log(rng, 8, 512) // groups)
    keep = rng.randint((groups + 1) // 2, groups)
    k = rng.randint(1, min(16, keep * (E // groups)))
    score = rng.choice(("sigmoid", "softmax"))
    return {"op": op, "T": min(_log(rng, 1, 16384), 4096 * 512 // E), "E": E, "k": k, "score": score, "groups": groups, "keep": keep,
            "best": rng.choice((1, 2)), "bias": rng.random() < 0.7, "renorm": rng.random() < 0.7,
            "x": rng.choice(("f32", "bf16"))}


def work(case):
    op, T = case["op"], case["T"]
    size = {"f32": 4, "bf16": 2, "none": 0}
    if op == "norm":
        H = case["H"]
        per = size[case["x"]] + size[case["res"]] + (size[case["res"]] or 0) + (1 if case["codes"] else 2)
        return {"bytes": T * H * per + 4 * H + (4 * T if case["codes"] else 0), "flops": T * H * (9 if case["codes"] else 5)}
    if op == "swiglu":
        F = case["F"]
        return {"bytes": T * F * (2 * size[case["x"]] + 1) + 4 * T, "flops": T * F * 10}
    if op == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": T * K + N * K + T * N * size[case["out"]] + 4 * T + 4 * N * (2 if case["bias"] else 1),
                "flops": 2 * T * N * K}
    E, k = case["E"], case["k"]
    return {"bytes": T * E * size[case["x"]] + 8 * T * k + (4 * E if case["bias"] else 0), "flops": T * E * (6 + 2 * k)}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _rows(g, T, n, dtype, pad, scale=1.0):
    """[T, n] of N(0, scale), as a part of rows that are `pad` wider."""
    full = torch.empty((T, n + pad), dtype=dtype, device=DEV)
    full.copy_(torch.randn((T, n + pad), generator=g, device=DEV) * scale)
    return full[:, :n]


def _route_logits(case, g, bias):
    """Router logits.  A row whose choice would hang on the last bits of a 32-bit score (two scores in
    its ranking that differ by less than 4e-6 of the row's largest, and are not equal) is drawn
    again: for such a row the plain form itself has no settled answer."""
    T, E, dt = case["T"], case["E"], DTYPES[case["x"]]
    logits = torch.randn((T, E), generator=g, device=DEV).mul_(1.5).to(dt)
    for _ in range(12):
        c = _scores(case, logits.double())
        c = c if bias is None else c + bias.double()
        tol = 4e-6 * c.abs().amax(1)
        gs = _group_scores(case, c)
        gap = -torch.diff(gs.sort(dim=1, descending=True)[0], dim=1)
        near = ((gap > 0) & (gap < tol[:, None])).any(1)
        top = _masked(case, c, gs).sort(dim=1, descending=True)[0][:, : case["k"] + 1]
        gap = -torch.diff(top, dim=1)
        near |= ((gap > 0) & (gap < tol[:, None])).any(1)
        new = torch.randn((T, E), generator=g, device=DEV).mul_(1.5).to(dt)
        logits = torch.where(near[:, None], new, logits)
    return logits


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, T = case["op"], case["T"]
    st = dict(case)
    empty = lambda *a: torch.empty(a[:-1], dtype=a[-1], device=DEV)  # noqa: E731
    if op == "norm":
        H, pad = case["H"], case["pad"]
        # attention or expert output on top of a residual stream with a few large channels
        st["x"] = _rows(g, T, H, DTYPES[case["x"]], pad)
        st["residual"] = None
        if case["res"] != "none":
            st["residual"] = _rows(g, T, H, DTYPES[case["res"]], pad, 3.0)
            st["residual"][:, :: max(1, H // 5)] *= 8
        st["gamma"] = 1.0 + 0.1 * torch.randn(H, generator=g, device=DEV)
        st["h"] = empty(T, H, DTYPES[case["res"]]) if st["residual"] is not None else None
        st["y"] = empty(T, H, BF16)  # the normalised rows, or the values the codes stand for
        st["q"] = empty(T, H, torch.int8) if case["codes"] else None
        st["s"] = empty(T, F32) if case["codes"] else None
    elif op == "swiglu":
        st["gu"] = _rows(g, T, 2 * case["F"], DTYPES[case["x"]], case["pad"], 1.5)
        st["q"], st["s"], st["y"] = empty(T, case["F"], torch.int8), empty(T, F32), empty(T, case["F"], BF16)
    elif op == "linear":
        N, K, pad = case["N"], case["K"], case["pad"]
        # codes of normal rows: their largest of several thousand values sits near four deviations
        def codes(rows):
            full = torch.empty((rows, K + pad), dtype=torch.int8, device=DEV)
            step = max(1, (1 << 26) // (K + pad))
            for i in range(0, rows, step):
                n = min(step, rows - i)
                full[i : i + n] = (torch.randn((n, K + pad), generator=g, device=DEV) * 32).round_().clamp_(-127, 127).to(torch.int8)
            return full[:, :K]

        st["q"], st["w"] = codes(T), codes(N)
        st["s"] = 0.02 + 0.02 * torch.rand(T, generator=g, device=DEV)
        st["ws"] = 5e-4 + 5e-4 * torch.rand(N, generator=g, device=DEV)
        st["bias"] = 0.1 * torch.randn(N, generator=g, device=DEV) if case["bias"] else None
        st["y"] = empty(T, N, DTYPES[case["out"]])
    else:
        E = case["E"]
        st["bias"] = 0.02 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
        st["logits"] = _route_logits(case, g, st["bias"])
        st["idx"] = empty(T, case["k"], torch.int32)
        st["gate"] = empty(T, case["k"], F32)
    return st


# ---------------------------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------------------------
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from quantized_expert_ffn_topk_amd import abi

    op, T = st["op"], st["T"]
    if op == "norm":
        x, res, h, q, y, H = st["x"], st["residual"], st["h"], st["q"], st["y"], st["H"]
        abi.moe_rmsnorm_quant(x, _dt(abi, x), x.stride(0), res, 0 if res is None else _dt(abi, res),
                              0 if res is None else res.stride(0), st["gamma"], T, H, EPS, h, H,
                              y if q is None else None, H, q, H, st["s"])
        if q is None:
            return h, y
        return h, torch.mul(q, st["s"].unsqueeze(1), out=y), st["s"]
    if op == "swiglu":
        gu, q, s, F = st["gu"], st["q"], st["s"], st["F"]
        abi.moe_swiglu_quant(gu, _dt(abi, gu), gu.stride(0), T, F, None, 0, q, F, s)
        return torch.mul(q, s.unsqueeze(1), out=st["y"]), s
    if op == "linear":
        q, w, y = st["q"], st["w"], st["y"]
        abi.moe_linear_int8(q, q.stride(0), st["s"], T, w, w.stride(0), st["ws"], st["bias"], st["N"], st["K"],
                            y, _dt(abi, y), st["N"])
        return y
    if "desc" not in st:  # a program fills its router's descriptor in once
        st["desc"] = abi.moe_route_desc(st["E"], st["k"], abi.SCORE_SIGMOID if st["score"] == "sigmoid" else abi.SCORE_SOFTMAX,
                                        st["groups"], st["keep"], st["best"], int(st["renorm"]), 2.5)
    x = st["logits"]
    abi.moe_route_select(st["desc"], x, _dt(abi, x), st["E"], st["bias"], T, st["idx"], st["gate"])
    return st["idx"], st["gate"]


def _dt(abi, t):
    return abi.DT_BF16 if t.dtype == BF16 else abi.DT_F32


def _quantise(y):
    """Codes of rows by their largest magnitude, as the values that they stand for, and the scales."""
    top = y.abs().amax(1, keepdim=True)
    s = top / 127.0
    q = torch.clamp(torch.round(y * torch.where(top > 0, 127.0 / top, 0.0)), -127, 127)
    return (q * s).to(BF16), s.squeeze(1)


def _run_plain(st):
    op = st["op"]
    if op == "norm":
        h = st["x"].float()
        if st["residual"] is not None:
            h = h + st["residual"].float()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * st["gamma"]
        out = None if st["residual"] is None else h.to(st["residual"].dtype)
        return (out, *_quantise(y)) if st["codes"] else (out, y.to(BF16))
    if op == "swiglu":
        g, u = st["gu"].float().chunk(2, dim=1)
        return _quantise(g * torch.sigmoid(g) * u)
    if op == "linear":
        y = (st["q"].float() @ st["w"].float().t()) * st["s"][:, None] * st["ws"]
        if st["bias"] is not None:
            y = y + st["bias"]
        return y.to(st["y"].dtype)
    p = _scores(st, st["logits"].float())
    c = p if st["bias"] is None else p + st["bias"]
    idx = _masked(st, c, _group_scores(st, c)).sort(dim=1, descending=True, stable=True)[1][:, : st["k"]]
    w = p.gather(1, idx)
    if st["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.to(torch.int32), w * 2.5


def _scores(case, logits):
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _group_scores(case, c):
    by = c.view(c.shape[0], case["groups"], -1)
    return by.sort(dim=2, descending=True)[0][:, :, : case["best"]].sum(2)


def _masked(case, c, gs):
    """c outside the `keep` best groups (the lower one where two are equal) at minus infinity."""
    G = case["groups"]
    stay = torch.zeros(gs.shape, dtype=torch.bool, device=c.device)
    stay.scatter_(1, gs.sort(dim=1, descending=True, stable=True)[1][:, : case["keep"]], True)
    return c.masked_fill(~stay.repeat_interleave(c.shape[1] // G, dim=1), -math.inf)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    st, op = prepare(case, seed), case["op"]

    def codes(v):
        m = v.abs().max(dim=1).values
        unit = (m / 127)[:, None]
        n = torch.where(unit > 0, v / unit, torch.zeros_like(v)).round()
        return n * unit, m / 127

    if op == "norm":
        h = st["x"].double()
        h = h if st["residual"] is None else st["residual"].double() + h
        v = st["gamma"].double() * (h / (h.pow(2).sum(1, keepdim=True) / case["H"] + EPS).sqrt())
        hh = None if st["residual"] is None else h
        return (hh, *codes(v)) if case["codes"] else (hh, v)
    if op == "swiglu":
        gate, up = st["gu"][:, : case["F"]].double(), st["gu"][:, case["F"] :].double()
        return codes(up * gate / (torch.exp(-gate) + 1))
    if op == "linear":
        y = torch.empty((case["T"], case["N"]), dtype=torch.float64, device=DEV)
        q, step = st["q"].double(), 4096
        for n in range(0, case["N"], step):
            y[:, n : n + step] = q @ st["w"][n : n + step].double().t().contiguous()
        y = st["ws"].double() * (st["s"].double()[:, None] * y)
        return y if st["bias"] is None else st["bias"].double() + y
    T, E, G, k = case["T"], case["E"], case["groups"], case["k"]
    x = st["logits"].double()
    if case["score"] == "sigmoid":
        p = torch.sigmoid(x)
    else:
        p = torch.softmax(x, dim=1)
    c = p if st["bias"] is None else st["bias"].double() + p
    each = c.reshape(T, G, E // G)
    rank = each.max(dim=2).values
    if case["best"] == 2 and E // G > 1:
        # the second best of a group: its best once the first place of the best is taken out
        at = each.argmax(dim=2, keepdim=True)
        rank = rank + each.scatter(2, at, -math.inf).max(dim=2).values
    # a group stays if fewer than `keep` stand before it
    order = torch.arange(G, device=DEV)
    before = (rank[:, None, :] > rank[:, :, None]) | ((rank[:, None, :] == rank[:, :, None]) & (order[None, None, :] < order[None, :, None]))
    c = c.masked_fill((before.sum(2) >= case["keep"])[:, :, None].expand(T, G, E // G).reshape(T, E), -math.inf)
    picks = []
    for _ in range(k):
        top = c.max(dim=1, keepdim=True).values
        first = torch.where(c == top, torch.arange(E, device=DEV), E).min(dim=1, keepdim=True).values
        picks.append(first)
        c = c.scatter(1, first, -math.inf)
    idx = torch.cat(picks, 1)
    w = torch.gather(p, 1, idx)
    return idx.to(torch.int32), (w / w.sum(1, keepdim=True) if case["renorm"] else w) * 2.5
