"""Operators of an FFN in 8-bit floating point, dense or by experts, as cases to measure: rows (or the
SwiGLU of rows) as E4M3 codes with a scale for each 128 values, the product of such codes with weights
of a scale for each 128 x 128, products grouped by expert with ragged sizes (E4M3 or bf16), the
grouping of routed rows, and the weighted sum that brings their outputs back to the tokens.

Sizes: hidden 6144 and 2048, FFN 2048, 256 and 64 experts with top-8 are this repository's layer
shapes; the dense FFN is 12288 wide; the token counts run from one decode step to a prefill of 4096.
"""
import math

import torch

own = False

DEV = "cuda"
F32, BF16, FP8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
DTYPES = {"f32": F32, "bf16": BF16, "fp8": FP8}
BLOCK = 128
TOP = 448.0  # the largest E4M3 value


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _quant(name, T, K, x, act, pad=0):
    return {"name": name, "op": "quant", "T": T, "K": K, "x": x, "act": act, "pad": pad}


def _linear(name, T, N, K, out, bias, pad=0):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "out": out, "bias": bias, "pad": pad}


def _grouped(name, T, k, E, N, K, x, out, skew, gather, pad=0):
    return {"name": name, "op": "grouped", "T": T, "k": k, "E": E, "N": N, "K": K, "x": x, "out": out,
            "skew": skew, "gather": gather, "pad": pad}


def _group(name, T, k, E, skew):
    return {"name": name, "op": "group", "T": T, "k": k, "E": E, "skew": skew}


def _combine(name, T, k, H, y, out, base, pad=0):
    return {"name": name, "op": "combine", "T": T, "k": k, "H": H, "y": y, "out": out, "base": base, "pad": pad}


def listed():
    return [
        # one decoded token in front of an E4M3 product
        _quant("quant_1x6144", 1, 6144, "bf16", "none"),
        # the experts' rows of a prefill of 4096 tokens between the two products: SwiGLU and codes
        _quant("quant_swiglu_32768x2048", 32768, 2048, "bf16", "swiglu"),
        # one decoded token, a square projection: a stream of weights
        _linear("linear_1x6144x6144", 1, 6144, 6144, "bf16", False),
        # an odd remainder of a prompt through an odd-sized head with bias, fp32 output, rows that end
        # inside a block and lie in wider ones
        _linear("linear_333x5003x2000_f32", 333, 5003, 2000, "f32", True, 16),
        # a prefill of 4096 tokens, gate and up of the dense FFN in one product
        _linear("linear_4096x24576x6144", 4096, 24576, 6144, "bf16", False),
        # a batch of 16 decoding sequences, gate and up of their experts: a stream of some hundred
        # experts' weights, one or a few rows each
        _grouped("grouped_fp8_16x8of256", 16, 8, 256, 4096, 6144, "fp8", "bf16", 0.5, True),
        # a prefill of 4096 tokens through the same experts
        _grouped("grouped_fp8_4096x8of256", 4096, 8, 256, 4096, 6144, "fp8", "bf16", 0.5, True),
        # an odd remainder of a prompt through bf16 experts of odd sizes, fp32 output
        _grouped("grouped_bf16_333x6of62", 333, 6, 62, 2051, 2044, "bf16", "f32", 1.0, False, 4),
        # the grouping of a batch of 16 decoding sequences
        _group("group_16x8of256", 16, 8, 256, 0.5),
        # the grouping of a prefill of 4096 tokens
        _group("group_4096x8of256", 4096, 8, 256, 0.5),
        # one decoded token's experts on top of the shared expert's output
        _combine("combine_1x8x6144", 1, 8, 6144, "bf16", "bf16", True),
        # a prefill's
        _combine("combine_4096x8x6144", 4096, 8, 6144, "bf16", "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Half of the widths are multiples of 64, a quarter of 8, a quarter any number."""
    n = _log(rng, lo, hi)
    return max(lo, n - n % rng.choice((64, 64, 8, 1)))


def draw(rng):
    op = rng.choice(("quant", "linear", "linear", "grouped", "grouped", "group", "combine"))
    if op == "quant":
        K = _width(rng, 128, 12288)
        return {"op": op, "T": min(_log(rng, 1, 32768), 32768 * 2048 // K), "K": K, "x": rng.choice(("bf16", "bf16", "f32")),
                "act": rng.choice(("none", "swiglu")), "pad": rng.choice((0, 0, 8, 3))}
    if op == "linear":
        N, K = _width(rng, 64, 24576), _width(rng, 64, 12288)
        T = max(1, min(_log(rng, 1, 4096), 4096 * 24576 * 6144 // (N * K)))
        return {"op": op, "T": T, "N": N, "K": K, "out": rng.choice(("bf16", "bf16", "f32")), "bias": rng.random() < 0.3,
                "pad": rng.choice((0, 0, 16, 3))}
    if op == "grouped":
        N, K = _width(rng, 64, 8192), _width(rng, 64, 8192)
        E = min(_log(rng, 4, 256), max(4, (1 << 31) // (N * K)))
        k = rng.randint(1, min(8, E))
        T = max(1, min(_log(rng, 1, 4096), (1 << 39) // (N * K * k)))
        return {"op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "x": rng.choice(("fp8", "fp8", "bf16")),
                "out": rng.choice(("bf16", "bf16", "f32")), "skew": rng.choice((0.0, 0.5, 1.5)),
                "gather": rng.random() < 0.5, "pad": rng.choice((0, 0, 16, 3))}
    if op == "group":
        E = _log(rng, 8, 512)
        return {"op": op, "T": _log(rng, 1, 16384), "k": rng.randint(1, min(16, E)), "E": E, "skew": rng.choice((0.0, 0.5, 1.5))}
    H, k = _width(rng, 128, 8192), rng.randint(1, 16)
    return {"op": op, "T": min(_log(rng, 1, 8192), 4096 * 8 * 6144 // (k * H)), "k": k, "H": H, "y": rng.choice(("bf16", "bf16", "f32")),
            "out": rng.choice(("bf16", "f32")), "base": rng.random() < 0.5, "pad": rng.choice((0, 0, 8, 3))}


SIZE = {"f32": 4, "bf16": 2, "fp8": 1, "none": 0}


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    op, T = case["op"], case["T"]
    if op == "quant":
        K, wide = case["K"], 2 if case["act"] == "swiglu" else 1
        return {"bytes": T * (K * (wide * SIZE[case["x"]] + 1) + 4 * _blocks(K)), "flops": T * K * (12 if wide == 2 else 3)}
    if op == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": T * (K + 4 * _blocks(K)) + N * K + 4 * _blocks(N) * _blocks(K) + T * N * SIZE[case["out"]] + (4 * N if case["bias"] else 0),
                "flops": 2 * T * N * K}
    if op == "grouped":
        N, K, E, M = case["N"], case["K"], case["E"], T * case["k"]
        size, scales = SIZE[case["x"]], 4 if case["x"] == "fp8" else 0
        # experts that get a row: by an even spread
        active = E * (1.0 - (1.0 - case["k"] / E) ** T)
        rows = T if case["gather"] else M
        return {"bytes": int(rows * (K * size + scales * _blocks(K)) + active * (N * K * size + scales * _blocks(N) * _blocks(K)) +
                             M * N * SIZE[case["out"]] + 4 * (E + 1) + (4 * M if case["gather"] else 0)),
                "flops": 2 * M * N * K}
    if op == "group":
        M = T * case["k"]
        return {"bytes": 12 * M + 4 * (case["E"] + 1), "flops": 4 * M}
    H, k = case["H"], case["k"]
    return {"bytes": T * (k * (H * SIZE[case["y"]] + 8) + H * SIZE[case["out"]] * (2 if case["base"] else 1)), "flops": 2 * T * k * H}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _rows(g, T, n, dtype, pad, scale=1.0):
    """[T, n] of N(0, scale), as a part of rows that are `pad` wider; made in pieces."""
    full = torch.empty((T, n + pad), dtype=dtype, device=DEV)
    step = max(1, (1 << 28) // (n + pad))
    for i in range(0, T, step):
        m = min(step, T - i)
        v = torch.randn((m, n + pad), generator=g, device=DEV) * scale
        full[i : i + m] = (v.clamp_(-TOP, TOP) if dtype == FP8 else v).to(dtype)
    return full[:, :n]


def _codes(g, T, K, pad):
    """E4M3 codes of normal rows: the largest of 128 values lies near 2.7 deviations, at code 448."""
    return _rows(g, T, K, FP8, pad, 150.0)


def _routing(g, T, k, E, skew):
    """Ids [T, k] of distinct experts, some experts more popular than others."""
    logits = torch.randn((T, E), generator=g, device=DEV) + skew * torch.randn(E, generator=g, device=DEV)
    return logits.sort(dim=1, descending=True)[1][:, :k].to(torch.int32).contiguous()


def _grouping(idx, E):
    """(offsets, rows, pos) of ids, as moe_group_rows gives them."""
    flat = idx.reshape(-1).long()
    order = flat.sort(stable=True)[1]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = (flat[:, None] == torch.arange(E, device=DEV)).sum(0).cumsum(0)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(flat.numel(), device=DEV)
    return offsets.to(torch.int32), (order // idx.shape[1]).to(torch.int32), pos.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, T = case["op"], case["T"]
    st = dict(case)
    empty = lambda *a: torch.empty(a[:-1], dtype=a[-1], device=DEV)  # noqa: E731
    scales = lambda n, m, lo: lo * (1.0 + torch.rand((n, m), generator=g, device=DEV))  # noqa: E731
    if op == "quant":
        K = case["K"]
        st["x"] = _rows(g, T, K * (2 if case["act"] == "swiglu" else 1), DTYPES[case["x"]], case["pad"], 1.5)
        st["q"], st["s"] = empty(T, K, FP8), empty(T, _blocks(K), F32)
    elif op == "linear":
        N, K = case["N"], case["K"]
        st["q"], st["w"] = _codes(g, T, K, case["pad"]), _codes(g, N, K, case["pad"])
        st["s"], st["ws"] = scales(T, _blocks(K), 4e-3), scales(_blocks(N), _blocks(K), 1e-4)
        st["bias"] = 0.1 * torch.randn(N, generator=g, device=DEV) if case["bias"] else None
        st["y"] = empty(T, N, DTYPES[case["out"]])
    elif op == "grouped":
        N, K, E, k = case["N"], case["K"], case["E"], case["k"]
        fp8 = case["x"] == "fp8"
        make = (lambda n: _codes(g, n, K, case["pad"])) if fp8 else (lambda n: _rows(g, n, K, BF16, case["pad"], 0.5))
        idx = _routing(g, T, k, E, case["skew"])
        st["offsets"], rows, _ = _grouping(idx, E)
        st["cap"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())  # rows of the largest group
        st["rows"] = rows if case["gather"] else None
        st["x"] = make(T if case["gather"] else T * k)
        st["w"] = make(E * N).unflatten(0, (E, N))
        st["s"] = scales(st["x"].shape[0], _blocks(K), 4e-3) if fp8 else None
        st["ws"] = scales(E * _blocks(N), _blocks(K), 1e-4).unflatten(0, (E, _blocks(N))) if fp8 else None
        st["y"] = empty(T * k, N, DTYPES[case["out"]])
        st["xtype"] = case["x"]
    elif op == "group":
        st["idx"] = _routing(g, T, case["k"], case["E"], case["skew"])
        st["offsets"] = empty(case["E"] + 1, torch.int32)
        st["rows"], st["pos"] = empty(T * case["k"], torch.int32), empty(T * case["k"], torch.int32)
    else:
        H, k = case["H"], case["k"]
        # a routed row lies anywhere among the grouped ones
        st["pos"] = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32)
        st["gate"] = torch.rand((T, k), generator=g, device=DEV) * (2.5 / k)
        st["rows"] = _rows(g, T * k, H, DTYPES[case["y"]], case["pad"])
        st["shared"] = _rows(g, T, H, DTYPES[case["out"]], case["pad"]) if case["base"] else None
        st["result"] = empty(T, H, DTYPES[case["out"]])
    return st


# ---------------------------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------------------------
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _dt(abi, t):
    return abi.DT_BF16 if t.dtype == BF16 else abi.DT_F32 if t.dtype == F32 else abi.DT_FP8


def _run_own(st):
    from quantized_expert_ffn_topk_amd import abi

    op, T = st["op"], st["T"]
    if op == "quant":
        x, q, s, K = st["x"], st["q"], st["s"], st["K"]
        abi.moe_quant_fp8(x, _dt(abi, x), x.stride(0), abi.ACT_SWIGLU if st["act"] == "swiglu" else abi.ACT_NONE, T, K, None,
                          q, K, s, s.stride(0))
        return q, s
    if op == "linear":
        q, s, w, ws, y = st["q"], st["s"], st["w"], st["ws"], st["y"]
        abi.moe_linear_fp8(q, q.stride(0), s, s.stride(0), T, w, w.stride(0), ws, ws.stride(0), st["bias"], st["N"], st["K"],
                           y, _dt(abi, y), st["N"])
        return y
    if op == "grouped":
        x, s, w, ws, y = st["x"], st["s"], st["w"], st["ws"], st["y"]
        abi.moe_grouped_linear(x, _dt(abi, x), x.stride(0), s, 0 if s is None else s.stride(0), x.shape[0], st["rows"], st["offsets"],
                               st["E"], y.shape[0], w, w.stride(1), w.stride(0), ws, 0 if ws is None else ws.stride(1),
                               0 if ws is None else ws.stride(0), st["N"], st["K"], y, _dt(abi, y), st["N"])
        return y
    if op == "group":
        abi.moe_group_rows(st["idx"], T, st["k"], st["E"], st["offsets"], st["rows"], st["pos"])
        return st["offsets"], st["rows"], st["pos"]
    y, base, out = st["rows"], st["shared"], st["result"]
    abi.moe_combine_rows(y, _dt(abi, y), y.stride(0), y.shape[0], st["pos"], st["gate"], base, 0 if base is None else base.stride(0),
                         T, st["k"], st["H"], out, _dt(abi, out), st["H"])
    return out


def _spread(s, K):
    """A scale for each block of 128, as one for each of K values."""
    return s.repeat_interleave(BLOCK, dim=-1)[..., :K]


def _run_plain(st):
    op, T = st["op"], st["T"]
    if op == "quant":
        K, v = st["K"], st["x"].float()
        if st["act"] == "swiglu":
            v = v[:, :K] * torch.sigmoid(v[:, :K]) * v[:, K:]
        by = torch.nn.functional.pad(v, (0, _blocks(K) * BLOCK - K)).view(T, -1, BLOCK)
        top = by.abs().amax(2)
        inv = torch.where(top > 0, TOP / top, 0.0)
        q = (v * _spread(inv, K)).clamp(-TOP, TOP).to(FP8)
        return q, top / TOP
    if op == "linear":
        N, K = st["N"], st["K"]
        x = st["q"].float() * _spread(st["s"], K)
        w = st["w"].float() * _spread(st["ws"].repeat_interleave(BLOCK, dim=0)[:N], K)
        y = x @ w.t()
        return (y if st["bias"] is None else y + st["bias"]).to(st["y"].dtype)
    if op == "grouped":
        N, K, E, M, cap = st["N"], st["K"], st["E"], st["y"].shape[0], st["cap"]
        x, w = st["x"].float(), st["w"].float()
        if st["xtype"] == "fp8":
            x, w = x * _spread(st["s"], K), w * _spread(st["ws"].repeat_interleave(BLOCK, dim=1)[:, :N], K)
        if st["rows"] is not None:
            x = x[st["rows"].long()]
        # every group padded to the largest one's rows
        first = st["offsets"][:-1].long()
        each = torch.arange(M, device=DEV)
        expert = (each[:, None] >= st["offsets"][1:].long()).sum(1)
        slot = expert * cap + each - first[expert]
        padded = torch.zeros((E * cap, K), device=DEV)
        padded[slot] = x
        y = torch.bmm(padded.view(E, cap, K), w.transpose(1, 2))
        return y.view(E * cap, N)[slot].to(st["y"].dtype)
    if op == "group":
        return _grouping(st["idx"], st["E"])
    y = st["rows"][st["pos"].long()].float().view(T, st["k"], -1)
    y = (y * st["gate"][:, :, None]).sum(1)
    return (y if st["shared"] is None else y + st["shared"].float()).to(st["result"].dtype)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _product(x, s, w, ws):
    """Rows of x with their blocks' scales times rows of w with theirs, block after block."""
    y = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device=DEV)
    of = torch.arange(w.shape[0], device=DEV) // BLOCK
    for b in range(_blocks(x.shape[1])):
        a, c = x[:, b * BLOCK : (b + 1) * BLOCK].double(), w[:, b * BLOCK : (b + 1) * BLOCK].double()
        y += (a @ c.t().contiguous()) * s[:, b].double()[:, None] * ws[of, b].double()
    return y


def exact(case, seed):
    st, op, T = prepare(case, seed), case["op"], case["T"]
    if op == "quant":
        K, v = case["K"], st["x"].double()
        if case["act"] == "swiglu":
            v = v[:, K:] * v[:, :K] / (1 + torch.exp(-v[:, :K]))
        q, s = torch.empty_like(v), torch.empty((T, _blocks(K)), dtype=torch.float64, device=DEV)
        for b in range(_blocks(K)):
            part = v[:, b * BLOCK : (b + 1) * BLOCK]
            top = part.abs().max(dim=1).values
            s[:, b] = top / 448
            z = torch.where(top[:, None] > 0, part * (448 / top[:, None]), 0.0)
            # E4M3 has three bits behind the leading one, the smallest step is 2^-9
            step = 2.0 ** (torch.floor(torch.log2(z.abs().clamp(min=2.0**-6))) - 3)
            q[:, b * BLOCK : (b + 1) * BLOCK] = torch.round(z / step) * step
        return q, s
    if op == "linear":
        y = torch.empty((T, case["N"]), dtype=torch.float64, device=DEV)
        step = 32 * BLOCK
        for n in range(0, case["N"], step):
            y[:, n : n + step] = _product(st["q"], st["s"], st["w"][n : n + step], st["ws"][n // BLOCK : (n + step) // BLOCK])
        return y if st["bias"] is None else y + st["bias"].double()
    if op == "grouped":
        y = torch.zeros((T * case["k"], case["N"]), dtype=torch.float64, device=DEV)
        at = st["offsets"].tolist()
        for e in range(case["E"]):
            if at[e] == at[e + 1]:
                continue
            which = torch.arange(at[e], at[e + 1], device=DEV) if st["rows"] is None else st["rows"][at[e] : at[e + 1]].long()
            if case["x"] == "fp8":
                y[at[e] : at[e + 1]] = _product(st["x"].view(torch.uint8)[which].view(FP8), st["s"][which], st["w"][e], st["ws"][e])
            else:
                y[at[e] : at[e + 1]] = st["x"][which].double() @ st["w"][e].double().t().contiguous()
        return y
    if op == "group":
        return None
    y = torch.zeros((T, case["H"]), dtype=torch.float64, device=DEV) if st["shared"] is None else st["shared"].double()
    pos = st["pos"].view(T, case["k"]).long()
    for i in range(case["k"]):
        y = y + st["gate"][:, i : i + 1].double() * st["rows"][pos[:, i]].double()
    return y
