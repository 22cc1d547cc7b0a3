"""GPU tests of block.py's E4M3 halves: a dense one, then a routed one with a shared expert, on one
residual stream, each step against the 64-bit form of what the step before gave; other streams, no
tokens, replays of a captured half, and refusals."""
import numpy as np
import pytest

from quantized_expert_ffn_topk_amd import abi
from tests import fp8_ref as ref
from tests import operators_ref as oref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from quantized_expert_ffn_topk_amd.block import Fp8DenseFFN, Fp8MoEFFN, quantise_weight_fp8  # noqa: E402

DEV = "cuda"
U = ref.U
H, F, E, K = 384, 200, 16, 4


def made(seed, *lead):
    g = torch.Generator().manual_seed(seed)
    gu, dn = torch.randn(*lead, 2 * F, H, generator=g) * 0.05, torch.randn(*lead, H, F, generator=g) * 0.05
    return [v.to(DEV) for pair in (quantise_weight_fp8(gu), quantise_weight_fp8(dn)) for v in pair]


def gamma(seed):
    return 1 + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(seed)).to(DEV)


def dense(max_tokens=8):
    return Fp8DenseFFN(gamma(1), *made(2), max_tokens=max_tokens)


def moe(max_tokens=8, shared=True, out_dtype=None):
    g = torch.Generator().manual_seed(3)
    router = (torch.randn(E, H, generator=g) * 0.05).bfloat16().to(DEV)
    bias = 0.02 * torch.randn(E, generator=g).to(DEV)
    route = abi.moe_route_desc(E, K, abi.SCORE_SIGMOID, 4, 2, 2, 1, 2.5)
    return Fp8MoEFFN(gamma(4), router, bias, *made(5, E), route, max_tokens, made(6) if shared else None, out_dtype=out_dtype)


def inputs(T, seed=7):
    g = torch.Generator().manual_seed(seed)
    return tuple(torch.randn(T, H, generator=g).mul_(f).bfloat16().to(DEV) for f in (1.0, 2.0))


def num(t):
    return t.double().cpu().numpy()


def values(q, s):
    return ref.scaled(q.view(torch.uint8).cpu().numpy(), s.cpu().numpy())


def weight(q, s):
    return ref.scaled_weights(q.view(torch.uint8).cpu().numpy(), s.cpu().numpy())


def close(got, x, w, bf16=True):
    want = x @ w.T
    assert (np.abs(got - want) <= ref.limit(x, w, 1, bf16, bf16)).all()


def swiglu_codes(qv, gu):
    act = oref.swiglu(gu)
    top = ref.spread(ref.block_max(act), F)
    step = np.maximum(np.abs(act) * 2.0 ** -4, top / 448 * 2.0 ** -10)
    assert (np.abs(qv - act) <= step * (1 + 2.0 ** -10) + 60 * U * top).all()


def normed(half, x, r, T):
    _, v = oref.rmsnorm(num(x), num(r), num(half.gamma), 1e-6)
    y = num(half.y[:T])
    assert (np.abs(y - v) <= np.abs(v) * (2.0 ** -8 + 2.0 ** -20) + 1e-37).all()
    q, s = ref.quant(y.astype(np.float32))
    assert np.array_equal(half.q[:T].view(torch.uint8).cpu().numpy()[y != 0], q[y != 0])
    return y


@pytest.mark.parametrize("T", [1, 7, 70])
@pytest.mark.parametrize("shared", [True, False])
def test_dense_then_routed_half_step_by_step(T, shared):
    d, m = dense(T), moe(T, shared)
    x, r = inputs(T)
    y1, h1 = d.forward(x, r)
    torch.cuda.synchronize()
    normed(d, x, r, T)
    close(num(d.gu[:T]), values(d.q[:T], d.s[:T]), weight(d.gate_up, d.s_gu))
    swiglu_codes(values(d.qh[:T], d.sh[:T]), num(d.gu[:T]))
    close(num(y1), values(d.qh[:T], d.sh[:T]), weight(d.down, d.s_dn))
    assert torch.equal(h1, (x.float() + r.float()).bfloat16())

    y2, h2 = m.forward(y1, h1)
    torch.cuda.synchronize()
    y = normed(m, y1, h1, T)
    rw = num(m.router)
    logits = num(m.logits[:T])
    assert (np.abs(logits - y @ rw.T) <= ref.limit(y, rw, 2, False, False)).all()
    idx, w, margin = oref.select(logits, num(m.bias), K, False, 4, 2, 2, True, 2.5)
    assert margin > 1e-6
    assert np.array_equal(m.idx[:T].cpu().numpy(), idx)
    np.testing.assert_allclose(m.w[:T].cpu().numpy(), w, rtol=2.0 ** -19)
    o, rows, pos = ref.group(idx, E)
    assert np.array_equal(m.offsets.cpu().numpy(), o) and np.array_equal(m.rows[:T * K].cpu().numpy(), rows)
    xv, qh, gu, yr = values(m.q[:T], m.s[:T])[rows], values(m.qh[:T * K], m.sh[:T * K]), num(m.gu[:T * K]), num(m.yr[:T * K])
    swiglu_codes(qh, gu)
    wg, wd = weight(m.gate_up, m.s_gu), weight(m.down, m.s_dn)
    for e in range(E):
        a, b = o[e], o[e + 1]
        if a < b:
            close(gu[a:b], xv[a:b], wg[e])
            close(yr[a:b], qh[a:b], wd[e])
    terms = num(m.w[:T])[:, :, None] * yr[pos]
    base = 0.0
    lim = K * U * np.abs(terms).sum(axis=1)
    if shared:
        v = values(m.shared.qh[:T], m.shared.sh[:T])
        sw = weight(m.shared.down, m.shared.s_dn)
        base = v @ sw.T
        lim = lim + ref.limit(v, sw, 1, True, True) + K * U * np.abs(base)
    want = terms.sum(axis=1) + base
    assert (np.abs(num(y2) - want) <= lim * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 1e-37).all()
    assert torch.equal(h2, (y1.float() + h1.float()).bfloat16())


@pytest.mark.parametrize("make", [dense, moe])
def test_halves_on_a_side_stream_and_of_no_tokens(make):
    half = make()
    x, r = inputs(8)
    want = half.forward(x, r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = half.forward(x, r, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = half.forward(x[:3], r[:3])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b[:3]) for a, b in zip(got[1:], want[1:]))
    y, h = half.forward(x[:0], r[:0])
    torch.cuda.synchronize()
    assert y.shape == (0, H) and h.shape == (0, H)


@pytest.mark.parametrize("make", [dense, moe])
def test_halves_captured_and_replayed_on_other_inputs(make):
    half = make()
    x, r = inputs(8)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = half.forward(x, r, torch.cuda.current_stream())
    for seed in (7, 8, 9):
        for t, v in zip((x, r), inputs(8, seed)):
            t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in got]
        want = half.forward(x, r)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, want))


def test_routed_half_with_fp32_output():
    a, b = moe(out_dtype=torch.float32), moe()
    x, r = inputs(8)
    y, z = a.forward(x, r)[0], b.forward(x, r)[0]
    torch.cuda.synchronize()
    assert y.dtype == torch.float32 and z.dtype == torch.bfloat16
    # the shared expert's output is rounded to bf16 in one of them, and the sum
    lim = 2.0 ** -8 * y.abs() + 2.0 ** -8 * (y.abs() + 1.0)
    assert ((y - z.float()).abs() <= lim).all()


def test_halves_refuse_what_does_not_fit():
    d, m = dense(4), moe(4)
    x, r = inputs(4)
    for half in (d, m):
        for bad in ((x[:1], r), (x[:, :H - 1], r), (x.half(), r), (x.cpu(), r), inputs(5)):
            with pytest.raises(ValueError):
                half.forward(*bad)
    gu, sg, dn, sd = made(2)
    for bad in ((gu.float(), sg, dn, sd), (gu, sg[:1], dn, sd), (gu, sg, dn[:, :1], sd), (gu, sg, dn, sd.cpu())):
        with pytest.raises(ValueError):
            Fp8DenseFFN(d.gamma, *bad, max_tokens=4)
    with pytest.raises(ValueError):
        Fp8MoEFFN(m.gamma, m.router.float(), None, *made(5, E), m.route, 4)
    with pytest.raises(ValueError):
        Fp8MoEFFN(m.gamma, m.router, m.bias[1:], *made(5, E), m.route, 4)
    with pytest.raises(ValueError):
        Fp8MoEFFN(m.gamma, m.router, None, *made(5, E - 1), m.route, 4)
