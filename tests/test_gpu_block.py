"""GPU test of the FFN halves of a block (block.py): a dense layer, then a
routed one, on one residual stream, against the same steps from the plain
forms and the oracle's expert layer; and their refusals."""
import numpy as np
import pytest

import oracle
from quantized_expert_ffn_topk_amd import abi, synth
from tests import operators_ref as ref
from tests.gpu_common import Case, rel_err

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda"


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def dense(seed, H, F, max_tokens):
    from quantized_expert_ffn_topk_amd.block import DenseFFN, quantise_weight
    g = torch.Generator().manual_seed(seed)
    gu = torch.randn(2 * F, H, generator=g) * 0.05
    dn = torch.randn(H, F, generator=g) * 0.05
    gamma = 1 + 0.1 * torch.randn(H, generator=g)
    qg, sg = quantise_weight(gu)
    qd, sd = quantise_weight(dn)
    d = DenseFFN(gamma.to(DEV), qg.to(DEV), sg.to(DEV), qd.to(DEV), sd.to(DEV), max_tokens)
    return d, (gamma.numpy(), qg.numpy(), sg.numpy(), qd.numpy(), sd.numpy())


def quant(v):
    a = np.abs(v).max(axis=1)
    safe = np.where(a > 0, a, 1.0)
    return np.rint(v * (127.0 / safe)[:, None]).clip(-127, 127), a / 127.0


def expert_rows(x, idx, w, c):
    """The oracle's experts for a given choice: shared + sum of w_i * expert idx_i."""
    out = np.zeros((x.shape[0], c.H))
    for t in range(x.shape[0]):
        qa, sa = oracle.quant_row(x[t])
        if c.shared is not None:
            out[t] += oracle.expert(qa, sa, c.shared, c.g)["y"]
        for e, we in zip(idx[t], w[t]):
            out[t] += float(we) * oracle.expert(qa, sa, c.distinct[c.emap[e]], c.g)["y"].astype(np.float64)
    return out


@pytest.mark.parametrize("T", [1, 3, 70])
def test_dense_then_routed_half_against_the_plain_steps(T):
    from quantized_expert_ffn_topk_amd.block import MoEFFN
    H, F, E, k = 512, 384, 32, 4
    d, (gamma, qg, sg, qd, sd) = dense(3, H, F, T)
    c = Case(5, T, H, 256, E, k, 1, r=2.5, n_distinct=3)
    lay = c.layer(max_tokens=T)
    route = abi.moe_route_desc(E, k, abi.SCORE_SIGMOID, 4, 2, 2, 1, 2.5)
    g2 = (1 + 0.1 * np.random.default_rng(6).standard_normal(H)).astype(np.float32)
    m = MoEFFN(torch.from_numpy(g2).to(DEV), lay, route)
    r = np.random.default_rng([7, T])
    x = ref.bf16(r.standard_normal((T, H)))
    res = ref.bf16(2 * r.standard_normal((T, H)))
    xt = torch.from_numpy(x).to(DEV).bfloat16()
    rt = torch.from_numpy(res).to(DEV).bfloat16()

    y1, h1 = d.forward(xt, rt)
    y2, h2 = m.forward(y1, h1)
    torch.cuda.synchronize()

    # dense half in 64 bits; a code may fall to the other side of a half where
    # the GPU's fp32 value does (one code of 127 steps, far inside 1 %)
    h, v = ref.rmsnorm(x, res, gamma, 1e-6)
    q, s = quant(v)
    gu = (q @ qg.astype(np.float64).T) * s[:, None] * sg.astype(np.float64)
    q2, s2 = quant(ref.swiglu(ref.bf16(gu)))
    want = (q2 @ qd.astype(np.float64).T) * s2[:, None] * sd.astype(np.float64)
    assert rel_err(y1.float().cpu().numpy(), want) < 1e-2
    assert np.array_equal(h1.float().cpu().numpy(), ref.bf16(x.astype(np.float32) + res))

    # routed half from the GPU's own dense output: norm, choice, experts
    y1n, h1n = y1.float().cpu().numpy(), h1.float().cpu().numpy()
    h, v = ref.rmsnorm(y1n, h1n, g2, 1e-6)
    yb = synth.bf16_bits_to_f32(bits(m.y[:T]))
    lim = np.abs(v) * (2.0 ** -8 + 2.0 ** -20) + 1e-37
    assert (np.abs(yb - v) <= lim).all()
    logits = yb.astype(np.float64) @ c.Wr.astype(np.float64).T
    idx, w, margin = ref.select(logits, c.b, k, False, 4, 2, 2, True, 2.5)
    assert margin > 1e-12
    assert np.array_equal(m.idx[:T].cpu().numpy(), idx)
    np.testing.assert_allclose(m.w[:T].cpu().numpy(), w, rtol=2.0 ** -22)
    out = expert_rows(yb, idx, m.w[:T].cpu().numpy(), c)
    assert rel_err(y2.cpu().numpy(), out) <= 2e-3
    assert np.array_equal(h2.float().cpu().numpy(), ref.bf16(y1n + h1n))
    lay.close()


def test_halves_on_a_side_stream_and_of_no_tokens():
    d, _ = dense(4, 256, 512, 8)
    x = torch.randn(8, 256, device=DEV).bfloat16()
    r = torch.randn(8, 256, device=DEV).bfloat16()
    want = d.forward(x, r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = d.forward(x, r, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    side.wait_stream(torch.cuda.current_stream())
    got = d.forward(x, r, side.cuda_stream)              # the raw handle
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y, h = d.forward(x[:0], r[:0])
    assert y.shape == (0, 256) and h.shape == (0, 256)


def test_halves_take_rows_of_wider_tensors():
    d, _ = dense(5, 256, 512, 4)
    wide = torch.randn(4, 512, device=DEV).bfloat16()
    r = torch.randn(4, 256, device=DEV)
    a = d.forward(wide[:, 128:384], r)
    b = d.forward(wide[:, 128:384].contiguous(), r)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert a[1].dtype == torch.float32


def test_halves_refuse_what_does_not_fit():
    from quantized_expert_ffn_topk_amd.block import DenseFFN, MoEFFN
    d, _ = dense(6, 256, 512, 4)
    x, r = torch.zeros(2, 256, device=DEV).bfloat16(), torch.zeros(2, 256, device=DEV).bfloat16()
    for bad in ((x[:1], r), (x[:, :255], r), (x.half(), r), (x.t().contiguous().t(), r),
                (torch.zeros(5, 256, device=DEV), torch.zeros(5, 256, device=DEV)), (x.cpu(), r)):
        with pytest.raises(ValueError):
            d.forward(*bad)
    with pytest.raises(ValueError):
        DenseFFN(d.gamma, d.gate_up.float(), d.s_gu, d.down, d.s_dn, 4)
    with pytest.raises(ValueError):
        DenseFFN(d.gamma, d.gate_up, d.s_gu[1:], d.down, d.s_dn, 4)
    c = Case(8, 2, 256, 256, 8, 2, 0, n_distinct=1)
    lay = c.layer()
    with pytest.raises(ValueError):
        MoEFFN(d.gamma, lay, abi.moe_route_desc(8, 3, 0, 1, 1, 1, 1, 1.0))
    lay.close()
