"""GPU tests of the operators around the MoE layer at the ends of their number ranges.

Tolerances.  U = 2^-24 as in the operators' other tests, TINY = 2^-149 the step of fp32's
subnormals.  A score below 2^-126 keeps that step: the exponential and the product with the
reciprocal round to it once each, so a score is within 1.5 of it beside the relative 20 U."""
import numpy as np
import pytest

from quantized_expert_ffn_topk_amd import abi
from tests import operators_ref as ref
from tests.test_gpu_operators import U, run_select

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda"
TINY = 2.0 ** -149


# ---------------------------------------------------------------------------
# scores below 2^-126: fp32 holds them as subnormals, they are in an order, and a row of them alone
# has weights
# ---------------------------------------------------------------------------
def low_logits(seed, T, E, top, step):
    """Rows of E different logits from `top` down in steps of `step`, each in an order of its own."""
    r = np.random.default_rng([seed, T, E])
    return np.stack([top - step * r.permutation(E) for _ in range(T)]).astype(np.float32)


def settled(p, G, best):
    """The scores of a row and the sums that its groups are ranked by lie further apart than they can be off."""
    off = lambda v, n: n * (20 * U * np.abs(v) + 1.5 * TINY)  # noqa: E731
    groups = -np.sort(-p.reshape(G, -1), axis=1)[:, :best].sum(axis=1)
    for v, n in ((np.sort(p), 1), (np.sort(groups), best)):
        if not (np.diff(v) > 2 * off(v[1:], n)).all():
            return False
    return True


@pytest.mark.parametrize("dt,E,step", [("f32", 64, 0.1), ("bf16", 16, 0.5)])
@pytest.mark.parametrize("G,tg,best", [(1, 1, 1), (8, 3, 1), (8, 5, 2)])
def test_select_sigmoid_rows_of_subnormal_scores(dt, E, step, G, tg, best):
    l = low_logits(1, 40, E, -86.0, step)
    p = ref.scores(l, False)
    k, checked = 6, 0
    idx, w = run_select(l, None, dt, k, False, G, tg, best, True)
    for t in range(l.shape[0]):
        if not settled(p[t], G, best):
            continue
        checked += 1
        iw, ww, _ = ref.select(l[t:t + 1], None, k, False, G, tg, best, True, 2.5)
        assert np.array_equal(idx[t], iw[0]), (t, idx[t], iw[0])
        pc = p[t, iw[0]]
        lim = ww[0] * ((40 + 2 * k) * U + 1.5 * TINY * (1 / pc + k / pc.sum()))
        assert (np.abs(w[t] - ww[0]) <= lim).all(), (t, w[t], ww[0])
    assert checked >= 20, checked


@pytest.mark.parametrize("dt,E,step", [("f32", 64, 0.13), ("bf16", 16, 0.5)])
@pytest.mark.parametrize("G,tg,best", [(1, 1, 1), (8, 3, 1), (8, 5, 2)])
def test_select_softmax_keeps_the_order_of_scores_far_below_the_largest(dt, E, step, G, tg, best):
    l = low_logits(2, 40, E, -88.0, step)
    l[:, 5] = 0.0                                        # one expert has all but nothing left over
    p = ref.scores(l, True)
    k, checked = 6, 0
    idx, w = run_select(l, None, dt, k, True, G, tg, best, False)
    for t in range(l.shape[0]):
        if not settled(p[t], G, best):
            continue
        checked += 1
        iw, ww, _ = ref.select(l[t:t + 1], None, k, True, G, tg, best, False, 2.5)
        assert np.array_equal(idx[t], iw[0]), (t, idx[t], iw[0])
        # a weight is 2.5 scores, rounded once more
        assert (np.abs(w[t] - ww[0]) <= ww[0] * (40 + 2 * k) * U + (2.5 * 1.5 + 0.5) * TINY).all()
    assert checked >= 20, checked


@pytest.mark.parametrize("softmax", [False, True])
def test_select_scores_below_the_smallest_number_are_zero(softmax):
    # below 2^-150 a score is 0 in fp32, whatever the logit: such experts are equal, and a row of them has weights 0
    l = np.full((3, 32), -120.0, np.float32)
    l[1, 20:] = np.finfo(np.float32).min
    l[2, 9:] = -np.inf
    if softmax:
        l[:, 31] = 0.0
    idx, w = run_select(l, None, "f32", 4, softmax, 1, 1, 1, not softmax)
    first = [31, 0, 1, 2] if softmax else [0, 1, 2, 3]
    assert idx.tolist() == [first] * 3
    assert w.tolist() == ([[2.5, 0, 0, 0]] * 3 if softmax else [[0.0] * 4] * 3)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_select_experts_without_a_score_come_last_and_weigh_exactly_nothing(dt):
    low = [-np.inf, -1000.0, -200.0, -199.5, np.nan, np.finfo(np.float32).min]
    l = np.array([low + [-90.0, 1.0, -81.0, -80.0, -79.5, 0.0]] * 2, np.float32)
    l[1] = l[1, ::-1]
    idx, w = run_select(l, None, dt, 12, False, 1, 1, 1, False, 1.0)
    # by score, then all scores of 0 by their number, the NaN behind them
    assert idx[0].tolist() == [7, 11, 10, 9, 8, 6, 0, 1, 2, 3, 5, 4]
    assert idx[1].tolist() == [4, 0, 1, 2, 3, 5, 6, 8, 9, 10, 11, 7]
    assert (w[:, :6] > 0).all() and (w[:, 6:] == 0).all()


# ---------------------------------------------------------------------------
# bf16 outputs at both ends of the range: rounded to nearest even, no tolerance where the fp32 value's
# bits are defined
# ---------------------------------------------------------------------------
def same_bits(got, want):
    """bf16 values held as fp32: equal bits, any NaN for a NaN."""
    got, want = got.astype(np.float32), want.astype(np.float32)
    nan = np.isnan(want)
    assert np.isnan(got[nan]).all()
    assert np.array_equal(got[~nan].view(np.uint32), want[~nan].view(np.uint32)), \
        list(zip(got[got != want][:4], want[got != want][:4]))


@pytest.mark.parametrize("T,N,K", [(6, 40, 100), (70, 4200, 48)])
def test_linear_bf16_subnormal_and_overflowing_outputs(T, N, K):
    from tests.test_gpu_operators import lin_inputs, run_linear
    q, s, w, ws, _ = lin_inputs(31, T, N, K)
    s[0::5] *= np.float32(1e-24)                         # y from 1e-42 to 1e-37
    s[1::5] *= np.float32(1e16)                          # y past fp32's largest number, and just below it
    s[2::5], s[4::5] = np.float32(np.inf), np.float32(np.nan)
    ws = (ws * np.float32(1e-18)).astype(np.float32)
    ws[1::3] *= np.float32(1e36)
    with np.errstate(over="ignore", invalid="ignore"):
        want = ref.linear(q, s, w, ws, None)
        same_bits(run_linear(q, s, w, ws, None, "bf16"), ref.bf16(want))
    got = run_linear(q, s, w, ws, None, "f32")
    nan = np.isnan(want)
    assert np.isnan(got[nan]).all() and np.array_equal(got[~nan].view(np.uint32), want[~nan].view(np.uint32))
    assert ((np.abs(want) < 2.0 ** -126) & (want != 0)).any() and np.isinf(want).any() and nan.any()


@pytest.mark.parametrize("H", [6, 300, 6144, 33001])
def test_norm_new_residual_of_subnormal_sums(H):
    from tests.test_gpu_operators import run_norm
    r = np.random.default_rng([32, H])
    x = (r.standard_normal((3, H)) * 1e-39).astype(np.float32)
    res = ref.bf16(r.standard_normal((3, H)) * 1e-39)
    res[1], x[2] = 0.0, -res[2]                          # sums that are subnormal, and exact zeros
    h = run_norm(x, res, None, "f32", "bf16")[0]
    same_bits(h, ref.bf16(x + res))
    assert np.array_equal(run_norm(x, res, None, "f32", "f32")[0], x + res)
