"""Plain 64-bit forms of the operators around the MoE layer, in numpy, and the
inputs of their tests.  Formulas only: no kernel's order of summation, no
fp32 steps except where the operator's definition names them (the epilogue of
the int8 product)."""
import numpy as np

from quantized_expert_ffn_topk_amd import synth


def bf16(a):
    """fp32/64 values rounded to bf16, as fp32."""
    return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(np.asarray(a, np.float32)))


def rmsnorm(x, res, gamma, eps):
    h = np.asarray(x, np.float64) + (0.0 if res is None else np.asarray(res, np.float64))
    with np.errstate(invalid="ignore"):
        v = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + float(np.float32(eps)))
    return h, v if gamma is None else v * np.asarray(gamma, np.float64)


def swiglu(gu):
    gu = np.asarray(gu, np.float64)
    F = gu.shape[1] // 2
    g, u = gu[:, :F], gu[:, F:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def check_codes(q, s, v, tol):
    """Codes and scales of rows v (fp64): s within tol of max|v|/127, every code
    within half a step (and 127*2*tol for the fp32 rounding of the value and of
    the multiplier) of v/s."""
    amax = np.abs(v).max(axis=1)
    np.testing.assert_allclose(s, amax / 127.0, rtol=tol, atol=2e-45)
    safe = np.where(amax > 0, amax, 1.0)
    off = np.abs(q.astype(np.float64) - v * (127.0 / safe)[:, None])
    assert off.max() <= 0.5 + 127 * 2 * tol, off.max()
    assert np.abs(q.astype(np.int32)).max() <= 127
    assert not q[amax == 0].any()


def linear(q, s, w, ws, bias):
    """The definition, with its fp32 epilogue: bits are defined.  (fp64 products
    and sums of codes are whole numbers far below 2^53: exact.)"""
    acc = q.astype(np.float64) @ w.astype(np.float64).T
    assert np.abs(acc).max(initial=0) < 2 ** 31
    y = acc.astype(np.float32) * s.astype(np.float32)[:, None] * ws.astype(np.float32)
    return y if bias is None else y + bias.astype(np.float32)


def scores(logits, softmax):
    l = np.asarray(logits, np.float64)
    nan = np.isnan(l)
    if not softmax:
        with np.errstate(over="ignore"):
            p = 1.0 / (1.0 + np.exp(-l))
        return np.where(nan, 0.0, p)
    m = np.where(nan, -np.inf, l).max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(m == np.inf, (l == np.inf) * 1.0, np.exp(l - m))
    e = np.where(nan | (l == -np.inf), 0.0, e)
    t = e.sum(axis=1, keepdims=True)
    return np.where(t > 0, e / np.where(t > 0, t, 1.0), 0.0)


def select(logits, bias, k, softmax, n_group, topk_group, group_best, renorm, scale):
    """(idx, w, margin): margin is the smallest nonzero difference of two
    neighbours in a ranking that the choice goes by, relative to the row's
    largest value -- where it is below fp32's errors the choice is open."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    p = scores(l, softmax)
    c = p + (0.0 if bias is None else np.asarray(bias, np.float64))
    c = np.where(np.isnan(l) | np.isnan(c), -np.inf, c)
    gs = E // n_group
    idx = np.zeros((T, k), np.int32)
    w = np.zeros((T, k))
    margin = np.inf

    def gaps(v, big):
        v = v[np.isfinite(v)]
        d = -np.diff(v)
        d = d[d > 0]
        return (d.min() / big) if d.size and big > 0 else np.inf

    for t in range(T):
        ct = c[t].copy()
        fin = np.abs(ct[np.isfinite(ct)])
        big = fin.max() if fin.size else 0.0
        if topk_group < n_group:
            top = -np.sort(-ct.reshape(n_group, gs), axis=1)[:, :group_best]
            with np.errstate(invalid="ignore"):
                score = top.sum(axis=1)
            score = np.where(np.isnan(score), -np.inf, score)
            order = np.lexsort((np.arange(n_group), -score))
            margin = min(margin, gaps(score[order], big))
            keep = np.zeros(n_group, bool)
            keep[order[:topk_group]] = True
            allowed = np.repeat(keep, gs)
        else:
            allowed = np.ones(E, bool)
        cand = np.flatnonzero(allowed)
        order = cand[np.lexsort((cand, -ct[cand]))]
        margin = min(margin, gaps(ct[order[:k + 1]], big))
        idx[t] = order[:k]
        w[t] = p[t, idx[t]]
        if renorm:
            den = w[t].sum()
            w[t] = w[t] / den if den > 0 else 0.0
    return idx, w * float(np.float32(scale)), margin
