"""GPU tests of the way through the experts: moe_group_rows (whole numbers), the products grouped
by expert in both types and moe_combine_rows, against their 64-bit forms within the bounds of
fp8_ref; groups that are empty, ragged, or end inside a tile; rows that belong to no group."""
import numpy as np
import pytest

from quantized_expert_ffn_topk_amd import abi
from tests import fp8_ref as ref
from tests import operators_ref as oref
from tests.test_gpu_fp8 import (CANARY, DEV, DT, TDT, check_canary, check_linear, dev_rows, linear_inputs, np_of,
                                out_rows)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = ref.U


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


# ---------------------------------------------------------------------------
# grouping
# ---------------------------------------------------------------------------
def run_group(idx, E, stream=None):
    T, k = idx.shape
    it = ints(idx)
    outs = [torch.full((n + 8,), CANARY, dtype=torch.int32, device=DEV) for n in (E + 1, T * k, T * k)]
    torch.cuda.synchronize()
    abi.moe_group_rows(it, T, k, E, *outs, stream)
    torch.cuda.synchronize()
    o, r, p = (v.cpu().numpy() for v in outs)
    assert (o[E + 1:] == CANARY).all() and (p[T * k:] == CANARY).all()
    assert (r[o[E]:] == CANARY).all()
    return o[:E + 1], r[:o[E]], p[:T * k].reshape(T, k)


def check_group(idx, E):
    got, want = run_group(idx, E), ref.group(idx, E)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (16, 8, 256), (5, 3, 7), (64, 2, 64), (333, 6, 62), (1000, 32, 1024),
                                   (4096, 8, 256), (8192, 8, 5), (8193, 8, 5), (4097, 16, 1024), (40000, 7, 300)])
@pytest.mark.parametrize("stray", [False, True])
def test_grouping(T, k, E, stray):
    r = np.random.default_rng([1, T, k, E])
    idx = r.integers(0, E, (T, k)).astype(np.int32)
    if stray:
        at = r.random((T, k)) < 0.2
        idx[at] = r.choice([-1, -(1 << 31), E, E + 1, (1 << 31) - 1], at.sum())
    check_group(idx, E)


@pytest.mark.parametrize("T", [2000, 20000])
def test_grouping_of_one_expert_and_of_none(T):
    idx = np.full((T, 8), 3, np.int32)
    check_group(idx, 9)
    check_group(np.full((T, 8), -1, np.int32), 9)
    check_group(idx, 3)


def test_grouping_of_no_tokens_gives_offsets_of_zeros():
    o = torch.full((10,), CANARY, dtype=torch.int32, device=DEV)
    abi.moe_group_rows(None, 0, 4, 9, o, None, None)
    torch.cuda.synchronize()
    assert not o.any()


# ---------------------------------------------------------------------------
# grouped products
# ---------------------------------------------------------------------------
class Inputs:
    """x [R,K], weights [E,N,K] and groups of the given sizes; the first group starts at `lead`."""

    def __init__(self, seed, sizes, N, K, xd, gather, lead=0, behind=0):
        r = np.random.default_rng([seed, N, K, sum(sizes), len(sizes)])
        self.E, self.N, self.K, self.xd = len(sizes), N, K, xd
        self.offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + lead
        self.M = int(self.offsets[-1]) + behind
        self.lead = lead
        self.R = max(1, self.M // 3) if gather else self.M
        self.rows = r.integers(0, self.R, self.M).astype(np.int32) if gather else None
        kb, nb = ref.blocks(K), ref.blocks(N)
        if xd == "fp8":
            pool = ref.codes(r, 1 << 14)
            self.x, self.w = pool[r.integers(0, 1 << 14, (self.R, K))], pool[r.integers(0, 1 << 14, (self.E, N, K))]
            self.s = (2.0 ** r.uniform(-9, -6, (self.R, kb))).astype(np.float32)
            self.ws = (2.0 ** r.uniform(-14, -11, (self.E, nb, kb))).astype(np.float32)
            self.xv, self.wv = ref.scaled(self.x, self.s), ref.scaled_weights(self.w, self.ws)
        else:
            self.x = oref.bf16(r.standard_normal((self.R, K)))
            self.w = oref.bf16(0.1 * r.standard_normal((self.E, N, K)))
            self.s = self.ws = None
            self.xv, self.wv = self.x.astype(np.float64), self.w.astype(np.float64)

    def run(self, out, pad=0, shift=0, spad=0, offsets=None, rows=None, stream=None, M=None):
        E, N, K, M = self.E, self.N, self.K, self.M if M is None else M
        xt = dev_rows(self.x, TDT[self.xd], pad, shift)
        wt = dev_rows(self.w.reshape(E * N, K), TDT[self.xd], pad, shift)
        kb, nb = ref.blocks(K), ref.blocks(N)
        st = wst = None
        if self.xd == "fp8":
            st, wst = dev_rows(self.s, torch.float32, spad), dev_rows(self.ws.reshape(E * nb, kb), torch.float32, spad)
        flat, y = out_rows(M, N, TDT[out], pad, shift)
        ot = ints(self.offsets if offsets is None else offsets)
        rt = None if self.rows is None else ints(self.rows if rows is None else rows)
        torch.cuda.synchronize()
        abi.moe_grouped_linear(xt, DT[self.xd], K + pad, st, kb + spad, self.R, rt, ot, E, M, wt, K + pad, N * (K + pad), wst,
                               kb + spad, nb * (kb + spad), N, K, y, DT[out], N + pad, stream)
        torch.cuda.synchronize()
        check_canary(flat, M, N, pad, shift)
        return np_of(y[:, :N])

    def check(self, y, out):
        o = self.offsets
        unit_fp8 = self.xd == "fp8" and out == "bf16" and self.M > 12 * self.E
        assert (y[:self.lead] == CANARY).all() and (y[o[-1]:] == CANARY).all()
        for e in range(self.E):
            if o[e] == o[e + 1]:
                continue
            at = ref.some_rows(o[e + 1] - o[e], o[e])
            x = self.xv[self.rows[at] if self.rows is not None else at]
            lim = ref.limit(x, self.wv[e], 1 if self.xd == "fp8" else 2, out == "bf16", unit_fp8)
            off = np.abs(y[at] - x @ self.wv[e].T)
            assert (off <= lim).all(), (e, float((off - lim).max()))


FEW = [1, 0, 3, 0, 0, 8, 9, 2, 1, 17, 0]
SOME = [20, 0, 33, 1, 64, 16, 5]
MANY = [70, 0, 129, 1, 64, 200, 65]


@pytest.mark.parametrize("xd", ["fp8", "bf16"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes", [FEW, SOME, MANY, [5], [300]])
@pytest.mark.parametrize("N,K", [(33, 100), (130, 513)])
def test_grouped_sizes(xd, out, gather, sizes, N, K):
    c = Inputs(1, sizes, N, K, xd, gather)
    c.check(c.run(out), out)


# groups of every size up to more than a tile's 256 rows, of so many channels that the tiles are 256 wide (E4M3 to
# fp32: 128 x 256); rows on 16 bytes, on 4, and on single ones
@pytest.mark.parametrize("xd", ["fp8", "bf16"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("K,pad,shift", [(256, 0, 0), (1100, 4, 4), (200, 3, 1), (60, 4, 0)])
@pytest.mark.parametrize("mean", [30, 140])
def test_grouped_tiles(xd, out, K, pad, shift, mean):
    sizes = {30: [64, 0, 1, 65, 130, 10, 5, 3], 140: [64, 0, 128, 129, 192, 193, 256, 300, 1]}[mean] * 4
    c = Inputs(8, sizes, 2600, K, xd, mean == 30)
    c.check(c.run(out, pad, shift, pad), out)


# few blocks in all, in blocks of 8, 16 and 32 rows; the last of more rows to an expert
@pytest.mark.parametrize("xd", ["fp8", "bf16"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", [[1], [7], [60], [129], [500], [3, 0, 0], [90, 0, 1, 40], [2, 3, 1, 0, 1, 2, 4, 3], [0, 1000]])
@pytest.mark.parametrize("N,K", [(250, 1300), (62, 77)])
def test_grouped_few_blocks(xd, out, sizes, N, K):
    c = Inputs(12, sizes, N, K, xd, len(sizes) > 1)
    c.check(c.run(out, 4, 4, 4), out)


# groups of 13 to 24 rows on average
@pytest.mark.parametrize("xd", ["fp8", "bf16"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_grouped_of_some_rows(xd, out):
    c = Inputs(13, [20, 0, 33, 1, 64, 16, 5, 8] * 4, 1100, 600, xd, True)
    c.check(c.run(out), out)


# many rows to an expert, on 16 bytes and on single ones
@pytest.mark.parametrize("xd", ["fp8", "bf16"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("K,pad,shift", [(256, 0, 0), (300, 3, 1)])
def test_grouped_of_many_rows(xd, out, K, pad, shift):
    c = Inputs(14, [400, 0, 257, 900], 2600, K, xd, True)
    c.check(c.run(out, pad, shift, pad), out)


# rows on 4 bytes whose length is not of whole words: the last row's last word is partly behind it
@pytest.mark.parametrize("xd", ["fp8", "bf16"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("K,pad", [(515, 1), (127, 1), (3, 1)])
@pytest.mark.parametrize("N", [66, 2600])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_rows_that_end_inside_a_word(xd, out, K, pad, N, gather):
    c = Inputs(10, [64, 0, 1, 65, 130, 193, 300, 40] * 3, N, K, xd, gather)
    c.check(c.run(out, pad), out)


# a few rows to an expert, with weights so many that they are read past the cache
@pytest.mark.parametrize("sizes", [[1, 0, 3, 2] * 8, [9, 0, 17, 5] * 8])
def test_grouped_streams_of_many_weights(sizes):
    c = Inputs(9, sizes, 4000, 4200, "fp8", True)
    c.check(c.run("bf16"), "bf16")


@pytest.mark.parametrize("xd", ["fp8", "bf16"])
@pytest.mark.parametrize("sizes", [FEW, MANY])
@pytest.mark.parametrize("pad,shift,spad", [(16, 16, 4), (3, 1, 1), (8, 0, 0)])
def test_grouped_strides_and_alignment(xd, sizes, pad, shift, spad):
    c = Inputs(2, sizes, 66, 300, xd, True)
    c.check(c.run("bf16", pad, shift, spad), "bf16")


@pytest.mark.parametrize("xd", ["fp8", "bf16"])
@pytest.mark.parametrize("sizes", [[0, 2, 0], [0, 0, 40], [90, 0, 0], [0, 0, 0]])
def test_rows_outside_all_groups_stay(xd, sizes):
    c = Inputs(3, sizes, 40, 200, xd, False, lead=3, behind=90)
    c.check(c.run("f32"), "f32")


@pytest.mark.parametrize("xd", ["fp8", "bf16"])
@pytest.mark.parametrize("E", [64, 65, 256, 257, 600, 1024])
def test_grouped_with_many_experts(xd, E):
    r = np.random.default_rng([4, E])
    sizes = r.choice([0, 0, 1, 2, 5, 11], E).tolist()
    c = Inputs(4, sizes, 17, 40, xd, True)
    c.check(c.run("bf16"), "bf16")
    sizes = r.choice([0, 0, 70, 130], E // 8).tolist() + [0] * (E - E // 8 - 1) + [75]
    c = Inputs(4, sizes, 17, 40, xd, True)
    c.check(c.run("f32"), "f32")


@pytest.mark.parametrize("xd", ["fp8", "bf16"])
def test_lists_that_are_none_touch_nothing_outside(xd):
    """Offsets and rows of any content: nothing outside of out's rows is written (the canaries), nothing
    outside of x is read (its end is its allocation's)."""
    c = Inputs(5, FEW, 40, 200, xd, True)
    r = np.random.default_rng(6)
    for _ in range(4):
        wild = r.choice([-(1 << 31), -1, 0, 5, c.M, c.M + 1, (1 << 31) - 1], c.E + 1)
        c.run("bf16", offsets=wild, rows=r.choice([-(1 << 31), -1, c.R, (1 << 31) - 1], c.M))


def test_grouped_on_a_side_stream_and_captured():
    c = Inputs(7, MANY, 130, 513, "fp8", True)
    want = c.run("bf16")
    assert np.array_equal(c.run("bf16", stream=torch.cuda.Stream()), want)
    xt, wt = dev_rows(c.x, torch.uint8), dev_rows(c.w.reshape(-1, c.K), torch.uint8)
    st, wst = torch.from_numpy(c.s).to(DEV), torch.from_numpy(c.ws).to(DEV)
    y = torch.zeros((c.M, c.N), dtype=torch.bfloat16, device=DEV)
    ot, rt = ints(c.offsets), ints(c.rows)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        abi.moe_grouped_linear(xt, abi.DT_FP8, c.K, st, 5, c.R, rt, ot, c.E, c.M, wt, c.K, c.N * c.K, wst, 5, 10, c.N, c.K, y,
                               abi.DT_BF16, c.N, torch.cuda.current_stream())
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(np_of(y), want)
    # other groups in the same arrays: a replay goes by what they hold then
    sizes = MANY[::-1]
    d = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    ot.copy_(ints(d))
    y.fill_(CANARY)
    g.replay()
    torch.cuda.synchronize()
    c.offsets = d
    c.check(np_of(y), "bf16")


# ---------------------------------------------------------------------------
# combining
# ---------------------------------------------------------------------------
def run_combine(y, yd, pos, w, base, out, pad=0, shift=0, in_place=False):
    T, k = pos.shape
    H = y.shape[1]
    yt = dev_rows(y, TDT[yd], pad, shift)
    flat, o = out_rows(T, H, TDT[out], pad, shift)
    bt = None if base is None else dev_rows(base, TDT[out], pad, shift)
    if in_place:
        o[:, :H].copy_(bt)
        bt = o
    pt, wt = ints(pos), torch.from_numpy(w).to(DEV)
    torch.cuda.synchronize()
    abi.moe_combine_rows(yt, DT[yd], H + pad, y.shape[0], pt, wt, bt, H + pad, T, k, H, o, DT[out], H + pad)
    torch.cuda.synchronize()
    check_canary(flat, T, H, pad, shift)
    return np_of(o[:, :H])


@pytest.mark.parametrize("yd,out", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,k,H,pad,shift", [(1, 8, 6144, 0, 0), (1, 1, 1, 0, 0), (3, 3, 7, 3, 1), (5, 32, 8, 0, 0), (20, 6, 513, 8, 8),
                                             (300, 2, 1000, 1, 3), (70000, 1, 9, 0, 0)])
@pytest.mark.parametrize("base", [None, "own", "out"])
def test_combine(yd, out, T, k, H, pad, shift, base):
    r = np.random.default_rng([8, T, k, H])
    R = T * k
    rnd = {"f32": lambda a: a.astype(np.float32), "bf16": oref.bf16}
    y = rnd[yd](r.standard_normal((R, H)))
    pos = r.permutation(R).reshape(T, k).astype(np.int32)
    stray = r.random((T, k)) < 0.1
    pos[stray] = r.choice([-1, R, -(1 << 31), (1 << 31) - 1], stray.sum())
    w = r.random((T, k)).astype(np.float32)
    b = None if base is None else rnd[out](r.standard_normal((T, H)))
    got = run_combine(y, yd, pos, w, b, out, pad, shift, base == "out")
    terms = np.where(stray[:, :, None], 0.0, w[:, :, None].astype(np.float64) * y[np.where(stray, 0, pos)])
    want = terms.sum(axis=1) + (0 if b is None else b)
    # k FMAs round the running sum
    lim = k * U * (np.abs(terms).sum(axis=1) + (0 if b is None else np.abs(b))) + 1e-37
    if out == "bf16":
        lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= lim).all()


def test_combine_passes_over_rows_that_nobody_wrote():
    """NaN in a row of y that no pos names, or in one whose place is outside, does not reach out."""
    y = np.full((4, 16), np.nan, np.float32)
    y[1] = 2.0
    pos = np.array([[1, -1], [4, 1]], np.int32)
    got = run_combine(y, "f32", pos, np.array([[0.5, 9.0], [9.0, 1.5]], np.float32), None, "f32")
    assert np.array_equal(got, np.repeat([[1.0], [3.0]], 16, axis=1).astype(np.float32))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 5, 100])
def test_a_run_through_the_experts(T):
    """Codes, grouping, gate and up, SwiGLU codes behind the groups' count, down, combine: every step against
    the 64-bit form of what the step before gave; some ids are no experts."""
    r = np.random.default_rng([9, T])
    H, F, E, k = 300, 200, 12, 4
    x = oref.bf16(r.standard_normal((T, H)))
    idx = np.argsort(r.random((T, E + 2)), axis=1)[:, :k].astype(np.int32)     # ids of 12 and 13 have no expert
    gate = r.random((T, k)).astype(np.float32)
    hb, fb = ref.blocks(H), ref.blocks(F)
    gu, dn = ref.codes(r, E, 2 * F, H), ref.codes(r, E, H, F)
    gus = (2.0 ** r.uniform(-13, -12, (E, ref.blocks(2 * F), hb))).astype(np.float32)
    dns = (2.0 ** r.uniform(-13, -12, (E, hb, fb))).astype(np.float32)
    M = T * k
    new = lambda *a, dt=torch.float32: torch.full(a, CANARY, dtype=dt, device=DEV)  # noqa: E731
    q, s = new(T, H, dt=torch.uint8), new(T, hb)
    off, rows, pos = new(E + 1, dt=torch.int32), new(M, dt=torch.int32), new(M, dt=torch.int32)
    h, qh, sh = new(M, 2 * F, dt=torch.bfloat16), new(M, F, dt=torch.uint8), new(M, fb)
    y, out = new(M, H, dt=torch.bfloat16), new(T, H)
    dev = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    xt, it, gt, gut, gust, dnt, dnst = dev(x).bfloat16(), ints(idx), dev(gate), dev(gu), dev(gus), dev(dn), dev(dns)
    torch.cuda.synchronize()
    abi.moe_quant_fp8(xt, abi.DT_BF16, H, abi.ACT_NONE, T, H, None, q, H, s, hb)
    abi.moe_group_rows(it, T, k, E, off, rows, pos)
    abi.moe_grouped_linear(q, abi.DT_FP8, H, s, hb, T, rows, off, E, M, gut, H, 2 * F * H, gust, hb, ref.blocks(2 * F) * hb,
                           2 * F, H, h, abi.DT_BF16, 2 * F)
    abi.moe_quant_fp8(h, abi.DT_BF16, 2 * F, abi.ACT_SWIGLU, M, F, off[E:], qh, F, sh, fb)
    abi.moe_grouped_linear(qh, abi.DT_FP8, F, sh, fb, M, None, off, E, M, dnt, F, H * F, dnst, fb, hb * fb, H, F, y,
                           abi.DT_BF16, H)
    abi.moe_combine_rows(y, abi.DT_BF16, H, M, pos, gt, None, 0, T, k, H, out, abi.DT_F32, H)
    torch.cuda.synchronize()
    o, rw, p = ref.group(idx, E)
    n = o[-1]
    assert np.array_equal(off.cpu().numpy(), o) and np.array_equal(rows.cpu().numpy()[:n], rw)
    assert np.array_equal(pos.cpu().numpy().reshape(T, k), p)
    assert np.array_equal(q.cpu().numpy(), ref.quant(x)[0])
    xv = ref.scaled(*ref.quant(x))[rw]
    hv, yv = np_of(h), np_of(y)
    assert (hv[n:] == CANARY).all() and (yv[n:] == CANARY).all() and (qh.cpu().numpy()[n:] == CANARY).all()
    qv = ref.scaled(qh.cpu().numpy(), sh.cpu().numpy())
    act = oref.swiglu(hv[:n])
    step = np.maximum(np.abs(act) * 2.0 ** -4, ref.spread(ref.block_max(act), F) / 448 * 2.0 ** -10)
    assert (np.abs(qv[:n] - act) <= step * (1 + 2.0 ** -10) + 60 * U * ref.spread(ref.block_max(act), F)).all()
    for e in range(E):
        a, b = o[e], o[e + 1]
        if a < b:
            for got, v, w in ((hv, xv, ref.scaled_weights(gu[e], gus[e])), (yv, qv, ref.scaled_weights(dn[e], dns[e]))):
                assert (np.abs(got[a:b] - v[a:b] @ w.T) <= ref.limit(v[a:b], w, 1, True, True)).all()
    terms = np.where(p[:, :, None] < 0, 0.0, gate[:, :, None].astype(np.float64) * yv[np.maximum(p, 0)])
    assert (np.abs(out.cpu().numpy() - terms.sum(axis=1)) <= k * U * np.abs(terms).sum(axis=1) + 1e-37).all()


# ---------------------------------------------------------------------------
# rows far apart: offsets that pass 32 bits, in bytes and in elements
# ---------------------------------------------------------------------------
def far(n, row, dtype, ld, fill=0):
    """[n, row] on the device, `ld` elements from one to the next."""
    flat = torch.full(((n - 1) * ld + row,), fill, dtype=dtype, device=DEV)
    return flat.as_strided((n, row), (ld, 1))


def on(view, a):
    view.copy_(torch.from_numpy(np.ascontiguousarray(a)))
    return view


# distances that copies by the load unit reach (up to 2^23 bytes between rows) and that they do not
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,ld", [(3, (1 << 31) + 4), (600, 1 << 22), (300, (1 << 23) + 4)])
def test_linear_of_rows_far_apart(out, T, ld):
    N, K = 150, 300
    q, s, w, ws, bias = linear_inputs(13, T, N, K)
    lds, ldo = (1 << 21) if T < 600 else 1 << 20, (1 << 30) + 2 if T == 3 else 1 << 22
    qt = on(far(T, K, torch.uint8, ld), q)
    st, wst = on(far(T, 3, torch.float32, lds), s), on(far(2, 3, torch.float32, 1 << 30), ws)
    wt = on(far(N, K, torch.uint8, ld if T == 600 else 1 << 24), w)
    y = far(T, N, TDT[out], ldo)
    torch.cuda.synchronize()
    abi.moe_linear_fp8(qt, ld, st, lds, T, wt, ld if T == 600 else 1 << 24, wst, 1 << 30, torch.from_numpy(bias).to(DEV), N, K, y,
                       DT[out], ldo)
    torch.cuda.synchronize()
    check_linear(np_of(y), q, s, w, ws, bias, out)


# R*ldx up to 2^31 is copied by the load unit, more is not; experts and rows of out lie further apart than 2^32 elements
@pytest.mark.parametrize("sizes", [[2, 1, 3], [40, 0, 70], [300, 0, 290]])
@pytest.mark.parametrize("ld", [1 << 20, 1 << 24])
def test_grouped_of_rows_far_apart(sizes, ld):
    c = Inputs(11, sizes, 150, 300, "fp8", True)
    stride, sstride, ldo = (1 << 32) + 4, (1 << 30) + 1, max(1 << 23, ((1 << 32) // c.M) & ~1)
    lds = (1 << 29) // c.R
    xt, st = on(far(c.R, c.K, torch.uint8, ld), c.x), on(far(c.R, 3, torch.float32, lds), c.s)
    wt, wst = far(c.E, c.N * c.K, torch.uint8, stride), far(c.E, 6, torch.float32, sstride)
    on(wt, c.w.reshape(c.E, -1)), on(wst, c.ws.reshape(c.E, -1))
    y = far(c.M, c.N, torch.bfloat16, ldo)
    ot, rt = ints(c.offsets), ints(c.rows)
    torch.cuda.synchronize()
    abi.moe_grouped_linear(xt, abi.DT_FP8, ld, st, lds, c.R, rt, ot, c.E, c.M, wt, c.K, stride, wst, 3, sstride, c.N, c.K, y,
                           abi.DT_BF16, ldo)
    torch.cuda.synchronize()
    c.check(np_of(y), "bf16")


def test_rows_and_combine_far_apart():
    T, K, ld = 5, 300, (1 << 30) + 1
    x = oref.bf16(np.random.default_rng(12).standard_normal((T, K)))
    xt, q, s = on(far(T, K, torch.bfloat16, ld), x), far(T, K, torch.uint8, ld), far(T, 3, torch.float32, ld)
    torch.cuda.synchronize()
    abi.moe_quant_fp8(xt, abi.DT_BF16, ld, abi.ACT_NONE, T, K, None, q, ld, s, ld)
    torch.cuda.synchronize()
    qw, sw = ref.quant(x)
    assert np.array_equal(np_of(q), qw) and np.array_equal(np_of(s), sw)
    del q, s
    y = far(T, K, torch.bfloat16, ld)
    torch.cuda.synchronize()
    abi.moe_combine_rows(xt, abi.DT_BF16, ld, T, ints(np.arange(T)[::-1]), torch.full((T,), 2.0, device=DEV), xt, ld, T, 1, K, y,
                         abi.DT_BF16, ld)
    torch.cuda.synchronize()
    want = oref.bf16((x + 2 * x[::-1]).astype(np.float32))          # exact in fp32 but for far exponents: one rounding
    assert (np.abs(np_of(y) - want) <= 2.0 ** -8 * np.abs(want)).all()
