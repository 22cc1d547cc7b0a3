"""GPU tests of the operators around the MoE layer through the C ABI: the RMS
norm with residual and int8 output, SwiGLU with int8 output, the int8 product,
and the selection of experts with groups, each against its plain 64-bit form.

Tolerances.  u = 2^-24 is half a unit in the last place of fp32's 24 bits, 2^-8
of bf16's 8.  A norm value takes an addition, a rounded 1/sqrt and two products:
under 6u of itself; SwiGLU takes the hardware's exp2 and reciprocal (one unit,
2u, each), a remainder and four products: under 16u.  Scales add a maximum
(exact) and a division."""
import numpy as np
import pytest

from quantized_expert_ffn_topk_amd import abi, synth
from tests import operators_ref as ref
from tests.gpu_common import Case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda"
U = 2.0 ** -24
NORM_TOL, SWIGLU_TOL = 8 * U, 20 * U
DT = {"f32": abi.DT_F32, "bf16": abi.DT_BF16}
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
CANARY = 77


def dev_rows(a, dtype, pad=0, shift=0):
    """a [T,n] on the device as `dtype`, rows `pad` apart beyond their length,
    `shift` elements into an allocation."""
    T, n = a.shape
    flat = torch.zeros(T * (n + pad) + shift, dtype=dtype, device=DEV)
    v = flat[shift:].view(T, n + pad)[:, :n]
    v.copy_(torch.from_numpy(np.ascontiguousarray(a)))
    return v


def out_rows(T, n, dtype, pad=0, shift=0):
    flat = torch.full((T * (n + pad) + shift + 64,), CANARY, dtype=dtype, device=DEV)
    return flat, flat[shift:shift + T * (n + pad)].view(T, n + pad)


def check_canary(flat, T, n, pad, shift):
    f = flat.float().cpu().numpy()
    body = f[shift:shift + T * (n + pad)].reshape(T, n + pad)
    assert (f[:shift] == CANARY).all() and (f[shift + T * (n + pad):] == CANARY).all()
    assert (body[:, n:] == CANARY).all()


def np_of(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


def check_bf16(got, want, tol):
    lim = np.abs(want) * (2.0 ** -8 + 2 * tol) + 1e-37
    assert (np.abs(got.astype(np.float64) - want) <= lim).all(), \
        float((np.abs(got - want) - lim).max())


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------
def run_norm(x, res, gamma, xd, rd, eps=1e-6, pad=0, shift=0, in_place=False, stream=None):
    T, H = x.shape
    xt = dev_rows(x, TDT[xd], pad, shift)
    rt = None if res is None else dev_rows(res, TDT[rd], pad, shift)
    gt = None if gamma is None else torch.from_numpy(gamma.astype(np.float32)).to(DEV)
    hf, h = out_rows(T, H, TDT[rd], pad, shift)
    yf, y = out_rows(T, H, torch.bfloat16, pad, shift)
    qf, q = out_rows(T, H, torch.int8, pad, shift)
    s = torch.full((T + 1,), float(CANARY), device=DEV)
    ld = H + pad
    torch.cuda.synchronize()
    abi.moe_rmsnorm_quant(xt, DT[xd], ld, rt, DT[rd], ld, gt, T, H, eps, rt if in_place else h, ld,
                          y, ld, q, ld, s, stream)
    torch.cuda.synchronize()
    for flat in ((yf, qf) if in_place else (hf, yf, qf)):
        check_canary(flat, T, H, pad, shift)
    assert float(s[T]) == CANARY
    hv = rt if in_place else h[:, :H]
    return np_of(hv), np_of(y[:, :H]), q[:, :H].cpu().numpy(), s[:T].cpu().numpy()


def norm_inputs(seed, T, H, xd, rd):
    r = np.random.default_rng([seed, T, H])
    x, res = r.standard_normal((T, H)), 3 * r.standard_normal((T, H))
    res[:, ::97] *= 20
    rnd = {"f32": lambda a: a.astype(np.float32), "bf16": ref.bf16}
    return rnd[xd](x), rnd[rd](res), (1 + 0.1 * r.standard_normal(H)).astype(np.float32)


def check_norm(out, x, res, gamma, rd, eps=1e-6):
    h, y, q, s = out
    hw, vw = ref.rmsnorm(x, res, gamma, eps)
    if rd == "f32":
        np.testing.assert_allclose(h, hw, rtol=U * 1.001, atol=0)
    else:
        check_bf16(h, hw, U)
    check_bf16(y, vw, NORM_TOL)
    ref.check_codes(q, s, vw, NORM_TOL)


@pytest.mark.parametrize("H", [1, 2, 7, 8, 9, 63, 64, 65, 511, 512, 513, 1000, 2047, 2048, 2049,
                               6144, 7001, 8192, 8193, 16385, 32768, 32769, 40003])
@pytest.mark.parametrize("xd,rd", [("bf16", "bf16"), ("f32", "bf16")])
def test_norm_widths(H, xd, rd):
    x, res, gamma = norm_inputs(1, 5, H, xd, rd)
    check_norm(run_norm(x, res, gamma, xd, rd), x, res, gamma, rd)


# on both sides of each length at which a row gets other threads
@pytest.mark.parametrize("H", [1024, 1025, 3328, 3329, 4096, 4097, 6145, 12288, 12289, 16384, 24576, 24577])
@pytest.mark.parametrize("xd,rd", [("bf16", "bf16"), ("f32", "f32")])
def test_norm_widths_between_shapes(H, xd, rd):
    x, res, gamma = norm_inputs(2, 5, H, xd, rd)
    check_norm(run_norm(x, res, gamma, xd, rd), x, res, gamma, rd)


@pytest.mark.parametrize("T", [1, 3, 4, 257])
@pytest.mark.parametrize("xd,rd", [("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (3, 1)])
def test_norm_tokens_strides_and_alignment(T, xd, rd, pad, shift):
    for H in (100, 2050):
        x, res, gamma = norm_inputs(2, T, H, xd, rd)
        check_norm(run_norm(x, res, gamma, xd, rd, pad=pad, shift=shift), x, res, gamma, rd)


@pytest.mark.parametrize("H", [5, 1003, 6145, 33000])
def test_norm_in_place_and_without_residual_or_gamma(H):
    x, res, gamma = norm_inputs(3, 6, H, "bf16", "bf16")
    check_norm(run_norm(x, res, gamma, "bf16", "bf16", in_place=True), x, res, gamma, "bf16")
    check_norm(run_norm(x, None, None, "bf16", "bf16"), x, None, None, "bf16")


def test_norm_each_output_alone_has_the_same_bits():
    T, H = 9, 1537
    x, res, gamma = norm_inputs(4, T, H, "bf16", "bf16")
    h0, y0, q0, s0 = run_norm(x, res, gamma, "bf16", "bf16")
    xt, rt = dev_rows(x, torch.bfloat16), dev_rows(res, torch.bfloat16)
    gt = torch.from_numpy(gamma).to(DEV)
    h, y = torch.empty_like(xt), torch.empty_like(xt)
    q, s = torch.empty((T, H), dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    args = (xt, abi.DT_BF16, H, rt, abi.DT_BF16, H, gt, T, H, 1e-6)
    abi.moe_rmsnorm_quant(*args, h, H, None, 0, None, 0, None)
    abi.moe_rmsnorm_quant(*args, None, 0, y, H, None, 0, None)
    abi.moe_rmsnorm_quant(*args, None, 0, None, 0, q, H, s)
    torch.cuda.synchronize()
    assert np.array_equal(np_of(h), h0) and np.array_equal(np_of(y), y0)
    assert np.array_equal(q.cpu().numpy(), q0) and np.array_equal(s.cpu().numpy(), s0)


@pytest.mark.parametrize("H", [6, 300, 6144, 33001])
def test_norm_rows_of_zeros_extremes_and_non_finite_values(H):
    x = np.zeros((8, H), np.float32)
    r = np.random.default_rng(5)
    x[1] = 1e-30 * r.standard_normal(H)                 # codes of a row far below eps
    x[2] = 1e30 * r.standard_normal(H)                  # squares beyond fp32
    x[3] = r.standard_normal(H)
    x[3, H // 2] = np.inf
    x[4] = r.standard_normal(H)
    x[4, H - 1] = np.nan
    x[5] = 3e38
    x[6, 0] = 1e-42                                     # a lone subnormal
    x[7] = -2.5
    h, y, q, s = run_norm(x, None, None, "f32", "f32")
    _, v = ref.rmsnorm(x, None, None, 1e-6)
    good = [0, 1, 2, 5, 6, 7]
    assert not q[0].any() and s[0] == 0 and not y[0].any()
    ref.check_codes(q[[1, 2, 5, 7]], s[[1, 2, 5, 7]], v[[1, 2, 5, 7]], NORM_TOL)
    # a value of 1e-39 is a subnormal: s keeps what bits it has, the code is whole
    assert q[6, 0] == 127 and not q[6, 1:].any() and abs(s[6] * 127 - v[6, 0]) <= 127 * 1.5e-45
    check_bf16(y[[1, 2, 5, 7]], v[[1, 2, 5, 7]], NORM_TOL)
    for t in (3, 4):
        assert np.isnan(s[t]) and not q[t].any()
    assert np.isnan(y[3]).any() and np.isnan(y[4]).any()
    assert np.array_equal(h[good], x[good])


# ---------------------------------------------------------------------------
# SwiGLU
# ---------------------------------------------------------------------------
def run_swiglu(gu, dt, pad=0, shift=0):
    T, F = gu.shape[0], gu.shape[1] // 2
    gt = dev_rows(gu, TDT[dt], pad, shift)
    yf, y = out_rows(T, F, torch.bfloat16, pad, shift)
    qf, q = out_rows(T, F, torch.int8, pad, shift)
    s = torch.full((T + 1,), float(CANARY), device=DEV)
    torch.cuda.synchronize()
    abi.moe_swiglu_quant(gt, DT[dt], 2 * F + pad, T, F, y, F + pad, q, F + pad, s)
    torch.cuda.synchronize()
    check_canary(yf, T, F, pad, shift)
    check_canary(qf, T, F, pad, shift)
    assert float(s[T]) == CANARY
    return np_of(y[:, :F]), q[:, :F].cpu().numpy(), s[:T].cpu().numpy()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,F,pad,shift", [(1, 1, 0, 0), (4, 7, 0, 0), (5, 8, 3, 1), (3, 513, 1, 3),
                                           (2, 2048, 0, 0), (6, 2049, 8, 8), (1, 12288, 0, 0),
                                           (3, 18431, 3, 1), (2, 32771, 0, 0)])
def test_swiglu(dt, T, F, pad, shift):
    r = np.random.default_rng([7, T, F])
    gu = (3 * r.standard_normal((T, 2 * F))).astype(np.float32)
    gu = ref.bf16(gu) if dt == "bf16" else gu
    y, q, s = run_swiglu(gu, dt, pad, shift)
    v = ref.swiglu(gu)
    check_bf16(y, v, SWIGLU_TOL)
    ref.check_codes(q, s, v, SWIGLU_TOL)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("F", [512, 1024, 1025, 3328, 3329, 4096, 4097, 6145, 8192, 8193, 12289, 16385, 24577])
def test_swiglu_widths_between_shapes(dt, F):
    test_swiglu(dt, 5, F, 3, 1)


@pytest.mark.parametrize("F", [40, 33003])
def test_swiglu_extremes(F):
    gu = np.zeros((6, 2 * F), np.float32)
    gu[1, :F], gu[1, F:] = np.linspace(-120, 120, F), 1.0        # the whole range of exp
    gu[2, :F], gu[2, F:] = -1e4, 1e4                             # exp(-g) overflows: 0
    gu[3, :F], gu[3, F:] = 1e20, 1e-15
    gu[4, :F], gu[4, F:] = 1.0, 1.0
    gu[4, F + 3] = np.inf
    gu[5, 2] = np.nan
    y, q, s = run_swiglu(gu, "f32")
    v = ref.swiglu(gu)
    ref.check_codes(q[:4], s[:4], v[:4], SWIGLU_TOL)
    check_bf16(y[:4], v[:4], SWIGLU_TOL)
    for t in (4, 5):
        assert np.isnan(s[t]) and not q[t].any()


# ---------------------------------------------------------------------------
# int8 product
# ---------------------------------------------------------------------------
def lin_inputs(seed, T, N, K):
    r = np.random.default_rng([seed, T, N, K])
    q = r.integers(-128, 128, (T, K)).astype(np.int8)
    w = r.integers(-128, 128, (N, K)).astype(np.int8)
    return (q, (0.01 + r.random(T)).astype(np.float32), w, (0.01 + r.random(N)).astype(np.float32),
            r.standard_normal(N).astype(np.float32))


def run_linear(q, s, w, ws, bias, od, pad=0, shift=0, stream=None):
    (T, K), N = q.shape, w.shape[0]
    qt, wt = dev_rows(q, torch.int8, pad, shift), dev_rows(w, torch.int8, pad, shift)
    st, wst = torch.from_numpy(s).to(DEV), torch.from_numpy(ws).to(DEV)
    bt = None if bias is None else torch.from_numpy(bias).to(DEV)
    of, o = out_rows(T, N, TDT[od], pad, shift)
    torch.cuda.synchronize()
    abi.moe_linear_int8(qt, K + pad, st, T, wt, K + pad, wst, bt, N, K, o, DT[od], N + pad, stream)
    torch.cuda.synchronize()
    check_canary(of, T, N, pad, shift)
    return np_of(o[:, :N])


def check_linear(got, q, s, w, ws, bias, od):
    want = ref.linear(q, s, w, ws, bias)
    want = ref.bf16(want) if od == "bf16" else want
    assert np.array_equal(got.astype(np.float32).view(np.uint32), want.view(np.uint32)), \
        int((got != want).sum())


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 64, 65, 127, 128, 200, 257])
@pytest.mark.parametrize("N,K", [(1, 1), (5, 15), (16, 16), (33, 17), (64, 64), (130, 200), (257, 512),
                                 (320, 1040), (100, 6144)])
def test_linear_shapes(T, N, K):
    q, s, w, ws, b = lin_inputs(1, T, N, K)
    check_linear(run_linear(q, s, w, ws, None, "f32"), q, s, w, ws, None, "f32")
    check_linear(run_linear(q, s, w, ws, b, "bf16"), q, s, w, ws, b, "bf16")


@pytest.mark.parametrize("T,N,K", [(1, 70, 333), (3, 129, 1024), (40, 65, 2047), (130, 200, 129),
                                   (300, 300, 768)])
@pytest.mark.parametrize("pad,shift", [(16, 16), (16, 3), (3, 0), (1, 5)])
def test_linear_strides_and_alignment(T, N, K, pad, shift):
    q, s, w, ws, b = lin_inputs(2, T, N, K)
    check_linear(run_linear(q, s, w, ws, b, "f32", pad, shift), q, s, w, ws, b, "f32")
    check_linear(run_linear(q, s, w, ws, None, "bf16", pad, shift), q, s, w, ws, None, "bf16")


@pytest.mark.parametrize("T,N,K", [(513, 1030, 512), (1024, 768, 2048), (700, 2600, 272),
                                   (2050, 520, 1088)])
def test_linear_many_tokens(T, N, K):
    q, s, w, ws, b = lin_inputs(3, T, N, K)
    check_linear(run_linear(q, s, w, ws, b, "bf16"), q, s, w, ws, b, "bf16")
    check_linear(run_linear(q, s, w, ws, None, "f32"), q, s, w, ws, None, "f32")


@pytest.mark.parametrize("T,N,K", [(513, 1030, 512), (200, 5003, 384), (384, 6144, 2050), (1999, 2001, 1040),
                                   (2047, 4090, 640), (4001, 4093, 520)])
@pytest.mark.parametrize("pad", [0, 16, 3])
def test_linear_every_tile_and_alignment(T, N, K, pad):
    # shapes that spread over the chip as 64 x 64, 64 x 128, 128 x 128, 128 x 256
    # and 256 x 256 tiles, whole and partial stages, aligned rows and others
    q, s, w, ws, b = lin_inputs(6, T, N, K)
    check_linear(run_linear(q, s, w, ws, b, "bf16", pad), q, s, w, ws, b, "bf16")
    check_linear(run_linear(q, s, w, ws, None, "f32", pad), q, s, w, ws, None, "f32")


# shapes that fill the chip best as 64 x 64, 64 x 128 or (longer K) 96 x 128,
# 192 x 128, 128 x 256, 192 x 256, 256 x 256 and 128 x 128 tiles, with every
# remainder of the stages' count that the kernels' rounds distinguish
@pytest.mark.parametrize("T,N,K", [(T, N, K) for T, N in ((66, 4170), (259, 6579))
                                   for K in (100, 256, 384, 520, 640, 768, 896, 1032, 1152, 1300, 1664)] +
                         [(T, N, K) for T, N in ((516, 7243), (780, 6620), (1030, 7200), (1545, 7250))
                          for K in (272, 640, 1032)] + [(110, 20001, K) for K in (4112, 4480, 4608)])
@pytest.mark.parametrize("pad", [0, 3])
def test_linear_tiles_at_every_count_of_stages(T, N, K, pad):
    q, s, w, ws, b = lin_inputs(9, T, N, K)
    od = "bf16" if K % 256 else "f32"
    check_linear(run_linear(q, s, w, ws, b, od, pad), q, s, w, ws, b, od)


# weights split among 4, 8 and 16 waves, in 16, 32 and 48 rows; tokens in 8, 16,
# 32 and 64, also more of them than one block takes; and as tiles
@pytest.mark.parametrize("T,N,K", [(5, 9001, 1100), (6, 13001, 1100), (13, 13001, 1100), (30, 13001, 1100), (33, 9001, 1100),
                                   (1, 4096, 1100), (8, 4100, 6100), (16, 9001, 1500), (32, 9001, 1500), (100, 300, 4500),
                                   (70, 1999, 1500), (100, 2500, 1500), (500, 700, 1500), (210, 1900, 1500)])
@pytest.mark.parametrize("pad", [0, 3])
def test_linear_splits_of_a_weight_stream(T, N, K, pad):
    q, s, w, ws, b = lin_inputs(10, T, N, K)
    check_linear(run_linear(q, s, w, ws, b, "bf16", pad), q, s, w, ws, b, "bf16")
    check_linear(run_linear(q, s, w, ws, None, "f32", pad), q, s, w, ws, None, "f32")


@pytest.mark.parametrize("T,N,K", [(7, 5001, 300), (12, 5001, 300), (24, 5001, 300), (50, 9001, 300), (64, 3000, 300)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 5)])
def test_linear_few_tokens_many_channels(T, N, K, pad, shift):
    q, s, w, ws, b = lin_inputs(8, T, N, K)
    check_linear(run_linear(q, s, w, ws, b, "bf16", pad, shift), q, s, w, ws, b, "bf16")
    check_linear(run_linear(q, s, w, ws, None, "f32", pad, shift), q, s, w, ws, None, "f32")


@pytest.mark.parametrize("T,N,K", [(3, 6200, 21700), (12, 6200, 21700), (12, 24600, 5505), (24, 6200, 21700),
                                   (24, 24577, 5504), (40, 6200, 21700), (40, 24577, 5504)])
def test_linear_weights_beyond_the_cache(T, N, K):
    check_large_weights(T, N, K)


# rows of whole lines, whose weights pass the cache
@pytest.mark.parametrize("T,N,K", [(8, 24600, 5504), (7, 6200, 21760), (5, 12200, 11136), (2, 16300, 8320), (12, 6200, 21760), (14, 12200, 11136), (14, 16300, 8320),
                                   (12, 24600, 5504), (30, 6200, 21760), (30, 12200, 11136), (30, 16300, 8320),
                                   (32, 24577, 5504), (50, 6200, 21760), (60, 24577, 5504), (60, 8500, 15872),
                                   (96, 24577, 5504), (128, 24577, 5504), (192, 24577, 5504), (250, 24577, 5504)])
def test_linear_weights_of_whole_lines_beyond_the_cache(T, N, K):
    check_large_weights(T, N, K)


def check_large_weights(T, N, K):
    r = np.random.default_rng([7, T, N])
    q, w = r.integers(-128, 128, (T, K), dtype=np.int8), r.integers(-128, 128, (N, K), dtype=np.int8)
    s, ws = (0.01 + r.random(T)).astype(np.float32), (0.01 + r.random(N)).astype(np.float32)
    check_linear(run_linear(q, s, w, ws, None, "bf16"), q, s, w, ws, None, "bf16")


@pytest.mark.parametrize("T", [1, 20, 300])
def test_linear_longest_sum_does_not_overflow(T):
    K = 131071
    q = np.full((T, K), -128, np.int8)
    w = np.full((3, K), -128, np.int8)
    w[1] = 127
    s, ws = np.ones(T, np.float32), np.ones(3, np.float32)
    check_linear(run_linear(q, s, w, ws, None, "f32"), q, s, w, ws, None, "f32")


def test_linear_row_scale_nan_stays_in_its_row():
    q, s, w, ws, _ = lin_inputs(4, 20, 40, 96)
    s[7] = np.nan
    got = run_linear(q, s, w, ws, None, "bf16")
    assert np.isnan(got[7]).all()
    assert not np.isnan(np.delete(got, 7, 0)).any()


def test_operators_row_offsets_beyond_32_bits():
    # rows 1.5e9 bytes apart: the third starts past 2^31, the fourth past 2^32
    T, n, ld = 4, 100, 1_500_000_000
    big = torch.empty(3 * ld + 4096, dtype=torch.int8, device=DEV)
    q, s, w, ws, _ = lin_inputs(5, T, 24, n)
    rows = torch.as_strided(big, (T, n), (ld, 1))
    st, wst = torch.from_numpy(s).to(DEV), torch.from_numpy(ws).to(DEV)
    out = torch.empty((T, 24), device=DEV)
    rows.copy_(torch.from_numpy(q))
    abi.moe_linear_int8(rows, ld, st, T, torch.from_numpy(w).to(DEV), n, wst, None, 24, n, out,
                        abi.DT_F32, 24)
    check_linear(out.cpu().numpy(), q, s, w, ws, None, "f32")
    # the same buffer as weights: N = 4 rows
    out = torch.empty((24, T), device=DEV)
    abi.moe_linear_int8(torch.from_numpy(w).to(DEV), n, wst, 24, rows, ld, st, None, T, n, out,
                        abi.DT_F32, T)
    check_linear(out.cpu().numpy(), w, ws, q, s, None, "f32")
    # codes of a norm into it, and a norm out of it
    x, _, gamma = norm_inputs(6, T, n, "bf16", "bf16")
    xt = dev_rows(x, torch.bfloat16)
    sc = torch.empty(T, device=DEV)
    abi.moe_rmsnorm_quant(xt, abi.DT_BF16, n, None, 0, 0, None, T, n, 1e-6, None, 0, None, 0, rows, ld, sc)
    ref.check_codes(rows.cpu().numpy(), sc.cpu().numpy(), ref.rmsnorm(x, None, None, 1e-6)[1], NORM_TOL)
    half = torch.as_strided(big.view(torch.bfloat16), (T, n), (ld // 2, 1))
    half.copy_(xt)
    y = torch.empty((T, n), dtype=torch.bfloat16, device=DEV)
    abi.moe_rmsnorm_quant(half, abi.DT_BF16, ld // 2, None, 0, 0, None, T, n, 1e-6, None, 0, y, n, None, 0, None)
    check_bf16(np_of(y), ref.rmsnorm(x, None, None, 1e-6)[1], NORM_TOL)


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------
def run_select(logits, bias, dt, k, softmax, G, tg, best, renorm, scale=2.5, pad=0, shift=0):
    T, E = logits.shape
    d = abi.moe_route_desc(E, k, abi.SCORE_SOFTMAX if softmax else abi.SCORE_SIGMOID, G, tg, best,
                           int(renorm), scale)
    lt = dev_rows(logits, TDT[dt], pad, shift)
    bt = None if bias is None else torch.from_numpy(bias.astype(np.float32)).to(DEV)
    idx = torch.full((T + 1, k), -5, dtype=torch.int32, device=DEV)
    w = torch.full((T + 1, k), -5.0, device=DEV)
    torch.cuda.synchronize()
    abi.moe_route_select(d, lt, DT[dt], E + pad, bt, T, idx, w)
    torch.cuda.synchronize()
    assert bool((idx[T] == -5).all()) and bool((w[T] == -5).all())
    return idx[:T].cpu().numpy(), w[:T].cpu().numpy()


def select_inputs(seed, T, E, bias, grid=None):
    r = np.random.default_rng([seed, T, E])
    l = 1.5 * r.standard_normal((T, E))
    l = np.round(l * grid) / grid if grid else l
    return l.astype(np.float32), (0.02 * r.standard_normal(E)).astype(np.float32) if bias else None


# fp32 scores differ from the 64-bit ones by a few units of 2^-24 of the row's
# largest: rows whose ranking hangs on less than 16 of them are left out
OPEN = 16 * U


def check_select(logits, bias, dt, k, softmax, G, tg, best, renorm, pad=0, shift=0):
    logits = ref.bf16(logits) if dt == "bf16" else logits
    idx, w = run_select(logits, bias, dt, k, softmax, G, tg, best, renorm, 2.5, pad, shift)
    checked = 0
    for t in range(logits.shape[0]):
        iw, ww, margin = ref.select(logits[t:t + 1], bias, k, softmax, G, tg, best, renorm, 2.5)
        if margin < OPEN:
            continue
        checked += 1
        assert np.array_equal(idx[t], iw[0]), (t, idx[t], iw[0])
        np.testing.assert_allclose(w[t], ww[0], rtol=(40 + 2 * k) * U, atol=1e-37)
    assert checked >= 0.9 * logits.shape[0]


@pytest.mark.parametrize("E,G,tg", [(1, 1, 1), (2, 2, 1), (8, 1, 1), (63, 1, 1), (60, 5, 3), (64, 8, 4),
                                    (128, 64, 7), (160, 8, 3), (256, 8, 4), (255, 5, 2), (256, 1, 1),
                                    (384, 3, 2), (512, 16, 16), (1000, 20, 9), (1024, 2, 1)])
@pytest.mark.parametrize("softmax", [False, True])
def test_select_shapes(E, G, tg, softmax):
    room = tg * (E // G)
    for i, k in enumerate(sorted({1, min(8, room), min(32, room)})):
        best = 2 if (i % 2 == 0 and E // G >= 2) else 1
        logits, bias = select_inputs(1, 37, E, i != 1)
        check_select(logits, bias, "f32", k, softmax, G, tg, best, i != 2)
        check_select(logits, bias, "bf16", k, softmax, G, tg, best, i == 2)


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 1)])
@pytest.mark.parametrize("T", [1, 2, 4, 5, 130])
def test_select_tokens_strides_and_alignment(T, pad, shift):
    logits, bias = select_inputs(2, T, 96, True)
    check_select(logits, bias, "f32", 6, False, 4, 2, 2, True, pad, shift)
    check_select(logits, bias, "bf16", 6, True, 4, 2, 2, True, pad, shift)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("G,tg,best", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_select_ties_go_to_the_lowest(softmax, G, tg, best):
    # logits on a grid of halves: many equal scores, and equal groups
    logits, _ = select_inputs(3, 200, 64, False, grid=2)
    idx, _ = run_select(logits, None, "bf16", 12, softmax, G, tg, best, True)
    want, _, _ = ref.select(logits, None, 12, softmax, G, tg, best, True, 2.5)
    assert np.array_equal(idx, want)
    same = np.zeros((3, 64), np.float32)
    idx, w = run_select(same, None, "f32", 10, softmax, G, tg, best, True)
    assert np.array_equal(idx, np.tile(np.arange(10, dtype=np.int32), (3, 1)))
    np.testing.assert_allclose(w, 0.25, rtol=60 * U)


@pytest.mark.parametrize("softmax", [False, True])
def test_select_masked_and_non_finite_logits(softmax):
    E, k = 40, 6
    l, bias = select_inputs(4, 9, E, True)
    l[0, 5:] = -np.inf                      # fewer experts left than k
    l[1] = -np.inf                          # none left
    l[2, ::3] = np.nan
    l[3] = np.nan
    l[4, 7] = np.inf
    l[5, [3, 30]] = np.inf
    l[6, :] = np.finfo(np.float32).min      # the type's lowest value throughout
    l[7, 9:] = np.finfo(np.float32).min
    for b in (None, bias):
        for G, tg, best in ((1, 1, 1), (4, 2, 2)):
            idx, w = run_select(l, b, "f32", k, softmax, G, tg, best, True)
            want, ww, _ = ref.select(l, b, k, softmax, G, tg, best, True, 2.5)
            assert np.array_equal(idx, want), (idx, want)
            np.testing.assert_allclose(w, ww, rtol=60 * U, atol=1e-37)
            assert np.isfinite(w).all()
            assert all(len(set(r)) == k for r in idx.tolist())


def test_select_non_finite_bias():
    l, b = select_inputs(5, 6, 32, True)
    b[3], b[9], b[20] = np.nan, np.inf, -np.inf
    for G, tg, best in ((1, 1, 1), (4, 2, 2)):
        idx, w = run_select(l, b, "f32", 5, False, G, tg, best, True)
        want, ww, _ = ref.select(l, b, 5, False, G, tg, best, True, 2.5)
        assert np.array_equal(idx, want)
        np.testing.assert_allclose(w, ww, rtol=60 * U)
        assert (idx[:, 0] == 9).all()


@pytest.mark.parametrize("T", [1, 3, 16, 40, 130])
def test_router_grouped_against_the_layers_own_and_the_64_bit_form(T):
    H, F, E, k = 512, 256, 64, 6
    c = Case(11, T, H, F, E, k, 0, r=2.5, n_distinct=2)
    lay = c.layer(max_tokens=T)
    x = lay.x_tensor(c.x)
    idx0, w0 = lay.router(x)
    idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    d = abi.moe_route_desc(E, k, abi.SCORE_SIGMOID, 1, 1, 1, 1, 2.5)
    abi.moe_router_topk_grouped(lay.ctx, d, x, T, lay.weights, idx, w)
    torch.cuda.synchronize()
    assert torch.equal(idx, idx0)
    np.testing.assert_allclose(w.cpu().numpy(), w0.cpu().numpy(), rtol=2 * U)
    logits = synth.bf16_bits_to_f32(c.x).astype(np.float64) @ c.Wr.astype(np.float64).T
    for softmax, G, tg, best, renorm in ((False, 8, 3, 2, True), (True, 4, 2, 1, False)):
        d = abi.moe_route_desc(E, k, int(softmax), G, tg, best, int(renorm), 1.5)
        abi.moe_router_topk_grouped(lay.ctx, d, x, T, lay.weights, idx, w)
        torch.cuda.synchronize()
        want, ww, margin = ref.select(logits, c.b, k, softmax, G, tg, best, renorm, 1.5)
        assert margin > 1e-12
        assert np.array_equal(idx.cpu().numpy(), want)
        np.testing.assert_allclose(w.cpu().numpy(), ww, rtol=2 * U)
        # the logits can still be read as after the layer's own router
        lg = lay.debug_read(2, (T, E), torch.float64)
        np.testing.assert_allclose(lg.cpu().numpy(), logits, rtol=1e-11, atol=1e-11)
    lay.close()


# ---------------------------------------------------------------------------
# streams, graphs, empty calls
# ---------------------------------------------------------------------------
def test_operators_of_no_rows_do_nothing():
    abi.moe_rmsnorm_quant(None, abi.DT_BF16, 8, None, 0, 0, None, 0, 8, 1e-6, None, 0, 1 << 20, 8, None, 0, None)
    abi.moe_swiglu_quant(None, abi.DT_BF16, 16, 0, 8, 1 << 20, 8, None, 0, None)
    abi.moe_linear_int8(None, 8, None, 0, None, 8, None, None, 4, 8, None, abi.DT_F32, 4)
    abi.moe_route_select(abi.moe_route_desc(8, 2, 0, 1, 1, 1, 1, 1.0), None, abi.DT_F32, 8, None, 0, None, None)


def test_operators_on_a_side_stream_and_in_a_graph():
    T, H, F, E, k = 6, 512, 384, 32, 4
    r = np.random.default_rng(21)
    x, res, gamma = norm_inputs(21, T, H, "bf16", "bf16")
    _, _, w, ws, _ = lin_inputs(22, T, 2 * F, H)
    xt, rt = dev_rows(x, torch.bfloat16), dev_rows(res, torch.bfloat16)
    gt, wt, wst = (torch.from_numpy(a).to(DEV) for a in (gamma, w, ws * 1e-4))
    lt = torch.from_numpy(r.standard_normal((T, E)).astype(np.float32)).to(DEV)
    d = abi.moe_route_desc(E, k, 0, 4, 2, 2, 1, 1.0)

    def outs():
        e = lambda *s, dt: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
        return (e(T, H, dt=torch.bfloat16), e(T, H, dt=torch.int8), e(T, dt=torch.float32),
                e(T, 2 * F, dt=torch.bfloat16), e(T, F, dt=torch.int8), e(T, dt=torch.float32),
                e(T, k, dt=torch.int32), e(T, k, dt=torch.float32))

    def chain(o, stream):
        h, q, s, gu, q2, s2, idx, gw = o
        abi.moe_rmsnorm_quant(xt, abi.DT_BF16, H, rt, abi.DT_BF16, H, gt, T, H, 1e-6, h, H, None, 0, q, H, s, stream)
        abi.moe_linear_int8(q, H, s, T, wt, H, wst, None, 2 * F, H, gu, abi.DT_BF16, 2 * F, stream)
        abi.moe_swiglu_quant(gu, abi.DT_BF16, 2 * F, T, F, None, 0, q2, F, s2, stream)
        abi.moe_route_select(d, lt, abi.DT_F32, E, None, T, idx, gw, stream)

    want = outs()
    chain(want, None)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), outs()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        chain(got, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = outs()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        chain(got, torch.cuda.current_stream())
    for i in range(4):
        xt.mul_(-1.0 if i % 2 == 0 else 1.0)            # other inputs, and back
        for o in got:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        chain(want, None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
