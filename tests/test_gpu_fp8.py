"""GPU tests of E4M3 rows and products through the C ABI: moe_quant_fp8 against its
own fp32 steps (bits are defined) and, for SwiGLU, the 64-bit value; moe_linear_fp8
against the 64-bit product, within the bounds of fp8_ref."""
import numpy as np
import pytest

from quantized_expert_ffn_topk_amd import abi
from tests import fp8_ref as ref
from tests import operators_ref as oref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda"
U = ref.U
DT = {"f32": abi.DT_F32, "bf16": abi.DT_BF16, "fp8": abi.DT_FP8}
TDT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}
CANARY = 77


def dev_rows(a, dtype, pad=0, shift=0):
    """a [T,n] on the device, rows `pad` apart beyond their length, `shift` elements into
    an allocation that ends with the last row."""
    T, n = a.shape
    flat = torch.zeros(T * (n + pad) - (pad if T else 0) + shift, dtype=dtype, device=DEV)
    v = flat[shift:].as_strided((T, n), (n + pad, 1), shift) if T else flat.view(0, n)
    v.copy_(torch.from_numpy(np.ascontiguousarray(a)))
    return v


def out_rows(T, n, dtype, pad=0, shift=0):
    flat = torch.full((T * (n + pad) + shift + 64,), CANARY, dtype=dtype, device=DEV)
    return flat, flat[shift:shift + T * (n + pad)].view(T, n + pad)


def check_canary(flat, T, n, pad, shift, rows=None):
    f = flat.float().cpu().numpy()
    body = f[shift:shift + T * (n + pad)].reshape(T, n + pad)
    assert (f[:shift] == CANARY).all() and (f[shift + T * (n + pad):] == CANARY).all()
    assert (body[:, n:] == CANARY).all()
    if rows is not None:
        assert (body[rows:] == CANARY).all()


def np_of(t):
    return t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()


# ---------------------------------------------------------------------------
# codes
# ---------------------------------------------------------------------------
def run_quant(x, xd, swiglu=False, pad=0, shift=0, count=None, stream=None):
    T, K = x.shape[0], x.shape[1] // (2 if swiglu else 1)
    nb = ref.blocks(K)
    xt = dev_rows(x, TDT[xd], pad, shift)
    qf, q = out_rows(T, K, torch.uint8, pad, shift)
    sf, s = out_rows(T, nb, torch.float32, pad, shift)
    ct = None if count is None else torch.tensor([count], dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    abi.moe_quant_fp8(xt, DT[xd], x.shape[1] + pad, abi.ACT_SWIGLU if swiglu else abi.ACT_NONE, T, K, ct, q, K + pad, s,
                      nb + pad, stream)
    torch.cuda.synchronize()
    rows = None if count is None else min(max(count, 0), T)
    check_canary(qf, T, K, pad, shift, rows)
    check_canary(sf, T, nb, pad, shift, rows)
    return q[:rows, :K].cpu().numpy(), s[:rows, :nb].cpu().numpy()


def same_scales(a, b):
    return np.array_equal(a.view(np.uint32)[~np.isnan(b)], b.view(np.uint32)[~np.isnan(b)]) and \
        np.array_equal(np.isnan(a), np.isnan(b))


def values(seed, T, n, xd, scale=1.0):
    v = np.random.default_rng([seed, T, n]).standard_normal((T, n)) * scale
    return v.astype(np.float32) if xd == "f32" else oref.bf16(v)


@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,pad,shift", [
    (1, 1, 0, 0), (3, 7, 0, 0), (2, 8, 3, 1), (5, 127, 0, 0), (5, 128, 0, 0), (5, 129, 5, 3), (1, 6144, 0, 0),
    (17, 1000, 8, 8), (300, 2048, 0, 0), (4, 12289, 1, 1), (1, 1 << 17, 0, 0)])
def test_codes_bit_for_bit(xd, T, K, pad, shift):
    x = values(1, T, K, xd, 3.0)
    q, s = run_quant(x, xd, pad=pad, shift=shift)
    qw, sw = ref.quant(x)
    assert same_scales(s, sw)
    assert np.array_equal(q, qw)


def test_codes_of_every_binade_and_special_blocks():
    """Blocks at both ends of the number range, of zeros, and with a NaN or an infinity in them."""
    r = np.random.default_rng(2)
    x = np.zeros((64, 256), np.float32)
    for i, e in enumerate(range(-149, 128, 9)):
        x[i] = np.ldexp(np.clip(r.standard_normal(256), -1.9, 1.9), e)
    x[40, 3] = np.nan
    x[41, 200] = np.inf
    x[42, 130] = -np.inf
    x[43] = 3.4e38
    x[44, 5] = -1e-45
    x[45, :128] = -0.0
    q, s = run_quant(x, "f32")
    qw, sw = ref.quant(x)
    assert same_scales(s, sw)
    live = (x != 0) | (np.isnan(np.repeat(sw, 128, axis=1)))
    assert np.array_equal(q[live], qw[live])
    assert (ref.decode(q[~live]) == 0).all()
    assert np.isnan(s[40, 0]) and not np.isnan(s[40, 1]) and not q[40, :128].any()


@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,pad,shift", [(1, 1, 0, 0), (3, 100, 3, 1), (7, 128, 0, 0), (33, 2048, 0, 0), (2, 12288, 8, 8),
                                           (5, 333, 1, 1)])
def test_swiglu_codes(xd, T, K, pad, shift):
    """v in fp32 is within 20u of the 64-bit value, the block's largest and the multiplier too: a code
    within half a step (2^-4 of itself, or 2^-10) and 3 * 20u of the multiplied value."""
    x = values(3, T, 2 * K, xd, 2.0)
    q, s = run_quant(x, xd, True, pad, shift)
    v = oref.swiglu(x)
    a = ref.block_max(v)
    np.testing.assert_allclose(s, a / 448, rtol=22 * U)
    p = v * ref.spread(448 / a, K)
    assert (np.abs(ref.decode(q) - p) <= np.maximum(np.abs(p) * 2.0 ** -4, 2.0 ** -10) + 60 * U * 448).all()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("count", [-3, 0, 1, 5, 40, 41, 1000])
def test_rows_behind_the_count_stay(swiglu, count):
    K = 200
    x = values(4, 41, K * (2 if swiglu else 1), "bf16")
    x[min(max(count, 0), 41):] = np.nan
    q, s = run_quant(x, "bf16", swiglu, count=count)
    q2, s2 = run_quant(x[:q.shape[0]], "bf16", swiglu) if q.shape[0] else (q, s)
    assert np.array_equal(q, q2) and np.array_equal(s, s2) and not np.isnan(s).any()


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def run_linear(q, s, w, ws, bias, out, pad=0, shift=0, spad=0, stream=None):
    T, K = q.shape
    N = w.shape[0]
    nb = ref.blocks(K)
    qt, wt = dev_rows(q, torch.uint8, pad, shift), dev_rows(w, torch.uint8, pad, shift)
    st, wst = dev_rows(s, torch.float32, spad), dev_rows(ws, torch.float32, spad)
    bt = None if bias is None else torch.from_numpy(bias).to(DEV)
    flat, y = out_rows(T, N, TDT[out], pad, shift)
    torch.cuda.synchronize()
    abi.moe_linear_fp8(qt, K + pad, st, nb + spad, T, wt, K + pad, wst, nb + spad, bt, N, K, y, DT[out], N + pad, stream)
    torch.cuda.synchronize()
    check_canary(flat, T, N, pad, shift)
    return np_of(y[:, :N])


def linear_inputs(seed, T, N, K):
    r = np.random.default_rng([seed, T, N, K])
    pool = ref.codes(r, 1 << 14)
    nb = ref.blocks(K)
    s = (2.0 ** r.uniform(-9, -6, (T, nb))).astype(np.float32)
    ws = (2.0 ** r.uniform(-14, -11, (ref.blocks(N), nb))).astype(np.float32)
    return pool[r.integers(0, 1 << 14, (T, K))], s, pool[r.integers(0, 1 << 14, (N, K))], ws, r.standard_normal(N).astype(np.float32)


def check_linear(y, q, s, w, ws, bias, out):
    at = ref.some_rows(q.shape[0])
    y, x, v = y[at], ref.scaled(q[at], s[at]), ref.scaled_weights(w, ws)
    want = x @ v.T
    lim = ref.limit(x, v, 1, out == "bf16", out == "bf16" and q.shape[0] > 32)
    if bias is not None:
        want = want + bias
        lim = lim + (2 * U + (2.0 ** -8 if out == "bf16" else 0)) * np.abs(bias)
    off = np.abs(y - want)
    assert (off <= lim).all(), float((off - lim).max())


SHAPES = [(1, 1, 1), (1, 16, 128), (2, 33, 64), (3, 130, 129), (8, 257, 1000), (9, 100, 384), (16, 129, 2000), (17, 64, 640),
          (32, 200, 255), (33, 65, 128), (40, 128, 127), (64, 64, 512), (65, 129, 513), (100, 300, 900), (130, 70, 1664),
          (200, 260, 300)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_linear_sizes(out, T, N, K):
    q, s, w, ws, bias = linear_inputs(5, T, N, K)
    check_linear(run_linear(q, s, w, ws, None, out), q, s, w, ws, None, out)


# Shapes whose rounds over the CUs cost least as tiles of 64x64, 64x128, 128x128, 128x256 and 256x256
# (fp32 outputs: up to 128x256); rows on 16 bytes, on 4, and on single ones (through registers).
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,N", [(64, 6100), (320, 5003), (512, 5000), (1100, 4600), (2100, 4700)])
@pytest.mark.parametrize("K,pad,shift", [(256, 0, 0), (520, 8, 8), (1300, 4, 4), (300, 3, 1), (100, 4, 0)])
def test_linear_tiles(out, T, N, K, pad, shift):
    q, s, w, ws, bias = linear_inputs(10, T, N, K)
    check_linear(run_linear(q, s, w, ws, bias, out, pad, shift, pad), q, s, w, ws, bias, out)


# Some rows, of so many channels that the blocks of a stream are 16, 32 and 64 channels wide, and a
# few more, where they are tiles.
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,N", [(33, 2040), (40, 4050), (64, 4100), (33, 8190), (200, 2250), (64, 9000), (300, 60), (2100, 7)])
@pytest.mark.parametrize("K,pad,shift", [(520, 8, 8), (1300, 4, 4), (700, 3, 1), (7, 0, 0)])
def test_linear_between_streams_and_tiles(out, T, N, K, pad, shift):
    q, s, w, ws, bias = linear_inputs(14, T, N, K)
    check_linear(run_linear(q, s, w, ws, bias, out, pad, shift, pad), q, s, w, ws, bias, out)


# rows on 4 bytes whose length is not of whole words: the last row's last word is partly behind it
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,N", [(40, 300), (320, 5003), (512, 5000), (1100, 4600), (2100, 4700)])
@pytest.mark.parametrize("K,pad", [(513, 3), (1302, 2), (127, 1), (3, 1)])
def test_linear_rows_that_end_inside_a_word(out, T, N, K, pad):
    q, s, w, ws, _ = linear_inputs(12, T, N, K)
    check_linear(run_linear(q, s, w, ws, None, out, pad), q, s, w, ws, None, out)


def test_linear_tiles_give_the_same_bits_in_every_shape():
    """Blocks' sums are added in their order whatever the tile: rows of a large product equal those of
    a smaller one."""
    q, s, w, ws, _ = linear_inputs(11, 2100, 4700, 1000)
    y = run_linear(q, s, w, ws, None, "bf16")
    for T in (512, 1100):
        assert np.array_equal(run_linear(q[:T], s[:T], w, ws, None, "bf16"), y[:T])


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift,spad", [(16, 16, 4), (3, 1, 1), (5, 0, 0), (8, 8, 2)])
@pytest.mark.parametrize("T,N,K", [(1, 50, 300), (20, 131, 1025), (70, 130, 1100)])
def test_linear_strides_alignment_and_bias(out, pad, shift, spad, T, N, K):
    q, s, w, ws, bias = linear_inputs(6, T, N, K)
    check_linear(run_linear(q, s, w, ws, bias, out, pad, shift, spad), q, s, w, ws, bias, out)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 12, 48])
def test_linear_long_rows(out, T):
    """More stages than a wave keeps weights' scales for, and the longest rows."""
    for N, K in ((20, 40000), (3, 1 << 17)):
        q, s, w, ws, _ = linear_inputs(7, T, N, K)
        check_linear(run_linear(q, s, w, ws, None, out), q, s, w, ws, None, out)


@pytest.mark.parametrize("T", [1, 20, 80])
def test_linear_of_codes_that_are_no_numbers(T):
    """A NaN code, or a NaN scale, reaches its own row or channel and no other."""
    q, s, w, ws, _ = linear_inputs(8, T, 150, 700)
    clean = run_linear(q, s, w, ws, None, "f32")
    q2, w2, s2, ws2 = q.copy(), w.copy(), s.copy(), ws.copy()
    q2[0, 699] = 0x7f
    w2[5, 3] = 0xff
    if T > 1:
        s2[1, 2] = np.nan
    ws2[1, 0] = np.nan                                 # channels 128 ..
    y = run_linear(q2, s2, w2, ws2, None, "f32")
    bad = np.zeros(y.shape, bool)
    bad[0] = bad[:, 5] = bad[:, 128:] = True
    if T > 1:
        bad[1] = True
    assert np.array_equal(np.isnan(y), bad)
    assert np.array_equal(y[~bad], clean[~bad])


def test_linear_twice_on_two_streams_and_captured():
    q, s, w, ws, bias = linear_inputs(9, 70, 300, 1000)
    a = run_linear(q, s, w, ws, bias, "bf16")
    side = torch.cuda.Stream()
    qt, wt = dev_rows(q, torch.uint8), dev_rows(w, torch.uint8)
    st, wst, bt = (torch.from_numpy(v).to(DEV) for v in (s, ws, bias))
    y = torch.zeros((70, 300), dtype=torch.bfloat16, device=DEV)
    y2 = torch.zeros_like(y)
    torch.cuda.synchronize()
    args = lambda o: (qt, 1000, st, 8, 70, wt, 1000, wst, 8, bt, 300, 1000, o, abi.DT_BF16, 300)  # noqa: E731
    abi.moe_linear_fp8(*args(y))
    abi.moe_linear_fp8(*args(y2), side)
    torch.cuda.synchronize()
    assert np.array_equal(np_of(y), a) and np.array_equal(np_of(y2), a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        abi.moe_linear_fp8(*args(y), torch.cuda.current_stream())
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(np_of(y), a)
