"""GPU tests of every kernel that the int8 product's choice can take, in both output types: each shape
first has to be one that takes the kernel it stands for, so that a change of the choice cannot
quietly leave one untested.  Likewise the two ways of the layer's router logits.

The product's bits are defined (exact sum, fp32 epilogue in a fixed order), so there is no tolerance."""
import numpy as np
import pytest

from quantized_expert_ffn_topk_amd import abi
from tests import int8_product_rule as rule

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda"
CANARY = 77.0


def codes(g, rows, K, pad):
    full = torch.randint(-128, 128, (rows, K + pad), generator=g, device=DEV, dtype=torch.int8)
    return full[:, :K]


def exact_sum(q, w):
    """fp64 products and sums of codes are whole numbers far below 2^53: exact in any order."""
    out = torch.empty((q.shape[0], w.shape[0]), dtype=torch.float64, device=DEV)
    qd, step = q.double(), 8192
    for n in range(0, w.shape[0], step):
        out[:, n:n + step] = qd @ w[n:n + step].double().t().contiguous()
    return out


def check(T, N, K, pad, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q, w = codes(g, T, K, pad), codes(g, N, K, pad)
    s, ws = (0.01 + torch.rand(n, generator=g, device=DEV) for n in (T, N))
    bias = torch.randn(N, generator=g, device=DEV)
    acc = exact_sum(q, w).float()
    for dtype, code, b in ((torch.float32, abi.DT_F32, None), (torch.bfloat16, abi.DT_BF16, bias),
                           (torch.float32, abi.DT_F32, bias)):
        out = torch.full((T + 1, N + 3), CANARY, dtype=dtype, device=DEV)
        torch.cuda.synchronize()
        abi.moe_linear_int8(q, K + pad, s, T, w, K + pad, ws, b, N, K, out, code, N + 3)
        torch.cuda.synchronize()
        want = (acc * s[:, None]) * ws
        want = (want if b is None else want + b).to(dtype)
        assert bool((out[T] == CANARY).all()) and bool((out[:, N:] == CANARY).all())
        bad = out[:T, :N] != want
        assert not bool(bad.any()), (dtype, int(bad.sum()), bad.nonzero()[:4].tolist())


# (way of the rows, weights with the non-temporal hint, tokens, channels of a tile), (T, N, K, pad)
TILES = [
    (("copies", False, 64, 64), (33, 8353, 528, 16)),
    (("copies", False, 64, 64), (65, 4149, 640, 0)),
    (("copies", False, 64, 128), (65, 16745, 528, 16)),
    (("copies", False, 64, 128), (68, 16443, 640, 0)),
    (("copies", False, 96, 128), (67, 17192, 1040, 16)),
    (("copies", False, 96, 128), (66, 17028, 1152, 0)),
    (("copies", False, 128, 128), (97, 17017, 3872, 16)),
    (("copies", False, 128, 128), (99, 16890, 4096, 0)),
    (("copies", False, 192, 128), (131, 22082, 528, 16)),
    (("copies", False, 192, 128), (136, 22015, 640, 0)),
    (("copies", False, 128, 256), (66, 32952, 528, 16)),
    (("copies", False, 128, 256), (67, 33647, 640, 0)),
    (("copies", False, 192, 256), (136, 33568, 528, 16)),
    (("copies", False, 192, 256), (134, 33242, 640, 0)),
    (("copies", False, 256, 256), (198, 34436, 528, 16)),
    (("copies", False, 256, 256), (198, 33253, 640, 0)),
    (("copies", True, 64, 64), (33, 15455, 6784, 0)),
    (("copies", True, 64, 64), (33, 31517, 3284, 44)),
    (("copies", True, 64, 128), (33, 19048, 5504, 0)),
    (("copies", True, 64, 128), (33, 37251, 2772, 44)),
    (("copies", True, 96, 128), (65, 20646, 5120, 0)),
    (("copies", True, 96, 128), (65, 21555, 4820, 44)),
    (("copies", True, 128, 128), (97, 24092, 4352, 0)),
    (("copies", True, 128, 128), (97, 24823, 4180, 44)),
    (("copies", True, 192, 128), (129, 19510, 5376, 0)),
    (("copies", True, 192, 128), (130, 31594, 3284, 44)),
    (("copies", True, 128, 256), (65, 33258, 4096, 0)),
    (("copies", True, 128, 256), (65, 33296, 3100, 100)),
    (("copies", True, 192, 256), (129, 37616, 2816, 0)),
    (("copies", True, 192, 256), (129, 36032, 2844, 100)),
    (("copies", True, 256, 256), (194, 37269, 2816, 0)),
    (("copies", True, 256, 256), (196, 39134, 2644, 44)),
    (("registers", False, 64, 64), (68, 4195, 531, 2)),
    (("registers", False, 64, 128), (33, 34637, 531, 2)),
    (("registers", False, 96, 128), (65, 16938, 1043, 2)),
    (("registers", False, 128, 128), (97, 16444, 4907, 2)),
    (("registers", False, 192, 128), (130, 23745, 531, 2)),
    (("registers", False, 128, 256), (66, 34207, 531, 2)),
    (("registers", False, 192, 256), (132, 33406, 531, 2)),
    (("registers", False, 256, 256), (195, 33161, 531, 2)),
]

# (hint, weight rows, tokens of a block, waves), (T, N, K, pad)
STREAMS = [
    ((False, 16, 8, 16), (1, 16, 531, 2)),
    ((False, 16, 8, 8), (1, 4104, 528, 16)),
    ((False, 48, 8, 8), (1, 8213, 531, 2)),
    ((False, 32, 8, 4), (1, 12317, 531, 2)),
    ((False, 16, 16, 8), (9, 16, 528, 16)),
    ((False, 32, 16, 8), (9, 4166, 531, 2)),
    ((False, 48, 16, 8), (9, 8208, 528, 16)),
    ((False, 32, 16, 4), (9, 12444, 531, 2)),
    ((False, 16, 32, 8), (2058, 17, 531, 2)),
    ((False, 32, 32, 8), (33, 2090, 531, 2)),
    ((False, 48, 32, 8), (33, 4230, 531, 2)),
    ((False, 32, 32, 4), (18, 12401, 531, 2)),
    ((False, 32, 64, 8), (33, 6266, 531, 2)),
    ((True, 16, 8, 8), (1, 5354, 19584, 0)),
    ((True, 16, 8, 8), (1, 8111, 12884, 44)),
    ((True, 32, 8, 4), (1, 31500, 3328, 0)),
    ((True, 32, 8, 4), (1, 38996, 2644, 44)),
    ((True, 48, 8, 8), (1, 10638, 9856, 0)),
    ((True, 48, 8, 8), (1, 11704, 8916, 44)),
    ((True, 64, 8, 4), (1, 15169, 6912, 0)),
    ((True, 64, 8, 4), (1, 15174, 6868, 44)),
    ((True, 32, 16, 8), (9, 7123, 14720, 0)),
    ((True, 32, 16, 8), (9, 7732, 13524, 44)),
    ((True, 48, 16, 8), (9, 11071, 9472, 0)),
    ((True, 48, 16, 8), (9, 12230, 8532, 44)),
    ((True, 48, 16, 4), (9, 21559, 4864, 0)),
    ((True, 48, 16, 4), (9, 39110, 2644, 44)),
    ((True, 64, 16, 4), (9, 14124, 7424, 0)),
    ((True, 64, 16, 4), (9, 14628, 7124, 44)),
    ((True, 32, 32, 8), (17, 6024, 17408, 0)),
    ((True, 32, 32, 8), (17, 7879, 13268, 44)),
    ((True, 48, 32, 8), (17, 9871, 10624, 0)),
    ((True, 48, 32, 8), (17, 12237, 8532, 44)),
    ((True, 48, 32, 4), (17, 31501, 3328, 0)),
    ((True, 48, 32, 4), (17, 37352, 2772, 44)),
    ((True, 64, 32, 4), (17, 15753, 6656, 0)),
    ((True, 64, 32, 4), (17, 15467, 6740, 44)),
    ((True, 32, 64, 8), (33, 6561, 16000, 0)),
    ((True, 32, 64, 8), (33, 6167, 16980, 44)),
]


@pytest.mark.parametrize("kernel,shape", TILES)
def test_every_tile_kernel(kernel, shape):
    T, N, K, pad = shape
    assert rule.kernel(T, N, K, K + pad, K + pad) == ("tiles",) + kernel
    check(T, N, K, pad, 1)


@pytest.mark.parametrize("kernel,shape", STREAMS)
def test_every_stream_kernel(kernel, shape):
    T, N, K, pad = shape
    assert rule.kernel(T, N, K, K + pad, K + pad) == ("stream",) + kernel
    check(T, N, K, pad, 2)


def test_the_shapes_reach_every_kernel_of_the_choice():
    ways = {(w, h) for w, h in (("copies", False), ("copies", True), ("registers", False))}
    assert {k for k, _ in TILES} == {(w, h, t[0], t[1]) for w, h in ways for t in rule.tiles()}
    assert len({k for k, _ in STREAMS}) == 26


# ---------------------------------------------------------------------------
# grouped selection behind logits that two launches' halves make: the selection adds them and keeps
# the sum
# ---------------------------------------------------------------------------
def logit_parts(T, H, E):
    """How many parts of H the router's logits come in, as kernels_router.hip's router_ksplit states it."""
    if T <= 16 or T >= 1024 or -(-E // 16) * -(-T // 16) >= 128:
        return 1
    h32 = H // 32
    return 2 if h32 % (16 if h32 % 16 else 32) == 0 else 1


@pytest.mark.parametrize("T,H,E,parts", [(17, 1024, 64, 2), (40, 2048, 100, 2), (100, 1024, 250, 2), (33, 6144, 48, 2),
                                         (16, 1024, 64, 1), (120, 1024, 256, 1), (40, 1280, 100, 1)])
def test_grouped_router_adds_both_halves_of_the_logits(T, H, E, parts):
    from quantized_expert_ffn_topk_amd import synth
    from tests import operators_ref as ref
    from tests.gpu_common import Case
    from tests.test_gpu_operators import U
    assert logit_parts(T, H, E) == parts
    k = 6
    c = Case(13, T, H, 256, E, k, 0, r=2.5, n_distinct=1)
    lay = c.layer(max_tokens=T)
    x = lay.x_tensor(c.x)
    logits = synth.bf16_bits_to_f32(c.x).astype(np.float64) @ c.Wr.astype(np.float64).T
    idx, w = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    G = next(g for g in (8, 5, 4, 2) if E % g == 0)
    for softmax, best, renorm, bias in ((False, 2, True, True), (True, 1, False, True), (False, 1, True, False)):
        d = abi.moe_route_desc(E, k, int(softmax), G, max(1, G // 2), best, int(renorm), 1.5)
        weights = lay.weights if bias else abi.moe_layer_weights(lay.weights.router_w, None, lay.weights.expert_ptrs, None)
        abi.moe_router_topk_grouped(lay.ctx, d, x, T, weights, idx, w)
        torch.cuda.synchronize()
        want, ww, margin = ref.select(logits, c.b if bias else None, k, softmax, G, max(1, G // 2), best, renorm, 1.5)
        assert margin > 1e-12
        assert np.array_equal(idx.cpu().numpy(), want)
        np.testing.assert_allclose(w.cpu().numpy(), ww, rtol=2 * U)
        # the whole logits can be read afterwards
        got = lay.debug_read(2, (T, E), torch.float64).cpu().numpy()
        np.testing.assert_allclose(got, logits, rtol=1e-11, atol=1e-11)
    lay.close()


@pytest.mark.parametrize("T", [6, 40])
@pytest.mark.parametrize("softmax", [False, True])
def test_grouped_router_of_tokens_that_are_not_finite(T, softmax):
    from quantized_expert_ffn_topk_amd import synth
    from tests import operators_ref as ref
    from tests.gpu_common import Case
    from tests.test_gpu_operators import U
    H, E, k, G = 1024, 64, 6, 8
    base = Case(14, T, H, 256, E, k, 0, r=2.5, n_distinct=1)
    bits = base.x.copy()
    bits[1, 7] = 0x7fc0                                  # NaN: every logit is NaN
    bits[2, 9] = 0x7f80                                  # inf: every logit is inf or -inf
    bits[3] = 0                                          # every logit is 0: all equal
    bits[4] = synth.f32_to_bf16_bits(synth.bf16_bits_to_f32(bits[4]) * np.float32(3e4))   # scores at both ends
    c = Case(14, T, H, 256, E, k, 0, r=2.5, n_distinct=1, x=bits)
    lay = c.layer(max_tokens=T)
    x = lay.x_tensor(c.x)
    idx, w = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    for best, renorm in ((2, True), (1, False)):
        d = abi.moe_route_desc(E, k, int(softmax), G, 4, best, int(renorm), 1.5)
        abi.moe_router_topk_grouped(lay.ctx, d, x, T, lay.weights, idx, w)
        torch.cuda.synchronize()
        got = lay.debug_read(2, (T, E), torch.float64).cpu().numpy()
        assert np.isnan(got[1]).all() and (got[3] == 0).all()
        # choice and weights from the logits that the router made
        want, ww, _ = ref.select(got, c.b, k, softmax, G, 4, best, renorm, 1.5)
        assert np.array_equal(idx.cpu().numpy(), want)
        np.testing.assert_allclose(w.cpu().numpy(), ww, rtol=2 * U, atol=2.0 ** -149)
        assert (w[1] == 0).all() and all(len(set(r)) == k for r in idx.tolist())
        assert not torch.isnan(w).any()
    lay.close()
