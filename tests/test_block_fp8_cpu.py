"""CPU tests of block.py's E4M3 halves: the rule of quantise_weight_fp8, and what the halves refuse
before any GPU is asked."""
import numpy as np
import pytest

from quantized_expert_ffn_topk_amd import abi
from tests import fp8_ref as ref

torch = pytest.importorskip("torch")

from quantized_expert_ffn_topk_amd.block import Fp8DenseFFN, Fp8MoEFFN, _fp8_weights, quantise_weight_fp8  # noqa: E402


def plain(w):
    """Codes and scales of weights [N,K] block by block: rows of one block each, by the rule of the rows."""
    N, K = w.shape
    q, s = np.zeros((N, K), np.uint8), np.zeros((ref.blocks(N), ref.blocks(K)), np.float32)
    for i in range(ref.blocks(N)):
        for j in range(ref.blocks(K)):
            part = w[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            a = np.float32(np.abs(part).max())
            s[i, j] = a / np.float32(448)
            if a > 0:
                pre = np.float32(2.0 ** 64) if a < 2.0 ** -96 else np.float32(1)
                q[128 * i:128 * i + 128, 128 * j:128 * j + 128] = ref.encode((part * pre) * (np.float32(448) / (a * pre)))
    return q, s


@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (129, 300), (256, 127)])
def test_quantise_weight_fp8_by_the_rule(N, K):
    r = np.random.default_rng([1, N, K])
    w = r.standard_normal((N, K)).astype(np.float32)
    w[:128, 128:256] *= 1e-38
    w[128:, 128:256] = 0
    q, s = quantise_weight_fp8(torch.from_numpy(w))
    qw, sw = plain(w)
    assert q.dtype == torch.float8_e4m3fn and q.is_contiguous() and s.shape == sw.shape
    np.testing.assert_array_equal(s.numpy(), sw)
    live = w != 0
    np.testing.assert_array_equal(q.view(torch.uint8).numpy()[live], qw[live])
    assert (ref.decode(q.view(torch.uint8).numpy()[~live]) == 0).all()


def test_quantise_weight_fp8_of_a_stack_and_of_what_is_not_finite():
    w = torch.randn(3, 130, 140)
    w[1, 129, 0] = float("inf")
    w[2, 0, 139] = float("nan")
    q, s = quantise_weight_fp8(w)
    for e in range(3):
        qe, se = quantise_weight_fp8(w[e])
        assert torch.equal(q[e].view(torch.uint8), qe.view(torch.uint8)) and torch.equal(s[e].isnan(), se.isnan())
    assert s[1].isnan().tolist() == [[False, False], [True, False]] and s[2].isnan().tolist() == [[False, True], [False, False]]
    assert (q[1, 128:, :128].float() == 0).all() and (q[2, :128, 128:].float() == 0).all()


def weights(E=None, H=256, F=128):
    lead = () if E is None else (E,)
    z = lambda *s: torch.zeros(lead + s).to(torch.float8_e4m3fn)  # noqa: E731
    o = lambda *s: torch.ones(lead + s)  # noqa: E731
    return z(2 * F, H), o(2, 2), z(H, F), o(2, 1)


def test_weights_that_do_not_fit_are_refused():
    gu, s, _, _ = weights()
    assert _fp8_weights(torch, gu, s, (256, 256), "w")[0].shape == (256, 256)
    for w, sc in ((gu.float(), s), (gu[:255], s), (gu, s[:1]), (gu, torch.ones(256))):
        with pytest.raises(ValueError):
            _fp8_weights(torch, w, sc, (256, 256), "w")


def test_halves_refuse_a_host():
    with pytest.raises(ValueError, match="not on a GPU"):
        Fp8DenseFFN(torch.ones(256), *weights(), max_tokens=4)
    route = abi.moe_route_desc(8, 2, abi.SCORE_SIGMOID, 1, 1, 1, 1, 1.0)
    with pytest.raises(ValueError, match="not on a GPU"):
        Fp8MoEFFN(torch.ones(256), torch.zeros(8, 256).bfloat16(), None, *weights(8), route, 4)
