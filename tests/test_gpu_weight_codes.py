"""GPU tests of quantise_weight_fp8: on the device its blocks of one row are moe_quant_fp8's, bit for bit, and its
matrices the host's."""
import numpy as np
import pytest

from quantized_expert_ffn_topk_amd import abi
from tests import fp8_ref as ref
from tests.test_weight_codes_cpu import between_codes

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from quantized_expert_ffn_topk_amd.block import quantise_weight_fp8  # noqa: E402


def bits(t):
    return t.cpu().view(torch.uint8).numpy()


@pytest.mark.parametrize("K", [128, 1000, 16384])
def test_blocks_of_one_row_are_the_activations(K):
    w = between_codes(11, ref.blocks(K))[:1, :K].copy()
    w[0, :100] *= 2.0 ** -120
    wt = torch.from_numpy(w).cuda()
    q, s = quantise_weight_fp8(wt)
    q2, s2 = torch.zeros((1, K), dtype=torch.uint8, device="cuda"), torch.zeros((1, ref.blocks(K)), device="cuda")
    torch.cuda.synchronize()
    abi.moe_quant_fp8(wt, abi.DT_F32, K, abi.ACT_NONE, 1, K, None, q2, K, s2, ref.blocks(K))
    torch.cuda.synchronize()
    assert np.array_equal(bits(s), bits(s2))
    assert np.array_equal(bits(q), bits(q2))


def test_matrices_on_the_device_are_the_hosts():
    w = torch.from_numpy(np.stack([between_codes(12 + i, 5)[:, :600] for i in range(3)]))
    for a, b in zip(quantise_weight_fp8(w.cuda()), quantise_weight_fp8(w)):
        assert np.array_equal(bits(a), bits(b))
