"""GPU tests of the codes in front of the E4M3 halves' products: their scales too are the quantiser's."""
import numpy as np
import pytest

from tests import fp8_ref as ref
from tests.test_gpu_block_fp8 import H, dense, inputs, moe, num

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T", [1, 7, 70])
def test_scales_in_front_of_the_first_product(T):
    """Each block's scale, bit for bit from the normed rows, in both halves."""
    x, r = inputs(T)
    for half in (dense(T), moe(T)):
        half.forward(x, r)
        torch.cuda.synchronize()
        q, s = ref.quant(num(half.y[:T]).astype(np.float32))
        assert np.array_equal(half.s[:T].cpu().numpy().view(np.uint32), s.view(np.uint32))
        assert half.s.shape == (T, ref.blocks(H)) and q.shape == (T, H)
