"""CPU tests of quantise_weight_fp8 where one rounding decides: values next to the middle between two codes."""
import numpy as np
import pytest

from tests import fp8_ref as ref
from tests.test_block_fp8_cpu import plain

torch = pytest.importorskip("torch")

from quantized_expert_ffn_topk_amd.block import quantise_weight_fp8  # noqa: E402


def between_codes(seed, blocks):
    """[128, 128*blocks]: each block's largest value is any number, the others lie at the middles between
    two codes, as near as fp32 comes, and one or two units of the last place to either side."""
    r = np.random.default_rng(seed)
    ties = ((ref.TABLE[:126] + ref.TABLE[1:127]) / 2)
    w = np.zeros((128, 128 * blocks), np.float32)
    for b in range(blocks):
        top = np.float32(r.uniform(0.001, 10))
        v = (r.choice(ties, (128, 128)) * (np.float64(top) / 448)).astype(np.float32)
        v = (v.view(np.int32) + r.integers(-2, 3, v.shape).astype(np.int32)).view(np.float32)
        v[r.integers(128), r.integers(128)] = top
        w[:, 128 * b:128 * b + 128] = v * r.choice([-1, 1], v.shape).astype(np.float32)
    return w


@pytest.mark.parametrize("seed", range(4))
def test_codes_next_to_the_middle_between_two(seed):
    w = between_codes(seed, 8)
    q, s = quantise_weight_fp8(torch.from_numpy(w))
    qw, sw = plain(w)
    np.testing.assert_array_equal(s.numpy(), sw)
    np.testing.assert_array_equal(q.view(torch.uint8).numpy(), qw)
