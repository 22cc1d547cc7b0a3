"""CPU tests of block.py: the rule of quantise_weight, and what the halves refuse before any GPU is
asked."""
import numpy as np
import pytest

from quantized_expert_ffn_topk_amd.block import quantise_weight
from tests import operators_ref as ref

torch = pytest.importorskip("torch")

U = 2.0 ** -24


def channels(K):
    """Rows of weights: ordinary, far below 2^-96, subnormal, near the largest number, and of zeros."""
    r = np.random.default_rng([1, K])
    w = r.standard_normal((7, K))
    for i, f in enumerate((1.0, 1e-3, 1e-30, 1e-37, 1e-41, 3e37)):
        w[i] *= f
    w[6] = 0.0
    return w.astype(np.float32)


# The multiplier is a rounded quotient and the code's product is rounded once more: 2 u.  Scales are
# one quotient; a subnormal one is off by half of 2^-149.
@pytest.mark.parametrize("K", [1, 4, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
def test_quantise_weight_by_the_rule_of_the_activations(K, dtype):
    w = channels(K)
    q, s = quantise_weight(torch.from_numpy(w).to(dtype))
    assert q.dtype == torch.int8 and s.dtype == torch.float32 and q.is_contiguous()
    ref.check_codes(q.numpy(), s.numpy(), w.astype(np.float64), 2 * U)
    top = np.abs(w).max(axis=1) > 0
    assert (np.abs(q.numpy()[top].astype(int)).max(axis=1) == 127).all()


def test_quantise_weight_of_a_tiny_channel_worked():
    q, s = quantise_weight(torch.tensor([[0.0, 1e-37, 5.05e-38, -2e-38], [0.0, 0.0, 0.0, 0.0]]))
    assert q.tolist() == [[0, 127, 64, -25], [0, 0, 0, 0]]
    np.testing.assert_allclose(s.numpy(), [1e-37 / 127, 0.0], rtol=1e-4)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_quantise_weight_marks_a_channel_that_is_not_finite(bad):
    w = torch.ones(3, 5)
    w[1, 3] = bad
    q, s = quantise_weight(w)
    assert q[1].tolist() == [0] * 5 and torch.isnan(s[1])
    assert (q[[0, 2]] == 127).all() and not torch.isnan(s[[0, 2]]).any()
