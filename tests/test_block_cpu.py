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


# ---------------------------------------------------------------------------
# everything of a half is on one GPU: a host address, or another GPU's, never reaches a kernel
# ---------------------------------------------------------------------------
def dense_parts(device, H=16, F=8):
    z = lambda *shape: torch.zeros(shape, dtype=torch.int8, device=device)  # noqa: E731
    o = lambda n: torch.ones(n, device=device)  # noqa: E731
    return o(H), z(2 * F, H), o(2 * F), z(H, F), o(H)


def layer_like(dev, H=16):
    from types import SimpleNamespace
    return SimpleNamespace(desc=SimpleNamespace(hidden=H, top_k=2, n_experts=8), dev=dev, max_tokens=4)


def route():
    from quantized_expert_ffn_topk_amd import abi
    return abi.moe_route_desc(8, 2, abi.SCORE_SIGMOID, 1, 1, 1, 1, 1.0)


def test_halves_refuse_host_tensors():
    from quantized_expert_ffn_topk_amd.block import DenseFFN, MoEFFN
    with pytest.raises(ValueError, match="GPU"):
        DenseFFN(*dense_parts("cpu"), max_tokens=4)
    with pytest.raises(ValueError, match="GPU"):
        MoEFFN(torch.ones(16), layer_like(torch.device("cuda", 0)), route())
