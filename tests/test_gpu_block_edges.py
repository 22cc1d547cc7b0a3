"""GPU tests of what block.py's halves refuse and how they stand to streams."""
import pytest

from tests.test_block_cpu import dense_parts, layer_like, route

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_routed_half_refuses_a_layer_of_another_gpu():
    from quantized_expert_ffn_topk_amd.block import MoEFFN
    with pytest.raises(ValueError, match="cuda:1"):
        MoEFFN(torch.ones(16, device="cuda:0"), layer_like(torch.device("cuda", 1)), route())


def test_halves_refuse_a_stream_of_another_gpu():
    from types import SimpleNamespace

    from quantized_expert_ffn_topk_amd.block import DenseFFN
    d = DenseFFN(*dense_parts("cuda:0"), max_tokens=4)
    x = torch.zeros(2, 16, device="cuda:0")
    other = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream"):
        d.forward(x, x, other)
