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


def test_dense_half_refuses_bad_weights_and_types_when_it_is_made():
    from quantized_expert_ffn_topk_amd.block import DenseFFN
    gamma, gu, s_gu, dn, s_dn = dense_parts("cuda")
    for bad in (dict(out_dtype=torch.float16), dict(out_dtype=torch.int8)):
        with pytest.raises(ValueError, match="out_dtype"):
            DenseFFN(gamma, gu, s_gu, dn, s_dn, 4, **bad)
    for parts in ((gamma, gu, s_gu, dn[0], s_dn), (gamma, gu.flatten(), s_gu, dn, s_dn)):
        with pytest.raises(ValueError):
            DenseFFN(*parts, 4)
    assert DenseFFN(gamma, gu, s_gu, dn, s_dn, 4, out_dtype=torch.float32).out_dtype == torch.float32


# ---------------------------------------------------------------------------
# tensors and streams
# ---------------------------------------------------------------------------
CYCLES = 60_000_000                    # some tens of milliseconds of one idle kernel


def weights(seed, H, F):
    from quantized_expert_ffn_topk_amd.block import quantise_weight
    g = torch.Generator().manual_seed(seed)
    gu, s_gu = quantise_weight(torch.randn(2 * F, H, generator=g) * 0.05)
    dn, s_dn = quantise_weight(torch.randn(H, F, generator=g) * 0.05)
    gamma = 1 + 0.1 * torch.randn(H, generator=g)
    return [a.cuda() for a in (gamma, gu, s_gu, dn, s_dn)]


def test_a_half_is_ready_on_every_stream_once_it_is_made():
    from quantized_expert_ffn_topk_amd.block import DenseFFN, MoEFFN
    parts = weights(1, 64, 32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for make in (lambda: DenseFFN(*parts, max_tokens=4),
                 lambda: MoEFFN(torch.ones(16, device="cuda"), layer_like(torch.device("cuda", 0)), route())):
        with torch.cuda.stream(side):
            torch.cuda._sleep(CYCLES)
            assert not side.query()
            make()
            assert side.query()


def test_a_half_and_its_inputs_may_be_dropped_while_another_stream_works():
    from quantized_expert_ffn_topk_amd.block import DenseFFN
    H, F, T = 2048, 1024, 64
    parts = weights(2, H, F)
    x, r = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, H, device="cuda").bfloat16()
    want = DenseFFN(*parts, max_tokens=T).forward(x, r)
    torch.cuda.synchronize()
    d = DenseFFN(*(a.clone() for a in parts), max_tokens=T)
    xc, rc = x.clone(), r.clone()
    sizes = [(a.numel() * a.element_size(), a.data_ptr()) for a in (*d._own, xc, rc)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    got = d.forward(xc, rc, side)
    del d, xc, rc
    used = {p for _, p in sizes}
    # what is allocated now, on the stream that all of it came from, is other memory
    others = [torch.full((n,), 85, dtype=torch.uint8, device="cuda") for n, _ in sizes]
    assert not side.query()
    assert not used & {o.data_ptr() for o in others}
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_half_in_a_graph_then_dropped():
    from quantized_expert_ffn_topk_amd.block import DenseFFN
    H, F, T = 512, 256, 5
    d = DenseFFN(*weights(3, H, F), max_tokens=T)
    x, r = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, H, device="cuda").bfloat16()
    d.forward(x, r)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = d.forward(x, r, torch.cuda.current_stream())
    for i in range(4):
        x.mul_(-1.0 if i % 2 == 0 else 0.5)
        for o in got:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = d.forward(x, r)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
    del g, got, d
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
