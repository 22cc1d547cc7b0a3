"""CPU tests of the operators around the MoE layer: every bad argument is
refused with E_INVAL before anything is enqueued (no GPU is needed to find
out), and the plain 64-bit forms that the GPU tests go by agree with worked
values and with their own definitions."""
import numpy as np
import pytest

from quantized_expert_ffn_topk_amd import abi
from tests import operators_ref as ref

P = 1 << 20                       # an aligned address that is never read


def refused(fn, *args):
    with pytest.raises(abi.MoEError) as ei:
        fn(*args)
    assert ei.value.status == abi.E_INVAL, str(ei.value)
    assert str(ei.value) != "E_INVAL: "


NORM = dict(x=P, x_dtype=1, ldx=64, residual=P, res_dtype=1, ldr=64, gamma=P, T=2, H=64, eps=1e-6,
            h_out=P, ldh=64, y_out=P, ldy=64, q=P, ldq=64, s=P)
SWIGLU = dict(gu=P, gu_dtype=1, ld=128, T=2, F=64, y_out=P, ldy=64, q=P, ldq=64, s=P)
LINEAR = dict(q=P, ldq=64, s=P, T=2, w=P, ldw=64, ws=P, bias=P, N=32, K=64, out=P, out_dtype=1, ldo=32)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x_dtype=2), dict(res_dtype=-1), dict(T=-1), dict(T=(1 << 20) + 1), dict(H=0),
    dict(H=(1 << 20) + 1), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(ldx=63), dict(ldr=63), dict(ldh=63), dict(ldy=63), dict(ldq=63), dict(s=None), dict(q=None),
    dict(h_out=None, y_out=None, q=None, s=None), dict(x=P + 1), dict(residual=P + 1),
    dict(gamma=P + 2), dict(h_out=P + 1), dict(y_out=P + 1), dict(s=P + 2),
    dict(residual=None, x_dtype=0), dict(x_dtype=0, x=P + 2)])
def test_norm_refusals(bad):
    refused(abi.moe_rmsnorm_quant, *dict(NORM, **bad).values())


@pytest.mark.parametrize("bad", [
    dict(gu=None), dict(gu_dtype=3), dict(T=-1), dict(T=(1 << 20) + 1), dict(F=0), dict(F=(1 << 20) + 1),
    dict(ld=127), dict(ldy=63), dict(ldq=63), dict(q=None), dict(s=None),
    dict(y_out=None, q=None, s=None), dict(gu=P + 1), dict(y_out=P + 1), dict(s=P + 1)])
def test_swiglu_refusals(bad):
    refused(abi.moe_swiglu_quant, *dict(SWIGLU, **bad).values())


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(s=None), dict(w=None), dict(ws=None), dict(out=None), dict(T=-1),
    dict(T=(1 << 20) + 1), dict(T=1 << 20, N=1 << 19, ldo=1 << 19), dict(N=0), dict(N=(1 << 20) + 1), dict(K=0), dict(K=131072), dict(ldq=63),
    dict(ldw=63), dict(ldo=31), dict(out_dtype=2), dict(s=P + 2), dict(ws=P + 1), dict(bias=P + 2),
    dict(out=P + 1), dict(out_dtype=0, out=P + 2)])
def test_linear_refusals(bad):
    refused(abi.moe_linear_int8, *dict(LINEAR, **bad).values())


ROUTE = dict(n_experts=64, top_k=8, score=0, n_group=8, topk_group=4, group_best=2, renorm=1, scale=2.5)


@pytest.mark.parametrize("bad", [
    dict(n_experts=0), dict(n_experts=1025), dict(top_k=0), dict(top_k=33), dict(score=2), dict(n_group=0),
    dict(n_group=7), dict(n_experts=130, n_group=65, topk_group=65), dict(topk_group=0),
    dict(topk_group=9), dict(topk_group=1, top_k=9), dict(group_best=0), dict(group_best=3),
    dict(n_experts=8, top_k=2), dict(renorm=2), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf"))])
def test_route_desc_refusals(bad):
    d = abi.moe_route_desc(*dict(ROUTE, **bad).values())
    refused(abi.moe_route_select, d, P, 0, 1100, P, 2, P, P)
    refused(abi.moe_router_topk_grouped, None, d, P, 2, abi.moe_layer_weights(), P, P)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(dt=5), dict(ld=63), dict(T=-1), dict(T=(1 << 20) + 1), dict(idx=None),
    dict(w=None), dict(logits=P + 2), dict(bias=P + 1), dict(idx=P + 2), dict(w=P + 1)])
def test_route_select_refusals(bad):
    d = abi.moe_route_desc(*ROUTE.values())
    a = dict(dict(logits=P, dt=0, ld=64, bias=P, T=2, idx=P, w=P), **bad)
    refused(abi.moe_route_select, d, *a.values())


def test_null_descriptor_and_context_are_refused():
    assert abi.lib().moe_route_select(None, None, 0, 8, None, 1, None, None, None) == abi.E_INVAL
    d = abi.moe_route_desc(*ROUTE.values())
    refused(abi.moe_router_topk_grouped, None, d, P, 2, abi.moe_layer_weights(), P, P)


def test_no_rows_need_no_pointers():
    abi.moe_rmsnorm_quant(None, 1, 64, None, 0, 0, None, 0, 64, 1e-6, None, 0, P, 64, None, 0, None)
    abi.moe_swiglu_quant(None, 1, 128, 0, 64, P, 64, None, 0, None)
    abi.moe_linear_int8(None, 64, None, 0, None, 64, None, None, 32, 64, None, 1, 32)
    abi.moe_route_select(abi.moe_route_desc(*ROUTE.values()), None, 0, 64, None, 0, None, None)


# ---------------------------------------------------------------------------
# the plain forms themselves
# ---------------------------------------------------------------------------
def test_reference_norm_worked_values():
    h, v = ref.rmsnorm(np.array([[3.0, -4.0]]), np.array([[0.0, 0.0]]), np.array([1.0, 2.0]), 1e-12)
    r = np.sqrt(12.5)
    np.testing.assert_allclose(v, [[3 / r, -8 / r]], rtol=1e-9)
    np.testing.assert_allclose(h, [[3, -4]])


def test_reference_swiglu_worked_values():
    np.testing.assert_allclose(ref.swiglu(np.array([[0.0, 1.0, 5.0, 2.0]])),
                               [[0.0, 2.0 / (1 + np.exp(-1.0))]], rtol=1e-15)


def test_reference_select_worked_values():
    # two groups of three; the second holds the best pair, the first the best one
    l = np.array([[3.0, -3.0, -3.0, 2.0, 2.0, -1.0]])
    idx, w, _ = ref.select(l, None, 2, False, 2, 1, 2, True, 1.0)
    assert idx.tolist() == [[3, 4]]
    np.testing.assert_allclose(w, [[0.5, 0.5]])
    idx, w, _ = ref.select(l, None, 2, False, 2, 1, 1, False, 2.0)
    assert idx.tolist() == [[0, 1]]
    s = 1 / (1 + np.exp(-np.array([3.0, -3.0])))
    np.testing.assert_allclose(w, [2 * s])
    idx, w, _ = ref.select(l, np.array([0, 0, 0, 0, 0, 9.0]), 1, True, 1, 1, 1, True, 1.0)
    assert idx.tolist() == [[5]] and w.tolist() == [[1.0]]


# ---- the direct calls' own conversions ---------------------------------------------
def test_direct_calls_take_numpy_arrays_and_integers():
    gu, q, s = np.zeros((0, 16), np.float32), np.zeros((0, 8), np.int8), np.zeros(0, np.float32)
    abi.moe_swiglu_quant(gu, abi.DT_F32, np.int64(16), 0, np.int32(8), None, 8, q, 8, s)
    abi.moe_swiglu_quant(P, abi.DT_F32, 16, 0, 8, None, 8, P, 8, P, stream=0)


@pytest.mark.parametrize("bad,error", [
    (dict(gu="x"), TypeError), (dict(gu=1.5), TypeError), (dict(gu=object()), TypeError),
    (dict(T="2"), TypeError), (dict(T=2.0), TypeError), (dict(T=None), TypeError),
    (dict(T=1 << 31), OverflowError), (dict(F=-(1 << 31) - 1), OverflowError), (dict(ld=1 << 63), OverflowError),
    (dict(stream="s"), AttributeError), (dict(stream=1.0), AttributeError)])
def test_direct_calls_refuse_what_they_cannot_convert(bad, error):
    with pytest.raises(error):
        abi.moe_swiglu_quant(**{**SWIGLU, **bad})
    # and nothing of it is left behind
    refused(lambda: abi.moe_swiglu_quant(**{**SWIGLU, "T": -1}))


def test_direct_calls_take_a_tensor_whose_address_fails_as_that_error():
    class Tensor:
        def data_ptr(self):
            raise RuntimeError("no storage")

    with pytest.raises(RuntimeError, match="no storage"):
        abi.moe_swiglu_quant(**{**SWIGLU, "gu": Tensor()})


def test_direct_calls_need_the_whole_description():
    with pytest.raises(TypeError):
        abi.moe_route_select(abi.moe_cache_event(), P, 0, 8, None, 1, P, P)
    with pytest.raises(TypeError):
        abi.moe_route_select(None, P, 0, 8, None, 1, P, P)
    with pytest.raises(TypeError):
        abi.calls().moe_linear_int8(P, 1)
