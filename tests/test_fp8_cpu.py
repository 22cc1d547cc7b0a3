"""CPU tests of the E4M3 and grouped operators: every bad argument is refused with E_INVAL before
anything is enqueued, through the direct calls and through ctypes, and the plain forms that the GPU
tests go by agree with worked values and with torch's own E4M3."""
import inspect

import numpy as np
import pytest

from quantized_expert_ffn_topk_amd import abi
from tests import fp8_ref as ref
from tests.test_operators_cpu import P, refused

QUANT = dict(x=P, x_dtype=1, ldx=256, act=1, T=2, K=128, count=P, q=P, ldq=128, s=P, lds=1)
LINEAR = dict(q=P, ldq=200, s=P, lds=2, T=2, w=P, ldw=200, ws=P, ldws=2, bias=P, N=32, K=200, out=P, out_dtype=1, ldo=32)
GROUPED = dict(x=P, x_dtype=2, ldx=200, s=P, lds=2, R=9, rows=P, offsets=P, E=3, M=20, w=P, ldw=200, w_stride=130 * 200, ws=P,
               ldws=2, ws_stride=4, N=130, K=200, out=P, out_dtype=1, ldo=130)
GROUP = dict(idx=P, T=2, k=4, E=8, offsets=P, rows=P, pos=P)
COMBINE = dict(y=P, y_dtype=1, ldy=64, R=8, pos=P, gate_w=P, base=P, ldb=64, T=2, k=4, H=64, out=P, out_dtype=1, ldo=64)

CASES = {
    "moe_quant_fp8": (QUANT, [
        dict(x=None), dict(q=None), dict(s=None), dict(x_dtype=2), dict(x_dtype=-1), dict(act=2), dict(act=-1), dict(T=-1),
        dict(T=(1 << 25) + 1), dict(K=0), dict(K=(1 << 17) + 1, ldx=1 << 20, ldq=1 << 20, lds=1 << 12), dict(ldx=255), dict(ldq=127),
        dict(lds=0), dict(T=1 << 25, K=1024, ldx=2048, ldq=1024, lds=8), dict(x=P + 1), dict(x_dtype=0, x=P + 2), dict(s=P + 2),
        dict(count=P + 2)]),
    "moe_linear_fp8": (LINEAR, [
        dict(q=None), dict(s=None), dict(w=None), dict(ws=None), dict(out=None), dict(T=-1), dict(T=(1 << 20) + 1), dict(N=0),
        dict(N=(1 << 20) + 1), dict(T=1 << 16, N=(1 << 19) + 8, ldo=1 << 20), dict(K=0), dict(K=(1 << 17) + 1, ldq=1 << 18, ldw=1 << 18, lds=1 << 11, ldws=1 << 11), dict(ldq=199),
        dict(ldw=199), dict(ldo=31), dict(lds=1), dict(lds=(1 << 21) + 1), dict(ldws=1), dict(out_dtype=2), dict(s=P + 2), dict(ws=P + 1), dict(bias=P + 2),
        dict(out=P + 1), dict(out_dtype=0, out=P + 2)]),
    "moe_grouped_linear": (GROUPED, [
        dict(x=None), dict(s=None), dict(offsets=None), dict(w=None), dict(ws=None), dict(out=None), dict(x_dtype=0), dict(x_dtype=3),
        dict(R=0), dict(rows=None), dict(E=0), dict(E=1025), dict(M=-1), dict(M=(1 << 25) + 1), dict(N=0), dict(K=0), dict(ldx=199),
        dict(ldw=199), dict(lds=1), dict(lds=1 << 29), dict(R=4, lds=1 << 62), dict(rows=None, R=20, lds=(1 << 21) + 1), dict(ldws=1), dict(ldo=129), dict(w_stride=130 * 200 - 1), dict(ws_stride=3), dict(out_dtype=2),
        dict(rows=P + 2), dict(offsets=P + 1), dict(s=P + 2), dict(ws=P + 2), dict(out=P + 1), dict(x_dtype=1, x=P + 1),
        dict(x_dtype=1, w=P + 1), dict(x_dtype=1, out_dtype=0, out=P + 2),
        dict(N=(1 << 17) + 1, ldo=1 << 18, w_stride=1 << 28, ws_stride=1 << 14),
        dict(N=1 << 10, M=(1 << 23) + 1, ldo=1 << 10, w_stride=1 << 28, ws_stride=1 << 14)]),
    "moe_group_rows": (GROUP, [
        dict(idx=None), dict(offsets=None), dict(rows=None), dict(pos=None), dict(T=-1), dict(T=(1 << 20) + 1), dict(k=0), dict(k=33),
        dict(E=0), dict(E=1025), dict(idx=P + 1), dict(offsets=P + 2), dict(rows=P + 2), dict(pos=P + 1)]),
    "moe_combine_rows": (COMBINE, [
        dict(y=None), dict(pos=None), dict(gate_w=None), dict(out=None), dict(y_dtype=2), dict(out_dtype=2), dict(R=-1), dict(T=-1),
        dict(T=(1 << 20) + 1), dict(k=0), dict(k=33), dict(H=0), dict(H=(1 << 20) + 1), dict(ldy=63), dict(ldb=63), dict(ldo=63),
        dict(y=P + 1), dict(base=P + 1), dict(out=P + 1), dict(pos=P + 2), dict(gate_w=P + 2)]),
}
EACH = [(name, bad) for name, (_, bads) in CASES.items() for bad in bads]


@pytest.fixture(params=["direct", "ctypes"])
def way(request, monkeypatch, tmp_path):
    if request.param == "ctypes":
        monkeypatch.setattr(abi, "_calls", None)
        monkeypatch.setattr(abi, "CALLS_PATH", str(tmp_path / "_calls.so"))
    assert inspect.ismodule(abi.calls()) == (request.param == "direct")


@pytest.mark.parametrize("name,bad", EACH)
def test_refusals(way, name, bad):
    refused(getattr(abi, name), *dict(CASES[name][0], **bad).values())


def test_calls_of_no_rows_need_no_pointers(way):
    abi.moe_quant_fp8(None, 1, 256, 1, 0, 128, None, None, 128, None, 1)
    abi.moe_linear_fp8(None, 200, None, 2, 0, None, 200, None, 2, None, 32, 200, None, 1, 32)
    abi.moe_grouped_linear(None, 2, 200, None, 2, 0, None, None, 3, 0, None, 200, 0, None, 2, 0, 130, 200, None, 1, 130)
    abi.moe_combine_rows(None, 1, 64, 0, None, None, None, 64, 0, 4, 64, None, 1, 64)


def test_calls_need_all_their_arguments(way):
    for name in CASES:
        with pytest.raises(TypeError):
            getattr(abi.calls(), name)(P, 1)


def test_the_bound_functions_are_named():
    m = abi.calls()
    assert set(CASES) < set(m.NAMES) and all(hasattr(m, n) for n in m.NAMES)
    with pytest.raises(TypeError):
        m.bind(1, 2, abi.check, abi.addr)


# ---------------------------------------------------------------------------
# the plain forms themselves
# ---------------------------------------------------------------------------
def test_codes_agree_with_torch():
    torch = pytest.importorskip("torch")
    f8 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(f8, ref.TABLE.astype(np.float32), equal_nan=True)
    r = np.random.default_rng(1)
    v = np.concatenate([r.standard_normal(20000) * 10.0 ** r.uniform(-4, 2, 20000), ref.TABLE[:127],
                        (ref.TABLE[:126] + ref.TABLE[1:127]) / 2]).astype(np.float32)   # every tie
    v = np.clip(np.concatenate([v, -v]), -448, 448)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(v), want)


def test_quant_worked_values():
    v = np.zeros((1, 130), np.float32)
    v[0, :4] = [7.0, -3.5, 0.4375, 1e-4]
    v[0, 129] = -0.5
    q, s = ref.quant(v)
    np.testing.assert_allclose(s, [[7 / 448, 0.5 / 448]], rtol=1e-7)
    assert ref.decode(q)[0, :4].tolist() == [448.0, -224.0, 28.0, 0.005859375] and ref.decode(q)[0, 129] == -448


def test_group_worked_values():
    o, r, p = ref.group(np.array([[2, 0], [5, 2], [0, -1]]), 3)
    assert o.tolist() == [0, 2, 2, 4] and r.tolist() == [0, 2, 0, 1] and p.tolist() == [[2, 0], [-1, 3], [1, -1]]


def test_eights_are_the_largest_of_eight_neighbours():
    x, w = np.arange(1.0, 18.0)[None], np.ones((2, 17))
    w[1, 7] = -10
    assert ref.eights(x, w).tolist() == [[8 + 16 + 17, 80 + 16 + 17]]
