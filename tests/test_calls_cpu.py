"""CPU tests of the operators' calls where the module of direct calls is not built: the build goes
on without it, and the same calls, with the same errors, go through ctypes."""
import inspect
import os

import numpy as np
import pytest

from quantized_expert_ffn_topk_amd import abi, build
from tests import test_operators_cpu as t


@pytest.fixture
def no_module(monkeypatch, tmp_path):
    monkeypatch.setattr(abi, "_calls", None)
    monkeypatch.setattr(abi, "CALLS_PATH", str(tmp_path / "_calls.so"))
    assert not inspect.ismodule(abi.calls())


def test_the_module_is_taken_where_it_is_built():
    assert inspect.ismodule(abi.calls())


def cases(fn):
    mark = [m for m in fn.pytestmark if m.name == "parametrize"][0]
    return mark.args[1]


def test_refusals_through_ctypes(no_module):
    for fn in (t.test_norm_refusals, t.test_swiglu_refusals, t.test_linear_refusals, t.test_route_desc_refusals,
               t.test_route_select_refusals):
        for bad in cases(fn):
            fn(bad)
    t.test_null_descriptor_and_context_are_refused()
    t.test_no_rows_need_no_pointers()


def test_conversions_through_ctypes(no_module):
    t.test_direct_calls_take_numpy_arrays_and_integers()
    for bad, error in cases(t.test_direct_calls_refuse_what_they_cannot_convert):
        t.test_direct_calls_refuse_what_they_cannot_convert(bad, error)
    t.test_direct_calls_take_a_tensor_whose_address_fails_as_that_error()
    t.test_direct_calls_need_the_whole_description()
    abi.moe_rmsnorm_quant(None, 1, 64, None, 0, 0, None, 0, 64, np.float32(1e-6), None, 0, t.P, 64, None, 0, None)
    for eps in ("1e-6", None):
        with pytest.raises(TypeError):
            abi.moe_rmsnorm_quant(**{**t.NORM, "eps": eps})


@pytest.mark.parametrize("without", ["header", "compiler"])
def test_build_goes_on_without_the_module(without, monkeypatch, tmp_path, capsys):
    lib, calls = tmp_path / "libmoe.so", tmp_path / "_calls.so"
    calls.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "CALLS", str(calls))
    monkeypatch.setattr(build, "_compile", lambda src: (src + ".o", ""))
    made = []

    def link(cmd, out, verbose):
        made.append(out)
        open(out, "w").close()

    monkeypatch.setattr(build, "_link", link)
    if without == "header":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    else:
        monkeypatch.setattr(build, "CXX", str(tmp_path / "none"))
    assert build.build(verbose=False) == str(lib)
    assert made == [str(lib)] and not os.path.exists(calls)
    assert "ctypes" in capsys.readouterr().out


def test_build_makes_the_module_where_it_can(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    assert build.build_calls(verbose=False) == build.CALLS and os.path.getsize(build.CALLS) > 0


class Failing:
    def data_ptr(self):
        raise AttributeError("storage is gone")


def test_addresses():
    class Flag(int):
        pass

    class Pointer:
        def data_ptr(self):
            return 77

    a = np.arange(4)
    assert [abi.addr(x) for x in (None, 5, True, Flag(9), Pointer(), a)] == [None, 5, 1, 9, 77, a.ctypes.data]
    assert abi.addr(a[2:]) == a.ctypes.data + 16
    for x in ("x", 1.5, object()):
        with pytest.raises(TypeError):
            abi.addr(x)


def test_an_error_inside_data_ptr_is_passed_on():
    with pytest.raises(AttributeError, match="storage is gone"):
        abi.addr(Failing())


def test_an_error_inside_data_ptr_is_passed_on_by_the_direct_calls():
    with pytest.raises(AttributeError, match="storage is gone"):
        abi.moe_swiglu_quant(**{**t.SWIGLU, "gu": Failing()})
