"""CPU tests of refusals of the E4M3 and grouped operators that depend on more than one argument, through the
direct calls and through ctypes."""
import pytest

from quantized_expert_ffn_topk_amd import abi
from tests.conftest import gpu_available
from tests.test_fp8_cpu import COMBINE, P, way  # noqa: F401
from tests.test_operators_cpu import refused


def in_place(**more):
    return dict(COMBINE, base=P, out=P, **more).values()


@pytest.mark.parametrize("ldb,ldo", [(64, 72), (72, 64), (1 << 40, 64)])
@pytest.mark.parametrize("dtype", [abi.DT_F32, abi.DT_BF16])
def test_a_sum_in_place_has_one_distance_of_rows(way, dtype, ldb, ldo):  # noqa: F811
    """base = out with another distance: a token's row would be read after another token's was written there."""
    refused(abi.moe_combine_rows, *in_place(out_dtype=dtype, ldb=ldb, ldo=ldo))


@pytest.mark.skipif(gpu_available(), reason="the addresses are none: for a host that goes no further than its missing GPU")
@pytest.mark.parametrize("more", [dict(ldb=72, ldo=72), dict(T=1, ldb=72, ldo=64)])
def test_a_sum_in_place_with_one_distance_or_one_token_is_taken(way, more):  # noqa: F811
    with pytest.raises(abi.MoEError) as ei:
        abi.moe_combine_rows(*in_place(**more))
    assert ei.value.status == abi.E_UNSUPPORTED
