"""CPU tests of the choice of a product's kernel: the rule at its borders."""
import itertools

import pytest

from tests import products_rule as rule


def test_rows_that_the_load_unit_copies():
    assert rule.copies(128, 128) and rule.copies(132, 4, 4) and rule.copies(1 << 23, 1 << 23)
    assert not rule.copies(130, 128) and not rule.copies(128, 130) and not rule.copies(128, 128, 2) and not rule.copies(128, 128, 1)
    assert not rule.copies((1 << 23) + 4, 128) and not rule.copies(128, (1 << 23) + 4) and not rule.copies(128, 128, 0, 130)
    assert rule.copies(1 << 20, 128, gathered=2048) and not rule.copies((1 << 20) + 4, 128, gathered=2048)
    assert rule.copies(1 << 30, 128, gathered=2) and not rule.copies(1 << 30, 128)


# up to 32 rows, and 12 to a group, the block's sums are the bf16 unit's; then fp32 outputs keep it
@pytest.mark.parametrize("N,K", [(1, 1), (256, 6144), (6144, 6144), (24576, 6144), (1 << 20, 128)])
@pytest.mark.parametrize("copied", [True, False])
def test_the_unit_of_few_and_of_many_rows(N, K, copied):
    for T in (1, 8, 9, 16, 17, 32, 33, 64, 1000, 1 << 15):
        assert rule.dense("f32", T, N, K, copied).unit == "f8x"
        assert rule.dense("bf16", T, N, K, copied).unit == ("f8x" if T <= 32 else "f8")
    if N <= 1 << 17:
        for E, rows in itertools.product((1, 8, 256), (1, 4, 5, 12, 13, 24, 64, 1000)):
            assert rule.grouped("fp8", "f32", E * rows, N, K, E, copied).unit == "f8x"
            assert rule.grouped("fp8", "bf16", E * rows, N, K, E, copied).unit == ("f8x" if rows <= 12 else "f8")
            assert rule.grouped("bf16", "bf16", E * rows, N, K, E, copied).unit == "bf16"
