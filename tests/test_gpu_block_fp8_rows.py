"""GPU tests of what block.py's E4M3 halves hold: a shared expert's rows are those between its products and no
others, and all are kept for the streams that work on them."""
import pytest

from tests import fp8_ref as ref
from tests.test_gpu_block_fp8 import F, dense, moe

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def tensors(*objects):
    return {a.data_ptr(): a for o in objects for a in vars(o).values() if isinstance(a, torch.Tensor)}


def test_the_shared_expert_has_no_rows_of_its_own_input():
    """max_tokens rows of the half's own bytes: all but the shared expert's gu, qh, sh are there without one too."""
    n = 1000
    size = lambda half: sum(a.numel() * a.element_size() for a in  # noqa: E731
                            tensors(half, *([half.shared] if half.shared else [])).values() if a.shape[0] == n)
    between = n * (2 * F * 2 + F + 4 * ref.blocks(F))
    assert size(moe(n, True)) - size(moe(n, False)) == between


def test_a_halfs_tensors_are_all_its_own():
    for half in (dense(), moe(), moe(shared=False)):
        parts = [half] + ([half.shared] if getattr(half, "shared", None) else [])
        assert {a.data_ptr() for a in half._own} == set(tensors(*parts))
