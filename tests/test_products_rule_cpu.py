"""CPU tests of the choice of a product's kernel: the rule at its borders, and the cases of products_cases held to it,
so that a change of the rule cannot take a kernel's cases away unseen."""
import itertools

import pytest

from tests import products_cases as pc
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


ALL = pc.DENSE + pc.GROUPED + pc.FAR + list(pc.TILES.values())


@pytest.mark.parametrize("case", ALL, ids=pc.label)
def test_a_case_takes_the_kernel_it_is_made_for(case):
    assert pc.name_of(pc.kernel(case)) == case["name"]


def reached(which):
    """(kernel, output) of the rule over a grid of sizes."""
    out = set()
    sizes = sorted({1 << i for i in range(18)} | {3 << i for i in range(16)} | {5003, 9003})
    for o, N, K, c in itertools.product(("bf16", "f32"), sizes, (1, 100, 1000, 4096, 9001, 1 << 17), (True, False)):
        for rows in sizes:
            if which == "dense":
                out.add((pc.name_of(rule.dense(o, rows, N, K, c)), o))
            else:
                for xd, E in itertools.product(("fp8", "bf16"), (1, 40)):
                    out.add((pc.name_of(rule.grouped(xd, o, rows, N, K, E, c)), o))
    return out


@pytest.mark.parametrize("which,cases", [("dense", pc.DENSE), ("grouped", pc.GROUPED)])
def test_every_kernel_has_a_case(which, cases):
    """Streams are the same code for both outputs but for their last store: a case of either will do."""
    have = {(c["name"], c["out"]) for c in cases}
    either = {n for n, _ in have}
    missing = {(n, o) for n, o in reached(which) if (n not in either if n.startswith("stream") else (n, o) not in have)}
    assert not missing


def test_far_cases_are_at_the_reach_of_copies():
    reach = {c["ldx"] * pc.rows_of_x(c) if c.get("gather") else c["ldx"] for c in pc.FAR if "copied" in pc.name_of(pc.kernel(c))}
    assert 1 << 23 in reach and max(reach) > (1 << 31) - 4 * 421
    for c in pc.FAR:
        rows = c["T"] if "T" in c else sum(c["sizes"])
        assert rows * c["ldo"] > 1 << 32


def test_the_bounds_on_tensors_are_the_references():
    import numpy as np
    torch = pytest.importorskip("torch")
    from tests import fp8_ref
    from tests.products_gpu import limit
    r = np.random.default_rng(1)
    for K in (1, 8, 77, 300):
        x, w = r.standard_normal((5, K)), r.standard_normal((7, K))
        for size, bf16, unit in ((1, False, False), (1, True, True), (2, True, False)):
            got = limit(torch.from_numpy(x), torch.from_numpy(w), size, bf16, unit).numpy()
            np.testing.assert_allclose(got, fp8_ref.limit(x, w, size, bf16, unit), rtol=1e-12)
