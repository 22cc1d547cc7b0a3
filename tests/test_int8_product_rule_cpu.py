"""CPU tests of the choice of the int8 product's tile: its figures, as they stand in the source, against
the measured times of all eight tiles (profiles/int8_product_tiles.csv)."""
import csv
import math
import os

import pytest

from quantized_expert_ffn_topk_amd import abi
from tests import int8_product_rule as rule

TIMES = os.path.join(os.path.dirname(abi.PKG), "profiles", "int8_product_tiles.csv")


def measured():
    with open(TIMES) as f:
        rows = list(csv.DictReader(line for line in f if not line.startswith("#")))
    names = [k for k in rows[0] if "x" in k]
    return names, [(r["set"], (int(r["T"]), int(r["N"]), int(r["K"])), [float(r[n]) for n in names]) for r in rows]


def losses(which):
    """Time of the tile that is taken over the fastest one's, for each shape."""
    names, rows = measured()
    assert names == ["%dx%d" % t[:2] for t in rule.tiles()]
    out = []
    for kind, shape, us in rows:
        if kind == which:
            assert not rule.is_stream(*shape[:2]), shape
            costs = rule.tile_costs(*shape)
            out.append(us[costs.index(min(costs))] / min(us))
    return out


# the repository's statement: 0.3 % on average, 8 % at most; twice that is no longer the same choice
@pytest.mark.parametrize("which,count", [("fit", 139), ("other", 100)])
def test_the_tile_taken_is_nearly_the_fastest(which, count):
    loss = losses(which)
    assert len(loss) == count
    assert math.exp(sum(map(math.log, loss)) / count) < 1.006
    assert max(loss) < 1.16


def test_every_tile_is_the_fastest_somewhere():
    _, rows = measured()
    assert {us.index(min(us)) for _, _, us in rows} == set(range(8))


def test_every_tile_is_taken_somewhere():
    _, rows = measured()
    assert {rule.tile(*shape) for _, shape, _ in rows} == {t[:2] for t in rule.tiles()}
