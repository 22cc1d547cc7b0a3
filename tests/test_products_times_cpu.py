"""CPU tests of the choice of the dense product's kernel against the measured times of the streams and tiles that more
than 32 rows can take (profiles/e4m3_product_kernels.csv)."""
import csv
import math
import os

import pytest

from quantized_expert_ffn_topk_amd import abi
from tests import products_rule as rule

TIMES = os.path.join(os.path.dirname(abi.PKG), "profiles", "e4m3_product_kernels.csv")


def losses(out, rows):
    """Time of the kernel that is taken over the fastest one's, for each shape."""
    with open(TIMES) as f:
        table = [r for r in csv.DictReader(line for line in f if not line.startswith("#")) if (r["out"], r["rows"]) == (out, rows)]
    loss = []
    for r in table:
        us = {n: float(v) for n, v in r.items() if "x" in n and v}
        k = rule.dense(out, int(r["T"]), int(r["N"]), int(r["K"]), rows == "copied")
        loss.append(us["%s%dx%d" % ("s" if k.way == "stream" else "", k.rows, k.channels)] / min(us.values()))
    return loss


# the repository's statement: 0.3, 0.7, 1.9 and 2 % on average and 14, 11, 21 and 22 % at most; twice that is no
# longer the same choice
@pytest.mark.parametrize("out,rows,mean,most", [("bf16", "copied", 1.006, 1.28), ("bf16", "registers", 1.014, 1.22),
                                                ("f32", "copied", 1.038, 1.42), ("f32", "registers", 1.04, 1.44)])
def test_the_kernel_taken_is_nearly_the_fastest(out, rows, mean, most):
    loss = losses(out, rows)
    assert len(loss) == 70
    assert math.exp(sum(map(math.log, loss)) / len(loss)) < mean and max(loss) < most
