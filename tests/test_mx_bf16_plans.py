"""The plans that the library chooses for products of bf16 rows with MXFP4 weights,
against the committed times of all of them (profiles/mx_bf16_plans.txt)."""

import math
import os

from perf import mx_bf16_plans as plans

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_chosen_plans_are_near_the_best():
    rows = plans.table(os.path.join(ROOT, "profiles", "mx_bf16_plans.txt"))
    found = plans.losses(rows)
    assert len(rows) == 447 and len(found) == 425
    assert math.exp(sum(math.log(f[0]) for f in found) / len(found)) <= 1.01
    assert found[0][0] <= 1.25


def test_geometry_of_a_plan():
    assert plans.geometry(plans.FORWARD, 333, 5500, 4096, "3x1") == (1, 3, 64, 66, 0)
    assert plans.geometry(plans.BACKWARD, 2048, 4096, 11008, "+2x0") == (0, 2, 64, 344, 256)
    assert plans.geometry(plans.GATED, 333, 2730, 2080, "1x2") == (2, 1, 33, 129, 129)
