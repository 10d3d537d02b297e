"""The mixture-of-experts block of examples/moe_block.py, serving and training,
against plain float64."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_block_example():
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    for name, off in m.main().items():
        # Errors of single elements over the root mean square of all: values
        # reach 5 times that. BF16 keeps 2^-9 of a value at each of up to six
        # roundings on the way (rows, activation, expert, combined row, result,
        # gradient), sums of many keep the root of their number: within 5 x 6 x
        # 2^-9 < 0.06. With 8-bit experts each code is off by up to half a step
        # of 1/127 of its row's largest (4 times the mean): weights, tokens and
        # activations each add up to 4 / 254 of a value in a sum of independent
        # errors, sqrt(3) x 4 / 254 / sqrt(3) (uniform) = 0.016 for one
        # standard deviation, and the largest of 24576 lies within 5 of them.
        assert off < (0.06 + 5 * 0.016 if name.startswith("serve") else 0.06), (name, off)
