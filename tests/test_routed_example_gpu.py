"""The block of examples/routed_block.py, serving and training, against plain
float64."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_routed_example():
    spec = importlib.util.spec_from_file_location("routed_block", os.path.join(ROOT, "examples", "routed_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    for name, off in m.main().items():
        # Errors of single elements over the root mean square of all: values reach 5
        # times that. BF16 rounds by up to 2^-8 of a value, 2^-8 / sqrt(3) for one standard
        # deviation, at each of up to seven roundings on the way (rows, activation,
        # expert, combined row of either rank, result, gradient): 5 x sqrt(7) x 2^-8 /
        # sqrt(3) of a root mean square, and 5 x 2^-8 for the last one on the largest
        # element: 0.05. A gradient of the router sums such errors over a row of 256, each
        # times a value: the sum's root mean square and theirs grow alike. With
        # 4-bit experts a weight of a Gaussian group of 32, whose largest is 2 standard deviations
        # of it and more (codes of up to 6, so steps of 0.5 to 2 of 2.2 standard deviations /
        # 6), is off by up to half a step: 0.5 x 2.2 / 6 / sqrt(3) = 0.106 of it for one
        # standard deviation below 4 / 6 of the largest, where 85% lie, twice that above: 0.13.
        # Two such products, after one another, h's and z's halves: sqrt(2) x 0.13 x
        # 5 = 0.92 at most for the block's result, less in h, where the residual joins.
        assert off < (0.05 + 0.92 if name.startswith("serve") else 0.05), (name, off)


def test_routed_example_serves_the_weights_that_its_codes_stand_for():
    """Compared with the products of the quantized weights, a serving step is off by its roundings alone: the limit of
    the training step above (it has no more of them)."""
    spec = importlib.util.spec_from_file_location("routed_block", os.path.join(ROOT, "examples", "routed_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    report = m.main()
    assert report["serve h"] < 0.05 and report["serve z"] < 0.05, report
