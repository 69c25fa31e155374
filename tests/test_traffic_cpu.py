"""The DRAM traffic that bench.py reports beside the sweeps' rates."""
import os
import sys

import pytest

ROOT = os.path.join(os.path.dirname(__file__), "..")


@pytest.mark.parametrize("prec", ["fp16x3", "fp16"])
@pytest.mark.parametrize("kernel", ["tc_lse", "tc_stats"])
def test_traffic_is_recorded_for_the_present_sweeps(kernel, prec):
    """A change that the sweeps do not see (wrappers of other kernels) leaves their figures valid; one
    that they do see wants the figures taken again."""
    sys.path.insert(0, ROOT)
    import bench
    assert (bench.recorded_traffic(kernel, prec) or 0) > 0
