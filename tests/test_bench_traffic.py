"""bench.py's measured DRAM traffic of the WKV7 backward belongs to the kernel sources
that it was taken on, by their hash: a change that reaches them (a declaration in a
header that they share will do) must bring a new figure, or the line reports null."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.mark.parametrize("which", ["TRAFFIC", "TRAFFIC_FP32"])
def test_the_figure_belongs_to_the_sources(which):
    import bench

    t = getattr(bench, which)
    assert bench.sources_sha256(t["sources"]) == t["sha256"]


def test_the_line_reports_it():
    import bench

    assert bench.measured_traffic(131072) > 0 and bench.measured_traffic_fp32(98304, 64) > 0
