"""The recorded DRAM figures of the benchmark's kernels are of the sources as they are: what other
kernels alone need has no place in the headers that these are compiled from."""

import pytest

import bench


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_figure_is_of_these_sources(kernel):
    assert bench.recorded_traffic(kernel) > 0
