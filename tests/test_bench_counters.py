"""The hardware counters that the bench line quotes for the ring kernels."""
import pytest

import bench
import workloads


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_COUNTERS))
def test_recorded_counters_describe_the_sources(kernel):
    """They are quoted only while the kernel's sources hash to what was
    captured: a change elsewhere must not take them from the line."""
    if bench.KERNEL_COUNTERS[kernel]["sha1"] is None:
        pytest.skip("no capture of the present kernel")
    w = workloads.FWDBWD_CAUSAL_128K
    traffic, tensor_pct = bench.recorded_counters(kernel, w.name, w.S, w.H)
    assert traffic is not None and tensor_pct is not None
